"""The calls around a paged cache held in 8 bits, as cases to be timed and compared: the write of new tokens with norms and position
rotation on the way, attention over the cache, and attention with a sliding window and first tokens that stay visible."""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one request, in the middle of a block
        {"name": "append_token", "op": "append", "batch": 1, "new": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "style": 0, "norm": False, "seq": 4097, "block": 64, "type": "bf16"},
        # a few drafted tokens of every request of a batch, head norms, part of the head turned
        {"name": "append_step", "op": "append", "batch": 32, "new": 5, "heads": 28, "kv_heads": 4, "dim": 128, "rot": 64, "style": 1, "norm": True, "seq": 4096, "block": 16, "type": "fp16"},
        # a long prompt
        {"name": "append_prompt", "op": "append", "batch": 1, "new": 16384, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "style": 0, "norm": True, "seq": 0, "block": 64, "type": "bf16"},
        # a few short requests
        {"name": "attend_short", "op": "attend", "batch": 3, "new": 1, "heads": 8, "kv_heads": 8, "dim": 64, "seq": 509, "block": 16, "type": "fp16"},
        # single-token decode of one long request
        {"name": "attend_token", "op": "attend", "batch": 1, "new": 1, "heads": 64, "kv_heads": 8, "dim": 128, "seq": 131071, "block": 64, "type": "bf16"},
        # single-token decode of a ragged batch
        {"name": "attend_batch", "op": "attend", "batch": 32, "new": 1, "heads": 32, "kv_heads": 8, "dim": 128, "seq": 16384, "block": 16, "type": "bf16"},
        # drafted chains over a ragged batch
        {"name": "attend_drafts", "op": "attend", "batch": 8, "new": 15, "heads": 32, "kv_heads": 8, "dim": 128, "seq": 8191, "block": 48, "type": "fp16"},
        # a model run in fp32
        {"name": "attend_fp32", "op": "attend", "batch": 4, "new": 3, "heads": 16, "kv_heads": 4, "dim": 64, "seq": 4093, "block": 32, "type": "fp32"},
        # a prompt's next piece behind a long cached one
        {"name": "attend_prompt", "op": "attend", "batch": 1, "new": 2039, "heads": 32, "kv_heads": 8, "dim": 128, "seq": 16384, "block": 64, "type": "bf16"},
        # decode of a batch in a layer with a window
        {"name": "window_batch", "op": "window", "batch": 64, "new": 1, "heads": 64, "kv_heads": 8, "dim": 128, "seq": 16384, "block": 64, "window": 1024, "sinks": 4, "type": "bf16"},
        # drafted chains there, an odd window
        {"name": "window_drafts", "op": "window", "batch": 16, "new": 7, "heads": 16, "kv_heads": 8, "dim": 128, "seq": 8191, "block": 16, "window": 509, "sinks": 0, "type": "fp16"},
        # a whole prompt there
        {"name": "window_prompt", "op": "window", "batch": 1, "new": 8179, "heads": 16, "kv_heads": 4, "dim": 128, "seq": 0, "block": 128, "window": 1024, "sinks": 4, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for k in w:
            most[c["op"], k] = max(most.get((c["op"], k), 0), w[k])
    while True:
        op = rng.choice(["append", "attend", "attend", "window"])
        kv = rng.choice([1, 2, 4, 8])
        c = {"op": op, "batch": _log(rng, 1, 256 if op == "append" else 64), "new": _log(rng, 1, 4096), "heads": kv * rng.choice([1, 2, 4, 7, 8]), "kv_heads": kv,
             "dim": rng.choice([64, 128, 128]), "seq": _log(rng, 1, 131072), "block": rng.choice([16, 32, 48, 64, 128])}
        if op == "append":
            c |= {"rot": c["dim"] // rng.choice([1, 1, 2]), "style": rng.choice([0, 1]), "norm": rng.choice([False, True])}
        if op == "window":
            c |= {"window": _log(rng, 16, 4096), "sinks": rng.choice([0, 1, 4, 64])}
        c["type"] = rng.choice(["fp32", "fp16", "bf16", "bf16"])
        if c["batch"] * (c["seq"] + c["new"]) * kv > 9e6 or c["batch"] * c["new"] > 65536:  # the cache of a few GB
            continue
        if op != "append" and c["batch"] * c["new"] * c["heads"] * (c["seq"] + c["new"]) > 1.2e9:  # scores of the plain form
            continue
        w = work(c)
        if all(w[k] <= most[op, k] for k in w):
            return c


def _mean(c):
    """Mean length and new tokens of a request: half to all of the case's."""
    part = 0.75 if c["batch"] > 1 else 1
    return c["seq"] * part, max(1, c["new"] * part)


def work(c):
    """Means over what prepare() draws."""
    size = {"fp32": 4, "fp16": 2, "bf16": 2}[c["type"]]
    seq, new = _mean(c)
    batch, heads, kv, d = c["batch"], c["heads"], c["kv_heads"], c["dim"]
    rows = batch * new
    if c["op"] == "append":
        n = rows * d
        return {"bytes": n * (2 * heads * size + 2 * kv * (size + 1)) + 8 * kv * batch * (new / c["block"] + 1), "flops": n * 9 * (heads + kv) + n * 3 * kv}
    # tokens that some row of a request sees, and those that a row sees on average
    if c["op"] == "attend":
        read, sees = seq + new, seq + (new + 1) / 2
    else:
        read = min(seq + new, c["window"] + new - 1 + c["sinks"])
        sees = min(seq + (new + 1) / 2, c["window"] + c["sinks"])
        if seq < c["window"] < seq + new:  # rows at the beginning see fewer
            ramp = c["window"] - seq
            sees = ((seq + c["window"]) / 2 * ramp + (c["window"] + c["sinks"]) * (new - ramp)) / new
    return {"bytes": batch * read * kv * (2 * d + 8 / c["block"]) + rows * 2 * heads * d * size, "flops": 4 * d * heads * rows * sees}


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n, g):
    """n counts from lo to hi, in an order of the seed's; one alone has all of it."""
    if n == 1:
        return torch.full((1,), hi, dtype=torch.int32, device="cuda")
    return torch.linspace(lo, hi, n, device="cuda", dtype=torch.float64).round().int()[torch.randperm(n, device="cuda", generator=g)]


def _starts(new):
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), new.cumsum(0).int()])


def _pages(need, width, total, g):
    """A table of pages in shuffled order."""
    order = torch.randperm(total, device="cuda", generator=g, dtype=torch.int32)
    first = need.cumsum(0) - need
    j = torch.arange(width, device="cuda")
    table = torch.where(j[None] < need[:, None], order[(first[:, None] + j[None]).clamp_max(total - 1)], -1)
    return table.int().contiguous()


def _power(a):
    """The least power of two s with a <= 448 s."""
    m, e = torch.frexp(a)  # a = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    s = torch.ldexp(torch.ones_like(a), e - 9 + (m > 0.875).int())
    return torch.where(a > 0, s, 2.0 ** -60).clamp(2.0 ** -60, 2.0 ** 40)


def _fill(codes, scales, g):
    """Codes and scales of keys or values with a few large channels, a magnitude for each token."""
    pages, kv, block, d = codes.shape
    step = max(1, (1 << 26) // (kv * block * d))
    for lo in range(0, pages, step):
        n = min(step, pages - lo)
        x = torch.randn(n, kv, block, d, device="cuda", generator=g)
        x[..., :4] *= 6
        x *= 0.5 + torch.rand(n, kv, block, 1, device="cuda", generator=g)
        s = _power(x.abs().amax((2, 3)))
        codes[lo:lo + n] = (x / s[:, :, None, None]).to(F8)
        scales[lo:lo + n] = s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    kv, hq, d, block, t = c["kv_heads"], c["heads"], c["dim"], c["block"], TYPES[c["type"]]
    lens = _spread((c["seq"] + 1) // 2, c["seq"], c["batch"], g)
    new = _spread((c["new"] + 1) // 2, c["new"], c["batch"], g)
    width = (c["seq"] + c["new"] + block - 1) // block
    pages = int(((lens + block - 1) // block + (new + block - 1) // block).sum())  # the same for every seed
    table = _pages((lens + new + block - 1) // block, width, pages, g)
    s = {"case": c, "len": lens, "new": new, "start": _starts(new), "table": table, "pages": pages}
    rows = int(new.sum())
    if own:
        import kv_cache_vector_tq_gb300 as tq
        cache = s["cache"] = tq.Cache8(pages, kv, block, d)
        s |= {"k8": cache.k, "v8": cache.v, "ks": cache.kscale, "vs": cache.vscale}
    else:
        s["k8"], s["v8"] = (torch.zeros(pages, kv, block, d, device="cuda").to(F8) for _ in range(2))
        s["ks"], s["vs"] = (torch.zeros(pages, kv, device="cuda") for _ in range(2))
    _fill(s["k8"], s["ks"], g)
    _fill(s["v8"], s["vs"], g)
    if c["op"] == "append":
        width = (hq + 2 * kv) * d  # a joint projection of q, k and v
        x = torch.randn(rows, width, device="cuda", generator=g) * (0.5 + torch.rand(rows, 1, device="cuda", generator=g))
        x.view(rows, -1, d)[:, hq:, :4] *= 10
        s["qkv"] = x.to(t)
        s["wq"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(t) if c["norm"] else None
        s["wk"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(t) if c["norm"] else None
        b = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), new.long())
        s["pos"] = (lens[b] + torch.arange(rows, device="cuda") - s["start"][b]).int()
        s["inv"] = torch.tensor(1e6 ** (-np.arange(0, c["rot"], 2) / c["rot"]), device="cuda", dtype=torch.float64)
        if own:
            s["freq"] = tq.tq_rope_frequencies(s["inv"].cpu().numpy())
        return s
    s["q"] = torch.randn(rows, hq, d, device="cuda", generator=g).to(t)
    if own:  # the workspace that a program keeps; its contents do not matter
        s["ws"] = torch.empty(tq.tq_cache8_attention_workspace_size(cache, c["batch"], hq, rows) // 4 + 4, device="cuda")
    return s


# ------------------------------------------------------------------ the operators in their plain form
def _turned(x, w, s):
    """Head norms where the model has them, and the rotation of x [rows, heads, d], in 32 bits."""
    c, y = s["case"], x.float()
    if c["norm"]:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    angle = s["pos"].double()[:, None] * s["inv"][None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot, half = c["rot"], c["rot"] // 2
    if c["style"] == 0:
        a, b = y[..., :half], y[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _store(x, codes, scales, s):
    """Rows x [rows, kv, d] in 32 bits into their blocks."""
    c, block, lens = s["case"], s["case"]["block"], s["len"].long()
    b = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), s["new"].long(), output_size=x.shape[0])
    at = lens[b] + torch.arange(x.shape[0], device="cuda") - s["start"][b]
    page, place = s["table"][b, at // block].long(), at % block
    need = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax")
    now = scales.index_copy(0, page, _power(need)[page])
    # the block in which a request's new tokens begin may hold some already: its scale does not shrink, and they are rounded again if it grows
    inside = lens % block
    on = inside > 0
    held, stays = s["table"][on, (lens // block)[on]].long(), torch.arange(block, device="cuda")[None] < inside[on][:, None]
    now[held] = torch.maximum(now[held], scales[held])
    kept = codes[held].float()
    again = (kept * (scales[held] / now[held])[:, :, None, None]).to(F8).float()
    codes[held] = torch.where(stays[:, None, :, None], again, kept).to(F8)
    codes[page, :, place] = (x / now[page][:, :, None]).to(F8)
    scales.copy_(now)


def _attend(s):
    c = s["case"]
    batch, hq, kv, block, d, new = c["batch"], c["heads"], c["kv_heads"], c["block"], c["dim"], c["new"]
    g, n = hq // kv, s["table"].shape[1] * c["block"]
    page = s["table"].clamp_min(0).long()
    k = (s["k8"][page].float() * s["ks"][page][..., None, None]).transpose(1, 2).reshape(batch, kv, n, d)
    v = (s["v8"][page].float() * s["vs"][page][..., None, None]).transpose(1, 2).reshape(batch, kv, n, d)
    i = torch.arange(new, device="cuda")
    t = torch.arange(n, device="cuda")
    row = (s["start"][:-1, None] + i[None]).clamp_max(s["q"].shape[0] - 1).long()
    real = i[None] < s["new"][:, None]
    q = (s["q"].float()[row] / math.sqrt(d)).view(batch, new, kv, g, d).permute(0, 2, 3, 1, 4).reshape(batch, kv, g * new, d)
    p = s["len"][:, None] + i[None]
    sees = t[None, None] <= p[..., None]
    if c["op"] == "window":
        sees &= (t[None, None] > p[..., None] - c["window"]) | (t < c["sinks"])
    z = (q @ k.transpose(-1, -2)).view(batch, kv, g, new, n)
    z = z.masked_fill(~sees[:, None, None], -math.inf)
    z = (z - z.amax(-1, keepdim=True)).exp()
    z = z / z.sum(-1, keepdim=True)
    # what no row of a request sees is left out of the sum, whatever it holds
    v = v.masked_fill((t[None] >= (s["len"] + s["new"])[:, None])[:, None, :, None], 0)
    out = (z.view(batch, kv, g * new, n) @ v).view(batch, kv, g, new, d).permute(0, 3, 1, 2, 4).reshape(batch, new, hq, d)
    return out[real].to(TYPES[c["type"]])


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if c["op"] == "append":
        hq, kv, d = c["heads"], c["kv_heads"], c["dim"]
        x = s["qkv"].view(-1, hq + 2 * kv, d)
        q, k, v = x[:, :hq], x[:, hq:hq + kv], x[:, hq + kv:]
        if own:
            import kv_cache_vector_tq_gb300 as tq
            out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
            tq.tq_cache8_append(q, k, v, s["wq"], s["wk"], 1e-6 if c["norm"] else 0.0, s["freq"], c["style"], s["pos"], s["start"], s["len"], s["table"], s["cache"], out)
        else:
            out = _turned(q, s["wq"], s).to(q.dtype)
            _store(_turned(k, s["wk"], s), s["k8"], s["ks"], s)
            _store(v.float(), s["v8"], s["vs"], s)
        return {"q": out, "k": s["k8"], "v": s["v8"], "ks": s["ks"], "vs": s["vs"]}
    if not own:
        return _attend(s)
    import kv_cache_vector_tq_gb300 as tq
    out = torch.empty_like(s["q"])
    tq.tq_cache8_attention(s["q"], s["start"], s["len"], s["table"], s["cache"], 1 / math.sqrt(c["dim"]), out, s["ws"], window=c.get("window", 0), sinks=c.get("sinks", 0))
    return out


# ------------------------------------------------------------------ the definitions, in 64 bits
def _exact_append(c, s):
    hq, kv, d, rot, block = c["heads"], c["kv_heads"], c["dim"], c["rot"], c["block"]
    x = s["qkv"].double().view(-1, hq + 2 * kv, d)
    y = x[:, :hq + kv].clone()
    if c["norm"]:
        w = torch.cat([s["wq"].double().expand(hq, d), s["wk"].double().expand(kv, d)])
        y = y / (y.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w
    turn = torch.polar(torch.ones(1, device="cuda", dtype=torch.float64), torch.outer(s["pos"].double(), s["inv"]))[:, None]
    if c["style"]:
        z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    out = {"q": y[:, :hq].contiguous()}
    start, lens, table = s["start"].tolist(), s["len"].tolist(), s["table"].cpu().numpy()
    for name, rows in (("k", y[:, hq:]), ("v", x[:, hq + kv:])):
        codes, scales = s[name + "8"].double(), s[name + "s"].double()
        for b, n in enumerate(lens):
            r = start[b]
            while r < start[b + 1]:
                at = n + r - start[b]
                page, place = int(table[b, at // block]), at % block
                m = min(block - place, start[b + 1] - r)
                new = rows[r:r + m].transpose(0, 1)
                top = new.abs().amax((1, 2)).clamp_min(1e-300)
                scale = torch.exp2(torch.ceil(torch.log2(top / 448)))
                scale = torch.where(scale / 2 * 448 >= top, scale / 2, torch.where(scale * 448 < top, scale * 2, scale)).clamp(2.0 ** -60, 2.0 ** 40)
                if place:
                    scale = torch.maximum(scale, scales[page])
                    codes[page, :, :place] = (codes[page, :, :place] * (scales[page] / scale)[:, None, None]).float().to(F8).double()
                scales[page] = scale
                codes[page, :, place:place + m] = new / scale[:, None, None]
                r += m
        out |= {name: codes, name + "s": scales}
    return out


def exact(case, seed):
    c = case
    if c["op"] == "append" and c["batch"] * (c["new"] // c["block"] + 2) > 4096:
        return None
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    if work(c)["flops"] > 4e12:
        return None
    hq, kv, d, block = c["heads"], c["kv_heads"], c["dim"], c["block"]
    g, outs, start = hq // kv, [], s["start"].tolist()
    for b, n in enumerate(s["len"].tolist()):
        lo, hi = start[b], start[b + 1]
        t = torch.arange(n + hi - lo, device="cuda")
        page, place = s["table"][b, t // block].long(), t % block
        p = n + torch.arange(hi - lo, device="cuda")
        hidden = t[None] > p[:, None]
        if c["op"] == "window":
            hidden = hidden | ((t[None] <= p[:, None] - c["window"]) & (t[None] >= c["sinks"]))
        heads = []
        for h in range(kv):
            k = s["k8"][page, h, place].double() * s["ks"][page, h].double()[:, None]
            v = s["v8"][page, h, place].double() * s["vs"][page, h].double()[:, None]
            q = s["q"][lo:hi, h * g:(h + 1) * g].double()
            z = torch.einsum("igd,td->git", q, k) / math.sqrt(d)
            heads.append((torch.softmax(z.masked_fill_(hidden, -math.inf), -1) @ v).transpose(0, 1))
        outs.append(torch.cat(heads, 1))
    return torch.cat(outs)
