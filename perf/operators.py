"""The serving operators around the packed cache, as cases to be timed and compared: block tables and slot maps, head norms with
the position rotation, the write of new tokens into pages, and attention of drafted tokens over a paged packed cache."""
import math

import numpy as np
import torch

own = False

D = 128  # head dimension of every packed cache here
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}

#: Lloyd-Max centroids of the normal distribution, positive half, for 1 to 4 bits.
HALF = {1: [0.7978846], 2: [0.4527800, 1.5104176],
        3: [0.2450942, 0.7560053, 1.3439093, 2.1519457],
        4: [0.1283951, 0.3880483, 0.6567591, 0.9423405, 1.2562312, 1.6180465, 2.0690172, 2.7326357]}


def centroids(b):
    h = np.array(HALF[b])
    return np.concatenate([-h[::-1], h])


def thresholds(b):
    c = centroids(b)
    return (c[1:] + c[:-1]) / 2


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a batch that has been running for a while: one token each, a page now and then
        {"name": "tables_step", "op": "tables", "batch": 32, "new": 1, "seq": 16384, "block": 16},
        # the admission of new prompts beside running requests
        {"name": "tables_prompts", "op": "tables", "batch": 257, "new": 1021, "seq": 16384, "block": 64},
        # one token of one request on its way into attention
        {"name": "norm_rope_token", "op": "norm_rope", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "style": 0, "type": "bf16", "out": "bf16"},
        # the drafted tokens of a batch
        {"name": "norm_rope_tree", "op": "norm_rope", "tokens": 509, "heads": 64, "kv_heads": 8, "dim": 128, "rot": 64, "style": 1, "type": "fp16", "out": "fp16"},
        # a long prompt
        {"name": "norm_rope_prompt", "op": "norm_rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "style": 0, "type": "bf16", "out": "fp16"},
        # the accepted tokens of a batch, into their pages
        {"name": "append_step", "op": "append", "batch": 32, "new": 3, "kv_heads": 8, "seq": 4096, "block": 16, "kbits": 4, "vbits": 4, "type": "fp16"},
        # a prompt, into its pages
        {"name": "append_prompt", "op": "append", "batch": 1, "new": 16384, "kv_heads": 8, "seq": 16384, "block": 64, "kbits": 3, "vbits": 3, "type": "fp16"},
        # a few short requests with small trees
        {"name": "tree_short", "op": "tree", "batch": 3, "heads": 8, "kv_heads": 8, "nodes": 7, "seq": 509, "block": 16, "kbits": 2, "vbits": 2, "type": "fp16", "mask": "tree"},
        # single-token decode over pages
        {"name": "tree_one_token", "op": "tree", "batch": 1, "heads": 32, "kv_heads": 8, "nodes": 1, "seq": 16384, "block": 64, "kbits": 4, "vbits": 4, "type": "bf16", "mask": "chain"},
        # ordinary trees over a ragged batch
        {"name": "tree_batch", "op": "tree", "batch": 8, "heads": 32, "kv_heads": 8, "nodes": 16, "seq": 8191, "block": 16, "kbits": 4, "vbits": 2, "type": "bf16", "mask": "tree"},
        # large trees
        {"name": "tree_wide", "op": "tree", "batch": 4, "heads": 64, "kv_heads": 8, "nodes": 63, "seq": 16384, "block": 128, "kbits": 3, "vbits": 3, "type": "fp16", "mask": "tree"},
        # a long context
        {"name": "tree_long", "op": "tree", "batch": 1, "heads": 64, "kv_heads": 8, "nodes": 32, "seq": 131072, "block": 64, "kbits": 3, "vbits": 3, "type": "bf16", "mask": "tree"},
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
        op = rng.choice(["tables", "norm_rope", "append", "tree", "tree"])
        if op == "tables":
            c = {"op": op, "batch": _log(rng, 1, 512), "new": _log(rng, 1, 2048), "seq": _log(rng, 16, 32768), "block": rng.choice([16, 32, 48, 64, 128, 256])}
        elif op == "norm_rope":
            dim = rng.choice([32, 64, 96, 128, 256])
            kv = rng.choice([1, 2, 4, 8])
            c = {"op": op, "tokens": _log(rng, 1, 16384), "heads": kv * rng.choice([1, 2, 4, 7, 8]), "kv_heads": kv, "dim": dim,
                 "rot": rng.choice([dim, dim // 2]), "style": rng.choice([0, 1]), "type": rng.choice(list(TYPES)), "out": rng.choice(list(TYPES))}
        elif op == "append":
            c = {"op": op, "batch": _log(rng, 1, 64), "new": _log(rng, 1, 4096), "kv_heads": rng.choice([1, 2, 4, 8]), "seq": _log(rng, 16, 16384),
                 "block": rng.choice([16, 32, 48, 64, 128]), "kbits": rng.randint(1, 4), "vbits": rng.randint(1, 4), "type": rng.choice(["fp32", "fp16"])}
            if c["batch"] * (c["new"] + c["seq"]) > 300000:
                continue
        else:
            kv = rng.choice([1, 2, 4, 8])
            c = {"op": op, "batch": _log(rng, 1, 16), "heads": kv * rng.choice([1, 2, 4, 8]), "kv_heads": kv, "nodes": _log(rng, 1, 100), "seq": _log(rng, 1, 131072),
                 "block": rng.choice([16, 32, 48, 64, 128]), "kbits": rng.randint(1, 4), "vbits": rng.randint(1, 4), "type": rng.choice(["fp32", "fp16", "bf16", "bf16"]),
                 "mask": rng.choice(["tree", "tree", "chain"])}
        w = work(c)
        if all(w[k] <= most[op, k] for k in w):
            return c


def work(c):
    """Means over what prepare() draws."""
    size = {"fp32": 4, "fp16": 2, "bf16": 2}
    if c["op"] == "tables":
        rows = c["batch"] * (c["new"] + 1) / 2
        taken = rows / c["block"] + c["batch"] / 2
        return {"bytes": rows * 12 + taken * 8 + c["batch"] * 20, "flops": rows * 4}
    if c["op"] == "norm_rope":
        n = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": n * (size[c["type"]] + size[c["out"]]) + c["tokens"] * 4, "flops": n * 9}
    if c["op"] == "append":
        n = c["batch"] * (c["new"] + 1) / 2 if c["batch"] > 1 else c["new"]
        n *= c["kv_heads"]
        return {"bytes": n * (2 * D * size[c["type"]] + 16 * (c["kbits"] + c["vbits"]) + 8), "flops": n * 4 * D * D}
    tokens = c["batch"] * c["seq"] * (0.75 if c["batch"] > 1 else 1)
    rows = c["batch"] * c["nodes"] * (0.75 if c["batch"] > 1 else 1)
    per = c["nodes"] * (0.75 if c["batch"] > 1 else 1)
    return {"bytes": tokens * c["kv_heads"] * (16 * (c["kbits"] + c["vbits"]) + 8) + rows * 2 * (c["heads"] + c["kv_heads"]) * D * size[c["type"]],
            "flops": 4 * D * c["heads"] * per * (tokens + rows)}


# ------------------------------------------------------------------ inputs
def _rotation(seed):
    q, r = np.linalg.qr(np.random.default_rng(seed).standard_normal((D, D)))
    return q * np.sign(np.diag(r))


def _codes(x, pi, b):
    """Codes of rows x and their norms, by the definition in 64 bits."""
    s = x.double().square().sum(-1).sqrt()
    v = (x.double() / s.clamp_min(1e-300)[:, None]) @ pi.T * math.sqrt(D)
    t = torch.tensor(thresholds(b), device=x.device, dtype=torch.float64)
    return torch.bucketize(v, t, right=True), s.float(), v


def _words(fields, b):
    """[n, m] codes of b bits as [n, m*b/32] words, the first code in the lowest bits."""
    n, m = fields.shape
    bits = (fields.int()[:, :, None] >> torch.arange(b, device=fields.device, dtype=torch.int32)) & 1
    bits = bits.reshape(n, m * b // 32, 32)
    return (bits << torch.arange(32, device=fields.device, dtype=torch.int32)).sum(-1, dtype=torch.int32)


def _fill(n, b, pair, pi, g):
    """Packed codes and norms of n rows with a few large channels, as keys and values have them."""
    codes, norm = [], []
    for lo in range(0, n, 1 << 18):
        x = torch.randn(min(n - lo, 1 << 18), D, device="cuda", generator=g)
        x[:, :4] *= 10
        s = x.square().sum(-1).sqrt()
        v = (x / s[:, None]) @ pi.float().T * math.sqrt(D)
        idx = torch.bucketize(v, torch.tensor(thresholds(b), device="cuda", dtype=torch.float32), right=True)
        if pair:
            idx = idx.view(-1, 2, D).transpose(1, 2).reshape(-1, 2 * D)
        codes.append(_words(idx, b).reshape(-1, 4 * b))
        norm.append(s)
    return torch.cat(codes), torch.cat(norm)


def _spread(lo, hi, n, g):
    """n counts from lo to hi, in an order of the seed's."""
    if n == 1:
        return torch.full((1,), hi, dtype=torch.int32, device="cuda")
    return torch.linspace(lo, hi, n, device="cuda", dtype=torch.float64).round().int()[torch.randperm(n, device="cuda", generator=g)]


def _lengths(c, g):
    """Ragged lengths: half to all of the case's length; one sequence alone has all of it."""
    return _spread((c["seq"] + 1) // 2, c["seq"], c["batch"], g)


def _pages(lens, block, g):
    """A table of pages in shuffled order for these lengths, and the number of pages."""
    need = (lens + block - 1) // block
    width, total = max(1, int(need.max())), max(1, int(need.sum()))
    order = torch.randperm(total, device="cuda", generator=g, dtype=torch.int32)
    first = need.cumsum(0) - need
    j = torch.arange(width, device="cuda")
    table = torch.where(j[None] < need[:, None], order[(first[:, None] + j[None]).clamp_max(total - 1)], -1)
    return table.int().contiguous(), total


def _starts(new):
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), new.cumsum(0).int()])


def _tree_masks(new, most, kind, g):
    """[rows, words] bits: the ancestors of every drafted token and itself; a random earlier token is its parent."""
    b = torch.repeat_interleave(torch.arange(new.numel(), device="cuda"), new.long())
    start = _starts(new)
    i = torch.arange(b.numel(), device="cuda") - start[b].long()
    up = (torch.rand(b.numel(), device="cuda", generator=g) * i).long().clamp_max(most)  # parent of node i: below i
    sees = torch.zeros(new.numel(), most, most, dtype=torch.bool, device="cuda")
    pad = torch.zeros(new.numel(), most, dtype=torch.long, device="cuda")
    pad[b, i] = up
    k = torch.arange(new.numel(), device="cuda")
    for t in range(most):
        if kind == "chain":
            sees[:, t, :t] = True
        elif t:
            sees[:, t] = sees[k, pad[:, t]]
        sees[:, t, t] = True
    words = (most + 31) // 32
    bits = torch.zeros(b.numel(), words * 32, dtype=torch.int64, device="cuda")
    bits[:, :most] = sees[b, i]
    w = (bits.view(-1, words, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int().contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "tables":
        lens, block = _lengths(c, g), c["block"]
        new = _spread(1, c["new"], c["batch"], g)
        held = (lens + block - 1) // block
        if c["batch"] > 1:  # one request has ended: its pages come back
            ended = new.argmin()
            lens[ended] = 0
            new[ended] = 0
        width = (c["seq"] + c["new"]) // block + 1
        total = c["batch"] * width
        order = torch.randperm(total, device="cuda", generator=g, dtype=torch.int32)
        first = held.cumsum(0) - held
        j = torch.arange(width, device="cuda")
        table = torch.where(j[None] < held[:, None], order[(first[:, None] + j[None]).clamp_max(total - 1)], -1)
        used = int(held.sum())
        ring = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        ring[:total - used] = order[used:]
        rows = int(new.sum())
        s |= {"len": lens, "new": new, "held": held.int(), "table": table.int().contiguous(), "ring": ring, "rows": rows + rows // 8,
              "state": torch.tensor([0, total - used], dtype=torch.int64, device="cuda")}
        if own:
            import kv_cache_vector_tq_gb300 as tq
            tq.lib()
        return s
    if c["op"] == "norm_rope":
        t, n, dim = TYPES[c["type"]], c["tokens"], c["dim"]
        width = (c["heads"] + 2 * c["kv_heads"]) * dim
        s["qkv"] = (torch.randn(n, width, device="cuda", generator=g) * (0.5 + torch.rand(n, 1, device="cuda", generator=g))).to(t)
        s["wq"] = (1 + 0.2 * torch.randn(dim, device="cuda", generator=g)).to(t)
        s["wk"] = (1 + 0.2 * torch.randn(dim, device="cuda", generator=g)).to(t)
        at = int(torch.randint(0, 131072 - 16384, (1,), device="cuda", generator=g))
        s["pos"] = torch.arange(at, at + n, device="cuda", dtype=torch.int32)
        s["inv"] = torch.tensor(1e6 ** (-np.arange(0, c["rot"], 2) / c["rot"]), device="cuda", dtype=torch.float64)
        if own:
            import kv_cache_vector_tq_gb300 as tq
            s["freq"] = tq.tq_rope_frequencies(s["inv"].cpu().numpy())
        return s
    pi = _rotation(seed)
    s["pi"] = torch.tensor(pi, device="cuda")
    kv, block = c["kv_heads"], c["block"]
    if own:
        import kv_cache_vector_tq_gb300 as tq

        # what a model's loading makes once for each layer: the device tables of its rotation and codebooks (1 to 5 ms each,
        # whatever is cached or asked later), nothing of a call's data; the rotation is the seed's here so that inputs differ
        def context(b):
            cb = tq.Codebook(d=D, b=b)
            cb.centroid[:1 << b] = centroids(b).tolist()
            cb.threshold[:(1 << b) - 1] = thresholds(b).tolist()
            return tq.Context(D, b, tq.TQ_MSE, tq.TQ_ROT_DENSE, pi, codebook=cb)

        kctx = context(c["kbits"])
        s["ctx"] = kctx, kctx if c["vbits"] == c["kbits"] else context(c["vbits"])
    lens = _lengths(c, g)
    if c["op"] == "append":
        t = TYPES[c["type"]]
        new = _spread(1, c["new"], c["batch"], g)
        table = _pages(lens + new, block, g)[0]
        pages = c["batch"] * ((c["seq"] + c["new"]) // block + 1)
        b = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), new.long())
        p = lens[b] + torch.arange(b.numel(), device="cuda") - _starts(new)[b]
        s["slots"] = table[b, (p // block).long()].long() * block + p % block
        n = b.numel()
        for name, bits in (("k", c["kbits"]), ("v", c["vbits"])):
            x = torch.randn(n, kv, D, device="cuda", generator=g)
            x[..., :4] *= 10
            x = x.to(t).view(-1, D)
            # a value on the border of two codes has no code of its own: such rows are drawn anew
            th = torch.tensor(thresholds(bits), device="cuda", dtype=torch.float64)
            for _ in range(6):
                v = _codes(x, s["pi"], bits)[2]
                near = (v[..., None] - th).abs().amin((-1, -2)) < 2e-5 if x.shape[0] < 1 << 15 else torch.cat([(u[..., None] - th).abs().amin((-1, -2)) < 2e-5 for u in v.split(1 << 14)])
                at = near.nonzero()[:, 0]
                if not at.numel():
                    break
                x[at] = torch.randn(at.numel(), D, device="cuda", generator=g).to(t)
            s["x" + name] = x.view(n, kv, D)
            if own:
                s["c" + name] = tq.CodeSet(s["ctx"][name == "v"], pages * kv * block, tq.TQ_LAYOUT_PAIR if name == "v" else tq.TQ_LAYOUT_TOKEN)
            else:
                s["c" + name] = torch.zeros(pages * kv * block, 4 * bits, dtype=torch.int32, device="cuda"), torch.zeros(pages * kv * block, device="cuda")
        return s
    t, hq = TYPES[c["type"]], c["heads"]
    table, pages = _pages(lens, block, g)
    new = _spread((c["nodes"] + 1) // 2, c["nodes"], c["batch"], g)
    rows = int(new.sum())
    s |= {"len": lens, "table": table, "start": _starts(new), "new": new}
    s["q"] = torch.randn(rows, hq, D, device="cuda", generator=g).to(t)
    s["k"] = torch.randn(rows, kv, D, device="cuda", generator=g).to(t)
    s["v"] = torch.randn(rows, kv, D, device="cuda", generator=g).to(t)
    s["k"][..., :4] *= 10
    s["v"][..., :4] *= 10
    s["mask"] = None if c["mask"] == "chain" else _tree_masks(new, c["nodes"], "tree", g)
    n = pages * kv * block
    for name, bits in (("k", c["kbits"]), ("v", c["vbits"])):
        codes, norm = _fill(n, bits, name == "v", s["pi"], g)
        if own:
            cs = tq.CodeSet(s["ctx"][name == "v"], n, tq.TQ_LAYOUT_PAIR if name == "v" else tq.TQ_LAYOUT_TOKEN)
            cs.codes[:codes.numel()] = codes.view(-1)
            cs.norm[:n] = norm
            s["c" + name] = cs
        else:
            s["c" + name] = codes, norm
    if own:  # the workspace that a program keeps; its contents do not matter
        s["ws"] = torch.empty(tq.tq_tree_attention_workspace_size(s["ctx"][0], c["batch"], hq, kv, rows) // 4 + 4, device="cuda")
    return s


# ------------------------------------------------------------------ the operators in their plain form
def _tables(s):
    c, block = s["case"], s["case"]["block"]
    need = (s["len"].long() + s["new"] + block - 1) // block
    take, give = (need - s["held"]).clamp_min(0), (s["held"] - need).clamp_min(0)
    head, tail = s["state"][0], s["state"][1]
    upto = take.cumsum(0)
    fits = (take == 0) | (upto <= tail - head)
    held = torch.where(fits, need, s["held"].long())
    taken = torch.where(fits, upto, 0).amax(0)
    new = torch.where(fits, s["new"], 0)
    ring, size = s["ring"].clone(), s["ring"].numel()
    j = torch.arange(s["table"].shape[1], device="cuda")
    fresh = fits[:, None] & (j[None] >= s["held"][:, None]) & (j[None] < need[:, None])
    at = (head + (upto - take)[:, None] + j[None] - s["held"][:, None]) % size
    table = torch.where(fresh, s["ring"][at], s["table"])
    back = (j[None] >= need[:, None]) & (j[None] < s["held"][:, None])
    to = (tail + (give.cumsum(0) - give)[:, None] + j[None] - need[:, None]) % size
    ring[to[back]] = s["table"][back]
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), new.cumsum(0)])
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(start[1:], r, right=True).clamp_max(c["batch"] - 1)
    p = s["len"][b] + r - start[b]
    live = r < start[-1]
    slots = torch.where(live, table[b, (p // block).clamp(0, table.shape[1] - 1)].long() * block + p % block, -1)
    return {"table": table, "ring": ring, "held": held.int(), "state": torch.stack([head + taken, tail + give.sum()]), "start": start.int(), "slots": slots,
            "pos": torch.where(live, p, 0).int()}


def _norm_rope(x, w, c, s):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    angle = s["pos"].double()[:, None] * s["inv"][None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot, half = c["rot"], c["rot"] // 2
    if c["style"] == 0:
        a, b = y[..., :half], y[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1).to(TYPES[c["out"]])


def _append(s, name, bits):
    c, x = s["case"], s["x" + name]
    kv, block = c["kv_heads"], c["block"]
    idx, norm, _ = _codes(x.view(-1, D), s["pi"], bits)
    codes, norms = s["c" + name]
    at = ((s["slots"] // block)[:, None] * kv + torch.arange(kv, device="cuda")) * block + (s["slots"] % block)[:, None]
    at = at.view(-1)
    norms[at] = norm
    if name == "k":
        codes[at] = _words(idx, bits)
        return codes, norms
    # a block holds two tokens: each takes its own bits out of it and puts its code there
    odd = (at % 2)[:, None, None]
    slot = torch.arange(2, device="cuda")
    w = codes.view(-1, 8 * bits)
    new = _words(torch.where(odd == slot, idx[:, :, None], 0).view(-1, 2 * D), bits)
    mine = _words(torch.where(odd == slot, (1 << bits) - 1, 0).expand(-1, D, 2).reshape(-1, 2 * D), bits)
    w.index_add_(0, at // 2, new - (w[at // 2] & mine))
    return codes, norms


def _unpack(words, b, pair):
    """Unit-variance values of packed vectors [n, 4b]: the codes' bits, then the codebook."""
    n = words.shape[0]
    step = 2 * b if pair else b
    at = torch.arange(D, device="cuda") * step
    w = words.view(-1, 8 * b) if pair else words
    last = w.shape[1] - 1
    if pair:
        at = (at[None] + torch.arange(2, device="cuda")[:, None] * b).view(-1)
    both = (w[:, at // 32].long() & 0xFFFFFFFF) | (w[:, (at // 32 + 1).clamp_max(last)].long() << 32)
    idx = (both >> (at % 32)) & ((1 << b) - 1)
    return torch.tensor(centroids(b), device="cuda", dtype=torch.float32)[idx].view(n, D)


def _tree(s):
    c = s["case"]
    batch, hq, kv, block = c["batch"], c["heads"], c["kv_heads"], c["block"]
    g, n, nodes = hq // kv, s["table"].shape[1] * block, c["nodes"]
    pi, scale = s["pi"].float(), 1 / math.sqrt(D)
    # the cache's vectors of every sequence and head, in order of position
    t = torch.arange(n, device="cuda")
    page = s["table"][:, t // block].clamp_min(0).long()
    at = ((page * kv)[:, None] + torch.arange(kv, device="cuda")[None, :, None]) * block + (t % block)[None, None]
    at = at.view(-1)
    ks, vs = s["ck"][1][at].view(batch, kv, n), s["cv"][1][at].view(batch, kv, n)
    k = _unpack(s["ck"][0], c["kbits"], False)[at].view(batch, kv, n, D)
    v = _unpack(s["cv"][0], c["vbits"], True)[at].view(batch, kv, n, D)
    # rows of q, padded to the longest sequence
    i = torch.arange(nodes, device="cuda")
    row = (s["start"][:-1, None] + i[None]).clamp_max(s["q"].shape[0] - 1).long()
    real = i[None] < s["new"][:, None]
    q = (s["q"].float()[row] * scale).view(batch, nodes, kv, g, D).permute(0, 2, 1, 3, 4).reshape(batch, kv, nodes * g, D)
    kn = s["k"].float()[row].permute(0, 2, 1, 3)
    vn = s["v"].float()[row].permute(0, 2, 1, 3)
    cached = (q @ pi.T) @ k.transpose(-1, -2) * (ks / math.sqrt(D))[:, :, None]
    cached = cached.masked_fill((t[None] >= s["len"][:, None])[:, None, None], -math.inf)
    drafted = q @ kn.transpose(-1, -2)
    if s["mask"] is None:
        sees = (i[:, None] >= i[None])[None].expand(batch, nodes, nodes)
    else:
        sees = ((s["mask"][row][..., i // 32] >> (i % 32)) & 1) != 0
    sees = (sees & real[:, None]).repeat_interleave(g, 1)[:, None]
    drafted = drafted.masked_fill(~sees, -math.inf)
    top = torch.maximum(cached.amax(-1), drafted.amax(-1))
    top = top.masked_fill(top == -math.inf, 0)[..., None]
    cached, drafted = (cached - top).exp(), (drafted - top).exp()
    total = (cached.sum(-1) + drafted.sum(-1))[..., None]
    out = (((cached * (vs / math.sqrt(D))[:, :, None]) @ v) @ pi + drafted @ vn) / total
    out = out.view(batch, kv, nodes, g, D).permute(0, 2, 1, 3, 4).reshape(batch, nodes, hq, D)
    return out[real].to(TYPES[c["type"]])


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if own:  # outputs are allocated in the pass, as the plain form's are
        import kv_cache_vector_tq_gb300 as tq
        if c["op"] == "tables":
            n, i32, i64 = s["rows"], torch.int32, torch.int64
            s = s | {"o": [torch.empty(m, dtype=t, device="cuda") for m, t in ((c["batch"], i32), (2, i64), (c["batch"] + 1, i32), (n, i64), (n, i32))]}
        elif c["op"] == "tree":
            s = s | {"out": torch.empty_like(s["q"])}
    if c["op"] == "tables":
        if not own:
            return _tables(s)
        held, after, start, slots, pos = s["o"]
        tq.tq_block_tables(s["len"], s["new"], s["held"], s["ring"], s["state"], s["table"], c["block"], held, after, start, slots, pos)
        return {"table": s["table"], "ring": s["ring"], "held": held, "state": after, "start": start, "slots": slots, "pos": pos}
    if c["op"] == "norm_rope":
        hq, kv, dim = c["heads"], c["kv_heads"], c["dim"]
        q = s["qkv"][:, :hq * dim].unflatten(1, (hq, dim))
        k = s["qkv"][:, hq * dim:(hq + kv) * dim].unflatten(1, (kv, dim))
        if not own:
            return _norm_rope(q, s["wq"], c, s), _norm_rope(k, s["wk"], c, s)
        qo = torch.empty(q.shape, dtype=TYPES[c["out"]], device="cuda")
        ko = torch.empty(k.shape, dtype=TYPES[c["out"]], device="cuda")
        tq.tq_qk_norm_rope(q, k, s["wq"], s["wk"], 1e-6, s["freq"], c["style"], s["pos"], qo, ko)
        return qo, ko
    if c["op"] == "append":
        if not own:
            (kc, kn), (vc, vn) = _append(s, "k", c["kbits"]), _append(s, "v", c["vbits"])
            return {"k": kc, "kn": kn, "v": vc, "vn": vn}
        for name, ctx in (("k", s["ctx"][0]), ("v", s["ctx"][1])):
            tq.tq_encode_slots(ctx, s["x" + name], s["slots"], c["block"], s["c" + name])
        return {"k": s["ck"].codes.view(-1, 4 * c["kbits"]), "kn": s["ck"].norm, "v": s["cv"].codes.view(-1, 4 * c["vbits"]), "vn": s["cv"].norm}
    if not own:
        return _tree(s)
    tq.tq_tree_attention(s["ctx"][0], s["ctx"][1], s["q"], s["k"], s["v"], s["start"], s["mask"], s["ck"], s["cv"], s["len"], s["table"], c["block"], 1 / math.sqrt(D), s["out"], s["ws"])
    return s["out"]


# ------------------------------------------------------------------ the definitions, in 64 bits
def _values64(words, b, pair):
    """Codebook values of packed vectors, bit by bit."""
    n = words.shape[0]
    w = words.view(-1, 8 * b) if pair else words
    bits = (w.long()[..., None] >> torch.arange(32, device="cuda")) & 1
    idx = (bits.view(w.shape[0], -1, b) << torch.arange(b, device="cuda")).sum(-1)
    if pair:
        idx = idx.view(-1, D, 2).transpose(1, 2)
    return torch.tensor(centroids(b), device="cuda")[idx.reshape(n, D)]


def exact(case, seed):
    c = case
    if c["op"] in ("tables",):
        return None
    s = prepare(c, seed)
    if c["op"] == "norm_rope":
        hq, kv, dim, rot = c["heads"], c["kv_heads"], c["dim"], c["rot"]
        x = s["qkv"][:, :(hq + kv) * dim].double().view(-1, hq + kv, dim)
        w = torch.cat([s["wq"].double().expand(hq, dim), s["wk"].double().expand(kv, dim)])
        y = x / (x.pow(2).sum(-1, keepdim=True) / dim + 1e-6).sqrt() * w
        turn = torch.polar(torch.ones(1, device="cuda", dtype=torch.float64), torch.outer(s["pos"].double(), s["inv"]))[:, None]
        if c["style"]:
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y[:, :hq].contiguous(), y[:, hq:].contiguous()
    kv, block = c["kv_heads"], c["block"]
    if c["op"] == "append":
        out = {"k": None, "v": None}
        h = torch.arange(kv, device="cuda")
        at = (s["slots"][:, None] // block * kv + h) * block + s["slots"][:, None] % block
        for name in "kv":
            norms = torch.zeros(s["c" + name][1].numel(), dtype=torch.float64, device="cuda")
            norms[at] = torch.linalg.vector_norm(s["x" + name].double(), dim=-1)
            out[name + "n"] = norms
        return out
    hq, g = c["heads"], c["heads"] // kv
    outs = []
    start = s["start"].tolist()
    for b, n in enumerate(s["len"].tolist()):
        t = torch.arange(n, device="cuda")
        page = s["table"][b, t // block].long()
        lo, hi = start[b], start[b + 1]
        new = torch.arange(hi - lo, device="cuda")
        if s["mask"] is None:
            sees = new[:, None] >= new[None]
        else:
            sees = (s["mask"][lo:hi].long()[:, new // 32] >> (new % 32) & 1).bool()
        heads = []
        for h in range(kv):
            at = (page * kv + h) * block + t % block
            kc, vc = s["ck"][0][at], s["cv"][0].view(-1, 2, 4 * c["vbits"])
            k = _values64(kc, c["kbits"], False) @ s["pi"] * (s["ck"][1][at].double() / math.sqrt(D))[:, None]
            pairs, where = torch.unique(at // 2, return_inverse=True)
            v = _values64(vc[pairs].reshape(-1, 4 * c["vbits"]), c["vbits"], True).view(-1, 2, D)[where, at % 2]
            v = v @ s["pi"] * (s["cv"][1][at].double() / math.sqrt(D))[:, None]
            k = torch.cat([k, s["k"][lo:hi, h].double()])
            v = torch.cat([v, s["v"][lo:hi, h].double()])
            q = s["q"][lo:hi, h * g:(h + 1) * g].double()
            z = torch.einsum("igd,td->igt", q, k) / math.sqrt(D)
            z[:, :, n:].masked_fill_(~sees[:, None], -math.inf)
            heads.append(torch.softmax(z, -1) @ v)
        outs.append(torch.cat(heads, 1))
    return torch.cat(outs)
