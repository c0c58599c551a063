"""The calls on an 8-bit paged cache against their definitions in 64 bits: appends with norms and position rotation,
attention, windows with first tokens that stay visible, and a server's steps of both."""

import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import kv_cache_vector_tq_gb300 as tq  # noqa: E402

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
LO, HI = 2.0 ** -60, 2.0 ** 40


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def least_scale(a):
    """The least power of two s with a <= 448 s, within [LO, HI] (float64 tensor)."""
    m, e = torch.frexp(a)
    e = (e - 9 + (m > 0.875).int()).clamp(-60, 40)  # (a = 0: below)
    s = ((e.long() + 1023) << 52).view(torch.float64)  # 2^e, bit for bit
    return torch.where(a > 0, s, LO)


def pages_for(need, block, g, spare=2):
    """A table of pages in shuffled order for these numbers of tokens, and the number of pages."""
    n = [(x + block - 1) // block for x in need]
    total = sum(n) + spare
    order = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((len(n), max(n + [1])), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(n):
        table[b, :k] = order[at:at + k]
        at += k
    return table, total


def filled(cache, g, spread=3):
    """Codes of every kind but NaN, scales over a few powers of two."""
    for codes, scale in ((cache.k, cache.kscale), (cache.v, cache.vscale)):
        codes.copy_((torch.randn(codes.shape, device="cuda", generator=g) * 60).clamp(-440, 440).to(F8))
        scale.copy_(torch.exp2(torch.randint(-spread - 6, spread - 5, scale.shape, device="cuda", generator=g).float()))


# ------------------------------------------------------------------ append
def turned(x, w, eps, inv, style, pos):
    y = x.double()
    if eps:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
        if w is not None:
            y = y * w.double()
    rot = 2 * len(inv)
    if not rot:
        return y
    ang = pos.double()[:, None] * torch.tensor(inv, device="cuda", dtype=torch.float64)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    y = y.clone()
    if style == tq.TQ_ROPE_HALF:
        a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def blocks_of(start, lens, table, block, b):
    """(first row, page, place, tokens) of every block that request b's new rows touch."""
    r = start[b]
    while r < start[b + 1]:
        at = lens[b] + r - start[b]
        m = min(block - at % block, start[b + 1] - r)
        yield r, int(table[b, at // block]), at % block, m
        r += m


def check_append(before, after, rows, exact, start, lens, table, block):
    """Codes and scales after an append of `rows` [n, Hkv, d] (float64); `exact`: the rows are the kernel's own, bit for bit."""
    codes0, scale0 = before
    codes1, scale1 = after
    want, wants = codes0.float(), scale0.clone()
    for b in range(len(lens)):
        for r, page, place, m in blocks_of(start, lens, table, block, b):
            new = rows[r:r + m].transpose(0, 1)  # [Hkv, m, d]
            top = new.abs().amax((1, 2))
            s = least_scale(top)
            got = scale1[page].double()
            if place:
                s = torch.maximum(s, scale0[page].double())
            if exact:
                assert torch.equal(got, s), (b, page)
            else:  # a magnitude within 1e-5 of the border may fall on either side
                near = (least_scale(top * (1 + 1e-5)) != least_scale(top * (1 - 1e-5)))
                assert (near | (got == s)).all(), (b, page)
                s = got
            if place:
                kept = codes0[page, :, :place].double() * (scale0[page].double() / s)[:, None, None]
                want[page, :, :place] = kept.float().to(F8).float()
            ideal = new / s[:, None, None]
            mine = codes1[page, :, place:place + m].double()
            if exact:
                assert torch.equal(mine, ideal.float().to(F8).double()), (b, page)
            else:
                # half a step (2^-4 of the number, 2^-10 below 2^-6) and what fp32 norms and rotations are off by
                tol = ideal.abs().clamp_min(2.0 ** -6) * 2.0 ** -4 + 2e-6 * top[:, None, None] / s[:, None, None]
                assert ((mine - ideal).abs() <= tol).all(), (b, page)
            want[page, :, place:place + m] = codes1[page, :, place:place + m].float()
            wants[page] = scale1[page]
    # whatever no new row touches is as it was, bit for bit
    assert torch.equal(codes1.float(), want) and torch.equal(scale1, wants)


CASES = [
    # lens, new, Hq, Hkv, d, rot, style, norm, block, type
    ([0], [1], 8, 2, 128, 128, 0, False, 16, "bf16"),
    ([15], [1], 4, 4, 128, 128, 0, True, 16, "fp16"),
    ([16], [1], 1, 1, 64, 64, 0, False, 16, "fp32"),
    ([5, 0, 31, 64], [3, 7, 0, 1], 12, 3, 128, 64, 1, True, 32, "bf16"),
    ([33, 1, 47], [100, 1, 17], 7, 1, 64, 32, 1, True, 48, "fp16"),
    ([130], [257], 16, 8, 128, 128, 0, True, 64, "bf16"),
    ([0, 63, 64, 65], [64, 65, 66, 1], 8, 8, 64, 64, 0, False, 64, "bf16"),
    ([100, 3], [300, 129], 4, 2, 128, 96, 1, False, 128, "fp32"),
    ([70], [500], 2, 2, 128, 16, 0, True, 256, "fp16"),
    ([0], [0], 2, 2, 128, 128, 0, True, 16, "bf16"),
    ([9] * 40, [2] * 40, 4, 1, 128, 128, 0, True, 16, "bf16"),
    ([1000], [33], 4, 2, 128, 0, 0, True, 16, "bf16"),
    ([17], [40], 4, 2, 128, 0, 0, False, 1024, "fp16"),
]


@pytest.mark.parametrize("lens,new,Hq,Hkv,d,rot,style,norm,block,ty", CASES)
def test_append(lens, new, Hq, Hkv, d, rot, style, norm, block, ty):
    g, t = gen(len(lens) + block), TYPES[ty]
    table, total = pages_for([a + b for a, b in zip(lens, new)], block, g)
    cache = tq.Cache8(total, Hkv, block, d)
    filled(cache, g)
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    rows = start[-1] + 3  # rows behind the last request's
    x = torch.randn(rows, Hq + 2 * Hkv, d, device="cuda", generator=g) * torch.exp2(3 * torch.randn(rows, 1, 1, device="cuda", generator=g))
    x = x.to(t)
    wq, wk = ((1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(t) if norm else None for _ in range(2))
    inv = 1e4 ** (-np.arange(0, rot, 2) / max(rot, 1))
    pos = torch.randint(0, 1 << 20, (rows,), device="cuda", generator=g).int()
    out = torch.full((rows, Hq, d), 7.0, device="cuda", dtype=t)
    k0, v0, ks0, vs0 = cache.k.clone(), cache.v.clone(), cache.kscale.clone(), cache.vscale.clone()
    args = (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], wq, wk, 1e-6 if norm else 0.0, tq.tq_rope_frequencies(inv) if rot else None,
            style, pos, i32(start), i32(lens), table, cache, out)
    tq.tq_cache8_append(*args)
    n, tab = start[-1], table.cpu().numpy()
    y = turned(x[:n, :Hq + Hkv].reshape(n, Hq + Hkv, d), None, 0, [], style, pos[:n])
    if norm:
        y = torch.cat([turned(x[:n, :Hq], wq, 1e-6, [], style, pos[:n]), turned(x[:n, Hq:Hq + Hkv], wk, 1e-6, [], style, pos[:n])], 1)
    y = turned(y, None, 0, inv, style, pos[:n])
    # half a step of the type, and fp32: a few roundings of the pair's larger element, an angle off by 2^-24 of a half turn
    tol = torch.finfo(t).eps / 2 * y[:, :Hq].abs() + 2e-6 * y[:, :Hq].abs().amax(-1, keepdim=True) if n else y[:, :Hq]
    if t is torch.float16:
        tol = tol + 2.0 ** -25
    assert ((out[:n].double() - y[:, :Hq]).abs() <= tol).all()
    assert (out[n:] == 7).all()
    check_append((k0, ks0), (cache.k, cache.kscale), y[:, Hq:], rot == 0 and not norm, start, lens, tab, block)
    check_append((v0, vs0), (cache.v, cache.vscale), x[:n, Hq + Hkv:].double(), True, start, lens, tab, block)
    assert cache.status.item() == 0
    # once more: nothing changes
    k1, v1, ks1, vs1 = cache.k.clone(), cache.v.clone(), cache.kscale.clone(), cache.vscale.clone()
    tq.tq_cache8_append(*args)
    for a, b in ((k1, cache.k), (v1, cache.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(ks1, cache.kscale) and torch.equal(vs1, cache.vscale)


def test_append_in_place_and_without_queries():
    g = gen(3)
    table, total = pages_for([40, 9], 16, g)
    a, b, c = (tq.Cache8(total, 2, 16) for _ in range(3))
    x = torch.randn(13, 8, 128, device="cuda", generator=g).bfloat16()
    start, lens, pos = i32([0, 10, 13]), i32([30, 6]), torch.arange(13, device="cuda").int()
    freq = tq.tq_rope_frequencies(1e4 ** (-np.arange(0, 128, 2) / 128))
    out = torch.empty(13, 4, 128, device="cuda", dtype=torch.bfloat16)
    rest = (None, None, 1e-6, freq, 0, pos, start, lens, table)
    tq.tq_cache8_append(x[:, :4], x[:, 4:6], x[:, 6:], *rest, a, out)
    tq.tq_cache8_append(None, x[:, 4:6], x[:, 6:], *rest, b, None)
    y = x.clone()
    tq.tq_cache8_append(y[:, :4], y[:, 4:6], y[:, 6:], *rest, c, y[:, :4])
    assert torch.equal(y[:, :4], out) and torch.equal(y[:, 4:], x[:, 4:])
    for o in (b, c):
        assert torch.equal(a.k.view(torch.uint8), o.k.view(torch.uint8)) and torch.equal(a.v.view(torch.uint8), o.v.view(torch.uint8))
        assert torch.equal(a.kscale, o.kscale) and torch.equal(a.vscale, o.vscale)


def append_plain(cache, x, start, lens, table):
    """x [rows, Hkv, d] as keys, turned by nothing, and as values."""
    tq.tq_cache8_append(None, x, x, None, None, 0.0, None, 0, torch.zeros(x.shape[0], device="cuda").int(), i32(start), i32(lens), table, cache, None)


def test_append_extremes():
    """Zeros, magnitudes at both ends of the scales, numbers on a border of two codes and of two scales."""
    block, table = 16, i32([[0, 1, 2, 3, 4, 5]])
    cache = tq.Cache8(6, 1, block, 64)
    x = torch.zeros(96, 1, 64, device="cuda")
    x[16:32] = 1e-30  # below the least scale's codes: 2^-60 · 2^-10 = 8.5e-22
    x[32:48] = 3e38
    x[48:64, :, 0] = 448.0  # scale 1
    x[48:64, :, 1] = 17.0   # halfway between 16 and 18: to the even code, 16
    x[64:80, :, 0] = float(np.nextafter(np.float32(448), np.float32(500)))  # scale 2
    x[80:, :, 0] = -3.0
    append_plain(cache, x, [0, 96], [0], table)
    s, k = cache.kscale[:, 0].tolist(), cache.k[:, 0].float()
    assert s[0] == s[1] == LO and (k[0] == 0).all() and (k[1] == 0).all()
    assert s[2] == HI and (k[2] == 448).all()
    assert s[3] == 1 and (k[3, :, 0] == 448).all() and (k[3, :, 1] == 16).all()
    assert s[4] == 2 and (k[4, :, 0] == 224).all()
    assert s[5] == 2.0 ** -7 and (k[5, :, 0] == -384).all()
    assert torch.equal(cache.k.float(), cache.v.float()) and torch.equal(cache.kscale, cache.vscale)


def test_append_numbers_that_are_none():
    """A NaN or an infinity marks its block, keeps codes numbers, and goes with the block's next beginning."""
    table = i32([[0, 1]])
    for bad in (math.nan, math.inf, -math.inf):
        cache = tq.Cache8(2, 2, 16, 64)
        x = torch.ones(20, 2, 64, device="cuda")
        x[3, 1, 5] = bad
        append_plain(cache, x, [0, 20], [0], table)
        assert cache.kscale[0, 1].isnan() and cache.vscale[0, 1].isnan()
        assert cache.kscale.isnan().sum() == 1 and cache.vscale.isnan().sum() == 1
        assert not cache.k.float().isnan().any() and not cache.v.float().isnan().any()
        append_plain(cache, x[:2], [0, 2], [4], table)  # inside the block: it stays marked
        assert cache.kscale[0, 1].isnan()
        append_plain(cache, x[:2], [0, 2], [0], table)  # the block begun anew
        assert cache.kscale[0, 1] == 2.0 ** -8 and cache.vscale[0, 1] == 2.0 ** -8


def test_append_outside_the_cache_and_the_table():
    """Bad pages and positions past the table are left out and reported; the others are stored."""
    cache = tq.Cache8(3, 1, 16, 64)
    x = torch.ones(64, 1, 64, device="cuda")
    append_plain(cache, x, [0, 64], [0], i32([[1, -1, 3, 2]]))
    assert cache.status.item() == 1 and (cache.k[1].float() != 0).all() and (cache.k[2].float() != 0).all() and (cache.k[0].float() == 0).all()
    cache = tq.Cache8(3, 1, 16, 64)
    append_plain(cache, x, [0, 64], [0], i32([[1, 2]]))
    assert cache.status.item() == 1 and (cache.k[0].float() == 0).all() and (cache.k[1:].float() != 0).all()


# ------------------------------------------------------------------ attention
def attend_ref(q, start, lens, table, cache, scale, window, sinks):
    """Rows of attention in 64 bits, and what each may be off by apart from its own rounding."""
    Hkv, block, d = cache.Hkv, cache.block, cache.d
    G, cap = q.shape[1] // Hkv, table.shape[1] * block
    out, off = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    # weights: one fp16 term (2^-11) for bf16, two (2^-22) otherwise
    term = 2.0 ** -11 if q.dtype is torch.bfloat16 else 2.0 ** -22
    tab = table.cpu().numpy()
    for b in range(len(lens)):
        lo, hi = start[b], start[b + 1]
        n = min(lens[b] + hi - lo, cap)
        if hi == lo:
            continue
        t = torch.arange(n, device="cuda")
        page = table[b].long()[t // block]
        there = (page >= 0) & (page < cache.pages)
        p = lens[b] + torch.arange(hi - lo, device="cuda")
        sees = (t[None] <= p[:, None]) & there[None]
        if window:
            sees &= (t[None] > p[:, None] - window) | (t[None] < sinks)
        page = torch.where(there, page, 0)
        for h in range(Hkv):
            k = cache.k[page, h, t % block].double() * cache.kscale[page, h].double()[:, None]
            v = cache.v[page, h, t % block].double() * cache.vscale[page, h].double()[:, None]
            v = torch.where(sees.any(0)[:, None], v, 0)
            qq = q[lo:hi, h * G:(h + 1) * G].double()
            z = torch.einsum("igd,td->igt", qq, k) * scale
            z = z.masked_fill(~sees[:, None], -math.inf)
            top = z.amax(-1, keepdim=True)
            w = torch.where(sees[:, None], (z - torch.where(top.isinf(), 0, top)).exp(), 0)
            w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
            out[lo:hi, h * G:(h + 1) * G] = w @ v
            # scores: fp32 sums of 8 products of 16 and two fp16 terms of q, 2^-20 of the sum of magnitudes each, and
            # the exponent's own rounding; sums over a warp's tokens: 2^-23 for every 16 of them
            most = (torch.einsum("igd,td->igt", qq.abs(), k.abs()).masked_fill(~sees[:, None], 0).amax(-1, keepdim=True) * scale)
            spread = w @ v.abs()
            off[lo:hi, h * G:(h + 1) * G] = spread * (term + 2.0 ** -19 * (1 + most) + n / 16 * 2.0 ** -23) + n * 2.0 ** -30 * v.abs().amax()
    return out, off


def attend(q, start, lens, table, cache, scale, window=0, sinks=0, rows=None, ws=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    if ws is None:  # what a workspace holds does not matter
        n = tq.tq_cache8_attention_workspace_size(cache, len(lens), q.shape[1], q.shape[0])
        ws = torch.full((n // 4 + 4,), math.nan, device="cuda")
    tq.tq_cache8_attention(q, i32(start), i32(lens), table, cache, scale, out, ws, window=window, sinks=sinks)
    return out


def close(out, ref, off, what=""):
    half = torch.finfo(out.dtype).eps / 2
    tiny = 2.0 ** -25 if out.dtype is torch.float16 else 0
    bad = (out.double() - ref).abs() - (half * ref.abs() + off * (1 + half) + tiny)
    assert (bad <= 0).all(), (what, float(bad.max()), torch.nonzero(bad > 0)[:4].tolist())


ATTEND = [
    # lens (before the rows), rows a request, Hq, Hkv, d, block, window, sinks
    ([0], [1], 1, 1, 128, 16, 0, 0),
    ([0, 1, 15, 16, 17], [1, 1, 1, 1, 1], 8, 2, 128, 16, 0, 0),
    ([127, 128, 129, 0], [1, 2, 3, 0], 8, 2, 64, 32, 0, 0),
    ([1000], [1], 32, 8, 128, 64, 0, 0),
    ([5000, 3], [1, 1], 7, 1, 64, 48, 0, 0),
    ([700, 40, 2000], [5, 3, 2], 14, 2, 128, 16, 0, 0),      # 35 rows a KV head in tiles of 32
    ([300], [9], 16, 8, 128, 128, 0, 0),                     # 18 rows
    ([0], [200], 4, 2, 128, 16, 0, 0),                       # a prompt from nothing
    ([511, 100], [65, 1], 8, 1, 64, 64, 0, 0),               # a prompt's piece beside a token
    ([900] * 33, [1] * 33, 4, 4, 64, 16, 0, 0),
    ([64] * 300, [1] * 300, 2, 1, 64, 16, 0, 0),             # more requests than threads
    ([1000, 2000, 10], [1, 1, 1], 8, 2, 128, 16, 100, 4),
    ([1000, 129, 300], [3, 20, 1], 8, 2, 64, 48, 1, 0),      # a window of the token itself
    ([3000], [40], 4, 2, 128, 64, 128, 130),                 # first tokens of two units
    ([0], [300], 4, 2, 128, 32, 37, 3),
    ([500], [1], 16, 2, 128, 16, 400, 100),                  # window and first tokens meet
    ([100], [1], 8, 2, 128, 16, 1000, 2),                    # a window longer than the cache
    ([4095], [1], 12, 1, 128, 1024, 0, 0),
    ([37, 90], [130, 64], 24, 2, 128, 16, 0, 0),             # 12 heads a KV head, many tiles
    ([2000, 1000, 1500], [15, 11, 8], 16, 4, 128, 48, 0, 0), # 60 rows at most
    ([300, 0, 127], [16, 128, 1], 2, 2, 64, 16, 0, 0),
    ([1000], [64], 8, 4, 64, 128, 0, 0),                     # 128 rows
    ([5000, 20], [33, 40], 6, 2, 128, 64, 700, 5),
    ([3000, 10, 0], [1, 1, 600], 8, 2, 128, 16, 0, 0),       # a prompt beside single tokens
    ([0], [1500], 4, 1, 128, 32, 256, 4),
    ([129], [777], 3, 1, 64, 48, 100, 0),
    ([0, 0], [256, 257], 1, 1, 128, 64, 0, 0),
    ([20000], [300], 2, 1, 128, 64, 0, 0),
    ([4000], [200], 2, 2, 64, 16, 4100, 200),
]


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("lens,new,Hq,Hkv,d,block,window,sinks", ATTEND)
def test_attention(lens, new, Hq, Hkv, d, block, window, sinks, ty):
    g, t = gen(sum(lens) + Hq), TYPES[ty]
    table, total = pages_for([a + b for a, b in zip(lens, new)], block, g)
    cache = tq.Cache8(total, Hkv, block, d)
    filled(cache, g)
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    rows = start[-1] + 2
    q = (torch.randn(rows, Hq + 3, d, device="cuda", generator=g) * 2).to(t)[:, 1:Hq + 1]  # a slice of a wider tensor
    # places that hold no token: NaN codes
    used = torch.zeros(total, block, dtype=torch.bool, device="cuda")
    for b, n in enumerate(a + c for a, c in zip(lens, new)):
        at = torch.arange(n, device="cuda")
        used[table[b].long()[at // block], at % block] = True
    for codes in (cache.k, cache.v):
        codes.view(torch.uint8).masked_fill_(~used[:, None, :, None], 0x7F)
    out = attend(q, start, lens, table, cache, 1 / math.sqrt(d), window, sinks)
    ref, off = attend_ref(q, start, lens, table, cache, 1 / math.sqrt(d), window, sinks)
    close(out[:start[-1]], ref[:start[-1]], off[:start[-1]])
    assert (out[start[-1]:] == 7).all() and cache.status.item() == 0
    assert torch.equal(out, attend(q, start, lens, table, cache, 1 / math.sqrt(d), window, sinks))  # the same every time


def test_attention_scales_far_apart():
    """Blocks whose V scales lie 2^60 apart, scores that differ by hundreds, rows of q of any magnitude."""
    g = gen(5)
    table, total = pages_for([200], 16, g)
    cache = tq.Cache8(total, 1, 16, 128)
    filled(cache, g)
    cache.vscale.copy_(torch.exp2(torch.linspace(-30, 30, total, device="cuda").round())[:, None])
    q = torch.randn(4, 2, 128, device="cuda", generator=g)
    q *= torch.tensor([1e-30, 1e-3, 30.0, 0.0], device="cuda")[:, None, None]
    for t in (torch.float32, torch.bfloat16):
        qq = q.to(t)
        out = attend(qq, [0, 4], [196], table, cache, 0.1)
        ref, off = attend_ref(qq, [0, 4], [196], table, cache, 0.1, 0, 0)
        close(out, ref, off)


def test_attention_rows_that_are_no_numbers_stay_alone():
    g = gen(6)
    table, total = pages_for([300, 300], 16, g)
    cache = tq.Cache8(total, 2, 16, 128)
    filled(cache, g)
    q = torch.randn(6, 8, 128, device="cuda", generator=g).half()
    args = ([0, 3, 6], [297, 290], table, cache, 0.1)
    good = attend(q, *args)
    bad = q.clone()
    bad[1, 2, 7], bad[4, 5] = math.nan, math.inf
    out = attend(bad, *args)
    assert out[1, 2].isnan().all() and out[4, 5].isnan().all()
    mask = torch.ones(6, 8, dtype=torch.bool, device="cuda")
    mask[1, 2] = mask[4, 5] = False
    assert torch.equal(out[mask], good[mask])
    # a marked block: rows that see one of its tokens, and no others
    cache.vscale[table[0, 1], 0] = math.nan
    out = attend(q, *args)
    assert out[:3, :4].isnan().all() and torch.equal(out[:3, 4:], good[:3, 4:]) and torch.equal(out[3:], good[3:])
    out, ref = attend(q, *args, window=260), attend_ref(q, *args, 260, 0)
    assert torch.isfinite(out).all()  # tokens up to 297 - 260 = 37 are hidden
    close(out, *ref)


def test_attention_pages_outside_the_cache():
    g = gen(7)
    table, total = pages_for([250, 90], 16, g)
    cache = tq.Cache8(total, 2, 16, 128)
    filled(cache, g)
    table[0, 3], table[0, 10], table[1, 0] = -5, total, 1 << 30
    q = torch.randn(5, 4, 128, device="cuda", generator=g).bfloat16()
    args = ([0, 2, 5], [248, 80], table, cache, 0.1)
    out, ref = attend(q, *args), attend_ref(q, *args, 0, 0)
    close(out, *ref)
    assert cache.status.item() == 1
    cache.status.zero_()
    # behind a window they are not looked up; a request of nothing but bad pages is zero
    out, ref = attend(q, *args, window=60), attend_ref(q, *args, 60, 0)
    close(out, *ref)
    assert cache.status.item() == 0
    table[:] = -1
    assert (attend(q, *args) == 0).all() and cache.status.item() == 1


def test_attention_past_the_table():
    """Rows past the table's capacity see what it holds; with a window, nothing at all."""
    g = gen(8)
    table, total = pages_for([64], 16, g)
    cache = tq.Cache8(total, 1, 16, 64)
    filled(cache, g)
    q = torch.randn(20, 2, 64, device="cuda", generator=g)
    out, ref = attend(q, [0, 20], [60], table, cache, 0.1), attend_ref(q, [0, 20], [60], table, cache, 0.1, 0, 0)
    close(out, *ref)
    out, ref = attend(q, [0, 20], [60], table, cache, 0.1, 4, 0), attend_ref(q, [0, 20], [60], table, cache, 0.1, 4, 0)
    close(out, *ref)
    assert (out[8:] == 0).all() and (out[:7] != 0).all()
    # lengths and offsets that make no sense touch nothing outside
    attend(q, [0, 20], [2 ** 31 - 5], table, cache, 0.1)
    attend(q, [-3, 99], [-7], table, cache, 0.1, 3, 3)
    attend(q, [0, 15, 5], [10, 10], table[:1].repeat(2, 1), cache, 0.1)


def test_offsets_past_32_bits():
    """A cache of more than 2^31 bytes a side: its last pages."""
    Hkv, block, d = 8, 64, 128
    total = (1 << 31) // (Hkv * block * d) + 8
    cache = tq.Cache8(total, Hkv, block, d)
    table = torch.arange(total - 6, total, device="cuda").int()[None].contiguous()
    g = gen(9)
    x = torch.randn(300, 4 * Hkv, d, device="cuda", generator=g).half()
    pos, out = torch.arange(300, device="cuda").int(), torch.empty(300, 2 * Hkv, d, device="cuda", dtype=torch.half)
    tq.tq_cache8_append(x[:, :16], x[:, 16:24], x[:, 24:], None, None, 0.0, None, 0, pos, i32([0, 300]), i32([0]), table, cache, out)
    assert torch.equal(out, x[:, :16])
    small = tq.Cache8(6, Hkv, block, d)
    tab = torch.arange(6, device="cuda").int()[None].contiguous()
    tq.tq_cache8_append(x[:, :16], x[:, 16:24], x[:, 24:], None, None, 0.0, None, 0, pos, i32([0, 300]), i32([0]), tab, small, out)
    assert torch.equal(cache.k[-6:].view(torch.uint8), small.k.view(torch.uint8)) and torch.equal(cache.vscale[-6:], small.vscale)
    for new in (1, 12, 100):
        a, b = (attend(x[:new, :16], [0, new], [299 - new], t, c, 0.1) for t, c in ((table, cache), (tab, small)))
        assert torch.equal(a, b)


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("B,new", [(152, 1), (76, 20), (38, 300)])
def test_long_sums_are_not_cut(B, new, ty):
    """Values of one sign over 70000 tokens, which every request shares, so that one CTA adds all of a tile up: how much
    of the result is missing."""
    n, Hq, Hkv, d, block, t = 70000, 4, 2, 128, 16, TYPES[ty]
    g = gen(18)
    width = (n + block - 1) // block
    cache = tq.Cache8(width, Hkv, block, d)
    filled(cache, g, 0)
    cache.v.copy_(cache.v.float().abs().to(F8))
    table = torch.randperm(width, generator=g, device="cuda").int()[None].repeat(B, 1)
    q = (0.25 * torch.randn(new, Hq, d, device="cuda", generator=g)).to(t)
    start, scale = [new * b for b in range(B + 1)], d ** -0.5
    out = attend(q.repeat(B, 1, 1), start, [n - new] * B, table, cache, scale).view(B, new, Hq, d)
    page, at = table[0].long()[torch.arange(n, device="cuda") // block], torch.arange(n, device="cuda") % block
    sees = torch.arange(n, device="cuda")[None] <= n - new + torch.arange(new, device="cuda")[:, None]
    dot, own, most = torch.zeros(B, device="cuda", dtype=torch.float64), 0, 0
    for h in range(Hkv):
        k, v = (c[page, h, at].double() * x[page, h].double()[:, None] for c, x in ((cache.k, cache.kscale), (cache.v, cache.vscale)))
        for j in range(h * 2, h * 2 + 2):
            z = q[:, j].double() @ k.T * scale
            ref = z.masked_fill(~sees, -math.inf).softmax(-1) @ v
            dot += ((out[:, :, j].double() - ref) * ref).sum((1, 2))
            own += ref.square().sum()
            most = max(most, (q[:, j].double().abs() @ k.abs().T).amax().item() * scale)
    # an addition cuts 2^-23 of the sum at most, which on average is half of the last; additions: of 16 tokens each, all
    # of a warp's (fp16 and bf16 rows that are few), those between two rests in fp32, or (fp32) none; scores: 16 additions
    terms = 1 if t is torch.bfloat16 else 2
    units = (n + 127) // 128
    steps = 2 if t is torch.float32 else 2 * units * terms if new == 1 else 4 * terms * min(units * (2 if new > 64 else 1), 256 if t is torch.float16 else 1024)
    # and the results' own rounding, half a step of either sign for each of as many results, four times its deviation
    count = new * Hq * d
    bound = steps / 2 * 2.0 ** -23 + 2.0 ** -19 * (1 + most) + 4 * torch.finfo(t).eps / 2 / math.sqrt(count)
    assert ((dot / own).abs() <= bound).all(), (float((dot / own).abs().max()), bound)


# ------------------------------------------------------------------ streams and graphs, and a server's steps
def test_captured_steps_serve_later_lengths():
    g = gen(10)
    B, Hq, Hkv, d, block, width = 3, 8, 2, 128, 16, 20
    order = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)
    eager, graphed = (tq.Cache8(B * width, Hkv, block, d) for _ in range(2))
    lens, start, pos = i32([0] * B), i32([0, 2, 4, 6]), i32([0] * 6)
    x = torch.empty(6, Hq + 2 * Hkv, d, device="cuda", dtype=torch.bfloat16)
    q, out = torch.empty(6, Hq, d, device="cuda", dtype=torch.bfloat16), torch.empty(6, Hq, d, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(tq.tq_cache8_attention_workspace_size(eager, B, Hq, 6) // 4 + 4, device="cuda")
    freq = tq.tq_rope_frequencies(1e4 ** (-np.arange(0, d, 2) / d))

    def step(cache):
        tq.tq_cache8_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], None, None, 1e-6, freq, 0, pos, start, lens, order, cache, q)
        tq.tq_cache8_attention(q, start, lens, order, cache, 0.1, out, ws, window=64, sinks=4)

    x.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(graphed)
        step(eager)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    at = [0, 37, 150]
    for k in range(12):
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        lens.copy_(i32(at))
        pos.copy_(i32([a + i for a in at for i in range(2)]))
        graph.replay()
        a = out.clone()
        step(eager)
        # request 1's and 2's first tokens were never written in either cache; they hold zeros with scale 0
        assert torch.equal(a, out)
        assert torch.equal(graphed.k.view(torch.uint8), eager.k.view(torch.uint8)) and torch.equal(graphed.kscale, eager.kscale)
        at = [v + (k % 3) for v in at]


# lens, rows a request, Hq, Hkv, d, block: calls of both kernels, with tiles that several CTAs have parts of
MIXED = [
    ([20000], [300], 2, 1, 128, 64),
    ([9000, 0, 400], [1, 700, 30], 8, 2, 64, 32),
    ([37, 90], [130, 64], 24, 2, 128, 16),
    ([6000, 100], [3, 1], 8, 2, 128, 16),
]


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("lens,new,Hq,Hkv,d,block", MIXED)
def test_many_runs_agree(lens, new, Hq, Hkv, d, block, ty):
    """The same call again and again, alone and beside itself on another stream: the same bits."""
    g = gen(13)
    table, total = pages_for([a + b for a, b in zip(lens, new)], block, g)
    cache = tq.Cache8(total, Hkv, block, d)
    filled(cache, g)
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = (2 * torch.randn(start[-1], Hq, d, device="cuda", generator=g)).to(TYPES[ty])
    n = tq.tq_cache8_attention_workspace_size(cache, len(lens), Hq, start[-1])
    first, at, size = i32(start), i32(lens), n // 4 + 4
    jobs = [(torch.cuda.Stream(), torch.empty(size, device="cuda"), [torch.empty_like(q) for _ in range(12)]) for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(12):
        for s, ws, outs in jobs:
            tq.tq_cache8_attention(q, first, at, table, cache, 0.1, outs[i], ws, stream=s)
    torch.cuda.synchronize()
    want = jobs[0][2][0]
    assert all(torch.equal(want, o) for _, _, outs in jobs for o in outs)
    ref, off = attend_ref(q, start, lens, table, cache, 0.1, 0, 0)
    close(want, ref, off)


@pytest.mark.parametrize("d,window,sinks", [(128, 0, 0), (64, 0, 0), (128, 200, 7)])
def test_captured_prompts_serve_later_lengths(d, window, sinks):
    """One captured call of up to 700 rows: prompts, pieces of them, single tokens and nothing at all."""
    g = gen(14)
    B, Hq, Hkv, block, width, rows = 3, 4, 2, 32, 80, 700
    cache = tq.Cache8(B * width, Hkv, block, d)
    filled(cache, g)
    table = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)
    q, out = (torch.zeros(rows, Hq, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ws = torch.empty(tq.tq_cache8_attention_workspace_size(cache, B, Hq, rows) // 4 + 4, device="cuda")
    start, lens = i32([0] * (B + 1)), i32([0] * B)

    def step():
        tq.tq_cache8_attention(q, start, lens, table, cache, 0.1, out, ws, window=window, sinks=sinks)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new, at in (([700, 0, 0], [0, 5, 5]), ([1, 1, 1], [2000, 3, 0]), ([0, 0, 0], [1, 2, 3]), ([128, 300, 129], [1000, 0, 2300]), ([0, 699, 1], [9, 1800, 40])):
        first = np.concatenate([[0], np.cumsum(new)]).tolist()
        q.copy_(torch.randn(q.shape, device="cuda", generator=g))
        start.copy_(i32(first))
        lens.copy_(i32(at))
        out.fill_(7.0)
        graph.replay()
        got = out.clone()
        out.fill_(7.0)
        step()
        assert torch.equal(got, out) and (got[first[-1]:] == 7).all()
        ref, off = attend_ref(q, first, at, table, cache, 0.1, window, sinks)
        close(got[:first[-1]], ref[:first[-1]], off[:first[-1]], new)
    assert cache.status.item() == 0


@pytest.mark.parametrize("ty", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new,Hq,Hkv,d,block,window,sinks", [
    ([2000, 700], [1, 3], 8, 2, 128, 16, 100, 4), ([3000, 50], [150, 20], 4, 2, 128, 16, 300, 20), ([5000], [400], 4, 1, 64, 48, 129, 0)])
def test_pages_behind_the_window_may_be_gone(lens, new, Hq, Hkv, d, block, window, sinks, ty):
    g = gen(15)
    table, total = pages_for([a + b for a, b in zip(lens, new)], block, g)
    cache = tq.Cache8(total, Hkv, block, d)
    filled(cache, g)
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = torch.randn(start[-1], Hq, d, device="cuda", generator=g).to(TYPES[ty])
    want = attend(q, start, lens, table, cache, 0.1, window, sinks)
    for b, n in enumerate(lens):  # first rows see tokens from n - window + 1 on, and the first ones
        gone = table[b, (sinks + block - 1) // block:max((n - window + 1) // block, 0)]
        for codes, scale in ((cache.k, cache.kscale), (cache.v, cache.vscale)):
            codes.view(torch.uint8)[gone.long()] = 0x7F
            scale[gone.long()] = math.nan
        gone.fill_(-1)
    assert torch.equal(want, attend(q, start, lens, table, cache, 0.1, window, sinks)) and cache.status.item() == 0


def test_requests_that_share_their_first_blocks():
    """A prefix held once: full blocks in several tables, twice in one of them, and appends behind it."""
    g = gen(16)
    B, Hq, Hkv, d, block = 4, 8, 2, 128, 16
    cache = tq.Cache8(60, Hkv, block, d)
    filled(cache, g)
    order = torch.randperm(60, generator=g, device="cuda").int()
    table = torch.stack([torch.cat([order[:10], order[10 + 12 * b:22 + 12 * b]]) for b in range(B)]).contiguous()
    table[3, 4] = table[3, 3]
    lens, new = [160, 160, 165, 170], [150, 1, 0, 9]
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    x = torch.randn(160, Hq + 2 * Hkv, d, device="cuda", generator=g).half()
    q, pos, k0 = torch.empty(160, Hq, d, device="cuda", dtype=torch.half), torch.arange(160, device="cuda").int(), cache.k[order[:10].long()].view(torch.uint8).clone()
    tq.tq_cache8_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], None, None, 0.0, None, 0, pos, i32(start), i32(lens), table, cache, q)
    assert torch.equal(q, x[:, :Hq]) and torch.equal(k0, cache.k[order[:10].long()].view(torch.uint8))
    out, ref = attend(q, start, lens, table, cache, 0.1), attend_ref(q, start, lens, table, cache, 0.1, 0, 0)
    close(out, *ref)


@pytest.mark.parametrize("Hq,Hkv,d,most", [(8, 2, 128, 1), (4, 1, 64, 40), (6, 3, 128, 130)])
def test_hundreds_of_ragged_requests(Hq, Hkv, d, most):
    g, r = gen(17), np.random.default_rng(17)
    B = 400
    new = r.integers(0, most + 1, B).tolist()
    lens = (r.integers(0, 300, B) * r.integers(0, 2, B)).tolist()
    table, total = pages_for([a + b for a, b in zip(lens, new)], 16, g)
    cache = tq.Cache8(total, Hkv, 16, d)
    filled(cache, g)
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = torch.randn(start[-1] + 5, Hq, d, device="cuda", generator=g).bfloat16()
    out = attend(q, start, lens, table, cache, 0.1)
    ref, off = attend_ref(q, start, lens, table, cache, 0.1, 0, 0)
    close(out[:start[-1]], ref[:start[-1]], off[:start[-1]])
    assert (out[start[-1]:] == 7).all() and cache.status.item() == 0


@pytest.mark.parametrize("Hq", [2, 40])
def test_tens_of_thousands_of_requests(Hq):
    """More requests than a CTA keeps offsets of: a token each, appended and attended to."""
    B, d, block, g = 40000, 64, 16, gen(19)
    cache = tq.Cache8(B, 1, block, d)
    filled(cache, g)
    table = torch.randperm(B, generator=g, device="cuda").int()[:, None].contiguous()
    lens = torch.randint(0, block, (B,), generator=g, device="cuda").int()
    start, pos, page = torch.arange(B + 1, device="cuda").int(), torch.zeros(B, device="cuda").int(), table[:, 0].long()
    x = torch.randn(B, Hq + 2, d, device="cuda", generator=g).half()
    q, old = torch.empty(B, Hq, d, device="cuda", dtype=torch.half), cache.vscale.clone()
    tq.tq_cache8_append(x[:, :Hq], x[:, Hq:Hq + 1], x[:, Hq + 1:], None, None, 0.0, None, 0, pos, start, lens, table, cache, q)
    assert torch.equal(q, x[:, :Hq])
    v = x[:, Hq + 1].double()
    s = torch.maximum(least_scale(v.abs().amax(1)), torch.where(lens > 0, old[page, 0].double(), 0))
    assert torch.equal(cache.vscale[page, 0].double(), s)
    assert torch.equal(cache.v[page, 0, lens.long()].float(), (v / s[:, None]).float().to(F8).float())
    ws = torch.empty(tq.tq_cache8_attention_workspace_size(cache, B, Hq, B) // 4 + 4, device="cuda")
    out = torch.empty_like(q)
    tq.tq_cache8_attention(q, start, lens, table, cache, 0.1, out, ws)
    k, v = (c[page, 0].double() * f[page].double()[..., None] for c, f in ((cache.k, cache.kscale), (cache.v, cache.vscale)))
    sees = (torch.arange(block, device="cuda")[None] <= lens[:, None])[:, None]
    z = (torch.einsum("bhd,btd->bht", q.double(), k) * 0.1).masked_fill(~sees, -math.inf)
    w = z.softmax(-1)
    most = (torch.einsum("bhd,btd->bht", q.double().abs(), k.abs()) * 0.1).masked_fill(~sees, 0).amax(-1, keepdim=True)
    close(out, w @ v, w @ v.abs() * (2.0 ** -22 + 2.0 ** -19 * (1 + most) + 2.0 ** -23) + block * 2.0 ** -30 * v.abs().amax())
    assert cache.status.item() == 0


def test_two_streams_with_workspaces_of_their_own():
    g = gen(11)
    jobs = []
    for k in range(2):
        table, total = pages_for([3000 + 700 * k, 500], 16, g)
        cache = tq.Cache8(total, 2, 16, 128)
        filled(cache, g)
        q = torch.randn(2, 8, 128, device="cuda", generator=g).half()
        ws = torch.empty(tq.tq_cache8_attention_workspace_size(cache, 2, 8, 2) // 4 + 4, device="cuda")
        lens, start = i32([2999 + 700 * k, 499]), i32([0, 1, 2])
        want = torch.empty_like(q)
        tq.tq_cache8_attention(q, start, lens, table, cache, 0.1, want, ws)
        jobs.append((torch.cuda.Stream(), q, start, lens, table, cache, ws, want, torch.empty_like(q)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, start, lens, table, cache, ws, want, out in jobs:
            tq.tq_cache8_attention(q, start, lens, table, cache, 0.1, out, ws, stream=s)
    torch.cuda.synchronize()
    for *_, want, out in jobs:
        assert torch.equal(want, out)


@pytest.mark.parametrize("ty", list(TYPES))
def test_server_steps(ty):
    """Prompts in pieces, then drafted chains of which some tokens are rejected: tables, append and attention together,
    against attention over the values as the cache holds them."""
    g, t = gen(12), TYPES[ty]
    B, Hq, Hkv, d, block, width = 3, 6, 2, 64, 16, 12
    pages = B * width
    cache = tq.Cache8(pages, Hkv, block, d)
    ring, state = torch.arange(pages, device="cuda").int(), torch.tensor([0, pages], device="cuda")
    table, held = i32([[-1] * width] * B), i32([0] * B)
    inv = 1e4 ** (-np.arange(0, d, 2) / d)
    freq = tq.tq_rope_frequencies(inv)
    keys = torch.zeros(B, width * block, Hkv, d, dtype=torch.float64, device="cuda")
    lens = [0] * B
    for step, new in enumerate([[40, 0, 100], [30, 17, 1], [4, 4, 4], [4, 4, 4], [1, 5, 0], [4, 4, 4]]):
        rows = sum(new)
        start, slots, pos = i32([0] * (B + 1)), torch.empty(rows, dtype=torch.int64, device="cuda"), i32([0] * rows)
        held2, state2 = torch.empty_like(held), torch.empty_like(state)
        tq.tq_block_tables(i32(lens), i32(new), held, ring, state, table, block, held2, state2, start, slots, pos)
        held, state = held2, state2
        x = torch.randn(rows, Hq + 2 * Hkv, d, device="cuda", generator=g).to(t)
        q, out = (torch.empty(rows, Hq, d, dtype=t, device="cuda") for _ in range(2))
        tq.tq_cache8_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], None, None, 1e-6, freq, 0, pos, start, i32(lens), table, cache, q)
        ws = torch.empty(tq.tq_cache8_attention_workspace_size(cache, B, Hq, rows) // 4 + 4, device="cuda")
        tq.tq_cache8_attention(q, start, i32(lens), table, cache, d ** -0.5, out, ws)
        first = start.tolist()
        ref, off = attend_ref(q, first, lens, table, cache, d ** -0.5, 0, 0)
        close(out, ref, off, step)
        # keys against what went in, every step until now: within a code's half step of the block's largest
        y = turned(x[:, Hq:Hq + Hkv], None, 1e-6, inv, 0, pos)
        for b in range(B):
            keys[b, lens[b]:lens[b] + new[b]] = y[first[b]:first[b + 1]]
            n = lens[b] + new[b]
            at = torch.arange(n, device="cuda")
            page = table[b].long()[at // block]
            held_keys = cache.k[page, :, at % block].double() * cache.kscale[page].double()[..., None]
            assert ((held_keys - keys[b, :n]).abs() <= keys[b, :n].abs() * 2.0 ** -4 * 1.1 + cache.kscale[page].double()[..., None] * 2.0 ** -9).all()
        lens = [a + (n if step < 2 else min(n, 2)) for a, n in zip(lens, new)]  # two drafted tokens stay
    assert cache.status.item() == 0


def test_other_device_stream_and_shape_refused():
    cache = tq.Cache8(2, 2, 16, 64)
    q, lens, start, table = torch.zeros(1, 2, 64, device="cuda"), i32([0]), i32([0, 1]), i32([[0]])
    ws = torch.zeros(tq.tq_cache8_attention_workspace_size(cache, 1, 2, 1) // 4 + 4, device="cuda")
    good = dict(q=q, row_start=start, lens=lens, table=table, cache=cache, scale=1.0, out=torch.empty_like(q), ws=ws)
    tq.tq_cache8_attention(**good)
    for change in (dict(q=q.cpu()), dict(lens=lens.cpu()), dict(table=table.long()), dict(table=table[0]), dict(out=q.half()), dict(q=q[..., :32]), dict(start=start[:1])):
        change = {"row_start" if k == "start" else k: v for k, v in change.items()}
        with pytest.raises(ValueError):
            tq.tq_cache8_attention(**{**good, **change})
    for change in (dict(scale=0.0), dict(window=-1), dict(sinks=-1), dict(ws=ws[:1])):
        with pytest.raises(tq.TqError):
            tq.tq_cache8_attention(**{**good, **change})
    with pytest.raises(ValueError):
        append_plain(cache, torch.zeros(1, 1, 64, device="cuda"), [0, 1], [0], table)
    with pytest.raises(ValueError):
        append_plain(cache, torch.zeros(1, 2, 128, device="cuda"), [0, 1], [0], table)
    n = ctypes.c_size_t()
    assert tq.lib().tq_cache8_attention_workspace_size(ctypes.byref(cache.desc), 1, 3, 1, ctypes.byref(n)) == tq.TQ_ERR_INVALID_ARG


def test_queries_and_their_output_go_together():
    cache, x = tq.Cache8(2, 2, 16, 64), torch.zeros(1, 2, 64, device="cuda")
    rest = (x, x, None, None, 0.0, None, 0, i32([0]), i32([0, 1]), i32([0]), i32([[0]]), cache)
    for q, out in ((x, None), (None, x), (x, x.half()), (x, x[..., :32])):
        with pytest.raises(ValueError):
            tq.tq_cache8_append(q, *rest, out)
    tq.tq_cache8_append(x, *rest, torch.empty_like(x))
    assert cache.status.item() == 0
