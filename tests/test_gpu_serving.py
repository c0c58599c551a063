"""Serving calls on the GPU against plain 64-bit restatements: block tables, norms with rotation, paged append,
drafted-token attention, and a run of them together as a server would make it."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import kv_cache_vector_tq_gb300 as tq
from kv_cache_vector_tq_gb300 import synth
from oracle import rotation as orot

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

D = 128
CTX = {}


def ctx(b, mode=None, seed=0):
    mode = tq.TQ_MSE if mode is None else mode
    if (b, mode, seed) not in CTX:
        G = synth.gaussian_matrix(seed, D)
        S = synth.qjl_matrix(seed, D) if mode == tq.TQ_PROD else None
        CTX[b, mode, seed] = tq.Context(D, b, mode, tq.TQ_ROT_DENSE, tq.tq_rotation_haar(G), S)
    return CTX[b, mode, seed]


def rotation(seed=0):
    return torch.tensor(orot.haar_rotation(synth.gaussian_matrix(seed, D)), device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ block tables
def tables_plain(lens, new, held, ring, head, tail, table, block, rows):
    """The definition, request by request."""
    size, taken, given = len(ring), 0, 0
    table, ring2 = [list(r) for r in table], list(ring)
    held2, start, slots, pos, best = [], [0], [], [], 0
    for b in range(len(lens)):
        need = -(-(lens[b] + new[b]) // block)
        good = lens[b] >= 0 and new[b] >= 0 and 0 <= held[b] <= len(table[b]) and need <= len(table[b])
        take, give = (max(need - held[b], 0), max(held[b] - need, 0)) if good else (0, 0)
        served = good and (take == 0 or taken + take <= tail - head)
        if served:
            for j in range(take):
                table[b][held[b] + j] = ring[(head + taken + j) % size]
            for j in range(give):
                ring2[(tail + given + j) % size] = table[b][need + j]
            if take:
                best = taken + take
        taken, given = taken + take, given + give
        held2.append(need if served else held[b])
        for i in range(new[b] if served else 0):
            p = lens[b] + i
            slots.append(table[b][p // block] * block + p % block)
            pos.append(p)
        start.append(len(slots))
    slots, pos = slots[:rows], pos[:rows]
    slots += [-1] * (rows - len(slots))
    pos += [0] * (rows - len(pos))
    return table, ring2, held2, [head + best, tail + given], start, slots, pos


def run_tables(lens, new, held, ring, head, tail, table, block, rows):
    B = len(lens)
    t, r = i32(table), i32(ring)
    o = (torch.full((B,), -7, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"),
         torch.full((B + 1,), -7, dtype=torch.int32, device="cuda"),
         torch.full((rows,), -7, dtype=torch.int64, device="cuda"), torch.full((rows,), -7, dtype=torch.int32, device="cuda"))
    state = torch.tensor([head, tail], device="cuda")
    for _ in range(2):  # repeated: the same answer
        tq.tq_block_tables(i32(lens), i32(new), i32(held), r, state, t, block, *o)
    return [x.tolist() for x in (t, r, *o)]


@pytest.mark.parametrize("B,block,most,newmost,seed", [(1, 16, 1, 1, 0), (5, 16, 100, 7, 1), (513, 64, 700, 70, 2),
                                                       (700, 48, 300, 200, 3), (3, 16, 40, 5000, 4), (4096, 16, 60, 3, 5)])
def test_block_tables(B, block, most, newmost, seed):
    r = np.random.default_rng(seed)
    lens = r.integers(0, most + 1, B)
    new = r.integers(0, newmost + 1, B)
    held = -(-lens // block) + r.integers(0, 3, B)  # some hold more than they need: rejected drafts
    gone = r.random(B) < 0.2
    lens[gone], new[gone] = 0, 0
    width = int(max(held.max(), (-(-(lens + new) // block)).max(), 1))
    total = B * width + 5
    order = r.permutation(total)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    head = int(r.integers(0, 3 * total))
    ring = np.full(total, -1)
    for j, page in enumerate(order[at:]):
        ring[(head + j) % total] = page
    args = ([int(x) for x in lens], [int(x) for x in new], [int(x) for x in held], [int(x) for x in ring], head, head + total - at,
            table.tolist(), block)
    rows = int(new.sum()) + 9
    assert run_tables(*args, rows) == list(tables_plain(*args, rows))
    assert run_tables(*args, rows // 2) == list(tables_plain(*args, rows // 2))  # fewer rows listed than there are
    # a ring that runs out part of the way through
    short = list(args)
    short[5] = head + max(0, (total - at) // 7)
    assert run_tables(*short, rows) == list(tables_plain(*short, rows))


def test_block_tables_odd_requests():
    """Negative numbers, more pages than a row holds, nothing at all: kept as they were, without rows."""
    args = ([-1, 5, 3, 0, 32], [2, -3, 400, 0, 1], [1, 1, 1, 0, 2], list(range(40, 60)), 0, 20, [[k, -1, -1] for k in range(4)] + [[4, 5, -1]], 16)
    got = run_tables(*args, 8)
    assert got == list(tables_plain(*args, 8))
    assert got[2] == [1, 1, 1, 0, 3] and got[4] == [0, 0, 0, 0, 0, 1]


def test_block_tables_lengths_past_32_bits():
    """A request that would pass 2^31 - 1 tokens keeps its pages and gets no rows, however many a table row holds."""
    big, block, width = 2 ** 31 - 1, 1 << 20, 2060
    held = [2048, 1, 2048]  # pages of big tokens; of one
    table = [[b * width + j for j in range(width)] for b in range(3)]
    args = ([big - 3, 5, big], [4, 2, 0], held, list(range(9000, 9008)), 0, 8, table, block)
    got = run_tables(*args, 4)
    assert got[2] == held and got[3] == [0, 8] and got[4] == [0, 0, 2, 2]
    assert got[5] == [width * block + 5, width * block + 6, -1, -1] and got[6] == [5, 6, 0, 0]
    args[1][0] = 3  # as many as there may be
    got = run_tables(*args, 4)
    assert got[4] == [0, 3, 5, 5] and got[6] == [big - 3, big - 2, big - 1, 5]
    assert got[5][2] == 2047 * block + (big - 1) % block


def test_block_tables_captured_serves_later_steps():
    """One captured step, its new held counts and state copied back inside the graph: steps with other lengths, each
    against the definition."""
    r, B, block, width, rows = np.random.default_rng(9), 6, 16, 9, 90
    pages = B * width
    ring, state = i32(r.permutation(pages).tolist()), torch.tensor([0, pages], device="cuda")
    table, held, lens, new = i32([[-1] * width] * B), i32([0] * B), i32([0] * B), i32([0] * B)
    held2, state2, start = torch.empty_like(held), torch.empty_like(state), i32([0] * (B + 1))
    slots, pos = torch.zeros(rows, dtype=torch.int64, device="cuda"), i32([0] * rows)

    def step():
        tq.tq_block_tables(lens, new, held, ring, state, table, block, held2, state2, start, slots, pos)
        held.copy_(held2)
        state.copy_(state2)

    side = torch.cuda.Stream()  # a first call outside of the capture: nothing new, nothing held
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    now = [0] * B
    for k in range(12):
        now = [0 if r.random() < 0.15 else n for n in now]  # some have ended
        add = [int(min(r.integers(0, 30), block * width - n)) for n in now]
        lens.copy_(i32(now))
        new.copy_(i32(add))
        want = tables_plain(now, add, held.tolist(), ring.tolist(), *state.tolist(), table.tolist(), block, rows)
        graph.replay()
        assert [x.tolist() for x in (table, ring, held, state, start, slots, pos)] == list(want), k
        now = [n + a for n, a in zip(now, add)]


# ------------------------------------------------------------------ norms and rotation
def norm_rope_plain(x, w, eps, inv, style, pos):
    """In 64 bits: the rows, and the size of what each value was made from."""
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.double()
    rot = 2 * len(inv)
    a = pos.double()[:, None] * torch.tensor(inv, device="cuda")[None]
    c, s = a.cos()[:, None], a.sin()[:, None]
    z, size = y.clone(), y.abs()
    if rot:
        i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if style == tq.TQ_ROPE_HALF else (slice(0, rot, 2), slice(1, rot, 2))
        z[..., i], z[..., j] = y[..., i] * c - y[..., j] * s, y[..., j] * c + y[..., i] * s
        size[..., i] = size[..., j] = y[..., i].abs() + y[..., j].abs()
    return z, size


TYPES = [torch.float32, torch.float16, torch.bfloat16]


def check_norm_rope(got, x, w, eps, inv, style, pos):
    z, size = norm_rope_plain(x, w, eps, inv, style, pos)
    # fp32 arithmetic: a sum of d squares by d/8 lanes of 8 and a tree (16 roundings at most), rsqrt, three products,
    # the sines (2 ulp and 2^-25 half turns of angle, 10^-7): 32 half steps of what the value was made from; then one
    # rounding to the output's type (its smallest step below the normal range)
    fi = torch.finfo(got.dtype)
    bound = 32 * 2.0 ** -24 * size + fi.eps / 2 * z.abs() + fi.tiny * fi.eps
    off = (got.double() - z).abs()
    assert (off <= bound).all(), (off / bound).max()


@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (256, 128), (96, 96), (32, 16), (128, 0), (160, 64), (224, 224)])
@pytest.mark.parametrize("style", [tq.TQ_ROPE_HALF, tq.TQ_ROPE_INTERLEAVED])
@pytest.mark.parametrize("ti,to", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32), (torch.float32, torch.float16)])
def test_qk_norm_rope(d, rot, style, ti, to):
    g = gen(d + rot)
    for N, Hq, Hkv in ((1, 8, 2), (37, 7, 1), (5, 1, 0), (3, 0, 5), (700, 16, 2)):
        qkv = torch.randn(N, (Hq + 2 * Hkv) * d, device="cuda", generator=g).to(ti)
        q, k = qkv[:, :Hq * d].unflatten(1, (Hq, d)) if Hq else qkv.new_empty(N, 0, d), qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d)) if Hkv else qkv.new_empty(N, 0, d)
        wq = (1 + torch.randn(d, device="cuda", generator=g)).to(ti)
        inv = 5e5 ** (-np.arange(0, rot, 2) / max(rot, 1))
        pos = torch.randint(-5, 2_000_000, (N,), device="cuda", generator=g, dtype=torch.int32)
        qo, ko = torch.empty(N, Hq, d, device="cuda", dtype=to), torch.empty(N, Hkv, d, device="cuda", dtype=to)
        tq.tq_qk_norm_rope(q, k, wq, None, 1e-6, tq.tq_rope_frequencies(inv) if rot else None, style, pos, qo, ko)
        check_norm_rope(qo, q, wq, 1e-6, inv, style, pos)
        check_norm_rope(ko, k, None, 1e-6, inv, style, pos)


def test_qk_norm_rope_in_place_and_odd_rows():
    """The inputs as outputs (v beside them stays); zero rows, tiny and huge ones, infinities and NaN."""
    g, d = gen(3), 128
    x = torch.randn(9, 6, d, device="cuda", generator=g)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e25
    x[3] *= 1e37
    x[4, 0, 5] = math.inf
    x[5, 1, 7] = math.nan
    keep = x.clone()
    inv = 1e4 ** (-np.arange(0, d, 2) / d)
    pos = torch.arange(9, device="cuda", dtype=torch.int32)
    tq.tq_qk_norm_rope(x[:, :3], x[:, 3:5], None, None, 1e-6, tq.tq_rope_frequencies(inv), 0, pos, x[:, :3], x[:, 3:5])
    assert torch.equal(x[:, 5], keep[:, 5])
    fine = torch.ones(9, 5, dtype=torch.bool, device="cuda")
    fine[4, 0] = fine[5, 1] = False
    z, size = norm_rope_plain(keep[:, :5], None, 1e-6, inv, 0, pos)
    assert ((x[:, :5].double() - z).abs() <= 34 * 2.0 ** -24 * size + 1e-38)[fine].all()
    assert x[4, 0, 5].isnan() and x[4, 0, 5 + 64].isnan() and x[5, 1].isnan().all()  # inf · 0; a NaN norm
    assert (x[4, 0].nan_to_num() == 0).all()


# ------------------------------------------------------------------ caches
def pages_for(lens, block, g, extra=3):
    need = [-(-n // block) for n in lens]
    total = sum(need) + extra
    order = torch.randperm(total, device="cuda", generator=g, dtype=torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def slots_of(table, b, first, count, block):
    p = torch.arange(first, first + count, device="cuda")
    return table[b, p // block].long() * block + p % block


def values(codes, b, seed=0, mode=None):
    """Every vector of a code set, dequantized in 64 bits: s·Πᵀŷ/√d with the codebook's own centroids."""
    c = ctx(b, mode, seed)
    idx = torch.from_numpy(tq.tq_unpack_indices(codes).astype(np.int64)).cuda()
    cen = torch.tensor(c.codebook.centroid[:1 << b], device="cuda", dtype=torch.float64)
    return cen[idx] @ rotation(seed) * (codes.norm[:codes.n].double() / math.sqrt(D))[:, None]


@pytest.mark.parametrize("b,layout,Hkv,block,ti", [(4, tq.TQ_LAYOUT_TOKEN, 8, 16, torch.float16), (1, tq.TQ_LAYOUT_PAIR, 8, 16, torch.float16),
                                                   (2, tq.TQ_LAYOUT_PAIR, 3, 32, torch.float32), (3, tq.TQ_LAYOUT_PAIR, 1, 48, torch.float16),
                                                   (4, tq.TQ_LAYOUT_PAIR, 17, 16, torch.float32), (3, tq.TQ_LAYOUT_TOKEN, 1, 2, torch.float32)])
def test_encode_slots_is_encode(b, layout, Hkv, block, ti):
    """The paged write stores what tq_encode stores, nothing else changes, skipped tokens are skipped."""
    g = gen(b + Hkv)
    for N in (1, 2, 3, 45, 700):
        pages = N // block + 3
        x = torch.randn(N, Hkv, D, device="cuda", generator=g).to(ti)
        x[0, 0] = 0
        slots = torch.randperm(pages * block, device="cuda", generator=g)[:N]
        if N == 45:
            slots = torch.arange(7, 7 + N, device="cuda")  # a run of neighbours, as a prompt makes them
        slots[N // 2] = -1
        if N > 3:
            slots[3] = pages * block + 5  # past the cache
        plain = tq.CodeSet(ctx(b), N * Hkv)
        tq.tq_encode(ctx(b), x.view(-1, D), plain)
        want = tq.tq_unpack_indices(plain).reshape(N, Hkv, D)
        out = tq.CodeSet(ctx(b), pages * block * Hkv, layout)
        out.codes.random_(-2 ** 31, 2 ** 31, generator=g)
        out.norm.uniform_(generator=g)
        before, norms = tq.tq_unpack_indices(out), out.norm.clone()
        tq.tq_encode_slots(ctx(b), x, slots, block, out)
        after = tq.tq_unpack_indices(out)
        s = slots.cpu().numpy()
        for i in range(N):
            if 0 <= s[i] < pages * block:
                v = (s[i] // block * Hkv + np.arange(Hkv)) * block + s[i] % block
                before[v] = want[i]
                norms[torch.from_numpy(v).cuda()] = plain.norm[i * Hkv:(i + 1) * Hkv]
        assert np.array_equal(before, after) and torch.equal(norms, out.norm)


@pytest.mark.parametrize("mode,b", [(tq.TQ_MIXED, 2), (tq.TQ_PROD, 3)])
@pytest.mark.parametrize("layout", [tq.TQ_LAYOUT_TOKEN, tq.TQ_LAYOUT_PAIR])
def test_encode_slots_other_modes(mode, b, layout):
    g, N, Hkv, block = gen(b), 37, 4, 16
    c = ctx(b, mode)
    x = torch.randn(N, Hkv, D, device="cuda", generator=g)
    slots = 5 + torch.arange(N, device="cuda")
    plain, out = tq.CodeSet(c, N * Hkv), tq.CodeSet(c, 4 * block * Hkv, layout)
    tq.tq_encode(c, x.view(-1, D), plain)
    tq.tq_encode_slots(c, x, slots, block, out)
    v = torch.from_numpy(((slots[:, None].cpu().numpy() // block * Hkv + np.arange(Hkv)) * block + slots[:, None].cpu().numpy() % block).reshape(-1))
    assert np.array_equal(tq.tq_unpack_indices(out)[v.numpy()], tq.tq_unpack_indices(plain))
    assert torch.equal(out.norm[v.cuda()], plain.norm[:N * Hkv])
    if mode == tq.TQ_PROD:
        assert torch.equal(out.rnorm[v.cuda()], plain.rnorm[:N * Hkv])
        assert torch.equal(out.qjl.view(-1, 4)[v.cuda()], plain.qjl.view(-1, 4)[:N * Hkv])


# ------------------------------------------------------------------ drafted-token attention
def tree_plain(q, k_new, v_new, start, mask, kc, vc, lens, table, block, Hkv, scale, kb, vb):
    """The definition in 64 bits: output, Σ p‖v‖/Σ p of every row, and the largest scale·‖q‖‖k‖."""
    K, V = values(kc, kb), values(vc, vb)
    rows, Hq, _ = q.shape
    out, size, top = torch.zeros(rows, Hq, D, device="cuda", dtype=torch.float64), torch.zeros(rows, Hq, device="cuda", dtype=torch.float64), 0.0
    G = Hq // Hkv
    for b in range(len(lens)):
        lo, hi, n = int(start[b]), int(start[b + 1]), int(lens[b])
        if hi == lo:
            continue
        t = torch.arange(n, device="cuda")
        page = torch.full((n,), b, device="cuda") if table is None else table[b, t // block].long()
        there = (page >= 0) & (page < kc.n // (Hkv * block))
        for h in range(Hkv):
            at = ((page * Hkv + h) * block + t % block)[there]
            k, v = K[at], V[at]
            sees = torch.ones(hi - lo, len(at), dtype=torch.bool, device="cuda")
            if k_new is not None:
                j = torch.arange(hi - lo, device="cuda")
                if mask is None:
                    m = j[:, None] >= j[None]
                else:
                    m = (j // 32 < mask.shape[1])[None] & ((mask[lo:hi].long()[:, (j // 32).clamp_max(mask.shape[1] - 1)] >> (j % 32) & 1) != 0)
                sees = torch.cat([sees, m], 1)
                k, v = torch.cat([k, k_new[lo:hi, h].double()]), torch.cat([v, v_new[lo:hi, h].double()])
            qq = q[lo:hi, h * G:(h + 1) * G].double()
            z = torch.einsum("igd,td->igt", qq, k) * scale
            z = torch.where(sees[:, None], z, -math.inf)
            p = torch.softmax(z, -1) if k.shape[0] else z
            p = torch.where(sees[:, None] & sees.any(-1)[:, None, None], p, 0)
            seen = torch.where(sees.any(0)[:, None], v, 0)
            out[lo:hi, h * G:(h + 1) * G] = p @ seen
            size[lo:hi, h * G:(h + 1) * G] = p @ seen.norm(dim=-1)
            if k.shape[0]:
                top = max(top, float(qq.norm(dim=-1).max() * k[sees.any(0)].norm(dim=-1).max() * scale) if sees.any() else 0.0)
    return out, size, top


def check_tree(got, want, size, top):
    """Error of a row in the 2-norm, relative to Σ p‖v‖/Σ p.  A score z is a sum of 128 products; a rounding of unit u
    in each operand moves it by about u·‖q‖‖k‖·scale/√128, 4 of those at most are allowed for, and moves p by as much
    (twice, above and below the line).  fp32: u = 2^-24, with 2·128 terms in the two sums.  16-bit types: the cached
    values are fp16 centroids (u = 2^-11) and so are the weights p (2^-11, twice as many roundings again for the row of
    v), then the output's own rounding."""
    fi = torch.finfo(got.dtype)
    if got.dtype == torch.float32:
        rel = 8 * 2.0 ** -24 * math.sqrt(256) * max(top, 1)
    else:
        rel = 8 * 2.0 ** -11 * max(top, 1) / math.sqrt(D) + 2 * 2.0 ** -11
    off = (got.double() - want).norm(dim=-1)
    bound = rel * size + fi.eps / 2 * want.norm(dim=-1) + fi.tiny * fi.eps * math.sqrt(D)
    assert (off <= bound).all(), float((off / bound).nan_to_num().max())
    # over the whole output: the library's bound for attention, and the type's rounding
    total = float((got.double() - want).norm() / want.norm().clamp_min(1e-300))
    assert total <= (2e-5 if got.dtype == torch.float32 else 2e-3 + fi.eps / 2), total


def tree_masks(new, kind, g, words):
    rows = []
    for T in new:
        sees = torch.zeros(T, words * 32, dtype=torch.bool)
        for t in range(T):
            if t and kind == "tree":
                sees[t] = sees[int(torch.randint(0, t, (1,), generator=g))]
            if kind == "random":
                sees[t, :T] = torch.rand(T, generator=g) < 0.4
            if t < words * 32 and kind != "random":
                sees[t, t] = True
        rows.append(sees)
    m = torch.cat(rows).view(-1, words, 32).long()
    w = (m << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int().cuda().contiguous()


def make_tree(dtype, kb, vb, Hq, Hkv, block, lens, new, seed=0, paged=True, outliers=True):
    g = gen(seed)
    lens, new = list(lens), list(new)
    rows = sum(new)
    s = {"start": i32(np.concatenate([[0], np.cumsum(new)]).tolist()), "lens": i32(lens)}
    table, pages = pages_for(lens, block, g)
    if not paged:
        table, pages = torch.arange(len(lens), device="cuda", dtype=torch.int32)[:, None], len(lens)
    s["K"], s["V"] = tq.CodeSet(ctx(kb), pages * block * Hkv), tq.CodeSet(ctx(vb), pages * block * Hkv, tq.TQ_LAYOUT_PAIR)
    for b, n in enumerate(lens):
        for name, bits in (("K", kb), ("V", vb)):
            x = torch.randn(n, Hkv, D, device="cuda", generator=g)
            if outliers:
                x[..., :4] *= 10
            tq.tq_encode_slots(ctx(bits), x.half(), slots_of(table, b, 0, n, block), block, s[name])
    s["table"] = table if paged else None
    s["q"] = torch.randn(rows, Hq, D, device="cuda", generator=g).to(dtype)
    s["k"], s["v"] = torch.randn(rows, Hkv, D, device="cuda", generator=g).to(dtype), torch.randn(rows, Hkv, D, device="cuda", generator=g).to(dtype)
    return s


def run_tree(s, kb, vb, block, mask=None, scale=1 / math.sqrt(D), drafts=True, out=None, ws=None, Hkv=None):
    q, B = s["q"], s["lens"].numel()
    Hkv = s["k"].shape[1]
    out = torch.full((q.shape[0], q.shape[1], D), 7.0, dtype=q.dtype, device="cuda") if out is None else out
    if ws is None:  # its contents do not matter: NaN
        ws = torch.full((tq.tq_tree_attention_workspace_size(ctx(kb), B, q.shape[1], Hkv, q.shape[0]) // 4 + 4,), math.nan, device="cuda")
    tq.tq_tree_attention(ctx(kb), ctx(vb), q, s["k"] if drafts else None, s["v"] if drafts else None, s["start"], mask, s["K"],
                         s["V"], s["lens"], s["table"], block, scale, out, ws, Hkv=Hkv)
    return out


def tree_case(dtype, kb, vb, Hq, Hkv, block, lens, new, mask=None, paged=True, drafts=True, seed=0):
    s = make_tree(dtype, kb, vb, Hq, Hkv, block, lens, new, seed, paged)
    m = None if mask is None else tree_masks(new, mask, torch.Generator().manual_seed(seed), (max(new) + 31) // 32)
    got = run_tree(s, kb, vb, block, m, drafts=drafts)
    assert ctx(kb).poll() == tq.TQ_OK
    check_tree(got, *tree_plain(s["q"], s["k"] if drafts else None, s["v"], s["start"], m, s["K"], s["V"], s["lens"], s["table"], block,
                                Hkv, 1 / math.sqrt(D), kb, vb))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kb,vb", [(1, 1), (2, 2), (3, 3), (4, 4), (4, 2), (1, 4), (3, 1), (2, 3)])
def test_tree_bits_and_types(dtype, kb, vb):
    tree_case(dtype, kb, vb, 8, 2, 16, [300, 17, 128], [5, 9, 1], "tree")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (7, 1), (6, 2), (32, 4), (40, 1)])
def test_tree_heads(dtype, Hq, Hkv):
    tree_case(dtype, 4, 3, Hq, Hkv, 32, [70, 1000], [11, 4], "tree")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,new", [([0], [1]), ([1], [1]), ([15, 16, 17], [1, 1, 1]), ([127, 128, 129], [2, 3, 1]),
                                      ([0, 0], [3, 40]), ([5, 600, 0, 33], [0, 3, 0, 2]), ([2000], [1]), ([257], [130]),
                                      ([0, 64], [300, 1])])
def test_tree_lengths(dtype, lens, new):
    tree_case(dtype, 4, 4, 8, 2, 16, lens, new)


@pytest.mark.parametrize("block", [16, 48, 64, 128, 256])
def test_tree_pages(block):
    tree_case(torch.float16, 3, 3, 4, 1, block, [777, 130, 511], [4, 1, 7], "tree")


@pytest.mark.parametrize("dtype", TYPES)
def test_tree_contiguous_cache_and_no_drafts(dtype):
    tree_case(dtype, 4, 4, 8, 2, 1024, [900, 1024, 1], [3, 1, 2], "tree", paged=False)
    tree_case(dtype, 2, 2, 8, 2, 512, [512, 3], [1, 1], paged=False, drafts=False)
    tree_case(dtype, 2, 4, 8, 2, 16, [300, 31], [4, 1], drafts=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_tree_many_splits(dtype):
    """Groups that several CTAs share, more units than CTAs and fewer."""
    tree_case(dtype, 4, 4, 4, 1, 64, [40000], [3], "tree")
    tree_case(dtype, 2, 2, 16, 8, 64, [5000, 3000, 1], [33, 64, 2], "tree")


@pytest.mark.parametrize("dtype", TYPES)
def test_tree_many_tiles_with_two_codebooks(dtype):
    """Many tiles for every CTA, K and V of different widths (a table each), pages of one chunk; wide and narrow tiles."""
    tree_case(dtype, 4, 2, 32, 8, 16, [6000, 5000, 7011, 4090], [16, 9, 12, 10], "tree")
    tree_case(dtype, 3, 4, 8, 8, 48, [30011, 9000], [9, 5], "tree")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kb,vb", [(1, 3), (2, 4), (3, 2), (4, 1)])
@pytest.mark.parametrize("new", [[4, 3, 1], [8, 5, 6], [16, 20, 9]])
def test_tree_rows_of_a_tile(dtype, kb, vb, new):
    """Tiles of 16, 32 and 64 rows (four query heads a KV head), each with every width of codes; sequences past one tile."""
    tree_case(dtype, kb, vb, 8, 2, 16, [777, 64, 3001], new, "tree")


@pytest.mark.parametrize("dtype", TYPES)
def test_tree_masks_and_empty_rows(dtype):
    """Random masks, rows that see nothing, drafted tokens past the mask's words."""
    tree_case(dtype, 4, 4, 8, 2, 16, [40, 0], [50, 33], "random")
    s = make_tree(dtype, 4, 4, 8, 2, 16, [0, 20], [4, 3])
    m = torch.zeros(7, 1, dtype=torch.int32, device="cuda")
    m[1, 0] = 0b0010
    got = run_tree(s, 4, 4, 16, m)
    assert (got[0] == 0).all() and (got[2:4] == 0).all()  # nothing cached, nothing seen
    assert (got[1].float() - s["v"][1].float().repeat_interleave(4, 0)).abs().max() <= 2 ** -7 * s["v"][1].float().abs().max()
    want = tree_plain(s["q"], s["k"], s["v"], s["start"], m, s["K"], s["V"], s["lens"], s["table"], 16, 2, 1 / math.sqrt(D), 4, 4)
    check_tree(got, *want)
    tree_long = make_tree(dtype, 4, 4, 8, 2, 16, [33], [70])
    m = torch.full((70, 2), -1, dtype=torch.int32, device="cuda")  # 64 tokens named, 70 there
    got = run_tree(tree_long, 4, 4, 16, m)
    t = tree_long
    check_tree(got, *tree_plain(t["q"], t["k"], t["v"], t["start"], m, t["K"], t["V"], t["lens"], t["table"], 16, 2, 1 / math.sqrt(D), 4, 4))


@pytest.mark.parametrize("dtype", TYPES)
def test_tree_masked_nan_and_infinity(dtype):
    """NaN and infinities in drafted rows touch the rows that see them, and no others; so do those in a row of q."""
    s = make_tree(dtype, 4, 4, 8, 2, 16, [40], [5])
    m = i32([[1], [2], [5], [8], [16]])  # row 2 sees drafted 0 and 2
    clean = run_tree(s, 4, 4, 16, m)
    s["k"][1, 0, 3] = math.nan
    s["v"][2, :, 9] = math.inf
    s["v"][3, 1, 0] = math.nan
    s["q"][4, 7, 2] = math.nan
    got = run_tree(s, 4, 4, 16, m)
    hit = torch.zeros(5, 8, dtype=torch.bool, device="cuda")
    hit[1, :4] = hit[2] = hit[3, 4:] = hit[4, 7] = True
    assert got[hit].isnan().any(-1).all() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", TYPES)
def test_tree_large_and_small_values(dtype):
    """Scores far apart and far from zero, values at the ends of the type's range."""
    s = make_tree(dtype, 4, 4, 4, 2, 16, [300], [6], outliers=False)
    big = 3e4 if dtype == torch.float16 else 1e18
    for scale, f, vf in ((1 / math.sqrt(D), 30.0, 1.0), (1e-6 / math.sqrt(D), 1.0, big), (0.3 / math.sqrt(D), 1.0, 1e-6 if dtype == torch.float16 else 1e-18)):
        t = dict(s, q=(s["q"] * f).to(dtype), v=(s["v"].clamp(-2, 2) * vf).to(dtype))
        got = run_tree(t, 4, 4, 16, scale=scale)
        want, size, top = tree_plain(t["q"], t["k"], t["v"], t["start"], None, t["K"], t["V"], t["lens"], t["table"], 16, 2, scale, 4, 4)
        rel = 8 * 2.0 ** -11 * max(top, 1) / math.sqrt(D) + 2 * 2.0 ** -11 if dtype != torch.float32 else 8 * 2.0 ** -24 * 16 * max(top, 1)
        fi = torch.finfo(dtype)
        bound = rel * size + fi.eps / 2 * want.norm(dim=-1) + fi.tiny * fi.eps * math.sqrt(D)
        off = (got.double() - want).norm(dim=-1)
        assert (off <= bound).all(), (scale, float((off / bound).max()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafted,cached", [(1e36, 1.0), (1e33, 1.0), (1.0, 1e35), (1e36, 1e35), (1e-24, 1e-24), (1e-24, 1.0)])
def test_tree_values_of_any_magnitude(dtype, drafted, cached):
    """Drafted and cached values from 1e-24 to 1e36, together and apart; a drafted row of zeros among them."""
    s = make_tree(dtype, 4, 4, 4, 2, 16, [300, 0, 40], [6, 5, 3], outliers=False)
    s["v"] = (s["v"].clamp(-2, 2).double() * drafted).to(dtype)
    s["v"][1] = 0
    s["V"].norm *= cached
    got = run_tree(s, 4, 4, 16)
    want, size, top = tree_plain(s["q"], s["k"], s["v"], s["start"], None, s["K"], s["V"], s["lens"], s["table"], 16, 2, 1 / math.sqrt(D), 4, 4)
    # as in check_tree, row by row
    rel = 8 * 2.0 ** -11 * max(top, 1) / math.sqrt(D) + 2 * 2.0 ** -11 if dtype != torch.float32 else 8 * 2.0 ** -24 * 16 * max(top, 1)
    fi = torch.finfo(dtype)
    bound = rel * size + fi.eps / 2 * want.norm(dim=-1) + fi.tiny * fi.eps * math.sqrt(D)
    off = (got.double() - want).norm(dim=-1)
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("factor", [0.0, 6e4, 1e30])
def test_tree_rows_of_q_do_not_depend_on_each_other(dtype, factor):
    """A row of zeros or of huge values in the same tile leaves small and ordinary rows what they are alone."""
    if dtype == torch.float16 and factor > 6e4:
        pytest.skip("past the type's range")
    s = make_tree(dtype, 4, 4, 8, 2, 16, [3, 70], [5, 4], outliers=False)
    # rows 0 and 6 stand apart; row 1 is small, with a key that is not; the others are ordinary
    q = s["q"].double().clamp(-1, 1)
    q[1] *= 1e-6 if dtype == torch.float16 else 1e-20
    s["q"] = q.to(dtype)
    big = torch.tensor([1], device="cuda")
    scale, kf = (35.0, 3e3) if dtype == torch.float16 else (3.5, 1e19)  # row 1: a score of about one
    s["k"][0] = (s["k"][0].double() * kf).to(dtype)
    m = i32([[1], [3], [4], [8], [16], [1], [2], [4], [8]])  # rows 0 and 1 see it
    t = dict(s, q=s["q"].clone())
    for r in (0, 6):
        t["q"][r] = (torch.sign(q[r]) * factor).to(dtype)
    got = run_tree(t, 4, 4, 16, m, scale=scale)
    rest = torch.tensor([1, 2, 3, 4, 5, 7, 8], device="cuda")
    for rows in (rest[1:], big):  # the bound goes by the largest scores: row 1's are apart
        keep = torch.zeros(9, 1, 1, dtype=torch.bool, device="cuda")
        keep[rows] = True
        want, size, top = tree_plain(torch.where(keep, t["q"], 0), s["k"], s["v"], s["start"], m, s["K"], s["V"], s["lens"], s["table"], 16, 2, scale, 4, 4)
        if rows is big:  # its own largest score
            top = float((s["q"][1].double().norm(dim=-1).max() * s["k"][0].double().norm(dim=-1).max()) * scale)
        else:
            top = float(q.norm(dim=-1).max() * max(values(s["K"], 4).norm(dim=-1).max(), s["k"][1:].double().norm(dim=-1).max()) * scale)
        rel = 8 * 2.0 ** -11 * max(top, 1) / math.sqrt(D) + 2 * 2.0 ** -11 if dtype != torch.float32 else 8 * 2.0 ** -24 * 16 * max(top, 1)
        off = (got.double() - want).norm(dim=-1)[rows]
        assert (off <= rel * size[rows] + torch.finfo(dtype).eps / 2 * want.norm(dim=-1)[rows]).all(), float((off / size[rows]).max())


@pytest.mark.parametrize("dtype,q,scale", [(torch.float32, 1e-36, 1e-4), (torch.bfloat16, 1e-36, 1e-4), (torch.float16, 1e-6, 1e-30),
                                           (torch.bfloat16, 1.0, 1e-36), (torch.float16, 1.0, 1e-38)])
def test_tree_scores_near_zero(dtype, q, scale):
    """Factors of q below the normal range: scores of zero, weights that are all one."""
    s = make_tree(dtype, 4, 4, 4, 2, 16, [70], [3], outliers=False)
    s["q"] = (s["q"].double() * q).to(dtype)
    got = run_tree(s, 4, 4, 16, scale=scale)
    check_tree(got, *tree_plain(s["q"], s["k"], s["v"], s["start"], None, s["K"], s["V"], s["lens"], s["table"], 16, 2, scale, 4, 4))


def one_term(x):
    """Rows as one fp16 in the rotated domain would hold them."""
    y = x.double() @ rotation().T
    up = torch.exp2(11 - torch.floor(torch.log2(y.abs().amax(-1, keepdim=True))))
    return (y * up).half().double() / up @ rotation()


def test_tree_second_terms_of_fp16_scores():
    """Large scores: q and the drafted keys count in two fp16 terms.  A score of up to `top` is off by 2^-23 of it for
    each operand's terms and for each of two truncated sums, and weights by twice that: 2^-20·top, doubled once more.
    One term of either breaks the bound."""
    Hkv, scale = 2, 8.0
    s = make_tree(torch.float16, 1, 1, 8, Hkv, 16, [40, 0, 9], [20, 64, 70], outliers=False)
    m = tree_masks([20, 64, 70], "tree", torch.Generator().manual_seed(1), 3)

    def plain(q, k):
        return tree_plain(q, k, s["v"], s["start"], m, s["K"], s["V"], s["lens"], s["table"], 16, Hkv, scale, 1, 1)

    want, size, top = plain(s["q"], s["k"])
    bound = 2.0 ** -19 * top * size + 2.0 ** -11 * want.norm(dim=-1)
    assert ((plain(one_term(s["q"]), s["k"])[0] - want).norm(dim=-1) > bound).any()
    assert ((plain(s["q"], one_term(s["k"]))[0] - want).norm(dim=-1) > bound).any()
    off = (run_tree(s, 1, 1, 16, m, scale=scale).double() - want).norm(dim=-1)
    assert (off <= bound).all(), float((off / bound).max())


def test_tree_second_terms_of_fp16_weights():
    """Two drafted tokens whose values cancel but for the difference of their weights: those count in two fp16 terms."""
    n = 32
    s = make_tree(torch.float16, 1, 1, 8, 2, 16, [0] * n, [2] * n, outliers=False)
    s["v"][1::2] = -s["v"][::2]
    m = i32([[3]] * (2 * n))
    scale = 0.01 / math.sqrt(D)
    got = run_tree(s, 1, 1, 16, m, scale=scale)
    want, size, _ = tree_plain(s["q"], s["k"], s["v"], s["start"], m, s["K"], s["V"], s["lens"], s["table"], 16, 2, scale, 1, 1)
    # sums and both terms are right to 2^-22 of Σ p‖v‖, eight of those; then the output's rounding
    bound = 2.0 ** -19 * size + 2.0 ** -11 * want.norm(dim=-1)
    z = (s["q"].double().view(n, 2, 2, 4, D)[:, :, :, :, None] * s["k"].double().view(n, 2, 2, D).transpose(1, 2)[:, None, :, None]).sum(-1) * scale
    w = (z.softmax(-1) * 50).half().double()  # one term
    one = ((w[..., :1] - w[..., 1:]) / w.sum(-1, keepdim=True) * s["v"][::2].double()[:, None, :, None]).reshape(2 * n, 8, D)
    assert ((one - want).norm(dim=-1) > bound).any()
    off = (got.double() - want).norm(dim=-1)
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("lens,new", [([0], [70]), ([0, 0, 0], [1, 64, 5]), ([0], [300])])
def test_tree_a_row_that_sees_itself_alone_is_its_value(lens, new):
    """fp16 rows: the value comes back but for 2^-20 of its norm (rotations in fp32, two fp16 terms) and one rounding."""
    s = make_tree(torch.float16, 2, 2, 8, 2, 16, lens, new)
    i = torch.cat([torch.arange(n) for n in new])
    m = torch.zeros(len(i), (max(new) + 31) // 32, dtype=torch.int64)
    m[torch.arange(len(i)), i // 32] = 1 << (i % 32)
    m = torch.where(m >= 2 ** 31, m - 2 ** 32, m).int().cuda()
    got = run_tree(s, 2, 2, 16, m).double().view(len(i), 2, 4, D)
    v = s["v"].double()
    bound = 2.0 ** -20 * v.norm(dim=-1, keepdim=True) + 2.0 ** -11 * v.abs()
    assert ((one_term(s["v"]) - v).abs() > bound).any()
    assert ((got - v[:, :, None]).abs() <= bound[:, :, None]).all()


def test_tree_fp32_to_fp32_rounding():
    """fp32 calls with moderate scores: sums of 128 and of all tokens in fp32.  A score is off by 8·2^-24·top (terms,
    norm, scale, exponent), weights by twice that, the sums and rotations by 16·2^-24 of Σ p‖v‖."""
    s = make_tree(torch.float32, 4, 4, 8, 2, 16, [700, 33, 0], [9, 30, 5], outliers=False)
    m = tree_masks([9, 30, 5], "tree", torch.Generator().manual_seed(2), 1)
    scale = 0.2 / math.sqrt(D)
    got = run_tree(s, 4, 4, 16, m, scale=scale)
    want, size, top = tree_plain(s["q"], s["k"], s["v"], s["start"], m, s["K"], s["V"], s["lens"], s["table"], 16, 2, scale, 4, 4)
    off = (got.double() - want).norm(dim=-1)
    assert (off <= 16 * 2.0 ** -24 * (1 + top) * size).all(), float((off / size).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B", [257, 700])
def test_tree_many_sequences(dtype, B):
    """More sequences than a CTA lays out at once: short and ragged, many without rows (a run of them across the first
    256), some with nothing cached."""
    r = np.random.default_rng(B)
    lens, new = r.integers(0, 300, B), r.integers(0, 4, B)
    lens[r.random(B) < 0.3] = 0
    new[200:256] = 0
    new[B // 2 + 130:B // 2 + 200] = 0
    new[-1] = 2
    tree_case(dtype, 3, 2, 4, 2, 16, lens.tolist(), new.tolist(), "tree")


def test_tree_rows_past_the_end_and_strides():
    """Rows behind the last sequence are left; q, k, v may be slices of one projection; bad offsets are cut."""
    s = make_tree(torch.bfloat16, 4, 4, 8, 2, 16, [100, 50], [3, 4])
    want = run_tree(s, 4, 4, 16)
    qkv = torch.full((12, 12, D), math.nan, dtype=torch.bfloat16, device="cuda")
    qkv[:7, :8], qkv[:7, 8:10], qkv[:7, 10:] = s["q"], s["k"], s["v"]
    t = dict(s, q=qkv[:, :8], k=qkv[:, 8:10], v=qkv[:, 10:])
    got = run_tree(t, 4, 4, 16)
    assert torch.equal(got[:7], want) and (got[7:] == 7).all()
    t = dict(s, start=i32([0, 3, 900]))  # the last sequence ends with the buffer
    assert torch.equal(run_tree(t, 4, 4, 16), want)


def test_tree_pages_outside_the_cache():
    """A page that is not one is left out and reported once; lengths past the table are cut."""
    s = make_tree(torch.float16, 4, 4, 8, 2, 16, [200, 70], [2, 3])
    bad = s["table"].clone()
    bad[0, 3], bad[1, 0] = 10_000_000, -5
    t = dict(s, table=bad)
    got = run_tree(t, 4, 4, 16)
    assert ctx(4).poll() == tq.TQ_ERR_INVALID_ARG and ctx(4).poll() == tq.TQ_OK
    check_tree(got, *tree_plain(t["q"], t["k"], t["v"], t["start"], None, t["K"], t["V"], t["lens"], bad, 16, 2, 1 / math.sqrt(D), 4, 4))
    t = dict(s, lens=i32([5000, 70]))
    cut = dict(s, lens=i32([s["table"].shape[1] * 16, 70]))
    assert torch.equal(run_tree(t, 4, 4, 16), run_tree(cut, 4, 4, 16))
    ctx(4).poll()


def test_tree_captured_serves_later_lengths():
    """A call captured into a graph reads lengths, offsets and masks when it is replayed; on another stream too."""
    s = make_tree(torch.bfloat16, 3, 3, 8, 2, 16, [900, 700], [5, 5])
    full = s["lens"].clone()
    ws = torch.zeros(tq.tq_tree_attention_workspace_size(ctx(3), 2, 8, 2, 10) // 4 + 4, device="cuda")
    out = torch.zeros(10, 8, D, dtype=torch.bfloat16, device="cuda")
    run_tree(s, 3, 3, 16, out=out, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_tree(s, 3, 3, 16, out=out, ws=ws)
    for lens, start in (([0, 1], [0, 1, 2]), ([400, 699], [0, 5, 10]), ([33, 0], [0, 0, 7]), (full.tolist(), [0, 9, 10])):
        s["lens"].copy_(i32(lens))
        s["start"].copy_(i32(start))
        out.fill_(7)
        graph.replay()
        n = start[-1]
        want = tree_plain(s["q"], s["k"], s["v"], s["start"], None, s["K"], s["V"], s["lens"], s["table"], 16, 2, 1 / math.sqrt(D), 3, 3)
        check_tree(out[:n], *(x[:n] if torch.is_tensor(x) else x for x in want))
        assert (out[n:] == 7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run_tree(s, 3, 3, 16)
    side.synchronize()
    assert torch.equal(other[:10], out)


def test_tree_waits_are_bounded():
    """With a wait limit of 0 every pipeline wait gives up before its first poll: the call returns, the status says so
    once, and the next call is right again."""
    c = tq.Context(D, 4, tq.TQ_MSE, tq.TQ_ROT_DENSE, tq.tq_rotation_haar(synth.gaussian_matrix(0, D)))
    for dtype, new in ((torch.bfloat16, [3, 2]), (torch.float16, [20, 9])):
        s = make_tree(dtype, 4, 4, 8, 2, 16, [700, 3000], new)
        ws = torch.zeros(tq.tq_tree_attention_workspace_size(c, 2, 8, 2, sum(new)) // 4 + 4, device="cuda")
        out = torch.zeros(sum(new), 8, D, dtype=dtype, device="cuda")

        def call():
            tq.tq_tree_attention(c, c, s["q"], s["k"], s["v"], s["start"], None, s["K"], s["V"], s["lens"], s["table"], 16,
                                 1 / math.sqrt(D), out, ws)

        c.set_wait_limit(0)
        call()
        assert c.poll() == tq.TQ_ERR_TIMEOUT and c.poll() == tq.TQ_OK
        c.set_wait_limit(1 << 22)
        call()
        assert c.poll() == tq.TQ_OK
        assert torch.equal(out, run_tree(s, 4, 4, 16))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_tree_factors_of_drafted_tiles_before_copied_norms(dtype):
    """A CTA's tiles of many short sequences: the place of a drafted tile's factors takes copied norms soon after."""
    tree_case(dtype, 4, 4, 8, 8, 16, [130 + 2 * k for k in range(64)], [1 + k % 4 for k in range(64)], "tree")


def test_tree_over_hadamard_rotated_caches():
    """A context with the randomized Hadamard rotation: the same answer as the decode call's over the same cache."""
    c = tq.Context(D, 4, tq.TQ_MSE, tq.TQ_ROT_HADAMARD, synth.hadamard_signs(3, D))
    g, B, Hq, Hkv, cap = gen(8), 2, 8, 2, 1008
    K, V = tq.CodeSet(c, B * Hkv * cap), tq.CodeSet(c, B * Hkv * cap, tq.TQ_LAYOUT_PAIR)
    for cs in (K, V):
        tq.tq_encode(c, torch.randn(B * Hkv * cap, D, device="cuda", generator=g), cs)
    q = torch.randn(B, Hq, D, device="cuda", generator=g)
    want = torch.empty(B, Hq, D, device="cuda")
    ws = torch.zeros(tq.tq_decode_workspace_size(c, B, Hq, Hkv, cap) // 4 + 4, device="cuda")
    tq.tq_decode_attention(c, c, q, K, V, B, Hq, Hkv, cap, cap, 1 / math.sqrt(D), want, ws)
    for dtype in TYPES:
        out = torch.empty(B, Hq, D, dtype=dtype, device="cuda")
        ws = torch.zeros(tq.tq_tree_attention_workspace_size(c, B, Hq, Hkv, B) // 4 + 4, device="cuda")
        tq.tq_tree_attention(c, c, q.to(dtype), None, None, i32([0, 1, 2]), None, K, V, i32([cap, cap]), None, cap,
                             1 / math.sqrt(D), out, ws, Hkv=Hkv)
        # the library's bound for attention on both sides, the roundings of q and of the output
        assert (out.float() - want).norm() <= (4e-3 + 2 * torch.finfo(dtype).eps) * want.norm()


def test_calls_at_once_on_two_streams():
    """Attention on two streams (a workspace each, one context pair) beside appends to a third cache: as one by one."""
    a = make_tree(torch.bfloat16, 4, 4, 32, 8, 16, [3000, 517, 2048], [7, 16, 1], 3)
    b = make_tree(torch.float16, 4, 4, 16, 2, 64, [9000, 33], [12, 30], 4)
    x = torch.randn(500, 8, D, device="cuda", generator=gen(5)).half()
    slots = torch.randperm(1024, device="cuda", generator=gen(6))[:500]
    codes = [tq.CodeSet(ctx(4), 1024 * 8, tq.TQ_LAYOUT_PAIR) for _ in range(2)]
    want = run_tree(a, 4, 4, 16), run_tree(b, 4, 4, 64)
    tq.tq_encode_slots(ctx(4), x, slots, 16, codes[0])
    ws = [torch.zeros(tq.tq_tree_attention_workspace_size(ctx(4), s["lens"].numel(), s["q"].shape[1], s["k"].shape[1], s["q"].shape[0]) // 4 + 4,
                      device="cuda") for s in (a, b)]
    outs = [[torch.zeros_like(w) for _ in range(8)] for w in want]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for k in range(8):
        with torch.cuda.stream(streams[0]):
            run_tree(a, 4, 4, 16, out=outs[0][k], ws=ws[0])
        with torch.cuda.stream(streams[1]):
            run_tree(b, 4, 4, 64, out=outs[1][k], ws=ws[1])
        with torch.cuda.stream(streams[2]):
            tq.tq_encode_slots(ctx(4), x, slots, 16, codes[1])
    torch.cuda.synchronize()
    for k in range(8):
        assert torch.equal(outs[0][k], want[0]) and torch.equal(outs[1][k], want[1])
    assert torch.equal(codes[0].codes, codes[1].codes) and torch.equal(codes[0].norm, codes[1].norm)
    assert ctx(4).poll() == tq.TQ_OK


def test_tree_is_deterministic():
    s = make_tree(torch.float16, 4, 4, 32, 8, 16, [3000, 100, 2500], [16, 3, 9])
    first = run_tree(s, 4, 4, 16)
    for _ in range(5):
        assert torch.equal(run_tree(s, 4, 4, 16), first)


def test_tree_agrees_with_decode():
    """One token per sequence over the contiguous cache is the decode step's attention."""
    s = make_tree(torch.float16, 4, 4, 8, 2, 512, [512, 512], [1, 1], paged=False)
    got = run_tree(s, 4, 4, 512, drafts=False)
    out = torch.empty(2, 8, D, device="cuda")
    ws = torch.zeros(tq.tq_decode_workspace_size(ctx(4), 2, 8, 2, 512) // 4 + 4, device="cuda")
    tq.tq_decode_attention(ctx(4), ctx(4), s["q"], s["K"], s["V"], 2, 8, 2, 512, 512, 1 / math.sqrt(D), out, ws)
    assert (got.float() - out).norm() <= 4e-3 * out.norm()


def test_refusals():
    c, prod, mixed = ctx(4), ctx(3, tq.TQ_PROD), ctx(2, tq.TQ_MIXED)
    s = make_tree(torch.float16, 4, 4, 8, 2, 16, [100], [3])
    ws = torch.zeros(tq.tq_tree_attention_workspace_size(c, 1, 8, 2, 3) // 4 + 4, device="cuda")
    out = torch.empty(3, 8, D, dtype=torch.float16, device="cuda")

    def call(kc=c, vc=c, K=s["K"], V=s["V"], block=16, scale=0.1, ws=ws, q=s["q"], table=s["table"], **kw):
        tq.tq_tree_attention(kc, vc, q, s["k"], s["v"], s["start"], None, K, V, s["lens"], table, block, scale, out, ws, **kw)

    call()

    def status(st, **kw):
        with pytest.raises(tq.TqError) as e:
            call(**kw)
        assert e.value.status == st, kw

    status(-2, block=8)
    status(-2, block=24)
    status(-1, block=0)
    status(-1, scale=0.0)
    status(-1, scale=math.nan)
    status(-1, ws=ws[:-16])
    status(-1, ws=ws[1:])
    status(-1, K=s["V"])
    status(-1, V=s["K"])
    status(-1, table=None, block=1 << 20)  # more than the cache holds
    status(-2, kc=prod, K=tq.CodeSet(prod, 1024))
    status(-2, kc=mixed, K=tq.CodeSet(mixed, 1024))
    status(-1, kc=ctx(3))
    status(-2, table=torch.empty(1, 2 ** 27 - 1, dtype=torch.int32, device="cuda"))  # 16 short of 2^31 places
    for kw in (dict(q=s["q"].transpose(0, 1)), dict(ws=ws.cpu()), dict(ws=ws[::2]), dict(q=s["q"].cpu()),
               dict(q=s["q"][:, :1, :64])):  # half a row of one head, the stride of a whole one
        with pytest.raises(ValueError):
            call(**kw)
    x = torch.randn(4, 2, D, device="cuda", dtype=torch.float16)
    slots = torch.arange(4, device="cuda")
    for st, kw in ((-2, dict(block=15)), (-1, dict(block=0)), (-1, dict(block=1 << 20))):
        with pytest.raises(tq.TqError) as e:
            tq.tq_encode_slots(c, x, slots, kw["block"], s["K"])
        assert e.value.status == st
    with pytest.raises(ValueError):
        tq.tq_encode_slots(c, x.bfloat16(), slots, 16, s["K"])
    wide = tq.Context(256, 4, tq.TQ_MSE, tq.TQ_ROT_DENSE, np.eye(256))
    with pytest.raises(tq.TqError) as e:
        tq.tq_encode_slots(wide, torch.randn(4, 2, 256, device="cuda"), slots, 16, tq.CodeSet(wide, 64))
    assert e.value.status == -2


def test_calls_that_take_no_bf16_refuse_it():
    """TQ_BF16 belongs to tq_qk_norm_rope and tq_tree_attention; the other calls refuse it, whatever else is right."""
    L, c, B, H, cap = tq.lib(), ctx(4), 1, 2, 64
    K, V = tq.CodeSet(c, B * H * cap), tq.CodeSet(c, B * H * cap, tq.TQ_LAYOUT_PAIR)
    x, out, slots = torch.zeros(B * H, D, device="cuda"), torch.empty(B, H, D, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = torch.zeros(tq.tq_decode_workspace_size(c, B, H, H, cap) // 4 + 4, device="cuda")
    k, v, a, o = tq.ctypes.byref(K.desc), tq.ctypes.byref(V.desc), x.data_ptr(), out.data_ptr()
    for dt, st in ((tq.TQ_BF16, tq.TQ_ERR_INVALID_ARG), (tq.TQ_F16, tq.TQ_OK)):
        assert L.tq_encode(c.handle, a, dt, 1, k, 0, 1, 0, None) == st
        assert L.tq_encode_slots(c.handle, a, dt, 1, H, slots.data_ptr(), 16, k, None) == st
        assert L.tq_decode_attention(c.handle, c.handle, a, dt, k, v, B, H, H, cap, cap, 0.1, o, ws.data_ptr(), ws.numel() * 4, None) == st
        assert L.tq_decode_step(c.handle, c.handle, a, dt, a, a, tq.TQ_F16, k, v, B, H, H, cap, cap, 0.1, o, ws.data_ptr(), ws.numel() * 4, None) == st
        assert L.tq_decode_step(c.handle, c.handle, a, tq.TQ_F16, a, a, dt, k, v, B, H, H, cap, cap, 0.1, o, ws.data_ptr(), ws.numel() * 4, None) == st
        assert L.tq_decode_attention_noalloc(c.handle, c.handle, a, dt, k, v, B, H, H, cap, cap, 0.1, o, None) == st
    torch.cuda.synchronize()


def test_tensors_of_another_device_are_refused(monkeypatch):
    x, pos = torch.ones(2, 1, D, device="cuda"), i32([0, 1])
    args = (x, x, None, None, 1e-6, None, 0, pos, torch.empty_like(x), torch.empty_like(x))
    tq.tq_qk_norm_rope(*args)
    monkeypatch.setattr(tq, "_T", tq._types()[:3] + (lambda: 1 + x.get_device(),))  # as if another were current
    with pytest.raises(ValueError, match="current device"):
        tq.tq_qk_norm_rope(*args)
    lens, n = i32([0]), torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="current device"):
        tq.tq_block_tables(lens, lens, lens, pos, n, lens[None], 16, pos, n.clone(), pos, n, pos)


# ------------------------------------------------------------------ together
def test_steps_of_a_server():
    """Three requests: prompts admitted, then rounds of drafted trees of which some tokens stay, over pages that come
    from and go back to one ring; every round against attention over all that was kept, in 64 bits."""
    g, block, kb, vb, Hq, Hkv, B, T = gen(11), 16, 4, 3, 8, 2, 3, 6
    r = np.random.default_rng(5)
    width, pages = 12, 30
    z32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, held, ring = z32(B), z32(B), torch.randperm(pages, device="cuda", generator=g, dtype=torch.int32)
    state, table = torch.tensor([0, pages], device="cuda"), torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    K, V = tq.CodeSet(ctx(kb), pages * block * Hkv), tq.CodeSet(ctx(vb), pages * block * Hkv, tq.TQ_LAYOUT_PAIR)
    freq = tq.tq_rope_frequencies(1e4 ** (-np.arange(0, D, 2) / D))
    w = (1 + 0.1 * torch.randn(2, D, device="cuda", generator=g)).to(torch.bfloat16)
    new = i32([37, 5, 64])
    for step in range(5):
        rows = int(new.sum())
        held2, state2, start = z32(B), torch.zeros_like(state), z32(B + 1)
        slots, pos = torch.zeros(rows, dtype=torch.int64, device="cuda"), z32(rows)
        tq.tq_block_tables(lens, new, held, ring, state, table, block, held2, state2, start, slots, pos)
        held, state = held2, state2
        qkv = torch.randn(rows, Hq + 2 * Hkv, D, device="cuda", generator=g).to(torch.bfloat16)
        q, k = torch.empty(rows, Hq, D, dtype=torch.float16, device="cuda"), torch.empty(rows, Hkv, D, dtype=torch.float16, device="cuda")
        tq.tq_qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], w[0], w[1], 1e-6, freq, 0, pos, q, k)
        v = qkv[:, Hq + Hkv:].half()
        mask = None if step == 0 else tree_masks(new.tolist(), "tree", torch.Generator().manual_seed(step), 1)
        s = {"q": q, "k": k, "v": v, "start": start, "lens": lens, "table": table, "K": K, "V": V}
        got = run_tree(s, kb, vb, block, mask)
        check_tree(got, *tree_plain(q, k, v, start, mask, K, V, lens, table, block, Hkv, 1 / math.sqrt(D), kb, vb))
        # the tokens that stay: all of a prompt, the first few of a tree (its slots are in order of position)
        stay = new if step == 0 else torch.minimum(new, i32(r.integers(0, T + 1, B).tolist()))
        n = torch.arange(rows, device="cuda")
        b = torch.searchsorted(start[1:].contiguous(), n.int(), right=True)
        put = torch.where(n - start[b] < stay[b], slots, -1)
        tq.tq_encode_slots(ctx(kb), k, put, block, K)
        tq.tq_encode_slots(ctx(vb), v.contiguous(), put, block, V)
        lens = lens + stay
        new = torch.full_like(lens, T)
        if step == 2:  # the first request ends, another takes its row
            lens[0], new[0] = 0, 0
        if step == 3:
            new[0] = 20
    free = ring[torch.arange(int(state[0]), int(state[1]), device="cuda") % pages]
    owned = torch.cat([table[b, :int(held[b])] for b in range(B)])
    assert sorted(torch.cat([free, owned]).tolist()) == list(range(pages))  # no page lost, none twice
