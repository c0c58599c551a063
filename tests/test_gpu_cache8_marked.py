"""Blocks of an 8-bit cache that were given a NaN or an infinity: rows that see one of their tokens are NaN, and no others."""

import math

import pytest

torch = pytest.importorskip("torch")
import kv_cache_vector_tq_gb300 as tq  # noqa: E402
from test_gpu_cache8 import TYPES, append_plain, attend, filled, gen, i32, pages_for  # noqa: E402

pytestmark = pytest.mark.gpu

BLOCK, REQUESTS, LEN = 16, 160, 2047  # requests of one table, so that a CTA has many units of a tile
# Hq, Hkv, d, rows a request: tiles of 8, 16, 32, 128 and 256 rows
SHAPES = [(8, 2, 128, 2), (8, 2, 64, 3), (8, 2, 128, 5), (8, 2, 128, 20), (8, 2, 64, 20), (8, 2, 64, 100), (4, 2, 128, 300)]


def setup(Hq, Hkv, d, new, ty):
    g = gen(new + d)
    table, total = pages_for([LEN + new], BLOCK, g)
    cache = tq.Cache8(total, Hkv, BLOCK, d)
    filled(cache, g)
    q = torch.randn(new, Hq, d, device="cuda", generator=g).to(TYPES[ty]).repeat(REQUESTS, 1, 1)
    return cache, table.repeat(REQUESTS, 1), q, [new * b for b in range(REQUESTS + 1)], [LEN] * REQUESTS


def check(cache, table, args, block, head, sees, **window):
    """Runs with this block of request 0's table marked against the run without: `sees` [rows a request]."""
    q, Hkv, page = args[0], cache.Hkv, int(table[0, block])
    clean = attend(*args, table, cache, 0.1, **window)
    assert torch.isfinite(clean).all()
    nan = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    G = q.shape[1] // Hkv
    nan[:, head * G:(head + 1) * G] = sees.repeat(REQUESTS)[:, None]
    assert nan.any() and not nan[:, head * G].all()
    for scale in (cache.kscale, cache.vscale):
        kept = scale[page, head].item()
        scale[page, head] = math.nan
        out = attend(*args, table, cache, 0.1, **window)
        scale[page, head] = kept
        assert out[nan].isnan().all()
        assert torch.equal(out[~nan], clean[~nan])


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("Hq,Hkv,d,new", SHAPES)
def test_a_block_that_later_rows_see(Hq, Hkv, d, new, ty):
    cache, table, q, start, lens = setup(Hq, Hkv, d, new, ty)
    block = (LEN + new // 2) // BLOCK
    sees = LEN + torch.arange(new, device="cuda") >= block * BLOCK
    check(cache, table, (q, start, lens), block, 1, sees)


@pytest.mark.parametrize("gone", [False, True])
@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("Hq,Hkv,d,new", SHAPES)
def test_a_block_that_earlier_rows_see(Hq, Hkv, d, new, ty, gone):
    """Behind the window of the later ones; `gone`: the page a unit further on lies outside the cache."""
    cache, table, q, start, lens = setup(Hq, Hkv, d, new, ty)
    block = 60
    last = block * BLOCK + BLOCK - 1
    window = LEN + new // 2 - last  # of the first half of the rows it still has the block's last token
    sees = LEN + torch.arange(new, device="cuda") - window < last
    if gone:
        table[:, block + 128 // BLOCK] = cache.pages
    check(cache, table, (q, start, lens), block, 0, sees, window=window, sinks=3)


@pytest.mark.parametrize("ty", list(TYPES))
def test_an_infinity_in_a_late_draft(ty):
    """Drafted tokens 14 to 17, the value of token 16 an infinity: tokens 14 and 15 are what they were."""
    g, t = gen(2), TYPES[ty]
    table, x = i32([[0, 1]]), torch.randn(18, 1, 64, device="cuda", generator=g).to(t)
    q = torch.randn(4, 4, 64, device="cuda", generator=g).to(t)
    outs = []
    for bad in (1.0, math.inf):
        cache = tq.Cache8(2, 1, 16, 64)
        append_plain(cache, x[:14], [0, 14], [0], table)
        y = x[14:].clone()
        y[2, 0, 5] = bad
        tq.tq_cache8_append(None, x[14:], y, None, None, 0.0, None, 0, i32([14, 15, 16, 17]), i32([0, 4]), i32([14]), table, cache, None)
        outs.append(attend(q, [0, 4], [14], table, cache, 0.1))
    assert torch.equal(outs[0][:2], outs[1][:2]) and torch.isfinite(outs[0]).all() and outs[1][2:].isnan().all()


# Hq, Hkv, d, rows, tokens before them, marked blocks: what a warp, a group or a CTA has is marked, and the first token,
# which another one has, weighs 2^200 and more times as much as what is not
JOINS = [
    (1, 1, 128, 1, 127, [2, 3]),                  # a warp of four
    (4, 2, 64, 2, 126, [2]),                      # half of what the warp has
    (8, 1, 128, 1, 999, list(range(8, 63))),      # parts of several CTAs, a warp joins them
    (8, 1, 64, 2, 3998, list(range(8, 250))),     # four warps do
    (8, 1, 128, 2, 3998, [200]),
    (2, 2, 128, 40, 88, [4, 5, 6, 7]),            # a group of softmax warps of two
    (2, 2, 64, 40, 88, [4]),
    (2, 2, 128, 40, 2960, list(range(8, 188))),   # parts of 128 rows
    (4, 2, 64, 200, 2800, list(range(8, 188))),   # parts of 256 rows
    (4, 2, 128, 200, 2800, [100]),
]


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("Hq,Hkv,d,new,n,blocks", JOINS)
def test_nothing_outweighs_a_marked_block(Hq, Hkv, d, new, n, blocks, ty):
    g = gen(n)
    table, total = pages_for([n + new], BLOCK, g)
    cache = tq.Cache8(total, Hkv, BLOCK, d)
    filled(cache, g)
    for scale in (cache.kscale, cache.vscale):
        scale.fill_(2.0 ** -6)
    cache.k.view(torch.uint8)[table[0, 0], :, 0] = 0x7E  # 448: a score of 4 · 7 · d / 10 against some ten at most
    q = (4 + 0.1 * torch.randn(new, Hq, d, device="cuda", generator=g)).to(TYPES[ty])
    pages = table[0, blocks].long()
    assert torch.isfinite(attend(q, [0, new], [n], table, cache, 0.1)).all()
    for scale in (cache.kscale, cache.vscale):
        kept = scale[pages].clone()
        scale[pages] = math.nan
        assert attend(q, [0, new], [n], table, cache, 0.1).isnan().all()
        scale[pages] = kept
