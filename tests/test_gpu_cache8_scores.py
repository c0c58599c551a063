"""Scores of an 8-bit cache's tokens so large that fp32 has no fractions left: the heaviest token is the result."""

import math

import pytest

torch = pytest.importorskip("torch")
import kv_cache_vector_tq_gb300 as tq  # noqa: E402
from test_gpu_cache8 import TYPES, attend, attend_ref, close, filled, gen, pages_for  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("n,new,Hq,Hkv,d,window", [
    (700, 2, 8, 2, 128, 0), (700, 5, 8, 2, 64, 0), (700, 40, 4, 2, 128, 0), (700, 40, 8, 2, 64, 300), (900, 200, 4, 2, 128, 0), (900, 200, 4, 2, 64, 129)])
def test_the_heaviest_token(n, new, Hq, Hkv, d, window, ty):
    g, t, block = gen(n + new + d), TYPES[ty], 16
    table, total = pages_for([n + new], block, g)
    cache = tq.Cache8(total, Hkv, block, d)
    filled(cache, g)
    cache.kscale.fill_(2.0 ** -6)
    q = torch.randn(new, Hq, d, device="cuda", generator=g).to(t)
    at = torch.arange(n + new, device="cuda")
    page, p = table[0].long()[at // block], n + torch.arange(new, device="cuda")
    sees = at[None] <= p[:, None]
    if window:
        sees &= at[None] > p[:, None] - window
    k, v = (c[page, :, at % block].double() * f[page].double()[..., None] for c, f in ((cache.k, cache.kscale), (cache.v, cache.vscale)))
    z = torch.einsum("ihgd,thd->ihgt", q.double().view(new, Hkv, Hq // Hkv, d), k).flatten(1, 2)
    top = z.masked_fill(~sees[:, None], -math.inf).topk(2, -1)
    ref = v.repeat_interleave(Hq // Hkv, 1)[top.indices[..., 0], torch.arange(Hq, device="cuda")[None]]
    # scores are 2^-20 of the sum of magnitudes off (ten times a score at most here): rows whose second score is as near
    # are left out
    clear = top.values[..., 0] - top.values[..., 1] > 2.0 ** -12 * top.values[..., 0].abs()
    assert clear.double().mean() > 0.95
    for power in (24, 27, 30, 40, 60):
        out = attend(q, [0, new], [n], table, cache, 2.0 ** power, window)
        assert torch.isfinite(out).all(), power
        # one weight is left: half a step of the output and of the weight's and the sum's fp32
        off = (out.double() - ref).abs() - ref.abs() * (torch.finfo(t).eps / 2 + 2.0 ** -20)
        assert (off[clear] <= 0).all(), (power, float(off[clear].max()))


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("n,new,Hq,Hkv,d", [(700, 5, 8, 2, 64), (700, 40, 4, 2, 128), (900, 200, 4, 2, 128), (900, 200, 4, 2, 64)])
def test_rows_of_large_scores_beside_others(n, new, Hq, Hkv, d, ty):
    """Scores of 2^21, or infinities, in one row of a tile: the others are right all the same, with infinities bit for bit."""
    g, t, scale = gen(new + d), TYPES[ty], 0.1 * 2.0 ** 8
    table, total = pages_for([n + new], 16, g)
    cache = tq.Cache8(total, Hkv, 16, d)
    filled(cache, g)
    q = (torch.randn(new, Hq, d, device="cuda", generator=g) * 2.0 ** -8).to(t)
    good, (ref, off) = attend(q, [0, new], [n], table, cache, scale), attend_ref(q, [0, new], [n], table, cache, scale, 0, 0)
    rest = torch.ones(new, Hq, dtype=torch.bool, device="cuda")
    rest[new // 2, 1] = rest[3, 0] = False
    close(good, ref, off)
    for factor in (2.0 ** 21, math.inf):
        bad = q.clone()
        bad[~rest] *= factor
        out = attend(bad, [0, new], [n], table, cache, scale)
        close(out[rest], ref[rest], off[rest], factor)
        if math.isinf(factor):
            assert torch.equal(out[rest], good[rest]) and out[~rest].isnan().all()
        else:
            assert torch.isfinite(out).all()
