"""Weights of an 8-bit cache's tokens far below one of their row's, and the sums they make."""

import math

import pytest

torch = pytest.importorskip("torch")
import kv_cache_vector_tq_gb300 as tq  # noqa: E402
from test_gpu_cache8 import TYPES, attend, gen  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,new", [(152, 1), (76, 20), (38, 300)])
def test_one_token_above_many_equal_ones(B, new, d, ty):
    """The first token 2^16 to 2^24 times as heavy as each of 65536 others, with a value like theirs, or none of its own:
    then they alone are the result.  Every request has the same cache, so that a CTA has all of a tile."""
    n, Hkv, block, t = 65536, 2, 64, TYPES[ty]
    width = (n + new + block) // block
    cache = tq.Cache8(width, Hkv, block, d)
    cache.kscale.fill_(1.0)
    cache.vscale.fill_(1.0)
    table = torch.randperm(width, generator=gen(d), device="cuda").int()[None].repeat(B, 1)
    cache.v.view(torch.uint8).fill_(0x38)  # 1
    first = table[0, 0]
    cache.k.view(torch.uint8)[first, :, 0, 3] = 0x7E  # 448
    q = torch.zeros(B * new, 2 * Hkv, d, device="cuda", dtype=t)
    q[:, :, 3] = 1
    many = n + torch.arange(new, device="cuda", dtype=torch.float64).repeat(B)[:, None, None]
    for orders, above in ((16, 64), (20, 64), (24, 64), (20, 128), (24, 128)):
        # a little less than half a step of six or seven bits above the power of two
        scale = (orders - math.log2((above + 0.49) / above)) * math.log(2) / 448
        w = math.exp(-448 * torch.tensor(scale).float().item())  # of each, the first token's being 1
        for own in (0.0, 1.0):
            cache.v.view(torch.uint8)[first, :, 0] = 0x38 if own else 0
            out = attend(q, [new * b for b in range(B + 1)], [n] * B, table, cache, scale)
            ref = (own + many * w) / (1 + many * w)
            # a weight: its terms of fp16 (half a step of 11 or 22 bits), and no finer than half of fp16's least step, 2^-25,
            # where the row's largest is 2^10 or more, 2^7 from 33 rows on (fp32 has the second term 2^12 times as large);
            # a score of 24 is three roundings of 2^-24 off, a power of two 2^-22
            term = 2.0 ** -12 if t is torch.bfloat16 else 2.0 ** -23
            least = 2.0 ** (-47 if t is torch.float32 else -35 if new == 1 else -32)
            weights = many * (w * (term + 2.0 ** -18) + least) / (own + many * w)
            # sums: fp32 rows 16 tokens at a time and a warp's quarter of them, half a step (2^-24) each; products of the
            # matrix units cut 2^-23 at most, those of a warp's quarter (few rows) or between two rests (256 and 1024 halves
            # of units, four products a term); sums of weights half a step for 64 tokens
            terms = 1 if t is torch.bfloat16 else 2
            halves = n / 64
            if t is torch.float32:
                sums = halves * 2.0 ** -24
            elif new == 1:
                sums = halves * terms * 2.0 ** -23
            else:
                sums = 4 * terms * min(halves, 256 if t is torch.float16 else 1024) * 2.0 ** -23
            sums += halves * 2.0 ** -24 + 2.0 ** -21  # (and the products of 16 tokens in themselves)
            off = ref * (weights + sums) * (1 + 2.0 ** -7)
            half = torch.finfo(t).eps / 2
            bad = (out.double() - ref).abs() - (half * ref + off * (1 + half))
            assert (bad <= 0).all(), (orders, above, own, float(((out.double() - ref) / ref).abs().max()))
