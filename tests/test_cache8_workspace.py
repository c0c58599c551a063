"""The workspace of attention over an 8-bit cache: one for the most requests and rows serves every smaller call."""

import ctypes
import os

import pytest

import kv_cache_vector_tq_gb300 as tq

ROWS = [0, 1, 8, 9, 40, 130, 600, 4096, 65536]


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 8, 128), (64, 8, 128), (2, 2, 64)])
def test_sizes_grow_with_requests_and_rows(Hq, Hkv, d):
    if not os.path.exists(tq.LIB_PATH):
        from kv_cache_vector_tq_gb300 import build
        build.build()
    a, n = 1 << 20, ctypes.c_size_t()  # an aligned address that nothing reads
    desc = tq.Cache8Desc(a, a, a, a, a, 4, Hkv, 16, d)
    last = None
    for B in (1, 2, 64, 512, 65536):
        sizes = []
        for rows in ROWS:
            assert tq.lib().tq_cache8_attention_workspace_size(ctypes.byref(desc), B, Hq, rows, ctypes.byref(n)) == tq.TQ_OK
            sizes.append(n.value)
        assert sizes == sorted(sizes)
        assert last is None or all(x <= y for x, y in zip(last, sizes)), B
        last = sizes


@pytest.mark.gpu
def test_one_workspace_for_all_calls():
    """A server's: 64 requests, 600 rows; then prompts of one, a few pieces, single tokens."""
    torch = pytest.importorskip("torch")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = tq.Cache8(64, 2, 64, 128)
    cache.k.view(torch.uint8).fill_(0x38)
    cache.v.view(torch.uint8).fill_(0x38)  # 1
    cache.kscale.fill_(1.0)
    cache.vscale.fill_(1.0)
    n = tq.tq_cache8_attention_workspace_size(cache, 64, 8, 600)
    guard = torch.full((n // 4 + 64,), 7.0, device="cuda")
    ws = guard[:n // 4]
    table = torch.arange(64, device="cuda").int().view(1, 64)
    for new in ([600], [599, 1], [1] * 64, [30] * 20, [0, 0, 3], [0] * 63 + [600]):
        B, rows = len(new), sum(new)
        for t in (torch.bfloat16, torch.float32):
            q, out = torch.ones(rows, 8, 128, device="cuda", dtype=t), torch.zeros(rows, 8, 128, device="cuda", dtype=t)
            start = i32([sum(new[:b]) for b in range(B + 1)])
            tq.tq_cache8_attention(q, start, i32([1000] * B), table.repeat(B, 1), cache, 0.1, out, ws)
            # one weight for all tokens: fp32's terms and sums are 1e-5 off at most, bf16 rounds to 1
            assert (out - 1).abs().max() <= 1e-5
    assert (guard[n // 4:] == 7).all()
