"""The serving calls' checks of their arguments and the host call, without a GPU.  Every refused call returns
before anything is launched, so its device addresses are made up."""

import ctypes
import os
import types

import numpy as np
import pytest

import kv_cache_vector_tq_gb300 as tq

A = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(tq.LIB_PATH):
        from kv_cache_vector_tq_gb300 import build
        build.build()
    return tq.lib()


TABLES = dict(len=A, new=A, held=A, B=4, block=16, ring=A, n=8, state=A, table=A, width=4, held_out=2 * A,
              state_out=2 * A, start=A, slots=A, pos=A, rows=5, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), -1), (dict(block=0), -1), (dict(n=0), -1), (dict(width=0), -1), (dict(rows=-1), -1),
    (dict(len=None), -1), (dict(new=None), -1), (dict(held=None), -1), (dict(ring=None), -1), (dict(state=None), -1),
    (dict(table=None), -1), (dict(held_out=None), -1), (dict(state_out=None), -1), (dict(start=None), -1),
    (dict(slots=None), -1), (dict(pos=None), -1), (dict(held_out=A), -1), (dict(state_out=A), -1),
    (dict(slots=A + 4), -1), (dict(state=A + 4), -1), (dict(B=4097), -2), (dict(B=4096, width=1 << 20), -2)])
def test_block_tables_refusals(L, change, status):
    assert L.tq_block_tables(*{**TABLES, **change}.values()) == status


NORM = dict(q=A, qs=4 * 128, k=A, ks=2 * 128, dt=1, N=3, Hq=4, Hkv=2, d=128, wq=A, wk=None, eps=1e-6, freq=A, rot=128,
            style=0, pos=A, qo=A, qos=512, ko=A, kos=256, odt=1, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dt=3), -1), (dict(odt=-1), -1), (dict(N=-1), -1), (dict(Hq=0, Hkv=0), -1), (dict(d=0), -1),
    (dict(rot=-16), -1), (dict(rot=144), -1), (dict(style=2), -1), (dict(eps=0.0), -1), (dict(eps=float("nan")), -1),
    (dict(qs=511), -1), (dict(ks=255), -1), (dict(qos=511), -1), (dict(kos=255), -1), (dict(q=None), -1),
    (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1), (dict(pos=None), -1), (dict(freq=None), -1),
    (dict(q=A + 8), -1), (dict(ko=A + 2), -1), (dict(wq=A + 4), -1), (dict(qs=516), -1), (dict(kos=257), -1),
    (dict(d=48, rot=48, qs=512), -2), (dict(d=288, rot=128, qs=2048, ks=2048, qos=2048, kos=2048), -2),
    (dict(rot=24), -2)])
def test_qk_norm_rope_refusals(L, change, status):
    assert L.tq_qk_norm_rope(*{**NORM, **change}.values()) == status


def test_nothing_to_do_is_fine(L):
    assert L.tq_qk_norm_rope(*{**NORM, "N": 0, "q": None, "k": None}.values()) == tq.TQ_OK


@pytest.fixture
def on_the_host(L, monkeypatch):
    """The binding as if the host were the current device, so that what it refuses by itself is seen without a GPU."""
    torch = pytest.importorskip("torch")
    types = {torch.float32: tq.TQ_F32, torch.float16: tq.TQ_F16, torch.bfloat16: tq.TQ_BF16}
    monkeypatch.setattr(tq, "_T", (torch, types, lambda dev: 0, lambda: -1))
    return torch


def test_binding_refuses_other_types_and_half_of_the_drafted_rows(on_the_host):
    torch = on_the_host
    x, pos = torch.zeros(2, 1, 128), torch.zeros(2, dtype=torch.int32)
    for q, out in ((x.double(), x), (x, x.double()), (x.int(), x)):
        with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
            tq.tq_qk_norm_rope(q, q, None, None, 1e-6, None, 0, pos, out, out)
    ctx = types.SimpleNamespace(d=128, handle=None)
    code = types.SimpleNamespace(desc=tq.Codes(), norm=x)

    def attend(q, k, v, **kw):
        tq.tq_tree_attention(ctx, ctx, q, k, v, pos, None, code, code, pos[:1], None, 16, 1.0, q, x, **kw)

    for k, v, kw in ((x, None, {}), (None, x, {}), (None, x, dict(Hkv=1)), (None, None, {})):
        with pytest.raises(ValueError, match="together"):
            attend(x, k, v, **kw)
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        attend(x.double(), x.double(), x.double())


def test_binding_refuses_code_sets_of_another_device(on_the_host):
    torch = on_the_host
    x, n = torch.zeros(2, 1, 128), torch.zeros(2, dtype=torch.int32)
    ctx = types.SimpleNamespace(d=128, handle=None)
    here = types.SimpleNamespace(desc=tq.Codes(), norm=torch.zeros(4))
    there = types.SimpleNamespace(desc=tq.Codes(), norm=types.SimpleNamespace(get_device=lambda: 1))
    for K, V, name in ((there, here, "K"), (here, there, "V")):
        with pytest.raises(ValueError, match=name + ": a code set on the current device"):
            tq.tq_tree_attention(ctx, ctx, x, x, x, n, None, K, V, n[:1], None, 16, 1.0, x, x)
    with pytest.raises(ValueError, match="codes: a code set on the current device"):
        tq.tq_encode_slots(ctx, x, n.long(), 16, there)


def test_null_contexts_are_refused(L):
    c = tq.Codes()
    n = ctypes.c_size_t()
    assert L.tq_encode_slots(None, A, 0, 1, 1, A, 16, ctypes.byref(c), None) == -1
    assert L.tq_tree_attention_workspace_size(None, 1, 1, 1, 1, ctypes.byref(n)) == -1
    assert L.tq_tree_attention(None, None, A, 128, A, 128, A, 128, 1, 1, A, None, 0, ctypes.byref(c), ctypes.byref(c), A,
                               A, 1, 16, 1, 1, 1, 1.0, A, A, 1 << 30, None) == -1


def test_rope_frequencies_are_fractions_of_a_turn(L):
    inv = np.concatenate([1e4 ** (-np.arange(0, 128, 2) / 128), [0.0, 2 * np.pi, -1.0, 7.0]])
    out = np.empty(inv.size, dtype=np.uint64)
    assert L.tq_rope_frequencies(inv.size, tq._ptr(inv), tq._ptr(out)) == tq.TQ_OK
    turn = inv / (2 * np.pi) % 1.0
    back = out.astype(np.float64) / 2.0 ** 64
    # a turn is two operations in 64 bits away; an angle close to a whole turn may come out on either side of it
    off = np.abs(back - turn)
    assert np.minimum(off, 1 - off).max() <= 4 * 2.0 ** -53
    assert L.tq_rope_frequencies(1, tq._ptr(np.array([np.inf])), tq._ptr(out)) == -1
    assert L.tq_rope_frequencies(-1, tq._ptr(inv), tq._ptr(out)) == -1
    assert L.tq_rope_frequencies(1, None, tq._ptr(out)) == -1
    assert L.tq_rope_frequencies(0, None, None) == tq.TQ_OK


def test_rope_frequencies_to_the_last_place(L):
    """Within one unit of frac(f/2π)·2^64, whose exact value is worked out in integers."""
    bits = 1300  # the smallest double has its last place at 2^-1074

    def arctan_of_inverse(n):  # the sum of (-1)^k / ((2k + 1) n^(2k + 1)), times 2^bits
        total, term, k = 0, (1 << bits) // n, 0
        while term:
            total += -(term // (2 * k + 1)) if k % 2 else term // (2 * k + 1)
            term, k = term // (n * n), k + 1
        return total

    pi = 16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239)
    inv = np.concatenate([1e6 ** (-np.arange(0, 128, 2) / 128), -1e4 ** (-np.arange(0, 64, 2) / 64),
                          [1.0, -1.0, 7.0, 0.0, 1e-30, -1e-30, 2 * np.pi, np.pi, 1000.5, 1e9, 1e12, 5e-324]])
    out = np.empty(inv.size, dtype=np.uint64)
    assert L.tq_rope_frequencies(inv.size, tq._ptr(inv), tq._ptr(out)) == tq.TQ_OK
    for f, got in zip(inv.tolist(), out.tolist()):
        n, d = f.as_integer_ratio()
        exact = (n << (bits + 63 + 64)) // (d * pi)  # f/2π·2^64 with 64 places behind the point
        off = ((got << 64) - exact) % (1 << 128)
        assert min(off, (1 << 128) - off) <= 1 << 64, (f, got)


def test_old_calls_keep_their_types(L):
    """bf16 is a type of the serving calls only; the encoder refuses it before it looks at anything else."""
    assert tq.TQ_BF16 == 2
