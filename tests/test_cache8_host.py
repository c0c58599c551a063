"""The 8-bit cache's calls: checks of their arguments, without a GPU.  Every refused call returns before anything is
launched, so its device addresses are made up."""

import ctypes
import os

import pytest

import kv_cache_vector_tq_gb300 as tq

A = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(tq.LIB_PATH):
        from kv_cache_vector_tq_gb300 import build
        build.build()
    return tq.lib()


CACHE = dict(d_k=A, d_v=A, d_kscale=A, d_vscale=A, d_status=A, pages=4, Hkv=2, block=16, d=128)
APPEND = dict(q=A, qs=4 * 128, k=A, ks=2 * 128, v=A, vs=2 * 128, dt=1, rows=3, Hq=4, wq=A, wk=None, eps=1e-6, freq=A,
              rot=128, style=0, pos=A, start=A, len=A, table=A, width=4, B=2, cache=None, qo=A, qos=512, stream=None)
ATTEND = dict(q=A, qs=4 * 128, dt=1, rows=3, start=A, len=A, table=A, width=4, B=2, Hq=4, cache=None, scale=1.0,
              window=0, sinks=0, out=A, ws=A, n=1 << 40, stream=None)
BAD_CACHE = [(dict(pages=0), -1), (dict(Hkv=0), -1), (dict(block=0), -1), (dict(d=0), -1), (dict(d_k=None), -1),
             (dict(d_v=A + 8), -1), (dict(d_kscale=None), -1), (dict(d_vscale=A + 2), -1), (dict(d_status=A + 1), -1),
             (dict(d=96), -2), (dict(d=256), -2), (dict(block=24), -2), (dict(block=1040), -2)]


def call(fn, args, change, cache):
    d = tq.Cache8Desc(**{**CACHE, **cache})
    return fn(*{**args, **change, "cache": ctypes.byref(d)}.values())


@pytest.mark.parametrize("cache,status", BAD_CACHE)
def test_bad_caches(L, cache, status):
    assert call(L.tq_cache8_append, APPEND, {}, cache) == status
    assert call(L.tq_cache8_attention, ATTEND, {}, cache) == status
    n = ctypes.c_size_t()
    d = tq.Cache8Desc(**{**CACHE, **cache})
    assert L.tq_cache8_attention_workspace_size(ctypes.byref(d), 2, 4, 3, ctypes.byref(n)) == status


@pytest.mark.parametrize("change,status", [
    (dict(dt=3), -1), (dict(rows=-1), -1), (dict(Hq=-1), -1), (dict(B=0), -1), (dict(width=0), -1), (dict(rot=-16), -1),
    (dict(rot=144), -1), (dict(style=2), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(eps=0.0), -1), (dict(qs=511), -1), (dict(ks=255), -1), (dict(vs=255), -1),
    (dict(qos=511), -1), (dict(q=None), -1), (dict(qo=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(pos=None), -1), (dict(start=None), -1), (dict(len=None), -1), (dict(table=None), -1), (dict(freq=None), -1),
    (dict(q=A + 8), -1), (dict(k=A + 8), -1), (dict(v=A + 8), -1), (dict(qo=A + 2), -1), (dict(wq=A + 4), -1),
    (dict(freq=A + 4), -1), (dict(pos=A + 2), -1), (dict(len=A + 1), -1), (dict(qs=516), -1), (dict(ks=257), -1),
    (dict(vs=260), -1), (dict(rot=24), -2), (dict(rows=2 ** 31 - 255), -2), (dict(width=2 ** 31 - 1), -2)])
def test_append_refusals(L, change, status):
    assert call(L.tq_cache8_append, APPEND, change, {}) == status


@pytest.mark.parametrize("change,status", [
    (dict(dt=3), -1), (dict(rows=-1), -1), (dict(Hq=0), -1), (dict(Hq=3), -1), (dict(B=0), -1), (dict(width=0), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(qs=511), -1), (dict(qs=516), -1), (dict(q=None), -1), (dict(out=None), -1),
    (dict(ws=None), -1), (dict(start=None), -1), (dict(len=None), -1), (dict(table=None), -1), (dict(q=A + 8), -1),
    (dict(out=A + 8), -1), (dict(ws=A + 8), -1), (dict(start=A + 2), -1), (dict(n=16), -1),
    (dict(rows=2 ** 29), -2), (dict(width=2 ** 31 - 1), -2)])
def test_attention_refusals(L, change, status):
    assert call(L.tq_cache8_attention, ATTEND, change, {}) == status


def test_nothing_to_do_is_fine(L):
    assert call(L.tq_cache8_append, APPEND, dict(rows=0, q=None, k=None, v=None, pos=None), {}) == tq.TQ_OK
    assert call(L.tq_cache8_attention, ATTEND, dict(rows=0, q=None, out=None, ws=None), {}) == tq.TQ_OK
    assert L.tq_cache8_append(*APPEND.values()) == tq.TQ_ERR_INVALID_ARG  # no cache
    assert L.tq_cache8_attention(*ATTEND.values()) == tq.TQ_ERR_INVALID_ARG


def test_sizes_past_what_the_kernels_count(L):
    for change, cache in ((dict(B=65537), {}), ({}, dict(pages=2 ** 30)), (dict(width=2 ** 20, qs=2 ** 12 * 128, Hq=2 ** 12), dict(Hkv=2 ** 12, block=1024, pages=1))):
        assert call(L.tq_cache8_attention, ATTEND, change, cache) == tq.TQ_ERR_UNSUPPORTED
    assert call(L.tq_cache8_append, APPEND, dict(B=65537), {}) == tq.TQ_ERR_UNSUPPORTED
