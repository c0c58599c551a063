"""TurboQuant hot path on GB300 (sm_103a): Python binding of the libtq C ABI.

The functions here marshal arguments (torch tensors -> device pointers, numpy
arrays -> host pointers) and call libtq.so; every step of the path runs in the
library's kernels.  The library is built in-tree by ``build.build()``; when it
is missing, ``lib()`` raises instead of falling back to anything else.
"""

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtq.so")

TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_CUDA, TQ_ERR_ALLOC, TQ_ERR_TIMEOUT = 0, -1, -2, -3, -4, -5
TQ_MSE, TQ_PROD, TQ_MIXED = 0, 1, 2
TQ_ROT_DENSE, TQ_ROT_HADAMARD = 0, 1
TQ_DENS_BETA, TQ_DENS_GAUSS = 0, 1
TQ_F32, TQ_F16, TQ_BF16 = 0, 1, 2
TQ_ROPE_HALF, TQ_ROPE_INTERLEAVED = 0, 1
TQ_LAYOUT_TOKEN, TQ_LAYOUT_PAIR = 0, 1

# every entry point of include/tq.h
EXPORTS = (
    "tq_version", "tq_status_string", "tq_last_cuda_error", "tq_codebook_build",
    "tq_rotation_haar", "tq_ctx_create", "tq_ctx_destroy", "tq_codes_layout", "tq_encode",
    "tq_scores_workspace_size", "tq_scores", "tq_decode_workspace_size",
    "tq_decode_attention", "tq_decode_step", "tq_decode_attention_noalloc", "tq_unpack_indices", "tq_status_poll",
    "tq_ctx_set_wait_limit", "tq_block_tables", "tq_rope_frequencies", "tq_qk_norm_rope", "tq_encode_slots",
    "tq_tree_attention_workspace_size", "tq_tree_attention",
)


class TqError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = _LIB.tq_status_string(status).decode() if _LIB else str(status)
        if status == TQ_ERR_CUDA and _LIB:
            msg += f" (cudaError {_LIB.tq_last_cuda_error()})"
        super().__init__(f"{fn}: {msg}")


class Codebook(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int), ("b", ctypes.c_int), ("density", ctypes.c_int),
        ("grid", ctypes.c_int), ("iters", ctypes.c_int),
        ("centroid", ctypes.c_double * 16), ("threshold", ctypes.c_double * 15),
        ("distortion", ctypes.c_double),
    ]


class Codes(ctypes.Structure):
    _fields_ = [
        ("d_codes", ctypes.c_void_p), ("d_norm", ctypes.c_void_p),
        ("d_qjl", ctypes.c_void_p), ("d_rnorm", ctypes.c_void_p),
        ("n", ctypes.c_int64), ("d", ctypes.c_int), ("b_mse", ctypes.c_int),
        ("mode", ctypes.c_int), ("layout", ctypes.c_int),
        ("words_per_vec", ctypes.c_int), ("qjl_words_per_vec", ctypes.c_int),
    ]


_LIB = None
_vp, _i, _i64, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


def lib():
    """Load libtq.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libtq.so is not built ({LIB_PATH}); run kv_cache_vector_tq_gb300.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    sig = {
        "tq_version": ([], ctypes.c_char_p),
        "tq_status_string": ([_i], ctypes.c_char_p),
        "tq_last_cuda_error": ([], _i),
        "tq_codebook_build": ([_i, _i, _i, _i, _i, P(Codebook)], _i),
        "tq_rotation_haar": ([_i, _vp, _vp], _i),
        "tq_ctx_create": ([_i, _i, _i, _i, _vp, _vp, P(Codebook), P(_vp)], _i),
        "tq_ctx_destroy": ([_vp], _i),
        "tq_codes_layout": ([_vp, _i, _i64, P(Codes), P(_sz), P(_sz), P(_sz), P(_sz)], _i),
        "tq_encode": ([_vp, _vp, _i, _i64, P(Codes), _i64, _i64, _i64, _vp], _i),
        "tq_scores_workspace_size": ([_vp, _i, P(_sz)], _i),
        "tq_scores": ([_vp, _vp, _i, P(Codes), _i64, _i64, _vp, _vp, _sz, _vp], _i),
        "tq_decode_workspace_size": ([_vp, _i, _i, _i, _i64, P(_sz)], _i),
        "tq_decode_attention": ([_vp, _vp, _vp, _i, P(Codes), P(Codes), _i, _i, _i, _i64, _i64,
                                 _f, _vp, _vp, _sz, _vp], _i),
        "tq_decode_step": ([_vp, _vp, _vp, _i, _vp, _vp, _i, P(Codes), P(Codes), _i, _i, _i, _i64,
                            _i64, _f, _vp, _vp, _sz, _vp], _i),
        "tq_decode_attention_noalloc": ([_vp, _vp, _vp, _i, P(Codes), P(Codes), _i, _i, _i, _i64,
                                         _i64, _f, _vp, _vp], _i),
        "tq_unpack_indices": ([P(Codes), _i64, _i64, _vp, _vp], _i),
        "tq_status_poll": ([_vp, _vp], _i),
        "tq_ctx_set_wait_limit": ([_vp, ctypes.c_uint32], _i),
        "tq_block_tables": ([_vp, _vp, _vp, _i, _i, _vp, _i64, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i64, _vp], _i),
        "tq_rope_frequencies": ([_i, _vp, _vp], _i),
        "tq_qk_norm_rope": ([_vp, _i64, _vp, _i64, _i, _i64, _i, _i, _i, _vp, _vp, _f, _vp, _i, _i, _vp, _vp, _i64,
                             _vp, _i64, _i, _vp], _i),
        "tq_encode_slots": ([_vp, _vp, _i, _i64, _i, _vp, _i, P(Codes), _vp], _i),
        "tq_tree_attention_workspace_size": ([_vp, _i, _i, _i, _i64, P(_sz)], _i),
        "tq_tree_attention": ([_vp, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _i, _i64, _vp, _vp, _i, P(Codes), P(Codes),
                               _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _sz, _vp], _i),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _LIB = L
    return L


def _check(fn, st):
    if st != TQ_OK:
        raise TqError(fn, st)


def _ptr(a):
    """Host pointer of a contiguous numpy array."""
    return a.ctypes.data_as(ctypes.c_void_p)


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


# ---------------------------------------------------------------- host calls
def tq_version():
    return lib().tq_version().decode()


def tq_codebook_build(d, b, density=TQ_DENS_BETA, grid=0, iters=0):
    cb = Codebook()
    _check("tq_codebook_build", lib().tq_codebook_build(d, b, density, grid, iters, ctypes.byref(cb)))
    return cb


def tq_rotation_haar(G):
    import numpy as np
    G = np.ascontiguousarray(G, dtype=np.float64)
    d = G.shape[0]
    Pi = np.empty((d, d), dtype=np.float64)
    _check("tq_rotation_haar", lib().tq_rotation_haar(d, _ptr(G), _ptr(Pi)))
    return Pi


class Context:
    """Owns a tq_ctx (device tables for one (d, b, mode, rotation)).  TQ_MIXED
    (b + 1/2 bits per coordinate) passes the b-bit and (b+1)-bit codebooks."""

    def __init__(self, d, b, mode, rot_kind, rot, S=None, codebook=None):
        import numpy as np
        rot = np.ascontiguousarray(rot, dtype=np.float64)
        S = None if S is None else np.ascontiguousarray(S, dtype=np.float64)
        self.d, self.b, self.mode, self.rot_kind = d, b, mode, rot_kind
        self.b_mse = b - 1 if mode == TQ_PROD else b
        if mode == TQ_MIXED:
            pair = (Codebook * 2)()
            pair[0] = tq_codebook_build(d, b) if codebook is None else codebook[0]
            pair[1] = tq_codebook_build(d, b + 1) if codebook is None else codebook[1]
            self.codebook = pair
        else:
            self.codebook = codebook if codebook is not None else tq_codebook_build(d, self.b_mse)
        h = ctypes.c_void_p()
        cbp = (ctypes.cast(self.codebook, ctypes.POINTER(Codebook)) if mode == TQ_MIXED
               else ctypes.byref(self.codebook))
        _check("tq_ctx_create", lib().tq_ctx_create(
            d, b, mode, rot_kind, _ptr(rot), _ptr(S) if S is not None else None, cbp, ctypes.byref(h)))
        self.handle = h

    def close(self):
        if self.handle:
            _check("tq_ctx_destroy", lib().tq_ctx_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_wait_limit(self, polls):
        """Bound of the context's pipeline waits (tq_ctx_set_wait_limit)."""
        _check("tq_ctx_set_wait_limit", lib().tq_ctx_set_wait_limit(self.handle, int(polls)))

    def poll(self, stream=None):
        st = lib().tq_status_poll(self.handle, _stream(stream))
        return st


class CodeSet:
    """Packed codes of n vectors in device memory (torch tensors)."""

    def __init__(self, ctx, n, layout=TQ_LAYOUT_TOKEN, device="cuda"):
        import torch
        desc = Codes()
        sizes = [ctypes.c_size_t() for _ in range(4)]
        _check("tq_codes_layout", lib().tq_codes_layout(ctx.handle, layout, n, ctypes.byref(desc),
                                                        *[ctypes.byref(s) for s in sizes]))
        cb, nb, qb, rb = (s.value for s in sizes)
        self.codes = torch.zeros(max(cb // 4, 4), dtype=torch.int32, device=device)
        self.norm = torch.zeros(max(nb // 4, 4), dtype=torch.float32, device=device)
        self.qjl = torch.zeros(max(qb // 4, 4), dtype=torch.int32, device=device) if qb else None
        self.rnorm = torch.zeros(max(rb // 4, 4), dtype=torch.float32, device=device) if rb else None
        desc.d_codes = self.codes.data_ptr()
        desc.d_norm = self.norm.data_ptr()
        desc.d_qjl = self.qjl.data_ptr() if self.qjl is not None else None
        desc.d_rnorm = self.rnorm.data_ptr() if self.rnorm is not None else None
        self.desc = desc
        self.n, self.layout, self.ctx = n, layout, ctx

    @property
    def words_per_vec(self):
        return self.desc.words_per_vec


# ---------------------------------------------------------------- device calls
def tq_encode(ctx, x, codes, offset=0, group_rows=None, group_stride=0, stream=None):
    import torch
    assert x.is_cuda and x.is_contiguous()
    dt = {torch.float32: TQ_F32, torch.float16: TQ_F16}[x.dtype]
    N = x.shape[0] if x.dim() == 2 else x.numel() // ctx.d
    gr = N if group_rows is None else group_rows
    _check("tq_encode", lib().tq_encode(ctx.handle, ctypes.c_void_p(x.data_ptr()), dt, N,
                                        ctypes.byref(codes.desc), offset, max(gr, 1), group_stride,
                                        _stream(stream)))


def tq_scores_workspace_size(ctx, M):
    n = ctypes.c_size_t()
    _check("tq_scores_workspace_size", lib().tq_scores_workspace_size(ctx.handle, M, ctypes.byref(n)))
    return n.value


def tq_scores(ctx, q, keys, out, ws, first=0, N=None, stream=None):
    N = keys.n - first if N is None else N
    M = q.shape[0]
    _check("tq_scores", lib().tq_scores(ctx.handle, ctypes.c_void_p(q.data_ptr()), M,
                                        ctypes.byref(keys.desc), first, N,
                                        ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(ws.data_ptr()),
                                        ws.numel() * ws.element_size(), _stream(stream)))


def tq_decode_workspace_size(kctx, B, Hq, Hkv, seq):
    n = ctypes.c_size_t()
    _check("tq_decode_workspace_size",
           lib().tq_decode_workspace_size(kctx.handle, B, Hq, Hkv, seq, ctypes.byref(n)))
    return n.value


def tq_decode_attention(kctx, vctx, q, K, V, B, Hq, Hkv, seq, cap, scale, out, ws, stream=None):
    import torch
    dt = {torch.float32: TQ_F32, torch.float16: TQ_F16}[q.dtype]
    _check("tq_decode_attention", lib().tq_decode_attention(
        kctx.handle, vctx.handle, ctypes.c_void_p(q.data_ptr()), dt, ctypes.byref(K.desc),
        ctypes.byref(V.desc), B, Hq, Hkv, seq, cap, float(scale), ctypes.c_void_p(out.data_ptr()),
        ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(), _stream(stream)))


def tq_decode_step(kctx, vctx, q, k_new, v_new, K, V, B, Hq, Hkv, seq, cap, scale, out, ws, stream=None):
    """Append k_new/v_new ([B, Hkv, d]) at position seq-1, then attend over seq tokens."""
    import torch
    dts = {torch.float32: TQ_F32, torch.float16: TQ_F16}
    assert k_new.dtype == v_new.dtype
    _check("tq_decode_step", lib().tq_decode_step(
        kctx.handle, vctx.handle, ctypes.c_void_p(q.data_ptr()), dts[q.dtype],
        ctypes.c_void_p(k_new.data_ptr()), ctypes.c_void_p(v_new.data_ptr()), dts[k_new.dtype],
        ctypes.byref(K.desc), ctypes.byref(V.desc), B, Hq, Hkv, seq, cap, float(scale),
        ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(),
        _stream(stream)))


def tq_decode_attention_noalloc(kctx, vctx, q, K, V, B, Hq, Hkv, seq, cap, scale, out, stream=None):
    """tq_decode_attention without a workspace (scratch built into the library)."""
    import torch
    dt = {torch.float32: TQ_F32, torch.float16: TQ_F16}[q.dtype]
    _check("tq_decode_attention_noalloc", lib().tq_decode_attention_noalloc(
        kctx.handle, vctx.handle, ctypes.c_void_p(q.data_ptr()), dt, ctypes.byref(K.desc),
        ctypes.byref(V.desc), B, Hq, Hkv, seq, cap, float(scale), ctypes.c_void_p(out.data_ptr()),
        _stream(stream)))


# ---------------------------------------------------------------- serving
# These calls are a few microseconds of GPU time each, so the binding looks at
# every tensor once and asks the runtime for as little as it can.
_T = None


def _types():
    """(torch, its type -> tq type, the raw current stream of a device, the current device), once torch is wanted."""
    global _T
    if _T is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        stream = raw if raw else (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        dev = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _T = torch, {torch.float32: TQ_F32, torch.float16: TQ_F16, torch.bfloat16: TQ_BF16}, stream, dev
    return _T


def _raw_stream(stream, dev):
    if stream is None:
        return _T[2](dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t, dtype, n, what, dev):
    """Device address of a contiguous tensor of this type with n elements or more, on this device."""
    if t.dtype is not dtype or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous CUDA tensor of {dtype} with {n} elements or more, on the current "
                         f"device, is wanted")
    return t.data_ptr()


def _heads(t, n, h, d, what, dev):
    """Address and token stride of a [n, h, d] tensor on this device whose heads are contiguous."""
    a, b, c = t.stride()
    if t.get_device() != dev or t.shape != (n, h, d) or c != 1 or (b != d and h > 1):
        raise ValueError(f"{what}: a CUDA tensor [{n}, {h}, {d}] with contiguous heads, on the current device, is wanted")
    return t.data_ptr(), a if n > 1 else h * d


def _codes(c, what, dev):
    """Descriptor of a code set on this device."""
    if c.norm.get_device() != dev:
        raise ValueError(f"{what}: a code set on the current device is wanted")
    return ctypes.byref(c.desc)


def _type(t, what):
    """The tq type of a tensor."""
    ty = _T[1].get(t.dtype)
    if ty is None:
        raise ValueError(f"{what}: float32, float16 or bfloat16 is wanted")
    return ty


def tq_block_tables(lens, new, held, ring, state, table, block, held_out, state_out, row_start, slots, pos,
                    stream=None):
    """Pages, slots and positions of one step's tokens (include/tq.h).  table [B, max_blocks], ring, lens, new, held,
    held_out, row_start and pos are int32, state, state_out and slots int64; pos and slots have one entry per row."""
    torch, _, _, cur = _types()
    dev = cur()
    i32, i64, B = torch.int32, torch.int64, lens.numel()
    _check("tq_block_tables", lib().tq_block_tables(
        _dev(lens, i32, B, "lens", dev), _dev(new, i32, B, "new", dev), _dev(held, i32, B, "held", dev), B, block,
        _dev(ring, i32, 1, "ring", dev), ring.numel(), _dev(state, i64, 2, "state", dev),
        _dev(table, i32, B * table.shape[-1], "table", dev), table.shape[-1], _dev(held_out, i32, B, "held_out", dev),
        _dev(state_out, i64, 2, "state_out", dev), _dev(row_start, i32, B + 1, "row_start", dev),
        _dev(slots, i64, 0, "slots", dev), _dev(pos, i32, slots.numel(), "pos", dev), slots.numel(), _raw_stream(stream, dev)))


def tq_rope_frequencies(inv_freq, device="cuda"):
    """Frequencies (radians per position, fp64) as 64-bit fractions of a turn, on the device (int64 words)."""
    import numpy as np
    import torch
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    out = np.empty(f.size, dtype=np.uint64)
    _check("tq_rope_frequencies", lib().tq_rope_frequencies(f.size, _ptr(f), _ptr(out)))
    return torch.from_numpy(out.view(np.int64)).to(device)


def tq_qk_norm_rope(q, k, wq, wk, eps, freq, style, pos, q_out, k_out, stream=None):
    """Head norms and position rotation of q [N, Hq, d] and k [N, Hkv, d] into q_out and k_out (include/tq.h).
    wq, wk: [d] of q's type or None; freq: tq_rope_frequencies or None (norms alone); outputs may be the inputs."""
    torch, _, _, cur = _types()
    dev = cur()
    (N, Hq, d), Hkv, ti, to = q.shape, k.shape[1], q.dtype, q_out.dtype
    if k.dtype is not ti or k_out.dtype is not to:
        raise ValueError("q and k, and q_out and k_out, are of one type")
    (qp, qs), (kp, ks) = _heads(q, N, Hq, d, "q", dev), _heads(k, N, Hkv, d, "k", dev)
    (qo, qos), (ko, kos) = _heads(q_out, N, Hq, d, "q_out", dev), _heads(k_out, N, Hkv, d, "k_out", dev)
    _check("tq_qk_norm_rope", lib().tq_qk_norm_rope(
        qp, qs, kp, ks, _type(q, "q"), N, Hq, Hkv, d, None if wq is None else _dev(wq, ti, d, "wq", dev),
        None if wk is None else _dev(wk, ti, d, "wk", dev), eps,
        None if freq is None else _dev(freq, torch.int64, 0, "freq", dev), 0 if freq is None else 2 * freq.numel(), style,
        _dev(pos, torch.int32, N, "pos", dev), qo, qos, ko, kos, _type(q_out, "q_out"), _raw_stream(stream, dev)))


def tq_encode_slots(ctx, x, slots, block, codes, stream=None):
    """tq_encode of x [N, Hkv, d] into a paged cache, token i at slots[i] (include/tq.h)."""
    torch, types, _, cur = _types()
    dev = cur()
    N, Hkv, d = x.shape
    if d != ctx.d:
        raise ValueError(f"x: rows of {ctx.d} elements are wanted")
    ti = x.dtype
    if ti is not torch.float32 and ti is not torch.float16:
        raise ValueError("x: float32 or float16 is wanted")
    _check("tq_encode_slots", lib().tq_encode_slots(
        ctx.handle, _dev(x, ti, 0, "x", dev), types[ti], N, Hkv, _dev(slots, torch.int64, N, "slots", dev), block,
        _codes(codes, "codes", dev), _raw_stream(stream, dev)))


def tq_tree_attention_workspace_size(kctx, B, Hq, Hkv, rows):
    n = ctypes.c_size_t()
    _check("tq_tree_attention_workspace_size",
           lib().tq_tree_attention_workspace_size(kctx.handle, B, Hq, Hkv, rows, ctypes.byref(n)))
    return n.value


def tq_tree_attention(kctx, vctx, q, k_new, v_new, row_start, mask, K, V, lens, table, block, scale, out, ws,
                      Hkv=None, stream=None):
    """Attention of drafted tokens q [rows, Hq, d] over a packed cache and each other (include/tq.h).  k_new, v_new
    [rows, Hkv, d] or None (Hkv is then given); mask [rows, words] int32 or None (a chain); table [B, max_blocks] or
    None (contiguous, cap = block)."""
    torch, _, _, cur = _types()
    dev = cur()
    rows, Hq, d = q.shape
    if d != kctx.d:
        raise ValueError(f"q: rows of {kctx.d} elements are wanted")
    ti = q.dtype
    if (k_new is None) != (v_new is None) or (k_new is None and Hkv is None):
        raise ValueError("k_new and v_new are given together, or neither of them and Hkv")
    B, Hkv = lens.numel(), k_new.shape[1] if k_new is not None else Hkv
    qp, qs = _heads(q, rows, Hq, d, "q", dev)
    kp = vp = None
    ks = vs = 0
    if k_new is not None:
        if k_new.dtype is not ti or v_new.dtype is not ti:
            raise ValueError("q, k_new and v_new are of one type")
        (kp, ks), (vp, vs) = _heads(k_new, rows, Hkv, d, "k_new", dev), _heads(v_new, rows, Hkv, d, "v_new", dev)
    i32 = torch.int32
    words, width = 0 if mask is None else mask.shape[1], 0 if table is None else table.shape[1]
    _check("tq_tree_attention", lib().tq_tree_attention(
        kctx.handle, vctx.handle, qp, qs, kp, ks, vp, vs, _type(q, "q"), rows, _dev(row_start, i32, B + 1, "row_start", dev),
        None if mask is None else _dev(mask, i32, rows * words, "mask", dev), words, _codes(K, "K", dev),
        _codes(V, "V", dev), _dev(lens, i32, B, "lens", dev),
        None if table is None else _dev(table, i32, B * width, "table", dev), width, block, B, Hq, Hkv, scale,
        _dev(out, ti, rows * Hq * d, "out", dev), _dev(ws, ws.dtype, 0, "ws", dev), ws.numel() * ws.element_size(),
        _raw_stream(stream, dev)))


def tq_unpack_indices(codes, first=0, count=None, with_bits=False):
    import numpy as np
    count = codes.n - first if count is None else count
    idx = np.zeros((count, codes.desc.d), dtype=np.uint8)
    bits = np.zeros((count, codes.desc.d), dtype=np.uint8) if with_bits else None
    _check("tq_unpack_indices", lib().tq_unpack_indices(ctypes.byref(codes.desc), first, count,
                                                        _ptr(idx), _ptr(bits) if with_bits else None))
    return (idx, bits) if with_bits else idx
