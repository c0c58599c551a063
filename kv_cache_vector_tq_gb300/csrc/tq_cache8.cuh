// A paged cache held in 8 bits: what its kernels share.
//
// Codes are e4m3 numbers (four significant bits, 2^-9 to 448), one scale for
// every page, KV head and side; a token at position p of a request stands at
// place p % block of page table[p / block].  The scales are powers of two, so
// that dividing by one is exact and a block whose scale grows is rounded again
// only where codes fall below 2^-6.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

constexpr float kC8Lo = 8.673617379884035e-19f;  // 2^-60: the least scale
constexpr float kC8Hi = 1099511627776.f;         // 2^40: the largest

// A request's rows and length, cut to what the buffers hold.
struct C8Seq {
  int start, T, len;
};
__device__ __forceinline__ int c8_row(const int32_t* row_start, int b, int rows) {
  return min(max(row_start[b], 0), rows);
}
__device__ __forceinline__ C8Seq c8_seq(const int32_t* row_start, const int32_t* len, int b, int rows) {
  C8Seq s;
  s.start = c8_row(row_start, b, rows);
  s.T = max(c8_row(row_start, b + 1, rows) - s.start, 0);
  s.len = max(len[b], 0);
  return s;
}

// The request of slot x, where request b has the slots from key(b) =
// row_start[b]·num / den + 2b or b (`each`) on: enough for its blocks or row tiles,
// since floor(x) + floor(y) <= floor(x + y), and found without a sum over the
// requests.  Whole warps call it with one x.
__device__ __forceinline__ int c8_key(const int32_t* row_start, int b, int rows, int num, int den, int each) {
  return (int)((uint32_t)(c8_row(row_start, b, rows) * num) / (uint32_t)den) + each * b;  // (rows · num < 2^31)
}
__device__ __forceinline__ int c8_find(const int32_t* row_start, int B, int rows, int num, int den, int each, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool below = at < n && c8_key(row_start, lo + at, rows, num, den, each) <= x;
    const uint32_t m = __ballot_sync(kFull, below);
    const int i = m ? 31 - __clz(m) : 0;
    lo += i * step;
    n = min(step, n - i * step);
  }
  return lo;
}

// ------------------------------------------------------------------ attention
//   out_r = Σ_t w_rt v̂_t / Σ_t w_rt / s_t',  w_rt = 2^(z_rt + log2 s_t' - M_r),
//   z_rt = scale·log2(e)·s_t·⟨q_r, code_t⟩,  s, s' the scales of t's block (K, V)
// over the tokens t that row r sees: t <= p_r, and with a window W: t > p_r - W or
// t < sinks.  The V scale stands inside the exponent, so that weights meet the codes
// themselves and stay within fp16 for any scale; the sum of weights takes it out
// again, one factor for the tokens of a block.
//
// Work: a tile is up to `tile` rows of a request and KV head, a row being one
// (token, query head of the KV head) pair; its units are the 128-token pieces of
// the cache that some row of it sees.  The units of all tiles, laid end to end (and
// for each tile a few more, for what its beginning and end cost), are
// shared evenly among the CTAs of a grid that fits the GPU once, whatever the
// lengths are: lengths live on the device, so a captured call serves later ones.  A
// tile that one CTA has all of is written out by it; parts go to the CTAs' records,
// and a second kernel joins them.
constexpr int kC8Unit = 128;
constexpr float kC8Log2e = 1.4426950408889634f;

// A part of a tile that was begun by a CTA and not ended: where the rest is.
struct C8Split {
  int h, row0, nrow, start;  // h < 0: none; the tile's rows of the request's, the request's first token row
  int64_t u0, u1, units;     // its counted units among all
};

struct C8Params {
  const void* q;
  int64_t qs;  // stride between tokens in elements
  int dtype;
  const int32_t *row_start, *len, *table;
  int rows, B, Hq, Hkv, G, max_blocks, block, d, window, sinks;
  int64_t pages;
  const uint8_t *k8, *v8;
  const float *kscale, *vscale;
  float zscale;  // scale·log2(e)
  void* out;
  int32_t* status;
  C8Split* split;  // [ctas]
  // [ctas][2]: a tile that goes on from the CTA before, one that begins here; in each
  // [tile][d + 4]: m, l, 2 pad, sums, or from 128 rows on (a thread of the kernel has a
  // row) [tile] of m, l, then [d / 4][tile] of four sums; with 128 rows [ctas] more behind
  // them (long sums of the second softmax group)
  float* rec;
  int ctas, tile, slots;
  int pad;         // what a tile's beginning and end cost, in units: the CTAs' shares count it
};

// The rows and the tokens of a tile.
struct C8Tile {
  int b, rt, row0, nrow;  // of the request's T·G rows
  int start, len;
  int i0, il;             // first and last token of the rows
  int lo, hi;             // tokens seen by some row: [lo, hi), and [0, sinks) with a window
  int su, lou, n;         // units of the first tokens, first unit of lo (0 where both are one run), units
};
__device__ __forceinline__ C8Tile c8_tile(const C8Params& p, const int32_t* row_start, const int32_t* len, int b, int rt) {
  C8Tile t;
  const C8Seq s = c8_seq(row_start, len, b, p.rows);
  t.b = b;
  t.rt = rt;
  t.start = s.start;
  t.len = s.len;
  const int all = s.T * p.G;  // (rows · Hq < 2^31)
  t.n = t.nrow = 0;
  if (rt < 0 || (int64_t)rt * p.tile >= all) return t;
  const int row0 = rt * p.tile;
  t.nrow = min(all - row0, p.tile);
  t.row0 = row0;
  t.i0 = row0 / p.G;
  t.il = (row0 + t.nrow - 1) / p.G;
  const int cap = p.max_blocks * p.block;
  t.hi = (int)min((int64_t)s.len + t.il + 1, (int64_t)cap);
  t.lo = 0;
  t.su = t.lou = 0;
  const int hiu = (t.hi + kC8Unit - 1) / kC8Unit;
  t.n = hiu;
  if (p.window > 0) {
    t.lo = (int)min(max((int64_t)s.len + t.i0 - p.window + 1, (int64_t)0), (int64_t)cap);
    t.su = (min(p.sinks, t.hi) + kC8Unit - 1) / kC8Unit;
    t.lou = t.lo / kC8Unit;
    if (t.lou <= t.su)
      t.lou = t.su = 0;
    else
      t.n = t.su + max(hiu - t.lou, 0);
  }
  if (t.n < 1) t.n = 1;  // rows past the capacity see nothing: the unit is empty, the rows zero
  return t;
}
// First token of unit u of a tile.
__device__ __forceinline__ int c8_unit(const C8Tile& t, int u) {
  return (u < t.su ? u : t.lou + (u - t.su)) * kC8Unit;
}
// The tile of slot x, the units of which stand in t.n (0: none).
__device__ __forceinline__ int c8_slot_b(const C8Params& p, const int32_t* row_start, int x) {
  int lo = 0, n = p.B;  // as c8_find, by one thread
  while (n > 1) {
    const int half = n >> 1;
    if (c8_key(row_start, lo + half, p.rows, p.G, p.tile, 1) <= x) {
      lo += half;
      n -= half;
    } else {
      n = half;
    }
  }
  return lo;
}
__device__ __forceinline__ int64_t c8_cut(int64_t c, int64_t units, int64_t n) { return c * units / n; }

// What a CTA begins with: its units, and the slot (and units before the slot) of
// the first.  Called by all threads of a CTA of NT threads; `copy`: shared memory for
// `room` numbers, where offsets and lengths are brought at once if they fit (looked up
// one after the other in memory they took 3 us).
struct C8Share {
  int64_t u0, u1, units, before;
  int slot, b;  // the first unit's slot and request
};
template <int NT>
__device__ __forceinline__ C8Share c8_share(const C8Params& p, int64_t (*sums)[NT / 32 + 1], int64_t* found, int32_t* copy, int room) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  C8Share s;
  const int32_t *row_start = p.row_start, *len = p.len;
  if (2 * p.B + 1 <= room) {
    for (int i = tid; i <= p.B; i += NT) {
      copy[i] = p.row_start[i];
      if (i < p.B) copy[p.B + 1 + i] = p.len[i];
    }
    row_start = copy;
    len = copy + p.B + 1;
    __syncthreads();
  }
  int64_t total = 0, mine = 0, before = 0;
  int mine_b = 0;
  // all slots are summed; where they are more threads than one pass has, they are
  // counted again for the place of the first unit
  for (int again = 0; again < 2; ++again) {
    int64_t carry = 0;
    for (int x0 = 0; x0 < p.slots; x0 += NT) {
      const int x = x0 + tid;
      if (again == 0 || p.slots > NT) {
        mine = 0;
        if (x < p.slots) {
          const int b = mine_b = c8_slot_b(p, row_start, x);
          const int n = c8_tile(p, row_start, len, b, x - c8_key(row_start, b, p.rows, p.G, p.tile, 1)).n;
          if (n > 0) mine = (int64_t)(n + p.pad) * p.Hkv;
        }
        int64_t in = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t a = __shfl_up_sync(kFull, in, o);
          if (lane >= o) in += a;
        }
        __syncthreads();
        if (lane == 31) sums[0][warp] = in;
        __syncthreads();
        int64_t base = 0, all = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
          if (w < warp) base += sums[0][w];
          all += sums[0][w];
        }
        before = carry + base + in - mine;
        carry += all;
      }
      if (again == 1) {
        if (x < p.slots && mine > 0 && before <= s.u0 && s.u0 < before + mine) {
          found[0] = x | ((int64_t)mine_b << 32);
          found[1] = before;
        }
      }
    }
    if (again == 0) {
      total = carry;
      s.units = total;
      s.u0 = c8_cut(blockIdx.x, total, p.ctas);
      s.u1 = c8_cut(blockIdx.x + 1, total, p.ctas);
    }
  }
  fence_proxy_async();  // (copies may take the place of offsets and lengths next)
  __syncthreads();
  s.slot = (int)(found[0] & 0xFFFFFFFFll);
  s.b = (int)(found[0] >> 32);
  s.before = found[1];
  return s;
}

// A run of units of one tile and KV head: units [first, first + n) of it.
struct C8Seg {
  C8Tile t;
  int h, first, n;
  int64_t u0;  // the tile's first counted unit among all
};
struct C8Walk {
  int64_t u, u1, before;
  int slot, b;
};
__device__ __forceinline__ C8Walk c8_walk(const C8Params& p, const C8Share& s) {
  return C8Walk{s.u0, s.u1, s.before, s.slot, s.u0 < s.u1 ? s.b : 0};
}
__device__ __forceinline__ bool c8_next(const C8Params& p, C8Walk& w, C8Seg& g) {
  while (w.u < w.u1 && w.slot < p.slots) {
    g.t = c8_tile(p, p.row_start, p.len, w.b, w.slot - c8_key(p.row_start, w.b, p.rows, p.G, p.tile, 1));
    const int64_t all = g.t.n > 0 ? (int64_t)(g.t.n + p.pad) * p.Hkv : 0;
    if (w.u < w.before + all) {
      // the first `pad` of a tile's counted units are no units
      const int nv = g.t.n + p.pad, at = (int)(w.u - w.before);
      g.h = at / nv;
      const int v0 = at - g.h * nv, cnt = (int)min((int64_t)(nv - v0), w.u1 - w.u);
      g.first = max(v0 - p.pad, 0);
      g.n = max(v0 + cnt - p.pad, 0) - g.first;
      g.u0 = w.before + (int64_t)g.h * nv;
      w.u += cnt;
      if (g.n > 0) return true;
      continue;
    }
    w.before += all;
    ++w.slot;
    while (w.b + 1 < p.B && c8_key(p.row_start, w.b + 1, p.rows, p.G, p.tile, 1) <= w.slot) ++w.b;
  }
  return false;
}

// N (2 or 4) numbers as T, to memory in one access.
template <typename T>
__device__ __forceinline__ uint32_t c8_pair(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    return pack_f16x2(a, b);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T, int N>
__device__ __forceinline__ void c8_store(T* p, const float (&x)[N]) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (N == 4)
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  } else if constexpr (N == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(c8_pair<T>(x[0], x[1]), c8_pair<T>(x[2], x[3]));
  } else {
    *reinterpret_cast<uint32_t*>(p) = c8_pair<T>(x[0], x[1]);
  }
}
template <int N>
__device__ __forceinline__ void c8_load(const float* p, float (&x)[N]) {
  if constexpr (N == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x;
    x[1] = v.y;
  }
}
// Two codes as fp16: the low 16 bits of w, or the high ones.
__device__ __forceinline__ uint32_t c8_wide(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t c8_wide_hi(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
// The power of two that takes a row's largest magnitude to [2^10, 2^11): its exponent.
__device__ __forceinline__ int c8_row_exp(float top) {
  return top > 0.f && top < INFINITY ? max((__float_as_int(top) >> 23) - 127 - 10, -100) : 0;
}
__device__ __forceinline__ float c8_pow2(int e) { return __int_as_float((127 + e) << 23); }
// A V scale as the exponents take it (a NaN stays one).
__device__ __forceinline__ float c8_vscale(float s) { return s < kC8Lo ? kC8Lo : s > kC8Hi ? kC8Hi : s; }
// Its inverse, which the sum of a block's weights meets: 0 for a NaN.  Rows that see the
// block have the NaN in their weights (the scale stands in their exponents too); those
// that do not have weights of 0, and 0 times a NaN would be one.
__device__ __forceinline__ float c8_inverse(float s) { return s == s ? 1.f / s : 0.f; }

template <typename... P, typename... A>
inline cudaError_t c8_launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

cudaError_t c8_attend_umma(const C8Params& p, cudaStream_t st);

}  // namespace tq
