// Rows of d elements, d/8 lanes each: loads, stores, norms and the position
// rotation, shared by the kernels that norm and turn queries and keys.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "tq_device.cuh"

namespace tq {

constexpr int kNrThreads = 256;

struct NormRopeParams {
  const void *q, *k, *wq, *wk;
  void *qo, *ko;
  const uint64_t* freq;
  const int32_t* pos;
  int64_t N, qs, ks, qos, kos;  // strides between tokens in elements
  int Hq, Hkv, d, rot, style;
  int chunk, chunks;  // heads per warp, warps per token
  float eps;
};

// Four elements as they lie in memory, and as fp32.
template <typename T>
using Raw4 = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;

template <typename T>
__device__ __forceinline__ void widen4(const Raw4<T>& r, float* v) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  } else {
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 f;
      if constexpr (std::is_same<T, __half>::value)
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else
        f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        w[i] = h2_bits(__floats2half2_rn(v[2 * i], v[2 * i + 1]));
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// LPR lanes per row (the power of two at or above d/8).  Rows come by asynchronous
// copies into slots of shared memory that are each lane's own (no barrier),
// kNrAhead lane groups of rows ahead of the one in use: 32 warps with eight times
// 512 bytes each cover the memory's latency several times over.
template <typename TI>
constexpr int kNrAhead = sizeof(TI) == 4 ? 4 : 8;

template <int BYTES>
__device__ __forceinline__ void nr_copy(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}

template <typename TI>
struct NrSlot {
  Raw4<TI> a, b;
};

// Cosines and sines of lane l's four pairs at a position (1 and 0 past `rot`).
__device__ __forceinline__ void turn_angles(uint64_t pos, const uint64_t* freq, int l, bool turns, float (&cs)[4],
                                            float (&sn)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (turns) {
      const uint64_t t = pos * freq[4 * l + e];
      sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f /* 2^-31 */, &sn[e], &cs[e]);
    }
  }
}

// The factors of a lane's pairs with the weights inside:
// z_a = r·(x_a·ca - x_b·sb), z_b = r·(x_b·cb + x_a·sa)
struct TurnFactors {
  float ca[4], sa[4], cb[4], sb[4];
};
template <typename TI, bool HALF>
__device__ __forceinline__ TurnFactors turn_factors(const TI* w, bool in, int ja, int jb, const float (&cs)[4],
                                                    const float (&sn)[4]) {
  using Raw = Raw4<TI>;
  TurnFactors f;
  float wv[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  if (in && w) {
    widen4<TI>(*reinterpret_cast<const Raw*>(w + ja), wv);
    widen4<TI>(*reinterpret_cast<const Raw*>(w + jb), wv + 4);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float wa = HALF ? wv[e] : wv[2 * e], wb = HALF ? wv[4 + e] : wv[2 * e + 1];
    f.ca[e] = wa * cs[e];
    f.sa[e] = wa * sn[e];
    f.cb[e] = wb * cs[e];
    f.sb[e] = wb * sn[e];
  }
  return f;
}

// Norm (with NORM) and rotation of a row over its LPR lanes; whole warps call it.
template <int LPR, bool HALF, bool NORM>
__device__ __forceinline__ void turn_row(float (&x)[8], const TurnFactors& f, bool turns, float inv_d, float eps,
                                         float (&z)[8]) {
  float ss = 0.f;
  if constexpr (NORM) {
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
  }
  float r = NORM ? rsqrtf(fmaf(ss, inv_d, eps)) : 1.f;
  if (NORM && __any_sync(kFull, !(ss < 1e36f))) {
    // squares past the fp32 range (or not numbers): once more with the row
    // scaled by the power of two that brings its largest magnitude to [1, 2)
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    int ex = 1;
    if (m > 0.f && m < INFINITY) frexpf(m, &ex);
    const float sc = ldexpf(1.f, 1 - ex);
    float s2 = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s2 = fmaf(x[e] * sc, x[e] * sc, s2);
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) s2 += __shfl_xor_sync(kFull, s2, o);
    if (!(ss < 1e36f)) {  // x·r without the large x meeting the weights first
      r = rsqrtf(fmaf(s2, inv_d, eps * sc * sc)) * sc;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= r;
      r = 1.f;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = HALF ? e : 2 * e, k = HALF ? 4 + e : 2 * e + 1;
    // a lane past `rot` has sines 0, and no product with them
    const float a = turns ? fmaf(x[i], f.ca[e], -x[k] * f.sb[e]) : x[i] * f.ca[e];
    const float b = turns ? fmaf(x[k], f.cb[e], x[i] * f.sa[e]) : x[k] * f.cb[e];
    z[i] = a * r;
    z[k] = b * r;
  }
}

// The rows of CTA `cta`; tokens from `live` on are left alone.  Without NORM the
// rows are turned only.
template <typename TI, typename TO, int LPR, bool HALF, bool NORM>
__device__ __forceinline__ void norm_rope_rows(const NormRopeParams& p, int64_t cta, int64_t live,
                                               NrSlot<TI> (*ring)[kNrThreads]) {
  constexpr int RPW = 32 / LPR, A = kNrAhead<TI>;
  using Raw = Raw4<TI>;
  using Slot = NrSlot<TI>;
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int64_t job = cta * (kNrThreads / 32) + (threadIdx.x >> 5);
  if (job >= p.N * p.chunks) return;  // whole warps
  int64_t n = job;
  int h0 = 0;
  if (p.chunks > 1) {
    n = job <= 0xFFFFFFFFll ? (int64_t)((uint32_t)job / (uint32_t)p.chunks) : job / p.chunks;
    h0 = (int)(job - n * p.chunks) * p.chunk;
  }
  if (n >= live) return;
  const int h1 = min(h0 + p.chunk, p.Hq + p.Hkv);
  const bool in = 8 * l < p.d, turns = 8 * l < p.rot;
  // this lane's elements: ja.., jb.. (four each); half-split: partners of one another
  const int ja = HALF && turns ? 4 * l : 8 * l, jb = HALF && turns ? (p.rot >> 1) + 4 * l : 8 * l + 4;
  const TI* qrow = static_cast<const TI*>(p.q) + n * p.qs;
  const TI* krow = static_cast<const TI*>(p.k) + n * p.ks;
  auto fetch = [&](int h, int slot) {  // this lane's piece of head h
    if (in && h < h1) {
      const TI* src = h < p.Hq ? qrow + (int64_t)h * p.d : krow + (int64_t)(h - p.Hq) * p.d;
      Slot& s = ring[slot][threadIdx.x];
      nr_copy<(int)sizeof(Raw)>(&s.a, src + ja);
      nr_copy<(int)sizeof(Raw)>(&s.b, src + jb);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");  // always, so that the groups count the heads
  };
#pragma unroll
  for (int a = 0; a < A; ++a) fetch(h0 + a * RPW + sub, a);
  float cs[4], sn[4];
  turn_angles((uint64_t)(int64_t)p.pos[n], p.freq, l, turns, cs, sn);
  const float inv_d = 1.f / (float)p.d;
  TurnFactors f;
  int of = -1;  // whose weights they hold: 1 q, 0 k

  int slot = 0;
#pragma unroll 1
  for (int hb = h0; hb < h1; hb += RPW) {
    const int h = hb + sub;
    const bool isq = h < p.Hq;
    if (of != (int)isq) {
      of = isq;
      f = turn_factors<TI, HALF>(static_cast<const TI*>(isq ? p.wq : p.wk), in, ja, jb, cs, sn);
    }
    asm volatile("cp.async.wait_group %0;\n" ::"n"(A - 1) : "memory");
    float x[8];
    {
      Slot s{};
      if (in && h < h1) s = ring[slot][threadIdx.x];
      widen4<TI>(s.a, x);
      widen4<TI>(s.b, x + 4);
    }
    fetch(h + A * RPW, slot);  // the slot's words are in registers
    if (++slot == A) slot = 0;
    float z[8];
    turn_row<LPR, HALF, NORM>(x, f, turns, inv_d, p.eps, z);
    if (in && h < h1) {
      TO* dst = isq ? static_cast<TO*>(p.qo) + n * p.qos + (int64_t)h * p.d
                    : static_cast<TO*>(p.ko) + n * p.kos + (int64_t)(h - p.Hq) * p.d;
      store4(dst + ja, z);
      store4(dst + jb, z + 4);
    }
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");
}

}  // namespace tq
