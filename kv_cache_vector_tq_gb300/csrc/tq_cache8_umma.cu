// Attention over the 8-bit paged cache on the fifth-generation tensor cores:
// prompts, their pieces and longer drafted chains of fp16 and bf16 calls.
// tq_cache8.cuh has the mathematics and the division of the work.
//
// A persistent CTA per SM; per unit of 128 tokens and 128 rows (token x query head)
// on the lanes of tensor memory:
//     S[row][token]  = Q·Kᵀ        A = Q (shared memory), B = K (shared memory)
//     P[row][token]  = 2^(z - M)   in fp16, over S in tensor memory
//     O[row][coord] += P·V         A = P (tensor memory), B = V (shared memory, row-contiguous)
// Rows on the lanes make a softmax row one thread's: no value changes lanes.  Codes
// become fp16 exactly on the way from the copied bytes to the operands, once for the
// rows of both halves.  Two halves of rows take turns (one's products run while the
// other's weights are made); with 128 rows or fewer (PAIR) both halves hold the same
// rows and every second unit each, and are joined at the tile's end.
// M is raised only before a weight passes 2^14, so that O is rarely rescaled.
// Weights are one fp16 term for bf16 outputs, two for fp16 (as in the kernel for few
// rows); both stand in the columns of their own scores.
//
// Warps: 0-3 and 4-7 softmax of the halves (thread = row), 8-11 codes to fp16, 12
// issues the products, 13 the copies (lane = 16 tokens, so pages may end anywhere on
// a multiple of 16).
#include "tq_cache8.cuh"

namespace tq {

namespace {

constexpr int kUmThreads = 512;
constexpr int kUmRegSoft = 192, kUmRegConv = 72, kUmRegRest = 56;
static_assert(8 * kUmRegSoft + 4 * kUmRegConv + 4 * kUmRegRest <= 16 * 128, "registers that the launch does not have would be waited for");
constexpr int kMeta = 4;                     // units whose scales are kept
constexpr uint32_t kUmLimit = 1u << 20;      // polls of a wait, a few microseconds each
constexpr uint32_t kUmLand = 1u << 14;       // a millisecond or more for copies under way

template <int D, bool PAIR>
struct Lay {
  static constexpr int kTile = 128 * D * 2;                 // 128 rows or tokens in fp16
  static constexpr int kRawTile = 128 * D;                  // as codes
  static constexpr int kRaws = D == 64 ? (PAIR ? 8 : 6) : (PAIR ? 4 : 2);
  static constexpr int kQ = 0, kK = kQ + (PAIR ? 1 : 2) * kTile, kV = kK + 2 * kTile, kRaw = kV + 2 * kTile;
  static constexpr int kMisc = kRaw + kRaws * kRawTile;
};

struct Misc {
  float4 meta[kMeta][8];       // K scale, log2 and inverse of the V scale of 16 tokens
  float2 raw_meta[kMeta][8];   // K and V scale as they are in memory
  uint32_t raw_valid[kMeta], valid[kMeta];
  uint64_t raw_full[8], raw_empty[8];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t meta_full[kMeta];
  uint64_t s_full[2], p_full[2], pv_done[2], q_full[2], pair, drain;
  int64_t sums[1][kUmThreads / 32 + 1], found[2];
  float m[128], l[128];        // of the second half, where the halves are joined
  uint32_t sent;               // tiles of codes asked for
  uint32_t tmem;
  int abort;
};
template <int D, bool PAIR>
constexpr int kUmSmem = Lay<D, PAIR>::kMisc + (int)sizeof(Misc);
static_assert(kUmSmem<128, true> <= 227 * 1024 && kUmSmem<128, false> <= 227 * 1024, "shared memory");

__device__ __forceinline__ bool um_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  if (poll_rest(bar, parity)) return true;
#pragma unroll 1
  for (uint32_t n = 1;; ++n) {
    if (n >= kUmLimit) {
      *abort_flag = 1;
      if (status) atomicOr(status, 2);
      return false;
    }
    if (poll_rest(bar, parity)) return true;
    if ((n & 15u) == 15u && *abort_flag) return false;
  }
}
__device__ __forceinline__ float um_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two fp32 numbers in one register pair, and arithmetic on both.
__device__ __forceinline__ uint64_t um_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 um_two(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t um_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t um_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Columns [a, b) of 32 as bits.
__device__ __forceinline__ uint32_t bits_of(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0u;
  return (b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

template <typename T, int D, bool PAIR>
__global__ void __launch_bounds__(kUmThreads, 1) c8_umma_kernel(const C8Params p) {
  using Ly = Lay<D, PAIR>;
  constexpr bool TWO = std::is_same<T, __half>::value;  // terms of a weight
  constexpr int REC = D + 4, NR = Ly::kRaws, KS = D / 16;
  extern __shared__ __align__(1024) unsigned char smem[];
  Misc& ms = *reinterpret_cast<Misc*>(smem + Ly::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  griddep_launch();
  if ((smem_u32(smem) & 1023u) != 0u) {  // the swizzled operands need it
    if (tid == 0) {
      if (p.status) atomicOr(p.status, 2);
      p.split[blockIdx.x].h = -1;
    }
    return;
  }
  volatile int* abort_flag = &ms.abort;
  if (tid == 0) {
    for (int i = 0; i < NR; ++i) {
      mbar_init(&ms.raw_full[i], 1);
      mbar_init(&ms.raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.k_full[i], 4);
      mbar_init(&ms.k_empty[i], 1);
      mbar_init(&ms.v_full[i], 4);
      mbar_init(&ms.v_empty[i], 1);
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.p_full[i], 4);
      mbar_init(&ms.pv_done[i], 1);
      mbar_init(&ms.q_full[i], 4);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&ms.meta_full[i], 1);
    mbar_init(&ms.pair, 8);
    mbar_init(&ms.drain, 1);
    ms.abort = 0;
    ms.sent = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(&ms.tmem, 512);
  tc_fence_before();
  const C8Share sh = c8_share<kUmThreads>(p, ms.sums, ms.found);  // (its barriers are these writes' too)
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  C8Walk walk = c8_walk(p, sh);
  C8Seg seg;
  const int firsts = p.window > 0 ? p.sinks : 0;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kUmRegSoft));
    // ---------------- softmax: half w, row r of the half
    const int w = warp >> 2, r = (warp & 3) * 32 + lane, wr0 = (warp & 3) * 32 + (PAIR ? 0 : w * 128);
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t tS = tl + 128 * w, tO = tl + 256 + 128 * w;
    uint32_t it = 0, gu = 0, met = 0;  // units of this half, units of the CTA, meetings of the halves
    bool ok = true;
    // both halves (bounded, as every wait here)
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.pair);
      return __all_sync(kFull, um_wait(&ms.pair, met++ & 1u, abort_flag, p.status));
    };
    C8Split split;
    split.h = -1;
    while (ok && c8_next(p, walk, seg)) {
      const C8Tile& t = seg.t;
      const int row = PAIR ? r : w * 128 + r;  // of the tile
      const int rho = t.row0 + row, tok = rho / p.G;
      const bool here = row < t.nrow, any = wr0 < t.nrow;  // the row, some row of the warp
      const int pos = here ? (int)min((int64_t)t.len + tok, (int64_t)INT32_MAX) : -1;
      const int64_t orow = ((int64_t)(t.start + tok) * p.Hq + seg.h * p.G + rho - tok * p.G) * D;
      // ---- the row of q, as an operand
      float cf;
      {
        uint4 x[D / 8];
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (int64_t)(t.start + tok) * p.qs +
                                                          (int64_t)(seg.h * p.G + rho - tok * p.G) * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) x[i] = here ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        auto two = [](uint32_t u) -> float2 {
          if constexpr (TWO)
            return __half22float2(*reinterpret_cast<const __half2*>(&u));
          else
            return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
        };
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = two(u[e]);
            top = um_max3(top, fabsf(f.x), fabsf(f.y));
          }
        }
        const int ex = c8_row_exp(top);
        cf = p.zscale * c8_pow2(ex);
        if (!PAIR || w == 0) {
          const float f = c8_pow2(-ex);
          unsigned char* dst = smem + Ly::kQ + (PAIR ? 0 : w * Ly::kTile) + r * 128;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 v = two(u[e]);
              h[e] = pack_f16x2(v.x * f, v.y * f);
            }
            *reinterpret_cast<uint4*>(dst + (i >> 3) * 16384 + (((i & 7) ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.q_full[w]);
        }
      }
      float M = -INFINITY, L = 0.f;
      const uint32_t it0 = it;
#pragma unroll 1
      for (int k = PAIR ? w : 0; k < seg.n; k += PAIR ? 2 : 1) {
        const uint32_t q = gu + k;
        ok = um_wait(&ms.s_full[w], it & 1u, abort_flag, p.status) &&
             um_wait(&ms.meta_full[q % kMeta], (q / kMeta) & 1u, abort_flag, p.status);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        tc_fence_after();
        if (any) {
          const float4* meta = ms.meta[q % kMeta];
          const uint32_t valid = ms.valid[q % kMeta];
          const int base = c8_unit(t, seg.first + k);
          const bool all = valid == 0xFFu && pos >= base + 127 && base + 127 < t.hi &&
                           (p.window == 0 || (int64_t)base > (int64_t)pos - p.window || base + 127 < firsts);
          const bool masked = !__all_sync(kFull, all);
          // columns that the row sees: [lo, hi) and [0, first)
          const int hi = min(min(pos, t.hi - 1) + 1 - base, 128);
          const int lo = p.window > 0 ? (int)max(min((int64_t)pos - p.window + 1 - base, (int64_t)128), (int64_t)0) : 0;
          const int first = min(firsts - base, hi);
          auto sees = [&](int c) -> uint32_t {
            uint32_t on = bits_of(lo - 32 * c, hi - 32 * c) | bits_of(0, first - 32 * c);
            if (!((valid >> (2 * c)) & 1u)) on &= 0xFFFF0000u;
            if (!((valid >> (2 * c + 1)) & 1u)) on &= 0x0000FFFFu;
            return on;
          };
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_nw(tS + 32 * c, s[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) wait_ld(s[c]);
          float top = -INFINITY;
          if (masked) {  // the scores to their end here
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t on = sees(c);
              const float4 m[2] = {meta[2 * c], meta[2 * c + 1]};
#pragma unroll
              for (int e = 0; e < 32; ++e)
                s[c][e] = __float_as_uint((on >> e) & 1u ? fmaf(__uint_as_float(s[c][e]), cf * m[e >> 4].x, m[e >> 4].y) : -INFINITY);
            }
          }
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const uint32_t* x = &s[g >> 1][(g & 1) * 16];
            auto v = [&](int e) { return __uint_as_float(x[e]); };
            const float y0 = um_max3(um_max3(v(0), v(1), v(2)), v(3), v(4)), y1 = um_max3(um_max3(v(5), v(6), v(7)), v(8), v(9));
            const float y2 = um_max3(um_max3(v(10), v(11), v(12)), v(13), v(14));
            const float y = fmaxf(um_max3(y0, y1, y2), v(15));
            const float4 m = meta[g];
            top = fmaxf(top, masked ? y : fmaf(y, cf * m.x, m.y));
          }
          const bool up = top > M + kC8Raise;
          if (__any_sync(kFull, up)) {
            const float nm = up ? top - kC8Fresh : M;
            const float f = !up ? 1.f : M == -INFINITY ? 0.f : ex2(M - nm);
            M = nm;
            L *= f;
            if (it > it0) {  // the sums so far, once the last product into them is done
              ok = __all_sync(kFull, um_wait(&ms.pv_done[w], (it - 1) & 1u, abort_flag, p.status));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16_nw(tO + 16 * c, o);
                wait_ld(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(tO + 16 * c, o);
              }
            }
          }
          const float use = M == -INFINITY ? 0.f : M;
          // the weights of 32 tokens in the place of their scores: 16 columns of
          // pairs, and 16 of the second terms
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t ph[16], pl[16];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const float4 m = meta[2 * c + g];
              const float a = masked ? 1.f : cf * m.x, b = masked ? -use : m.y - use;
              const uint64_t aa = um_pack(a, a), bb = um_pack(b, b);
              uint64_t sum = 0;  // of even and of odd tokens
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 z = um_two(um_fma2(um_pack(__uint_as_float(s[c][16 * g + 2 * e]), __uint_as_float(s[c][16 * g + 2 * e + 1])), aa, bb));
                const float w0 = ex2(z.x), w1 = ex2(z.y);
                sum = um_add2(sum, um_pack(w0, w1));
                if constexpr (TWO)
                  split2(w0, w1, ph[8 * g + e], pl[8 * g + e]);
                else
                  ph[8 * g + e] = pack_f16x2(w0, w1);
              }
              const float2 both = um_two(sum);
              L = fmaf(both.x + both.y, m.z, L);
            }
            tmem_st16(tS + 32 * c, ph);
            if constexpr (TWO) tmem_st16(tS + 32 * c + 16, pl);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full[w]);
        ++it;
      }
      if (!ok) break;
      gu += seg.n;
      // ---- the rows' sums, once the half's last product is done
      const bool mine = it > it0;
      if (mine) {
        ok = __all_sync(kFull, um_wait(&ms.pv_done[w], (it - 1) & 1u, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
      }
      if (M == -INFINITY && L != L) M = 0.f;  // all scores are no numbers: the NaN goes on
      const bool whole = seg.first == 0 && seg.n == t.n;
      float* rec = p.rec + (((int64_t)blockIdx.x * 2 + (seg.first == 0)) * p.tile + row) * REC;
      auto put = [&](int col, const float (&o)[16], float inv) {  // 16 of the row's sums
        if (!here) return;
        if (whole) {
          T* to = static_cast<T*>(p.out) + orow + col;
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (TWO) {
              h[e] = pack_f16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
            } else {
              const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
              h[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
          }
          reinterpret_cast<uint4*>(to)[0] = make_uint4(h[0], h[1], h[2], h[3]);
          reinterpret_cast<uint4*>(to)[1] = make_uint4(h[4], h[5], h[6], h[7]);
        } else {
          float4* to = reinterpret_cast<float4*>(rec + 4 + col);
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      };
      if constexpr (!PAIR) {
        if (any) {
          if (here && !whole) *reinterpret_cast<float2*>(rec) = make_float2(M, L);
          const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            float f[16];
            tmem_ld16_nw(tO + 16 * c, o);
            wait_ld(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = L == 0.f ? 0.f : __uint_as_float(o[e]);
            put(16 * c, f, inv);
          }
        }
      } else {
        // the second half's sums through the place of q, which both have done with
        float* buf = reinterpret_cast<float*>(smem + Ly::kQ);  // [D/2][128]
        if (w == 1) {
          ms.m[r] = mine ? M : -INFINITY;
          ms.l[r] = mine ? L : 0.f;
        }
        if (!(ok = meet())) break;
        float f0 = 1.f, f1 = 0.f;
        if (w == 0) {
          const float m1 = ms.m[r], top = fmaxf(M, m1);
          f0 = M == -INFINITY ? 0.f : ex2(M - top);
          f1 = m1 == -INFINITY ? 0.f : ex2(m1 - top);
          L = (f0 == 0.f ? 0.f : L * f0) + (f1 == 0.f ? 0.f : ms.l[r] * f1);
          M = top;
          if (here && !whole) *reinterpret_cast<float2*>(rec) = make_float2(M, L);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 1
        for (int part = 0; ok && part < 2; ++part) {
          if (w == 1 && any && mine) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[16];
              tmem_ld16_nw(tO + part * (D / 2) + 16 * c, o);
              wait_ld(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) buf[(16 * c + e) * 128 + r] = __uint_as_float(o[e]);
            }
          }
          if (!(ok = meet())) break;
          if (w == 0 && any) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[16];
              float f[16];
              tmem_ld16_nw(tO + part * (D / 2) + 16 * c, o);
              wait_ld(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                f[e] = f0 == 0.f ? 0.f : __uint_as_float(o[e]) * f0;
                if (f1 != 0.f) f[e] = fmaf(buf[(16 * c + e) * 128 + r], f1, f[e]);
              }
              put(part * (D / 2) + 16 * c, f, inv);
            }
          }
          if (!(ok = meet())) break;
        }
        if (!ok) break;
      }
      tc_fence_before();
      if (seg.first == 0 && !whole) {
        split.b = t.b;
        split.rt = t.rt;
        split.h = seg.h;
        split.u0 = seg.u0;
        split.u1 = seg.u0 + t.n;
      }
    }
    split.units = sh.units;
    if (tid == 0) {
      if (!ok) split.h = -1;
      p.split[blockIdx.x] = split;
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kUmRegConv));
    // ---------------- codes to fp16 operands
    const int ct = tid - 256;
    constexpr int CH = D / 16;  // 16-code pieces of a token
    uint32_t gu = 0, rs = 0, rph = 0;
    bool ok = true;
    while (ok && c8_next(p, walk, seg)) {
#pragma unroll 1
      for (int k = 0; k < seg.n; ++k) {
        const uint32_t q = gu + k, st = q & 1u, ph = (q >> 1) & 1u;
        const int base = c8_unit(seg.t, seg.first + k);
        uint32_t valid = 0;
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
          ok = um_wait(&ms.raw_full[rs], rph, abort_flag, p.status) &&
               um_wait(side ? &ms.v_empty[st] : &ms.k_empty[st], ph ^ 1u, abort_flag, p.status);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          if (side == 0 && warp == 8) {
            if (lane < 8) {
              const float2 sc = ms.raw_meta[q % kMeta][lane];
              const float vs = c8_vscale(sc.y);
              ms.meta[q % kMeta][lane] = make_float4(sc.x, log2f(vs), 1.f / vs, 0.f);
            }
            if (lane == 0) ms.valid[q % kMeta] = ms.raw_valid[q % kMeta];
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.meta_full[q % kMeta]);
          }
          if (side == 0) valid = ms.raw_valid[q % kMeta];  // (rewritten once K's bytes are given back)
          const bool part = side == 1 && !(valid == 0xFFu && base + 127 < seg.t.hi && (base >= seg.t.lo || base + 127 < firsts));
          const unsigned char* raw = smem + Ly::kRaw + rs * Ly::kRawTile;
          unsigned char* dst = smem + (side ? Ly::kV : Ly::kK) + st * Ly::kTile;
#pragma unroll 4
          for (int i = 0; i < CH; ++i) {
            const int x = ct + 128 * i, tk = x / CH, cc = x % CH;
            uint4 c = *reinterpret_cast<const uint4*>(raw + tk * D + cc * 16);
            if (part) {  // what no row sees may be anything, and 0 times it a NaN
              const int at = base + tk;
              if (!(((valid >> (tk >> 4)) & 1u) && at < seg.t.hi && (at >= seg.t.lo || at < firsts))) c = make_uint4(0u, 0u, 0u, 0u);
            }
            const uint4 lo = make_uint4(c8_wide(c.x), c8_wide_hi(c.x), c8_wide(c.y), c8_wide_hi(c.y));
            const uint4 hi = make_uint4(c8_wide(c.z), c8_wide_hi(c.z), c8_wide(c.w), c8_wide_hi(c.w));
            unsigned char* row = dst + (cc >> 2) * 16384 + tk * 128;
            const int ch = 2 * (cc & 3), sw = tk & 7;
            // lanes of the second 64 coordinates store their pieces the other way round: no bank twice
            const bool odd = (cc >> 2) & 1;
            *reinterpret_cast<uint4*>(row + (((ch + odd) ^ sw) << 4)) = odd ? hi : lo;
            *reinterpret_cast<uint4*>(row + (((ch + 1 - odd) ^ sw) << 4)) = odd ? lo : hi;
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(side ? &ms.v_full[st] : &ms.k_full[st]);
            mbar_arrive(&ms.raw_empty[rs]);
          }
          if (++rs == NR) {
            rs = 0;
            rph ^= 1u;
          }
        }
        if (!ok) break;
      }
      gu += seg.n;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kUmRegRest));
    if (warp == 12) {
      // ---------------- products
      constexpr uint32_t idesc = umma_idesc_f16(128, 128), idesc_p = umma_idesc_f16(128, D) | (1u << 16);  // V contiguous along N
      const uint64_t dq = umma_desc_sw128(smem_u32(smem + Ly::kQ)), dk = umma_desc_sw128(smem_u32(smem + Ly::kK));
      // V: 64 coordinates a 128-byte row, the next 64 coordinates 16384 bytes on
      const uint64_t dv = (umma_desc_sw128(smem_u32(smem + Ly::kV)) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(16384 >> 4) << 16);
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(kFull, um_wait(bar, parity, abort_flag, p.status));
      };
      uint32_t gu = 0, qn = 0, it[2] = {0, 0};
      // scores of unit q (of the CTA) for half w
      auto scores = [&](uint32_t q, int w, bool last) -> bool {
        const uint32_t st = q & 1u;
        if (!wait(&ms.k_full[st], (q >> 1) & 1u)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = dq + (PAIR ? 0 : (uint32_t)w * (Ly::kTile / 16)), b = dk + st * (Ly::kTile / 16);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) / 16;
            umma_f16(tmem + 128 * w, a + o, b + o, idesc, ks ? 1u : 0u);
          }
          umma_commit(&ms.s_full[w]);
          if (last) umma_commit(&ms.k_empty[st]);
        }
        __syncwarp();
        return true;
      };
      auto values = [&](uint32_t q, int w, bool fresh, bool last) -> bool {
        const uint32_t st = q & 1u;
        if (!wait(&ms.p_full[w], it[w] & 1u) || !wait(&ms.v_full[st], (q >> 1) & 1u)) return false;
        ++it[w];
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b = dv + st * (Ly::kTile / 16);
          const uint32_t a = tmem + 128 * w, d = tmem + 256 + 128 * w;
          if constexpr (TWO) {  // remainders first: not truncated against a large sum
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) umma_f16_ts(d, a + 16 + 32 * (ks >> 1) + 8 * (ks & 1), b + ks * 128, idesc_p, (ks || !fresh) ? 1u : 0u);
          }
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) umma_f16_ts(d, a + 32 * (ks >> 1) + 8 * (ks & 1), b + ks * 128, idesc_p, (TWO || ks || !fresh) ? 1u : 0u);
          umma_commit(&ms.pv_done[w]);
          if (last) umma_commit(&ms.v_empty[st]);
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      while (ok && c8_next(p, walk, seg)) {
        ok = wait(&ms.q_full[0], qn & 1u) && (PAIR || wait(&ms.q_full[1], qn & 1u));
        ++qn;
        if (!ok) break;
        if constexpr (!PAIR) {
          ok = scores(gu, 0, false) && scores(gu, 1, true);
          for (int k = 0; ok && k < seg.n; ++k)
            for (int w = 0; ok && w < 2; ++w) {
              ok = values(gu + k, w, k == 0, w == 1);
              if (ok && k + 1 < seg.n) ok = scores(gu + k + 1, w, w == 1);
            }
        } else {
          ok = scores(gu, 0, true) && (seg.n < 2 || scores(gu + 1, 1, true));
          for (int k = 0; ok && k < seg.n; ++k) {
            ok = values(gu + k, k & 1, k < 2, true);
            if (ok && k + 2 < seg.n) ok = scores(gu + k + 2, k & 1, true);
          }
        }
        gu += seg.n;
      }
      if (elect_one()) umma_commit(&ms.drain);  // every product issued completes before tensor memory is released
      for (uint32_t k = 0; k < kSpinLimitDev && !mbar_try_wait(&ms.drain, 0u); ++k) {
      }
    } else if (warp == 13) {
      // ---------------- copies: lane = 16 tokens of the unit, scales one unit ahead, pages two
      uint32_t gu = 0, rs = 0, rph = 1, sent = 0;
      bool ok = true;
      while (ok && c8_next(p, walk, seg)) {
        const C8Tile& t = seg.t;
        auto look = [&](int k, int& page, int& off) {
          page = -1;
          off = 0;
          if (lane < 8 && k < seg.n) {
            const int t0 = c8_unit(t, seg.first + k) + 16 * lane;
            if (t0 < t.hi && (t0 + 16 > t.lo || t0 < firsts)) {
              const int j = t0 / p.block;
              off = t0 - j * p.block;
              page = __ldg(p.table + (int64_t)t.b * p.max_blocks + j);
              if (page < 0 || page >= p.pages) {
                page = -1;
                if (p.status) atomicOr(p.status, 1);
              }
            }
          }
        };
        auto scales = [&](int page) -> float2 {
          const int64_t blk = (int64_t)page * p.Hkv + seg.h;
          return page >= 0 ? make_float2(__ldg(p.kscale + blk), __ldg(p.vscale + blk)) : make_float2(0.f, 1.f);
        };
        int pg0, off0, pg1, off1;
        look(0, pg0, off0);
        look(1, pg1, off1);
        float2 sc0 = scales(pg0);
#pragma unroll 1
        for (int k = 0; k < seg.n; ++k) {
          const uint32_t q = gu + k;
          int pg2, off2;
          look(k + 2, pg2, off2);
          const float2 sc1 = scales(pg1);
          const uint32_t valid = __ballot_sync(kFull, pg0 >= 0);
          const int64_t at = (((int64_t)pg0 * p.Hkv + seg.h) * p.block + off0) * D;
#pragma unroll 1
          for (int side = 0; side < 2; ++side) {
            ok = __all_sync(kFull, um_wait(&ms.raw_empty[rs], rph, abort_flag, p.status));
            if (!ok) break;
            if (side == 0) {
              if (lane < 8) ms.raw_meta[q % kMeta][lane] = sc0;
              if (lane == 0) ms.raw_valid[q % kMeta] = valid;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&ms.raw_full[rs], (uint32_t)__popc(valid) * 16 * D);
            __syncwarp();
            if (pg0 >= 0)
              bulk_g2s(smem + Ly::kRaw + rs * Ly::kRawTile + lane * 16 * D, (side ? p.v8 : p.k8) + at, 16 * D, &ms.raw_full[rs]);
            ++sent;
            if (++rs == NR) {
              rs = 0;
              rph ^= 1u;
            }
          }
          if (!ok) break;
          pg0 = pg1;
          off0 = off1;
          sc0 = sc1;
          pg1 = pg2;
          off1 = off2;
        }
        gu += seg.n;
      }
      if (lane == 0) ms.sent = sent;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // every copy issued lands before the CTA exits: each slot's last phase (bounded)
    if (tid == 0) {
      const uint32_t n = ms.sent;
      for (uint32_t q = n > NR ? n - NR : 0u; q < n; ++q)
        for (uint32_t k = 0; k < kUmLand && !mbar_try_wait(&ms.raw_full[q % NR], (q / NR) & 1u); ++k) {
        }
    }
    __syncthreads();
  }
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D, bool PAIR>
cudaError_t run_umma(const C8Params& p, cudaStream_t st) {
  static PerDeviceValue attr;
  const cudaError_t e = smem_attr_once(attr, (const void*)c8_umma_kernel<T, D, PAIR>, kUmSmem<D, PAIR>);
  return e != cudaSuccess ? e : c8_launch(c8_umma_kernel<T, D, PAIR>, dim3(p.ctas), kUmThreads, kUmSmem<D, PAIR>, st, p);
}
template <typename T>
cudaError_t run_umma_d(const C8Params& p, cudaStream_t st) {
  if (p.tile == 128) return p.d == 64 ? run_umma<T, 64, true>(p, st) : run_umma<T, 128, true>(p, st);
  return p.d == 64 ? run_umma<T, 64, false>(p, st) : run_umma<T, 128, false>(p, st);
}

}  // namespace

// p.tile: 128 (both halves hold the same rows) or 256
cudaError_t c8_attend_umma(const C8Params& p, cudaStream_t st) {
  return p.dtype == TQ_F16 ? run_umma_d<__half>(p, st) : run_umma_d<__nv_bfloat16>(p, st);
}

}  // namespace tq
