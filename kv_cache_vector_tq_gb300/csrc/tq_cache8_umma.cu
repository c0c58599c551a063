// Attention over the 8-bit paged cache on the fifth-generation tensor cores:
// prompts, their pieces and longer drafted chains of fp16 and bf16 calls.
// tq_cache8.cuh has the mathematics and the division of the work.
//
// A persistent CTA per SM; per half of a unit (64 of its 128 tokens), with 128 rows
// (token x query head) on the lanes of tensor memory:
//     S[row][token]  = Q·Kᵀ        A = Q, B = K (shared memory)
//     P[row][token]  = 2^(z - M)   in fp16, over S
//     O[row][coord] += P·V         A = P (tensor memory), B = V (shared memory, row-contiguous)
// Rows on the lanes make a softmax row one thread's: no value changes lanes.  Two
// groups of softmax warps take a half of every unit each, with sums of their own
// that are joined at the tile's end, or (WIDE: more than 128 rows a request and KV
// head) 128 rows each, so that K and V are converted once for 256.  From the weights
// of one place of scores to the next scores in it it is some 2000 clocks (the slowest
// warp, two products, three waits), more than a group takes for its next weights:
// WIDE tiles have four places.  With the same rows in both groups Q is in tensor
// memory instead (three places): its products take two thirds of the time that way
// and leave shared memory to the codes' way to fp16 (exact), which there is made for
// half as many rows (64 rows over 32 x 16384: 240 against 277 us when it was measured, 203 now).
// M is raised only before a weight passes 2^15, so that O is rarely rescaled (kUmRaise).
// Weights are one fp16 term for bf16 outputs, two for fp16 (as in the kernel for few
// rows); both stand in the columns of their own scores.
//
// Warps: 0-3 and 4-7 softmax (thread = row), 8-11 K's codes to fp16, 12-15 V's, 16
// and 17 issue the products, 18 and 19 the copies (lane = 16 tokens, so pages may
// end anywhere on a multiple of 16).
//
// Measured (bf16, d = 128, 32/8 heads): a prompt's piece of 2039 tokens behind 16384 450 us,
// 1293 TFLOP/s of the 1882 that a plain matrix product gets; tensor pipe 57 % active,
// issue slots 65 % (fp16, with its second terms: 558 us).  A unit of 256 rows takes 3500 clocks, its products 2560 (1536 the
// scores, whose operands are both in shared memory, 64 columns at a time; 128 at a time
// would take 1024 and slow the codes' way to fp16 by half).  Prompt of 8179 with a window
// of 1024, 16/4 heads: 122 us (528 TFLOP/s; nine units a tile, its ends cost four more).
// Spills: <bf16, 128, false> 140 bytes a thread, the others none or 16.
#include "tq_cache8.cuh"

namespace tq {

namespace {

constexpr int kUmThreads = 640, kUmMma = 16, kUmCopy = 18;
constexpr int kUmRegSoft = 128, kUmRegConv = 64;  // the rest keep the launch's 96
static_assert(8 * kUmRegSoft + 8 * kUmRegConv + 4 * 96 <= 20 * 96, "registers that the launch does not have would be waited for");
constexpr int kMeta = 8;                     // units whose scales are kept (copies are four units ahead of the products at most, those of what is converted)
constexpr uint32_t kUmLimit = 1u << 20;      // polls of a wait, a few microseconds each
constexpr uint32_t kUmLand = 1u << 14;       // a millisecond or more for copies under way
// Tensor memory's sums are cut, not rounded, where they are longer than the products added
// to them: after so many products of 64 tokens they go to fp32 sums in the CTA's record, and
// begin anew (fp16 over 65536 tokens, 2048 rows: 1e-4 to 3e-4 short without, half of its
// rounding or more; bf16 has a quarter of the products for its rounding).
template <bool TWO>
constexpr int kChain = TWO ? 256 : 1024;
// M is raised before a weight passes 2^15, and then so that the row's largest is 2^7.  A
// higher fresh maximum leaves more binary orders to fp16's least step, a lower one fewer
// raises, for each of which a whole warp rescales its sums (a prompt's piece of 2039 behind
// 16384: eight orders between the two 453 us, six 468, four 486, three 491).
constexpr float kUmRaise = 15.f, kUmFresh = 7.f;
// A weight's exponent comes of the product in one rounding, with the maximum that was
// rounded by itself; for maxima past this the two could differ by what takes a weight out
// of fp16's range.  (All rows of a warp then: a choice by the row costs 2 % everywhere.  A
// row whose maximum is an infinity is a NaN either way, and asks for nothing.)
constexpr float kUmFar = 1048576.f;
// Tensor memory columns: places of scores (and Q behind three of them), the two sums
constexpr uint32_t kMostPlaces = 4, kColQ = 192, kColO = 256;

template <int D, bool WIDE>
struct Lay {
  static constexpr int kTile = 128 * D * 2;   // 128 rows or tokens in fp16
  static constexpr int kRawTile = 128 * D;    // as codes
  static constexpr int kRaws = D == 64 ? 8 : WIDE ? 2 : 4;  // K and V in turn
  static constexpr int kQTiles = WIDE ? 2 : 1;
  static constexpr int kQ = 0, kK = kQ + kQTiles * kTile, kV = kK + 2 * kTile, kRaw = kV + 2 * kTile;
  static constexpr int kMisc = kRaw + kRaws * kRawTile;
};

struct Misc {
  float4 meta[kMeta][8];       // K scale, log2 and inverse of the V scale of 16 tokens
  uint32_t valid[kMeta];       // which of the unit's 16 tokens are there, a bit each
  uint64_t raw_full[8], raw_empty[8];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t meta_full[kMeta];
  uint64_t s_full[kMostPlaces], s_empty[kMostPlaces], p_full[kMostPlaces], pv_done[2], q_full, o_done, pair, drain;
  int64_t sums[1][kUmThreads / 32 + 1], found[2];
  float m[128], l[128];        // of the second group, where the two are joined
  uint32_t sent[2];            // tiles of codes asked for, K and V
  uint32_t tmem;
  int abort;
};
template <int D, bool WIDE>
constexpr int kUmSmem = Lay<D, WIDE>::kMisc + (int)sizeof(Misc);
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
// One look at a phase.
__device__ __forceinline__ bool um_look(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// um_wait for a warp whose lanes wait for different barriers: looks only (a poll that
// suspends would do so for the lanes that have theirs as well).  What one lane's barrier
// has made visible to it is used by all: the warp's barrier at the end hands it on (a
// vote orders no memory).
__device__ __forceinline__ bool um_wait_lanes(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  bool got = um_look(bar, parity);
#pragma unroll 1
  for (uint32_t n = 1; !__all_sync(kFull, got); ++n) {
    if (n >= (kUmLimit << 4)) {
      *abort_flag = 1;
      if (status) atomicOr(status, 2);
      return false;
    }
    got = got || um_look(bar, parity);
    if ((n & 255u) == 255u && __any_sync(kFull, *abort_flag != 0)) return false;
  }
  __syncwarp();
  return true;
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

template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(kUmThreads, 1) c8_umma_kernel(const C8Params p) {
  using Ly = Lay<D, WIDE>;
  constexpr bool TWO = std::is_same<T, __half>::value;  // terms of a weight
  constexpr int REC = D + 4, NR = Ly::kRaws, KS = D / 16, PER = WIDE ? 4 : 2;  // scores of 64 tokens and 128 rows a unit
  constexpr uint32_t kPlaces = WIDE ? 4 : 3;
  extern __shared__ __align__(1024) unsigned char smem[];
  Misc& ms = *reinterpret_cast<Misc*>(smem + Ly::kMisc);
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;  // (the warp's number in a uniform register)
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
      mbar_init(&ms.pv_done[i], 1);
    }
    for (int i = 0; i < (int)kMostPlaces; ++i) {
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.s_empty[i], 1);
      mbar_init(&ms.p_full[i], 4);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&ms.meta_full[i], 1);
    mbar_init(&ms.q_full, 8);
    mbar_init(&ms.o_done, 1);
    mbar_init(&ms.pair, 8);
    mbar_init(&ms.drain, 2);
    ms.abort = 0;
    ms.sent[0] = ms.sent[1] = 0;
    fence_mbar_init();
  }
  if (warp == kUmMma) tmem_alloc(&ms.tmem, 512);
  tc_fence_before();
  const C8Share sh = c8_share<kUmThreads>(p, ms.sums, ms.found, reinterpret_cast<int32_t*>(smem + Ly::kQ), Ly::kTile / 4);  // (its barriers are these writes' too)
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, ms.tmem, 0);
  C8Walk walk = c8_walk(p, sh);
  C8Seg seg;
  const int firsts = p.window > 0 ? p.sinks : 0;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kUmRegSoft));
    // ---------------- softmax: row r of the group's rows, tokens 64w.. of every unit or (WIDE) all
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16), tO = tl + kColO + 128 * w;
    uint32_t gu = 0, done = 0, buf = (uint32_t)w, bph = 0, met = 0, segs = 0;  // units and this group's scores so far, place of the next ones and its phase, meetings, segments
    bool ok = true;
    // both groups (bounded, as every wait here)
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.pair);
      return __all_sync(kFull, um_wait(&ms.pair, met++ & 1u, abort_flag, p.status));
    };
    C8Split split;
    split.h = -1;
    while (ok && c8_next(p, walk, seg)) {
      const C8Tile& t = seg.t;
      const int row = WIDE ? 128 * w + r : r, rho = t.row0 + row, tok = rho / p.G;
      const bool here = row < t.nrow, any = row - lane < t.nrow;  // the row, some row of the warp
      // tokens that the row sees: from .. upto, and the first ones (a row that is none sees
      // what the last one does, so that its warp masks no more than others: a prompt's last
      // tile took a seventh longer where it saw nothing)
      const int pos = (int)min((int64_t)t.len + min(tok, t.il), (int64_t)INT32_MAX);
      const int upto = min(pos, t.hi - 1), from = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
      // ---- the warp's 32 rows of q, as an operand: read along rows (a thread's own row
      // takes a look-up in L1 for every lane)
      float cf = 0.f;
      {
        constexpr int LPR = D / 8, RPI = 32 / LPR, NI = 32 / RPI;  // lanes of a row, rows of an access, accesses
        const int c8 = lane % LPR, r0 = row - lane + lane / LPR;   // piece of a row, first row
        uint4 x[NI];
        int at = t.row0 + r0, tk = at / p.G, gg = at - tk * p.G;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if (r0 + RPI * i < t.nrow)
            x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (int64_t)(t.start + tk) * p.qs +
                                                        (int64_t)(seg.h * p.G + gg) * D) + c8);
          gg += RPI;
          while (gg >= p.G) {
            gg -= p.G;
            ++tk;
          }
        }
        auto two = [](uint32_t u) -> float2 {
          if constexpr (TWO)
            return __half22float2(*reinterpret_cast<const __half2*>(&u));
          else
            return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
        };
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          if constexpr (TWO) {  // fp16 already
            cf = p.zscale;
            continue;
          }
          float top = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = two(u[e]);
            top = um_max3(top, fabsf(f.x), fabsf(f.y));
          }
#pragma unroll
          for (int o = LPR / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
          const int ex = c8_row_exp(top);
          const float f = c8_pow2(-ex), mine = __shfl_sync(kFull, p.zscale * c8_pow2(ex), (lane % RPI) * LPR);
          if (lane / RPI == i) cf = mine;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = two(u[e]);
            u[e] = pack_f16x2(v.x * f, v.y * f);
          }
          x[i] = make_uint4(u[0], u[1], u[2], u[3]);
        }
        if constexpr (WIDE) {  // to shared memory: 64 coordinates, then the others
          unsigned char* to = smem + Ly::kQ + w * Ly::kTile + (c8 >> 3) * 16384;
          const int rr = r - lane + lane / LPR;  // of the group's 128 rows
#pragma unroll
          for (int i = 0; i < NI; ++i)
            *reinterpret_cast<uint4*>(to + (rr + RPI * i) * 128 + (((c8 & 7) ^ ((rr + RPI * i) & 7)) << 4)) = x[i];
          fence_proxy_async();
        } else {  // to tensor memory, each group its half of the coordinates: turned in a place of the warp's own
          constexpr int PC = D / 16;  // 16-byte pieces
          unsigned char* mine = smem + Ly::kQ + warp * (Ly::kTile / 8);
          if (c8 / PC == w)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const int lr = lane / LPR + RPI * i;
              *reinterpret_cast<uint4*>(mine + lr * (PC * 16) + (((c8 % PC) ^ (lr & (PC - 1))) << 4)) = x[i];
            }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < PC; i += 2) {  // eight columns of pairs
            const uint4 a = *reinterpret_cast<const uint4*>(mine + lane * (PC * 16) + ((i ^ (lane & (PC - 1))) << 4));
            const uint4 b = *reinterpret_cast<const uint4*>(mine + lane * (PC * 16) + (((i + 1) ^ (lane & (PC - 1))) << 4));
            const uint32_t h8[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            tmem_st8(tl + kColQ + w * (4 * PC) + 4 * i, h8);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.q_full);
      }
      constexpr int TILE = WIDE ? 256 : 128;
      auto record = [&]() -> float* { return p.rec + ((int64_t)blockIdx.x * 2 + (seg.first == 0)) * (TILE * REC); };
      // a long sum of the row so far stands there too (of the second group with the same
      // rows behind the records), its maximum behind the records' own; with what tensor
      // memory holds it goes there (`away`) or to tensor memory
      auto long_sum = [&](bool first, bool away, float m) {
        float* base = WIDE || w == 0 ? record() : p.rec + ((int64_t)p.ctas * 2 + blockIdx.x) * (TILE * REC);
        float* top = base + 2 * TILE + row;
        const float hm = here && !first ? *top : -INFINITY, scale = hm == -INFINITY ? 0.f : ex2(hm - m);
        if (here && away) *top = m;
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          float4* at = reinterpret_cast<float4*>(base) + TILE * (1 + 4 * c) + row;
          uint32_t o[16];
          tmem_ld16_nw(tO + 16 * c, o);
          wait_ld(o);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(o[4 * e + i]);
            if (scale != 0.f) {
              const float4 v = at[TILE * e];
              f[0] = fmaf(v.x, scale, f[0]);
              f[1] = fmaf(v.y, scale, f[1]);
              f[2] = fmaf(v.z, scale, f[2]);
              f[3] = fmaf(v.w, scale, f[3]);
            }
            if (here && away) at[TILE * e] = make_float4(f[0], f[1], f[2], f[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[4 * e + i] = away ? 0u : __float_as_uint(f[i]);
          }
          tmem_st16(tO + 16 * c, o);
        }
        tmem_wait_st();
      };
      const int halves = (WIDE ? 2 : 1) * seg.n;  // of units, this group's
      float M = -INFINITY, L = 0.f;
      bool far = false;  // some row's maximum is past kUmFar: scores to their end first, then the differences
#pragma unroll 1
      for (int k = 0, rest = kChain<TWO>; ok && k < halves; rest += kChain<TWO>) {
        if (k > 0) {  // a rest: the last product is done (the one before it is when the next scores are there)
          ok = __all_sync(kFull, um_wait(&ms.s_full[buf], bph, abort_flag, p.status) &&
                                     um_wait(&ms.pv_done[w], (done - 1) & 1u, abort_flag, p.status));
          if (!ok) break;
          tc_fence_after();
          if (any) long_sum(k == kChain<TWO>, true, M);
        }
#pragma unroll 1
        for (; k < min(halves, rest); ++k, ++done) {
          const int unit = WIDE ? k >> 1 : k, part = WIDE ? k & 1 : w;  // of the segment; which 64 tokens
          const uint32_t q = gu + unit, tS = tl + 64 * buf;
          // (lanes wait for one or the other: with the converting warps' reads and writes
          // before it, a poll takes 200 clocks even where it finds its phase complete)
          ok = um_wait_lanes(lane & 1 ? &ms.meta_full[q % kMeta] : &ms.s_full[buf], lane & 1 ? (q / kMeta) & 1u : bph, abort_flag,
                             p.status);
          if (!ok) break;
          tc_fence_after();
          if (any) {
            uint32_t s[2][32];
            tmem_ld32_nw(tS, s[0]);
            tmem_ld32_nw(tS + 32, s[1]);
            const float4* meta = ms.meta[q % kMeta] + 4 * part;
            const uint32_t valid = (ms.valid[q % kMeta] >> (4 * part)) & 15u;
            const int base = c8_unit(t, seg.first + unit) + 64 * part;
            const bool all = valid == 15u && base + 63 <= upto && (base >= from || base + 63 < firsts);
            const bool masked = far || !__all_sync(kFull, all);
            wait_ld(s[0]);
            wait_ld(s[1]);
            if (masked) {  // the scores to their end here
              // columns that the row sees: [lo, hi) and [0, first)
              const int hi = min(upto + 1 - base, 64), lo = min(max(from - base, 0), 64);
              const int first = min(firsts - base, hi);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t on = bits_of(lo - 32 * c, hi - 32 * c) | bits_of(0, first - 32 * c);
                if (!((valid >> (2 * c)) & 1u)) on &= 0xFFFF0000u;
                if (!((valid >> (2 * c + 1)) & 1u)) on &= 0x0000FFFFu;
                const float4 m[2] = {meta[2 * c], meta[2 * c + 1]};
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  s[c][e] = __float_as_uint((on >> e) & 1u ? fmaf(__uint_as_float(s[c][e]), cf * m[e >> 4].x, m[e >> 4].y) : -INFINITY);
              }
            }
            float a[4], b[4], iv[4], top = -INFINITY;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const uint32_t* x = &s[g >> 1][(g & 1) * 16];
              auto v = [&](int e) { return __uint_as_float(x[e]); };
              const float y0 = um_max3(um_max3(v(0), v(1), v(2)), v(3), v(4)), y1 = um_max3(um_max3(v(5), v(6), v(7)), v(8), v(9));
              const float y2 = um_max3(um_max3(v(10), v(11), v(12)), v(13), v(14));
              const float y = fmaxf(um_max3(y0, y1, y2), v(15));
              const float4 m = meta[g];
              a[g] = masked ? 1.f : cf * m.x;
              b[g] = masked ? 0.f : m.y;
              iv[g] = m.z;
              top = fmaxf(top, fmaf(y, a[g], b[g]));
            }
            const bool up = top - M > kUmRaise;
            if (__any_sync(kFull, up)) {
              const float nm = up ? top - kUmFresh : M;
              const float f = !up ? 1.f : M == -INFINITY ? 0.f : ex2(M - nm);
              M = nm;
              L *= f;
              far = __any_sync(kFull, fabsf(M) > kUmFar && fabsf(M) < INFINITY);
              if (far && !masked) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                  s[e >> 5][e & 31] = __float_as_uint(fmaf(__uint_as_float(s[e >> 5][e & 31]), a[e >> 4], b[e >> 4]));
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                  a[g] = 1.f;
                  b[g] = 0.f;
                }
              }
              if (k > 0) {  // the sums so far, once the last product into them is done (the one before it was when these scores' place was free)
                ok = __all_sync(kFull, um_wait(&ms.pv_done[w], (done - 1) & 1u, abort_flag, p.status));
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
            float sum64 = 0.f;  // of the weights: one rounding into the row's for 64
            // the weights of 32 tokens: 16 columns of pairs, then those of the second terms
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t ph[16], pl[16];
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const float bg = b[2 * c + g] - use;
                const uint64_t aa = um_pack(a[2 * c + g], a[2 * c + g]), bb = um_pack(bg, bg);
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
                sum64 = fmaf(both.x + both.y, iv[2 * c + g], sum64);
              }
              tmem_st16(tS + 16 * c, ph);
              if constexpr (TWO) tmem_st16(tS + 32 + 16 * c, pl);
            }
            L += sum64;
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.p_full[buf]);
          buf += 2;  // the next of this group's scores
          if (buf >= kPlaces) {
            buf -= kPlaces;
            bph ^= 1u;
          }
        }
      }
      if (!ok) break;
      gu += seg.n;
      // ---- the rows' sums, once the last product is done
      // (a barrier of the segments' own: a group may be two units ahead of its products
      // here, and a wait by parity tells one phase from the next only)
      ok = __all_sync(kFull, um_wait(&ms.o_done, segs++ & 1u, abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      if (M == -INFINITY && L != L) M = 0.f;  // all scores are no numbers: the NaN goes on
      const bool whole = seg.first == 0 && seg.n == t.n;
      const int64_t orow = ((int64_t)(t.start + tok) * p.Hq + seg.h * p.G + rho - tok * p.G) * D;
      if (any && halves > kChain<TWO>) long_sum(false, false, M);
      float* rec = record();
      auto half8 = [&](const float* o, float inv) -> uint4 {  // eight sums as outputs
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = c8_pair<T>(o[2 * e] * inv, o[2 * e + 1] * inv);
        return make_uint4(h[0], h[1], h[2], h[3]);
      };
      auto put = [&](int col, const float (&o)[16], float inv) {  // 16 of the row's sums
        if (whole) {
          const uint4 a = half8(o, inv), b = half8(o + 8, inv);
          if (!here) return;
          T* to = static_cast<T*>(p.out) + orow + col;
          reinterpret_cast<uint4*>(to)[0] = a;
          reinterpret_cast<uint4*>(to)[1] = b;
        } else if (here) {
          float4* to = reinterpret_cast<float4*>(rec) + TILE * (1 + (col >> 2)) + row;
#pragma unroll
          for (int e = 0; e < 4; ++e) to[TILE * e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      };
      if constexpr (WIDE) {
        if (any) {
          if (here && !whole) *reinterpret_cast<float2*>(rec + 2 * row) = make_float2(M, L);
          const float inv = L == 0.f ? 0.f : 1.f / L;
          // 64 coordinates at a time; whole rows are turned where the warp's own q was, so
          // that stores go along rows
          unsigned char* turn = smem + Ly::kQ + w * Ly::kTile + (warp & 3) * 4096;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            float f[16];
            tmem_ld16_nw(tO + 16 * c, o);
            wait_ld(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = L == 0.f ? 0.f : __uint_as_float(o[e]);
            if (!whole) {
              put(16 * c, f, inv);
              continue;
            }
            const uint4 a = half8(f, inv), b = half8(f + 8, inv);
            *reinterpret_cast<uint4*>(turn + lane * 128 + (((2 * c) & 7) ^ (lane & 7)) * 16) = a;
            *reinterpret_cast<uint4*>(turn + lane * 128 + (((2 * c + 1) & 7) ^ (lane & 7)) * 16) = b;
            if ((c & 3) != 3) continue;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int lr = 4 * i + (lane >> 3), c8 = lane & 7;
              const int64_t to = __shfl_sync(kFull, orow, lr);
              const uint4 v = *reinterpret_cast<const uint4*>(turn + lr * 128 + ((c8 ^ (lr & 7)) << 4));
              if (row - lane + lr < t.nrow) reinterpret_cast<uint4*>(static_cast<T*>(p.out) + to + 64 * (c >> 2))[c8] = v;
            }
            __syncwarp();
          }
        }
      } else {
        // the second group's sums go to the first through shared memory, half of the columns at a time
        float* buf_join = reinterpret_cast<float*>(smem + Ly::kQ);  // [D/2][128], where q was
        if (w == 1) {
          ms.m[r] = M;
          ms.l[r] = L;
          if (any) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[16];
              tmem_ld16_nw(tO + 16 * c, o);
              wait_ld(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) buf_join[(16 * c + e) * 128 + r] = __uint_as_float(o[e]);
            }
          }
        }
        if (!(ok = meet())) break;
        float f0 = 0.f, f1 = 0.f, inv = 0.f;
        if (w == 0) {
          const float m1 = ms.m[r], top = fmaxf(M, m1);
          f0 = M == -INFINITY ? 0.f : ex2(M - top);
          f1 = m1 == -INFINITY ? 0.f : ex2(m1 - top);
          L = L * f0 + ms.l[r] * f1;  // (a NaN goes on with a factor of 0)
          inv = L == 0.f ? 0.f : 1.f / L;
          if (here && !whole) *reinterpret_cast<float2*>(rec + 2 * row) = make_float2(top, L);
        }
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
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
                if (f1 != 0.f) f[e] = fmaf(buf_join[(16 * c + e) * 128 + r], f1, f[e]);
              }
              put(part * (D / 2) + 16 * c, f, inv);
            }
          }
          if (!(ok = meet())) break;
          if (part == 0) {
            if (w == 1 && any) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[16];
                tmem_ld16_nw(tO + D / 2 + 16 * c, o);
                wait_ld(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) buf_join[(16 * c + e) * 128 + r] = __uint_as_float(o[e]);
              }
            }
            if (!(ok = meet())) break;
          }
        }
        if (!ok) break;
      }
      tc_fence_before();
      if (seg.first == 0 && !whole) {
        split.row0 = t.row0;
        split.nrow = t.nrow;
        split.start = t.start;
        split.h = seg.h;
        split.u0 = seg.u0;
        split.u1 = seg.u0 + t.n + p.pad;
      }
    }
    split.units = sh.units;
    if (tid == 0) {
      if (!ok) split.h = -1;
      p.split[blockIdx.x] = split;
    }
  } else if (warp < kUmMma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kUmRegConv));
    // ---------------- codes to fp16 operands: K by one group of warps, V by the other
    const bool is_v = warp >= 12;
    const int ct = tid & 127;
    constexpr int CH = D / 16, STEP = 128 / CH;  // 16-code pieces of a token, tokens that the threads take at a time
    const int tk = ct / CH, cc = ct % CH;
    // lanes of the second 64 coordinates store their two pieces the other way round: no bank twice
    const bool odd = (cc >> 2) & 1;
    const int to0 = ((2 * (cc & 3) + odd) ^ (tk & 7)) << 4, to1 = ((2 * (cc & 3) + 1 - odd) ^ (tk & 7)) << 4;
    uint64_t* full = is_v ? ms.v_full : ms.k_full;
    uint64_t* empty = is_v ? ms.v_empty : ms.k_empty;
    uint32_t q = 0, rs = is_v, rph = 0;
    bool ok = true;
    while (ok && c8_next(p, walk, seg)) {
#pragma unroll 1
      for (int k = 0; k < seg.n; ++k, ++q) {
        const uint32_t st = q & 1u, ph = (q >> 1) & 1u;
        if constexpr (WIDE)  // (these warps are ahead, and looks would take issue slots from the others: 540 -> 515 us)
          ok = __all_sync(kFull, um_wait(&ms.raw_full[rs], rph, abort_flag, p.status) && um_wait(&empty[st], ph ^ 1u, abort_flag, p.status));
        else
          ok = um_wait_lanes(lane & 1 ? &empty[st] : &ms.raw_full[rs], lane & 1 ? ph ^ 1u : rph, abort_flag, p.status);
        if (!ok) break;
        uint32_t valid = 0xFFu;
        bool part = false;
        int base = 0;
        if (is_v) {
          valid = ms.valid[q % kMeta];
          base = c8_unit(seg.t, seg.first + k);
          part = !(valid == 0xFFu && base + 127 < seg.t.hi && (base >= seg.t.lo || base + 127 < firsts));
        }
        const unsigned char* raw = smem + Ly::kRaw + rs * Ly::kRawTile + ct * 16;
        unsigned char* row = smem + (is_v ? Ly::kV : Ly::kK) + st * Ly::kTile + (cc >> 2) * 16384 + tk * 128;
        auto one = [&](int i, bool there) {
          uint4 c = *reinterpret_cast<const uint4*>(raw + i * 2048);
          if (!there) c = make_uint4(0u, 0u, 0u, 0u);
          const uint4 lo = make_uint4(c8_wide(c.x), c8_wide_hi(c.x), c8_wide(c.y), c8_wide_hi(c.y));
          const uint4 hi = make_uint4(c8_wide(c.z), c8_wide_hi(c.z), c8_wide(c.w), c8_wide_hi(c.w));
          *reinterpret_cast<uint4*>(row + to0 + i * (STEP * 128)) = odd ? hi : lo;
          *reinterpret_cast<uint4*>(row + to1 + i * (STEP * 128)) = odd ? lo : hi;
        };
        if (!part) {
#pragma unroll 4
          for (int i = 0; i < CH; ++i) one(i, true);
        } else {  // what no row sees may be anything, and 0 times it a NaN
#pragma unroll 1
          for (int i = 0; i < CH; ++i) {
            const int t = tk + STEP * i, at = base + t;
            one(i, ((valid >> (t >> 4)) & 1u) && at < seg.t.hi && (at >= seg.t.lo || at < firsts));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[st]);
          mbar_arrive(&ms.raw_empty[rs]);
        }
        rs += 2;
        if (rs >= NR) {
          rs -= NR;
          rph ^= 1u;
        }
      }
    }
  } else if (warp == kUmMma) {
    // ---------------- scores, of 64 tokens at a time.  (Scores and sums have a warp
    // each: one for both took twice the products' own time.)
    constexpr uint32_t idesc = umma_idesc_f16(128, 64);
    const uint64_t dk = umma_desc_sw128(smem_u32(smem + Ly::kK)), dq = umma_desc_sw128(smem_u32(smem + Ly::kQ));
    uint32_t q = 0, buf = 0, bph = 1, qn = 0;  // scores so far, place of the next scores and its phase, tiles
    bool ok = true;
    while (ok && c8_next(p, walk, seg)) {
      if (!(ok = __all_sync(kFull, um_wait(&ms.q_full, qn++ & 1u, abort_flag, p.status)))) break;
#pragma unroll 1
      for (int k = 0; k < PER * seg.n; ++k) {
        const uint32_t at = q % PER, u = q / PER, st = u & 1u;
        const bool lk = (lane & 1) && at == 0;  // odd lanes look for K, with a unit's first scores
        ok = um_wait_lanes(lk ? &ms.k_full[st] : &ms.s_empty[buf], lk ? (u >> 1) & 1u : bph, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b = dk + st * (Ly::kTile / 16) + (WIDE ? at >> 1 : at) * (8192 / 16);
          const uint64_t a = dq + (at & 1u) * (Ly::kTile / 16);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) / 16;
            if constexpr (WIDE)
              umma_f16(tmem + 64 * buf, a + o, b + o, idesc, ks ? 1u : 0u);
            else
              umma_f16_ts(tmem + 64 * buf, tmem + kColQ + 8 * ks, b + o, idesc, ks ? 1u : 0u);
          }
          umma_commit(&ms.s_full[buf]);
          if (at == PER - 1) umma_commit(&ms.k_empty[st]);
        }
        __syncwarp();
        ++q;
        if (++buf == kPlaces) {
          buf = 0;
          bph ^= 1u;
        }
      }
    }
    if (elect_one()) umma_commit(&ms.drain);  // every product issued completes before tensor memory is released
  } else if (warp == kUmMma + 1) {
    // ---------------- weights with values
    constexpr uint32_t idesc = umma_idesc_f16(128, D) | (1u << 16);  // V contiguous along N
    // V: 64 coordinates a 128-byte row, the next 64 coordinates 16384 bytes on
    const uint64_t dv = (umma_desc_sw128(smem_u32(smem + Ly::kV)) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(16384 >> 4) << 16);
    uint32_t q = 0, buf = 0, bph = 0;
    bool ok = true;
    while (ok && c8_next(p, walk, seg)) {
#pragma unroll 1
      for (int k = 0; k < PER * seg.n; ++k) {
        const uint32_t at = q % PER, u = q / PER, st = u & 1u, w = q & 1u;
        const bool lv = (lane & 1) && at == 0;
        ok = um_wait_lanes(lv ? &ms.v_full[st] : &ms.p_full[buf], lv ? (u >> 1) & 1u : bph, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b = dv + st * (Ly::kTile / 16) + (WIDE ? at >> 1 : at) * (8192 / 16);
          const uint32_t a = tmem + 64 * buf, d = tmem + kColO + 128 * w;
          const uint32_t on = k < 2 ? 0u : 1u;
          if constexpr (TWO) {  // remainders first: not truncated against a large sum
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) umma_f16_ts(d, a + 32 + 8 * ks, b + ks * 128, idesc, ks ? 1u : on);
          }
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) umma_f16_ts(d, a + 8 * ks, b + ks * 128, idesc, TWO || ks ? 1u : on);
          umma_commit(&ms.s_empty[buf]);
          umma_commit(&ms.pv_done[w]);
          if (at == PER - 1) umma_commit(&ms.v_empty[st]);
          if (k == PER * seg.n - 1) umma_commit(&ms.o_done);
        }
        __syncwarp();
        ++q;
        if (++buf == kPlaces) {
          buf = 0;
          bph ^= 1u;
        }
      }
    }
    if (elect_one()) umma_commit(&ms.drain);
  } else if (warp < kUmCopy + 2) {
    // ---------------- copies, K by one warp and V by the other: lane = 16 tokens of
    // the unit; the first lane of a run inside one page copies the run (a copy takes
    // some 100 clocks to issue).  Pages are read two units ahead, scales (V's warp) one
    const bool is_v = warp != kUmCopy;
    const uint8_t* codes = is_v ? p.v8 : p.k8;
    uint32_t q = 0, rs = is_v, rph = 1, sent = 0;
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
              if (p.status && is_v) atomicOr(p.status, 1);
            }
          }
        }
      };
      auto scales = [&](int page) -> float2 {
        const int64_t blk = (int64_t)page * p.Hkv + seg.h;
        return is_v && page >= 0 ? make_float2(__ldg(p.kscale + blk), __ldg(p.vscale + blk)) : make_float2(0.f, 1.f);
      };
      int pg0, off0, pg1, off1;
      look(0, pg0, off0);
      look(1, pg1, off1);
      float2 sc0 = scales(pg0);
#pragma unroll 1
      for (int k = 0; k < seg.n; ++k, ++q) {
        int pg2, off2;
        look(k + 2, pg2, off2);
        const float2 sc1 = scales(pg1);
        const uint32_t valid = __ballot_sync(kFull, pg0 >= 0);
        // runs: a lane goes on from the one before it where the page is the same
        const int before = __shfl_up_sync(kFull, pg0, 1);
        const bool leads = pg0 >= 0 && (lane == 0 || before != pg0 || off0 == 0);
        const uint32_t starts = __ballot_sync(kFull, leads || pg0 < 0);  // (lanes from 8 on have no page)
        const uint32_t run = __ffs(starts >> ((lane + 1) & 31));
        const int64_t at = (((int64_t)pg0 * p.Hkv + seg.h) * p.block + off0) * D;
        ok = __all_sync(kFull, um_wait(&ms.raw_empty[rs], rph, abort_flag, p.status));
        if (!ok) break;
        if (is_v && lane == 0) ms.valid[q % kMeta] = valid;
        if (lane == 0) mbar_arrive_expect_tx(&ms.raw_full[rs], (uint32_t)__popc(valid) * 16 * D);
        __syncwarp();
        if (leads) bulk_g2s(smem + Ly::kRaw + rs * Ly::kRawTile + lane * 16 * D, codes + at, run * 16 * D, &ms.raw_full[rs]);
        if (is_v) {  // the unit's scales, for the softmax
          if (lane < 8) {
            const float vs = c8_vscale(sc0.y);
            ms.meta[q % kMeta][lane] = make_float4(sc0.x, log2f(vs), c8_inverse(vs), 0.f);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.meta_full[q % kMeta]);
        }
        ++sent;
        rs += 2;
        if (rs >= NR) {
          rs -= NR;
          rph ^= 1u;
        }
        pg0 = pg1;
        off0 = off1;
        sc0 = sc1;
        pg1 = pg2;
        off1 = off2;
      }
    }
    if (lane == 0) ms.sent[is_v] = sent;
  }

  if (warp == kUmMma || warp == kUmMma + 1)
    for (uint32_t k = 0; k < kSpinLimitDev && !mbar_try_wait(&ms.drain, 0u); ++k) {
    }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // every copy issued lands before the CTA exits: each slot's last phase (bounded)
    if (warp >= kUmCopy && warp < kUmCopy + 2 && lane == 0) {
      constexpr uint32_t H = NR / 2;  // places of a side
      const uint32_t side = warp - kUmCopy, n = ms.sent[side];
      for (uint32_t q = n > H ? n - H : 0u; q < n; ++q)
        for (uint32_t k = 0; k < kUmLand && !mbar_try_wait(&ms.raw_full[2 * (q % H) + side], (q / H) & 1u); ++k) {
        }
    }
    __syncthreads();
  }
  if (warp == kUmMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D, bool WIDE>
cudaError_t run_umma(const C8Params& p, cudaStream_t st) {
  static PerDeviceValue attr;
  const cudaError_t e = smem_attr_once(attr, (const void*)c8_umma_kernel<T, D, WIDE>, kUmSmem<D, WIDE>);
  return e != cudaSuccess ? e : c8_launch(c8_umma_kernel<T, D, WIDE>, dim3(p.ctas), kUmThreads, kUmSmem<D, WIDE>, st, p);
}
template <typename T>
cudaError_t run_umma_d(const C8Params& p, cudaStream_t st) {
  if (p.tile == 256) return p.d == 64 ? run_umma<T, 64, true>(p, st) : run_umma<T, 128, true>(p, st);
  return p.d == 64 ? run_umma<T, 64, false>(p, st) : run_umma<T, 128, false>(p, st);
}

}  // namespace

// p.tile: 128 or 256 (WIDE)
cudaError_t c8_attend_umma(const C8Params& p, cudaStream_t st) {
  return p.dtype == TQ_F16 ? run_umma_d<__half>(p, st) : run_umma_d<__nv_bfloat16>(p, st);
}

}  // namespace tq
