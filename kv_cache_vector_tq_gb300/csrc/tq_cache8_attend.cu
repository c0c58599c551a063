// Attention over the 8-bit paged cache (tq_cache8_attention) for few rows a request:
// single tokens, drafted chains, and every fp32 call.  tq_cache8.cuh has the
// mathematics and the division of the work.
//
// A warp takes 32 tokens of a unit, 16 at a time on the rows of mma.m16n8k16 and up
// to 8·NT rows (token x query head) on its columns:
//     Sᵀ[token][row] = K·Q̂ᵀ,   Oᵀ[coord][row] += Vᵀ·P
// Codes become fp16 exactly (every e4m3 number is one) on the way from shared
// memory to the operands.  The order of the coordinates along a contraction, of the
// coordinates in Oᵀ and of the 16 tokens is free: a lane's bytes are 16 in a row (of
// K's coordinates 16c.. and 64 on, of V's 16 of a row's), and rows of 128 bytes in
// TMA's swizzle meet no bank twice (kTok, kPart).  P's transposition from the layout
// of a result to that of an operand is one movmatrix for 8 tokens.
// Bytes come by TMA, a box for 16 tokens of K or V, kStages groups of tokens ahead in
// a ring of each warp's own, so that no warp waits for another inside a tile; the
// warps' states are joined at its end.
// Rounding: q is scaled by a power of two into fp16's range, which holds fp16 and
// bf16 numbers whole; fp32 rows are two fp16 terms (2^-22).  Weights are one fp16
// term for bf16 outputs (2^-12 against the output's 2^-9; two take 137 us for the 32 single
// tokens below and 164 for 140 with rows for a tile of 32), two for fp16 and fp32, where
// one would cost as much as the output's own rounding or more; the second one of
// fp32 calls is 2^12 times as large and has sums of its own, so that it keeps its bits
// for weights far below the row's largest too.
// Measured (bf16, d = 128): 32 single tokens over up to 16384, 32/8 heads: 133 us, 6.1
// TB/s of the 6.8 that a copy gets, issue slots 37 % used; one over 131072, 64/8 heads:
// 54 us, of which 40 are its bytes and the rest a share's start, the states' and the
// parts' joins; 64 with a window of 1024, 64/8 heads: 45 us for 137 MB, the same.
// Spills: <fp32, 128, 4> 240 bytes a thread, the other fp32 ones and the 16-bit <128, 4> 52
// at most, the rest none.
#include "tq_cache8.cuh"

namespace tq {

namespace {

constexpr int kAtThreads = 128, kAtWarps = 4;  // two CTAs an SM
constexpr uint32_t kAtPolls = 1u << 20;          // polls of a wait
// M is raised before a weight passes 2^14, and then so that the row's largest is 2^10: a
// fresh maximum that high leaves 34 binary orders to fp16's least step (weights 24 orders
// below one other's were 0.2 % off with 2^6), and four to the next raise, which costs
// nothing here (2^6, 2^8, 2^10, 2^11: 32 long single tokens 133 us each time).
constexpr float kAtRaise = 14.f, kAtFresh = 10.f;

template <typename T>
constexpr int kQTerms = sizeof(T) == 4 ? 2 : 1;  // fp16 terms of q
template <typename T>
constexpr int kPTerms = std::is_same<T, __nv_bfloat16>::value ? 1 : 2;  // of the weights
template <typename T, int D, int NT>
constexpr int kStages = (D == 64 ? 6 : 3) - (kQTerms<T> == 2 && NT == 4 ? 1 : 0);
template <int D>
constexpr int kSlot = 64 * D;  // 32 tokens' K and V codes
template <typename T, int D, int NT>  // the rings, and in their place the warps' states; aligned in the kernel
constexpr int kAtSmem = kAtWarps * (kStages<T, D, NT> * kSlot<D> > 8 * NT * (D + 4) * 4 ? kStages<T, D, NT> * kSlot<D> : 8 * NT * (D + 4) * 4) + 1024;
// Token of row g of an operand's 8, and place of lane g's part of a V row.
template <int D>
__device__ __forceinline__ int kTok(int g) { return D == 128 ? (g >> 1) | ((g & 1) << 2) : g; }

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float4*>(p);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    float2 a, b;
    if constexpr (std::is_same<T, __half>::value) {
      a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
      b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    } else {
      a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
      b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    }
    return make_float4(a.x, a.y, b.x, b.y);
  }
}
// Weights as two fp16 terms, the second kLow times as large: weights far below the largest
// keep their bits (in fp16's own range a second term is no finer than 2^-24).  A weight is
// 2^14 at most, what its first term leaves 2^2: within the range.  (32 single tokens over up
// to 16384 147 -> 152 us, a prompt of 512 over 4096 269 -> 300 us; a weight 2^-24 times
// another's is 2^-23 off, with the second term in fp16's own range 2^-11.)
constexpr float kLow = 4096.f;
__device__ __forceinline__ void split2_low(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  hi = h2_bits(h);
  lo = pack_f16x2((x0 - __low2float(h)) * kLow, (x1 - __high2float(h)) * kLow);
}
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kAtThreads, 2)
    c8_attend_kernel(const C8Params p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr int QT = kQTerms<T>, PT = kPTerms<T>, ST = kStages<T, D, NT>;
  constexpr int TILE = 8 * NT, KP = D / 64, KS = D / 16, SLOT = kSlot<D>, REC = D + 4;
  constexpr bool QREG = NT * QT <= 2;  // q's operands stay in registers
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint2 qf[NT][QT][KS][32];
  __shared__ float4 s_scale[kAtWarps][ST][2];  // of 16 tokens: K scale, log2 and inverse of the V scale
  __shared__ __align__(8) uint64_t s_full[kAtWarps][ST];
  __shared__ float s_c[TILE];
  __shared__ int s_pos[TILE];
  __shared__ int64_t s_sums[1][kAtThreads / 32 + 1], s_found[2];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  if (tid < kAtWarps * ST) mbar_init(&s_full[0][0] + tid, 1);
  fence_mbar_init();
  griddep_wait();
  griddep_launch();
  const C8Share sh = c8_share<kAtThreads>(p, s_sums, s_found, reinterpret_cast<int32_t*>(smem), kAtWarps * ST * SLOT / 4);  // (its barriers are the mbarriers' too)
  C8Split split;
  split.h = -1;
  unsigned char* ring = smem + warp * (ST * SLOT);
  uint32_t cs = 0, cph = 0, ps = 0;  // slot and phase of the next group to be read, slot of the next one to be asked for
  uint32_t under_way = 0;            // groups asked for and not read
  bool dead = false;
  C8Walk walk = c8_walk(p, sh);
  C8Seg seg;
  while (c8_next(p, walk, seg)) {
    const C8Tile& t = seg.t;
    const int h = seg.h, first = seg.first, n = seg.n;  // units here
    const int firsts = p.window > 0 ? p.sinks : 0;
    // pages of 16 groups of tokens, a lane for 16 tokens, 16 groups ahead
    int pgA, offA, pgB, offB;
    auto pages = [&](int i, int& pg, int& off) {
      pg = -1;
      off = 0;
      if (i < n) {
        const int t0 = c8_unit(t, first + i) + 32 * warp + 16 * (lane & 1);
        if (t0 < t.hi && (t0 + 16 > t.lo || t0 < firsts)) {
          const int j = t0 / p.block;
          off = t0 - j * p.block;
          pg = p.table[(int64_t)t.b * p.max_blocks + j];
          if (pg < 0 || pg >= p.pages) {
            pg = -1;
            if (p.status) atomicOr(p.status, 1);
          }
        }
      }
    };
    pages(lane >> 1, pgB, offB);
    // lane 0, 1: K of the group's tokens, 2, 3: V; pages and scales of the next group to be asked for
    int pg = -1, off = 0;
    float sc = 1.f;
    auto look = [&](int i) {
      if ((i & 15) == 0) {
        pgA = pgB;
        offA = offB;
        pages(i + 16 + (lane >> 1), pgB, offB);
      }
      const int from = 2 * (i & 15) + (lane & 1);
      pg = __shfl_sync(kFull, pgA, from);
      off = __shfl_sync(kFull, offA, from);
      sc = 1.f;
      if (lane < 4 && pg >= 0) sc = __ldg((lane < 2 ? p.kscale : p.vscale) + (int64_t)pg * p.Hkv + h);
    };
    auto put_scale = [&](int slot, int part) {
      float* to = reinterpret_cast<float*>(&s_scale[warp][slot][part & 1]);
      if (part < 2) {
        to[0] = sc;
      } else {
        const float vs = c8_vscale(sc);
        to[1] = log2f(vs);
        to[2] = c8_inverse(vs);
      }
    };
    uint32_t live = 0;  // two bits a group asked for: which of its tokens are there, the last group's in bits 0 and 1
    auto issue = [&](int i) {
      const uint32_t there = __ballot_sync(kFull, pg >= 0) & 3u;
      live = (live << 2) | there;
      if (lane < 4) put_scale((int)ps, lane);
      if (lane == 0) mbar_arrive_expect_tx(&s_full[warp][ps], (uint32_t)__popc(there) * 32 * D);
      __syncwarp();
      if (lane < 4 && pg >= 0)
        tma_load_3d(ring + ps * SLOT + (lane >> 1) * (32 * D) + (lane & 1) * (16 * D), lane < 2 ? &kmap : &vmap, 0, off,
                    pg * p.Hkv + h, &s_full[warp][ps]);
      if (++ps == ST) ps = 0;
      ++under_way;
      if (i + 1 < n) look(i + 1);
    };
    // the first groups all at once, lanes 4·i.. for group i; no copy waits for a scale
    if (!dead) {
      const int count = min(ST, n), i = lane >> 2;
      pgA = pgB;
      offA = offB;
      pages(16 + (lane >> 1), pgB, offB);
      const int from = 2 * i + (lane & 1);
      pg = __shfl_sync(kFull, pgA, from);
      off = __shfl_sync(kFull, offA, from);
      if (i >= count) pg = -1;
      const uint32_t there = __ballot_sync(kFull, pg >= 0);
#pragma unroll
      for (int k = 0; k < ST; ++k)
        if (k < count) live = (live << 2) | ((there >> (4 * k)) & 3u);
      const int at = (int)ps + i < ST ? (int)ps + i : (int)ps + i - ST;
      if (i < count && (lane & 3) == 0)
        mbar_arrive_expect_tx(&s_full[warp][at], (uint32_t)__popc((there >> (4 * i)) & 3u) * 32 * D);
      __syncwarp();
      const int part = lane & 3;
      if (pg >= 0) {
        tma_load_3d(ring + at * SLOT + (part >> 1) * (32 * D) + (part & 1) * (16 * D), part < 2 ? &kmap : &vmap, 0, off,
                    pg * p.Hkv + h, &s_full[warp][at]);
        sc = __ldg((part < 2 ? p.kscale : p.vscale) + (int64_t)pg * p.Hkv + h);
      }
      if (i < count) put_scale(at, part);
      ps = (int)ps + count < ST ? ps + count : ps + count - ST;
      under_way += count;
      if (count < n) look(count);
    }
    // ---- the rows of q, as operands
#pragma unroll 1
    for (int r = warp; r < TILE; r += kAtWarps) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      const int rho = t.row0 + r, i = rho / p.G;
      if (r < t.nrow && 4 * lane < D)
        x = load4(static_cast<const T*>(p.q) + (int64_t)(t.start + i) * p.qs + (int64_t)(h * p.G + rho - i * p.G) * D + 4 * lane);
      float top = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      const int ex = c8_row_exp(top);
      const float f = c8_pow2(-ex);
      x.x *= f;
      x.y *= f;
      x.z *= f;
      x.w *= f;
      if (4 * lane < D) {
        // coordinates 4·lane..: operand word (k-step) 4·(lane/16) + lane % 4 of lane 4r + (lane/4) % 4
        uint2 hi, lo;
        split2(x.x, x.y, hi.x, lo.x);
        split2(x.z, x.w, hi.y, lo.y);
        const int ks = 4 * (lane >> 4) + (lane & 3), to = 4 * (r & 7) + ((lane >> 2) & 3);
        qf[r >> 3][0][ks][to] = hi;
        if (QT == 2) qf[r >> 3][QT - 1][ks][to] = lo;
      }
      if (lane == 0) {
        s_c[r] = p.zscale * c8_pow2(ex);
        s_pos[r] = r < t.nrow ? (int)min((int64_t)t.len + i, (int64_t)INT32_MAX) : -1;
      }
    }
    __syncthreads();
    uint2 bq[QREG ? NT : 1][QREG ? QT : 1][QREG ? KS : 1];
    if constexpr (QREG) {
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int y = 0; y < QT; ++y)
#pragma unroll
          for (int k = 0; k < KS; ++k) bq[x][y][k] = qf[x][y][k][lane];
    }
    float cf[NT][2], M[NT][2], L[NT][2], O[NT][KS][4];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        cf[x][e] = s_c[8 * x + 2 * c + e];
        M[x][e] = -INFINITY;
        L[x][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[x][i][e] = 0.f;
    }
    // tokens that every row of the tile sees: up to seen, and from every on or within the first ones
    const int64_t seen = (int64_t)t.len + t.i0;
    const int64_t every = p.window > 0 ? (int64_t)t.len + t.il - p.window + 1 : 0;
#pragma unroll 1
    for (int i = 0; i < n && !dead; ++i) {
      for (uint32_t k = 0; !mbar_try_wait(&s_full[warp][cs], cph); ++k)
        if (k >= kAtPolls) {  // (never, while copies land)
          dead = true;
          break;
        }
      dead = __any_sync(kFull, dead);
      if (dead) break;
      const uint32_t there = (live >> (2 * (min(n - i, ST) - 1))) & 3u;
      const unsigned char* sl = ring + cs * SLOT;
      if (there) {
        const int t0 = c8_unit(t, first + i) + 32 * warp;
        const float4 sc0 = s_scale[warp][cs][0], sc1 = s_scale[warp][cs][1];
        // ---- scores
        float z[2][NT][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int x = 0; x < NT; ++x) z[hf][x][0] = z[hf][x][1] = z[hf][x][2] = z[hf][x][3] = 0.f;
          const int r = kTok<D>(g);
          const unsigned char* row = sl + (16 * hf + r) * D;
          const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
#pragma unroll
          for (int x = 0; x < KP; ++x) {
            const uint4 ka = *reinterpret_cast<const uint4*>(row + (((c + 4 * x) ^ sw) << 4));
            const uint4 kb = *reinterpret_cast<const uint4*>(row + 8 * D + (((c + 4 * x) ^ sw) << 4));
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t a0 = c8_wide(wa[j]), a1 = c8_wide(wb[j]), a2 = c8_wide_hi(wa[j]), a3 = c8_wide_hi(wb[j]);
#pragma unroll
              for (int y = 0; y < NT; ++y)
#pragma unroll
                for (int q = 0; q < QT; ++q) {
                  const uint2 bb = QREG ? bq[QREG ? y : 0][QREG ? q : 0][QREG ? 4 * x + j : 0] : qf[y][q][4 * x + j][lane];
                  mma16816(z[hf][y], a0, a1, a2, a3, bb.x, bb.y);
                }
            }
          }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              z[hf][x][e] = fmaf(z[hf][x][e], cf[x][e & 1] * (hf ? sc1.x : sc0.x), hf ? sc1.y : sc0.y);
        const bool masked = !(there == 3u && t0 + 31 <= seen && t0 + 31 < t.hi && (t0 >= every || t0 + 31 < firsts));
        if (masked) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int at = t0 + 16 * hf + kTok<D>(g) + 8 * (e >> 1), pos = s_pos[8 * x + 2 * c + (e & 1)];
                const bool sees = ((there >> hf) & 1u) && at < t.hi && at <= pos &&
                                  (p.window == 0 || (int64_t)at > (int64_t)pos - p.window || at < firsts);
                if (!sees) z[hf][x][e] = -INFINITY;
              }
        }
        bool up = false;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            // (the difference: of large scores M + 14 may round to M + 16, past fp16's range)
            up |= fmaxf(fmaxf(z[0][x][e], z[0][x][e + 2]), fmaxf(z[1][x][e], z[1][x][e + 2])) - M[x][e] > kAtRaise;
        if (__any_sync(kFull, up)) {
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(fmaxf(z[0][x][e], z[0][x][e + 2]), fmaxf(z[1][x][e], z[1][x][e + 2]));
#pragma unroll
              for (int o = 4; o <= 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
              if (top - M[x][e] > kAtRaise) {
                float m = top - kAtFresh;
                if (top - m > kAtRaise) m = top;  // (rounded, of a large score)
                const float f = M[x][e] == -INFINITY ? 0.f : ex2(M[x][e] - m);
                M[x][e] = m;
                L[x][e] *= f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                  O[x][k][e] *= f;
                  O[x][k][e + 2] *= f;
                }
              }
            }
        }
        // ---- weights, transposed
        uint32_t bp[2][NT][PT][2];
        float sum[NT][2];  // of the weights: one rounding into the row's for both halves
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float m = M[x][e & 1];
              w[e] = ex2(z[hf][x][e] - (m == -INFINITY ? 0.f : m));
            }
            const float iv = hf ? sc1.z : sc0.z;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sum[x][e] = fmaf(w[e] + w[e + 2], iv, hf ? sum[x][e] : 0.f);
              if (hf) L[x][e] += sum[x][e];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if constexpr (PT == 2) {
                uint32_t hi, lo;
                if constexpr (QT == 2)
                  split2_low(w[2 * e], w[2 * e + 1], hi, lo);
                else
                  split2(w[2 * e], w[2 * e + 1], hi, lo);
                bp[hf][x][0][e] = transpose8(hi);
                bp[hf][x][PT - 1][e] = transpose8(lo);
              } else {
                bp[hf][x][0][e] = transpose8(pack_f16x2(w[2 * e], w[2 * e + 1]));
              }
            }
          }
        // ---- values
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t wv[4][D / 32];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = (D == 128 ? c + 4 * (x & 1) : 2 * c + (x & 1)) + 8 * (x >> 1);  // the tokens of operand rows 2c, 2c + 1
            const unsigned char* row = sl + 32 * D + (16 * hf + r) * D;
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(row + ((kTok<D>(g) ^ (r & 7)) << 4));
              wv[x][0] = v.x;
              wv[x][1] = v.y;
              wv[x][D / 32 - 2] = v.z;
              wv[x][D / 32 - 1] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(row + ((((g >> 1) ^ (r >> 1)) & 3) << 4) + ((g & 1) << 3));
              wv[x][0] = v.x;
              wv[x][1] = v.y;
            }
            if (masked) {  // what no row sees may be anything, and 0 times it a NaN
              const int at = t0 + 16 * hf + r;
              if (!(((there >> hf) & 1u) && at < t.hi && (at >= t.lo || at < firsts)))
#pragma unroll
                for (int k = 0; k < D / 32; ++k) wv[x][k] = 0;
            }
          }
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const uint32_t lo = __byte_perm(wv[0][k], wv[1][k], o ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(wv[2][k], wv[3][k], o ? 0x7362 : 0x5140);
              const uint32_t a0 = c8_wide(lo), a1 = c8_wide_hi(lo), a2 = c8_wide(hi), a3 = c8_wide_hi(hi);
#pragma unroll
              for (int x = 0; x < NT; ++x) {
                if constexpr (QT == 2) {
                  // fp32: 16 tokens by themselves, since the matrix units cut what a long sum
                  // has no bits for (64 requests over 65536: 2e-5 to 6e-5 off, 6e-7 this way, for
                  // 140 -> 145 us of 32 single tokens over up to 16384); their second terms first
                  float part[4] = {0.f, 0.f, 0.f, 0.f};
                  mma16816(part, a0, a1, a2, a3, bp[hf][x][PT - 1][0], bp[hf][x][PT - 1][1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) part[e] *= 1.f / kLow;
                  mma16816(part, a0, a1, a2, a3, bp[hf][x][0][0], bp[hf][x][0][1]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) O[x][2 * k + o][e] += part[e];
                } else {
#pragma unroll
                  for (int q = 0; q < PT; ++q) mma16816(O[x][2 * k + o], a0, a1, a2, a3, bp[hf][x][q][0], bp[hf][x][q][1]);
                }
              }
            }
          }
        }
      }
      if (++cs == ST) {
        cs = 0;
        cph ^= 1u;
      }
      --under_way;
      __syncwarp();  // the slot has been read
      if (i + ST < n) issue(i + ST);
    }
    __syncthreads();  // the rings are free: the warps' states go there
    float* mg = reinterpret_cast<float*>(smem) + warp * (TILE * REC);
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = L[x][e];
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
        float* to = mg + (8 * x + 2 * c + e) * REC;
        // (a row all of whose scores are no numbers has no maximum: its NaN goes on)
        if (g == 0) *reinterpret_cast<float2*>(to) = make_float2(M[x][e] == -INFINITY && l != l ? 0.f : M[x][e], l);
#pragma unroll
        for (int k = 0; k < KS; ++k)
          *reinterpret_cast<float2*>(to + 4 + kTok<D>(g) * (D / 8) + 2 * k) = make_float2(O[x][k][e], O[x][k][e + 2]);
      }
    }
    __syncthreads();
    const bool whole = first == 0 && n == t.n;
#pragma unroll 1
    for (int r = warp; r < t.nrow; r += kAtWarps) {
      constexpr int E = D / 32;  // coordinates of a lane
      const float* from = reinterpret_cast<const float*>(smem) + r * REC;
      float m[kAtWarps], top = -INFINITY, l = 0.f, o[E];
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        m[w] = from[w * (TILE * REC)];
        top = fmaxf(top, m[w]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        const float f = m[w] == -INFINITY ? 0.f : ex2(m[w] - top), lw = from[w * (TILE * REC) + 1];
        if (f != 0.f || lw != lw) {  // (a NaN goes on, whatever outweighs it)
          l = fmaf(lw, f, l);
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = fmaf(from[w * (TILE * REC) + 4 + E * lane + e], f, o[e]);
        }
      }
      if (whole) {
        const int rho = t.row0 + r, i = rho / p.G;
        T* to = static_cast<T*>(p.out) + ((int64_t)(t.start + i) * p.Hq + h * p.G + rho - i * p.G) * D + E * lane;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= inv;
        c8_store<T, E>(to, o);
      } else {
        float* to = p.rec + (((int64_t)blockIdx.x * 2 + (first == 0)) * TILE + r) * REC;
        if (lane == 0) *reinterpret_cast<float2*>(to) = make_float2(top, l);
        c8_store<float, E>(to + 4 + E * lane, o);
      }
    }
    if (first == 0 && !whole) {
      split.row0 = t.row0;
      split.nrow = t.nrow;
      split.start = t.start;
      split.h = h;
      split.u0 = seg.u0;
      split.u1 = seg.u0 + t.n + p.pad;
    }
    fence_proxy_async();  // before copies take the states' place
    __syncthreads();
  }
  split.units = sh.units;
  if (tid == 0) p.split[blockIdx.x] = split;
  if (dead) {  // copies under way land before the CTA ends (bounded)
    if (lane == 0 && p.status) atomicOr(p.status, 2);
    for (; under_way; --under_way) {
      for (uint32_t k = 0; k < kAtPolls / 64 && !mbar_try_wait(&s_full[warp][cs], cph); ++k) {
      }
      if (++cs == ST) {
        cs = 0;
        cph ^= 1u;
      }
    }
  }
}

// The parts k0, k0 + every, .. of row r (part 0: of the CTA that began the tile), in
// the warp's running maximum, sum and sums of values, AT of them in flight; whole warps.
template <int D, int AT>
__device__ __forceinline__ void join_row(const C8Params& p, const C8Split& s, int parts, int r, int k0, int every, float& M, float& L,
                                         float (&o)[D / 32]) {
  constexpr int REC = D + 4, E = D / 32;
  const int lane = threadIdx.x & 31, c0 = blockIdx.x;
  const int64_t step = 2 * (int64_t)p.tile * REC;
  const float* own = p.rec + (((int64_t)c0 * 2 + 1) * p.tile + r) * REC;
  const float* more = p.rec + (int64_t)r * REC;  // of CTA k: + k·step
#pragma unroll 1
  for (; k0 < parts; k0 += every * AT) {
    // a lane looks at the maximum and the sum of a part
    const int k = k0 + every * lane;
    bool on = lane < AT && k < parts;
    if (on && k > 0 && s.units < p.ctas) on = c8_cut(c0 + k + 1, s.units, p.ctas) != c8_cut(c0 + k, s.units, p.ctas);
    const uint32_t asked = __ballot_sync(kFull, on);
    float m = -INFINITY, l = 0.f;
    if (on) {
      const float2 ml = *reinterpret_cast<const float2*>(k == 0 ? own : more + (c0 + k) * step);
      m = ml.x;
      l = ml.y;
    }
    float a[AT][E];
#pragma unroll
    for (int q = 0; q < AT; ++q) {
      const int kq = k0 + every * q;
      const float* at = (kq == 0 ? own : more + (c0 + kq) * step) + 4 + E * lane;
#pragma unroll
      for (int e = 0; e < E; ++e) a[q][e] = 0.f;
      if ((asked >> q) & 1u) c8_load<E>(at, a[q]);
    }
    on = on && l != 0.f;  // saw nothing (a NaN goes on)
    float top = on ? m : -INFINITY;
#pragma unroll
    for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
    const float nm = fmaxf(M, top), use = nm == -INFINITY ? 0.f : nm;
    const float fa = M == -INFINITY ? 0.f : ex2(M - use);
    const float f = on ? ex2(m - use) : 0.f;
    float ls = on ? l * f : 0.f;
#pragma unroll
    for (int i = 16; i; i >>= 1) ls += __shfl_xor_sync(kFull, ls, i);
    L = L * fa + ls;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= fa;
#pragma unroll
    for (int q = 0; q < AT; ++q) {
      const float fk = __shfl_sync(kFull, f, q);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fk == 0.f ? o[e] : fmaf(a[q][e], fk, o[e]);
    }
    M = nm;
  }
}

// The parts of the tiles that several CTAs worked on.  The CTAs of blockIdx.x join the
// rows of the tile that CTA blockIdx.x there began and did not end.  They are let in
// while the kernel before is under way, and wait beside its own.
// Few rows a tile: a warp a row.  A long request's parts are some 40, and four warps
// join a row where they are more than one has in flight (one token over 131072: 56 ->
// 53 us).
constexpr int kJoinThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) c8_join_kernel(const C8Params p) {
  constexpr int E = D / 32, W = kJoinThreads / 32, AT = 12;  // coordinates of a lane, warps, records in flight
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const C8Split s = p.split[blockIdx.x];
  if (s.h < 0) return;
  const int parts = (int)((s.u1 * p.ctas - 1) / s.units) - (int)blockIdx.x + 1;
  float M, L, o[E];
  auto begin = [&]() {
    M = -INFINITY;
    L = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
  };
  auto put = [&](int r) {
    const int rho = s.row0 + r, i = rho / p.G;
    T* to = static_cast<T*>(p.out) + ((int64_t)(s.start + i) * p.Hq + s.h * p.G + rho - i * p.G) * D + E * lane;
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= inv;
    c8_store<T, E>(to, o);
  };
  if (parts <= AT) {
#pragma unroll 1
    for (int r = W * blockIdx.y + warp; r < s.nrow; r += W * gridDim.y) {
      begin();
      join_row<D, AT>(p, s, parts, r, 0, 1, M, L, o);
      put(r);
    }
    return;
  }
  __shared__ float s_m[W], s_l[W], s_o[W][D];
#pragma unroll 1
  for (int r0 = 2 * blockIdx.y; r0 < s.nrow; r0 += 2 * gridDim.y) {
    const int r = r0 + (warp >> 2);
    begin();
    if (r < s.nrow) join_row<D, AT>(p, s, parts, r, warp & 3, 4, M, L, o);
    __syncthreads();  // the rows before have been read
    if (lane == 0) {
      s_m[warp] = L == 0.f ? -INFINITY : M;
      s_l[warp] = L;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][E * lane + e] = o[e];
    __syncthreads();
    if ((warp & 3) == 0 && r < s.nrow) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, s_m[warp + w]);
      begin();
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = s_m[warp + w] == -INFINITY ? 0.f : ex2(s_m[warp + w] - top);
        if (f == 0.f && s_l[warp + w] == s_l[warp + w]) continue;  // (a NaN goes on)
        L = fmaf(s_l[warp + w], f, L);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(s_o[warp + w][E * lane + e], f, o[e]);
      }
      put(r);
    }
  }
}

// From 128 rows a tile on: the parts are two or three where the tiles are many.  A warp
// takes 8 rows and 32 coordinates, a lane 8 coordinates of a row: the records' four
// sums of 8 rows stand together (and those of 32 where the kernel before stores them;
// with rows of d + 4 numbers instead, a store met 32 lines: prompt of 8179 with a window
// 130 against 122 us).  No shared memory, so that CTAs find room beside that kernel's
// (with some, 5 to 20 us more).
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 3) c8_join_wide_kernel(const C8Params p) {
  constexpr int REC = D + 4, W = kJoinThreads / 32, AT = 4, CG = D / 32;  // records in flight, column groups
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x;
  const C8Split s = p.split[c0];
  if (s.h < 0) return;
  const int parts = (int)((s.u1 * p.ctas - 1) / s.units) - c0 + 1;
  const int64_t size = (int64_t)p.tile * REC;
#pragma unroll 1
  for (int u = W * blockIdx.y + warp; u < (s.nrow + 7) / 8 * CG; u += W * gridDim.y) {
    const int r = 8 * (u / CG) + (lane >> 2), c8 = 4 * (u % CG) + (lane & 3);  // row, eight coordinates
    const bool here = r < s.nrow;
    float M = -INFINITY, L = 0.f, o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < parts; k0 += AT) {
      float m[AT], l[AT], a[AT][2][4];
#pragma unroll
      for (int q = 0; q < AT; ++q) {
        const int k = k0 + q;
        const bool on = here && k < parts &&
                        (k == 0 || s.units >= p.ctas || c8_cut(c0 + k + 1, s.units, p.ctas) != c8_cut(c0 + k, s.units, p.ctas));
        const float* rec = p.rec + ((int64_t)(c0 + k) * 2 + (k == 0)) * size;
        m[q] = -INFINITY;
        l[q] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) a[q][e >> 2][e & 3] = 0.f;
        if (on) {
          const float2 ml = *reinterpret_cast<const float2*>(rec + 2 * r);
          m[q] = ml.x;
          l[q] = ml.y;
#pragma unroll
          for (int e = 0; e < 2; ++e) c8_load<4>(rec + 4 * ((int64_t)p.tile * (1 + 2 * c8 + e) + r), a[q][e]);
        }
      }
      float top = M;
#pragma unroll
      for (int q = 0; q < AT; ++q)
        if (l[q] != 0.f) top = fmaxf(top, m[q]);  // (0: saw nothing; a NaN goes on)
      const float use = top == -INFINITY ? 0.f : top, fa = M == -INFINITY ? 0.f : ex2(M - use);
      M = top;
      L *= fa;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= fa;
#pragma unroll
      for (int q = 0; q < AT; ++q) {
        const float f = l[q] != 0.f ? ex2(m[q] - use) : 0.f;
        if (f == 0.f && l[q] == l[q]) continue;  // (a NaN goes on)
        L = fmaf(l[q], f, L);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(a[q][e >> 2][e & 3], f, o[e]);
      }
    }
    if (here) {
      const int rho = s.row0 + r, i = rho / p.G;
      const float inv = L == 0.f ? 0.f : 1.f / L;
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = c8_pair<T>(o[2 * e] * inv, o[2 * e + 1] * inv);
      *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + ((int64_t)(s.start + i) * p.Hq + s.h * p.G + rho - i * p.G) * D + 8 * c8) =
          make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

template <typename T, int D, int NT>
cudaError_t run_attend(const C8Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t st) {
  static PerDeviceValue attr;
  const cudaError_t e = smem_attr_once(attr, (const void*)c8_attend_kernel<T, D, NT>, kAtSmem<T, D, NT>);
  return e != cudaSuccess ? e
                          : c8_launch(c8_attend_kernel<T, D, NT>, dim3(p.ctas), kAtThreads, kAtSmem<T, D, NT>, st, p, kmap, vmap);
}
template <typename T, int D>
cudaError_t run_attend_d(const C8Params& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  cudaError_t e = p.tile == 8    ? run_attend<T, D, 1>(p, k, v, st)
                  : p.tile == 16 ? run_attend<T, D, 2>(p, k, v, st)
                  : p.tile == 32 ? run_attend<T, D, 4>(p, k, v, st)
                                 : c8_attend_umma(p, st);
  if (e != cudaSuccess) return e;
  if (p.tile <= 32) return c8_launch(c8_join_kernel<T, D>, dim3(p.ctas, p.tile / 4), kJoinThreads, 0, st, p);
  if constexpr (sizeof(T) == 2) e = c8_launch(c8_join_wide_kernel<T, D>, dim3(p.ctas, 16), kJoinThreads, 0, st, p);
  return e;
}
template <typename T>
cudaError_t run_attend_t(const C8Params& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  return p.d == 64 ? run_attend_d<T, 64>(p, k, v, st) : run_attend_d<T, 128>(p, k, v, st);
}

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// Rows of a tile, by a mean request's rows: the smallest that hold them.  From 33 on
// fp16 and bf16 rows go to the fifth-generation tensor cores (8 requests over 8191, 32/8
// heads of 128, up to 12 and 15 tokens: 47 us, with two 32-row tiles each 71 to 90; of up
// to 6 and 8, where these take 51 to 59, the tensor cores' tile would take 45; 32 requests
// over 2048 with heads of 64: 46 to 52 and 43 to 50).  One size for a whole call: a piece of
// 512 beside 255 single tokens takes 1114 us, the two in calls of their own 847.
int tile_rows(int64_t rows, int B, int G, bool umma) {
  const int64_t mean = (rows * G + B - 1) / B;
  return mean <= 8 ? 8 : mean <= 16 ? 16 : mean <= 32 || !umma ? 32 : mean <= 128 ? 128 : 256;
}
// CTAs of the grid: as many as fit at once.
int grid_ctas(int tile) { return num_sms() * (tile <= 32 ? 2 : 1); }

}  // namespace

size_t cache8_ws_bytes(int d, int B, int Hq, int Hkv, int64_t rows) {
  const int tile = tile_rows(rows, B, Hq / Hkv, true);  // (no fewer than the other kernel's)
  const size_t ctas = (size_t)num_sms() * 2, parts = (size_t)grid_ctas(tile) * 2;
  return al256(ctas * sizeof(C8Split)) + (parts + (tile == 128 ? parts / 2 : 0)) * tile * (d + 4) * 4;
}

tq_status launch_cache8_attention(const Cache8AttendArgs& a, cudaStream_t stream) {
  const tq_cache8& c = *a.cache;
  C8Params p{};
  p.q = a.q;
  p.qs = a.q_stride;
  p.dtype = a.dtype;
  p.row_start = a.row_start;
  p.len = a.len;
  p.table = a.table;
  p.rows = (int)a.rows;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = c.Hkv;
  p.G = a.Hq / c.Hkv;
  p.max_blocks = a.max_blocks;
  p.block = c.block;
  p.d = c.d;
  p.window = a.window;
  p.sinks = a.window > 0 ? a.sinks : 0;
  p.pages = c.pages;
  p.k8 = c.d_k;
  p.v8 = c.d_v;
  p.kscale = c.d_kscale;
  p.vscale = c.d_vscale;
  p.zscale = a.scale * kC8Log2e;
  p.out = a.out;
  p.status = c.d_status;
  p.tile = tile_rows(a.rows, a.B, p.G, a.dtype != TQ_F32);
  p.ctas = grid_ctas(p.tile);
  // (of 1 to 5: 128 rows with 3 46.7 us for 8 x 15 drafted, with 5 45.7; 8 to 32 rows with 1
  // 20.9 us for 16 x 7 with a window, with 2 17.7, with 3 19.0)
  p.pad = p.tile == 256 ? 3 : p.tile == 128 ? 5 : 2;
  p.split = static_cast<C8Split*>(a.ws);
  p.rec = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + al256((size_t)num_sms() * 2 * sizeof(C8Split)));
  const int64_t slots = a.rows * p.G / p.tile + a.B;
  const int64_t most = (int64_t)a.max_blocks * c.block / kC8Unit + 2 + p.pad;  // counted units of a tile
  if (slots > INT32_MAX || most * p.Hkv > INT32_MAX || c.pages > INT32_MAX / p.Hkv) return TQ_ERR_UNSUPPORTED;
  p.slots = (int)slots;
  CUtensorMap kmap, vmap;
  tq_status ms = pages_tensor_map(&kmap, c.d_k, c.pages * c.Hkv, c.block, c.d);
  if (ms == TQ_OK) ms = pages_tensor_map(&vmap, c.d_v, c.pages * c.Hkv, c.block, c.d);
  if (ms != TQ_OK) return ms;
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.dtype) {
    case TQ_F32: e = run_attend_t<float>(p, kmap, vmap, stream); break;
    case TQ_F16: e = run_attend_t<__half>(p, kmap, vmap, stream); break;
    case TQ_BF16: e = run_attend_t<__nv_bfloat16>(p, kmap, vmap, stream); break;
  }
  return e == cudaSuccess ? TQ_OK : set_cuda_error(e);
}

}  // namespace tq
