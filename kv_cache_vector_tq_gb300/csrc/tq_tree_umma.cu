// Attention of drafted tokens over a packed cache on the fifth-generation
// tensor cores (fp16 and bf16 inputs).  tq_tree.cuh has the mathematics and
// the division of the work into units of 128 tokens.
//
// A persistent CTA per SM; per unit, with 128 rows (drafted token x query
// head) on the lanes of tensor memory:
//     S[row][token] = Q̂·K̂ᵀ       A = Q̂ (tensor memory), B = K̂ (shared memory)
//     P = 2^(S·s_k·c - M)·s_v     in fp16, over S's own columns
//     O[row][coord] += P·V̂        A = P (tensor memory), B = V̂ᵀ (shared memory)
// K̂ and V̂ are the codebook's fp16 pairs (α·c) in the 128-byte swizzle; the
// norms are applied to the score and to the weight in fp32, so no rounding
// depends on them.  M is the running maximum of log2 weight times s_v, raised
// only when a weight would pass 2^14 (the sums are rescaled then, which is
// rare); subtracting log2 of the tile's largest s_v keeps any magnitude of the
// values inside fp16.
// Rounding of the operands: for fp16 outputs Q̂ and P are split into two fp16
// terms each (two products), since one rounding of either costs as much as the
// output's own; bf16 outputs round sixteen times coarser and take one term.
//
// Warps: 0-3 softmax (thread = row), 4-7 K̂ (thread = token: 64 table lookups
// of two codes, 16 swizzled 16-byte stores), 8-11 V̂ᵀ (thread = 8 tokens x 16
// coordinates; PAIR blocks hold two tokens of a coordinate side by side, which
// is V̂ᵀ's order), 12 issues the products, 13 the bulk copies of the packed
// tiles (per 16 tokens, so pages may end anywhere on a multiple of 16).
// Lookup tables are replicated per lane (one bank each) and aligned so that an
// address is one shift and one and-or.
#include "tq_tree.cuh"

namespace tq {

namespace {

constexpr int kThreads = 14 * 32;
constexpr int kOp = 128 * 256;            // bytes of one 128 x 128 fp16 operand
constexpr int kNormSlots = 4;
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384;  // tensor memory: S/P x 2, O, Q̂ (hi 64 | lo 64)
constexpr float kLazyUp = 14.f;           // raise M before a weight passes 2^14
constexpr float kShift = 6.f;             // a fresh maximum sits at weight 2^6: small weights keep their bits longer

// Shared memory by absolute address (dynamic shared memory starts at 1024, the
// system's reserved bytes): raw tiles, [the K table], the V table (or both) at
// 64 KB, the operands, norms and barriers.
constexpr uint32_t kBase = 1024;
constexpr uint32_t kLutV = 65536;
constexpr uint32_t kOps = kLutV + 32768;  // K̂ x 2, V̂ x 2
constexpr uint32_t kNorms = kOps + 4 * kOp;  // [slot][K | V][128] fp32
constexpr uint32_t kBars = kNorms + 3072;     // three norm slots here, the fourth below the tables
constexpr uint32_t kEnd = 1024 + 227 * 1024;
constexpr uint32_t kRaw = kBase + 1024;       // the fourth norm slot comes first

__host__ __device__ constexpr uint32_t lut_bytes(int b) { return (1u << (2 * b)) * 128u; }
__host__ __device__ constexpr uint32_t raw_v_off(int kb) { return 2048u * kb; }
__host__ __device__ constexpr uint32_t raw_bytes(int kb, int vb) { return 2048u * kb + 16u * (128u * vb + 16u); }

struct Bars {
  uint64_t raw_full[3], raw_empty[3];
  uint64_t kh_full[2], kh_empty[2], vh_full[2], vh_empty[2];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t n_full[kNormSlots], n_empty[kNormSlots];
  uint64_t q_full, drain;
  uint32_t valid[kNormSlots];  // 16-token chunks of the tile that are there
  uint32_t tmem;
  int abort;
};
static_assert(kBars + sizeof(Bars) <= kEnd, "shared memory");

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Two fp32 values in one 64-bit register: one instruction per pair.
__device__ __forceinline__ uint64_t pk2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void up2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Tensor-memory loads complete; the loaded registers pass through, so that
// nothing that uses them moves ahead of the wait.
template <int N>
__device__ __forceinline__ void wait_ld(uint32_t (&r)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Table entry of the 2B-bit field at bit `off` (a constant once unrolled) of
// w: the field moved to bits 7.., then one and-or with the lane's table base.
template <int B, int N>
__device__ __forceinline__ uint32_t look(const uint32_t (&w)[N], int off, uint32_t base) {
  constexpr uint32_t m = ((1u << (2 * B)) - 1u) << 7;
  const int i = off >> 5, s = off & 31;
  uint32_t x;
  if (s + 2 * B > 32)
    x = __funnelshift_r(w[i], w[i + 1 < N ? i + 1 : i], s) << 7;
  else if (s >= 7)
    x = w[i] >> (s - 7);
  else
    x = w[i] << (7 - s);
  return lds32((x & m) | base);
}

// K̂ row of token t: 16 chunks of 8 coordinates.
template <int B>
__device__ __forceinline__ void dequant_k(uint32_t raw, uint32_t op, uint32_t lut, int t) {
  const uint32_t row = op + t * 128, sw = (uint32_t)(t & 7) << 4;
  if constexpr (B == 4) {
    // 16-byte pieces in an order that differs between lanes: rows are 64 bytes,
    // eight lanes reading the same piece would meet in two banks of eight
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = (i + (t >> 1)) & 3;  // coordinates 32x..
      const uint4 u = lds128(raw + t * 64 + 16 * x);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      const uint32_t at = row + ((x >> 1) << 14);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t c = (uint32_t)(4 * (x & 1) + e) << 4;
        const uint32_t v0 = look<4>(w, 32 * e, lut), v1 = look<4>(w, 32 * e + 8, lut);
        const uint32_t v2 = look<4>(w, 32 * e + 16, lut), v3 = look<4>(w, 32 * e + 24, lut);
        sts128(at + (c ^ sw), v0, v1, v2, v3);
      }
    }
  } else {
    uint32_t w[4 * B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const uint4 u = lds128(raw + t * (16 * B) + 16 * i);
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = look<B>(w, (8 * c + 2 * e) * B, lut);
      sts128(row + ((c >> 3) << 14) + (((c & 7) << 4) ^ sw), v[0], v[1], v[2], v[3]);
    }
  }
}

// V̂ᵀ: 8 tokens (group c8 of block blk) of coordinates 16·cg..+15.
template <int B>
__device__ __forceinline__ void dequant_v(uint32_t raw, uint32_t op, uint32_t lut, int c8, int cg, int blk) {
  uint32_t w[4][B];
  const uint32_t src = raw + (blk * 8 + c8) * (128 * B + 16) + cg * (4 * B);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (B == 4) {
      const uint4 u = lds128(src + p * 128);
      w[p][0] = u.x;
      w[p][1] = u.y;
      w[p][2] = u.z;
      w[p][3] = u.w;
    } else {
#pragma unroll
      for (int i = 0; i < B; ++i) w[p][i] = lds32(src + p * (32 * B) + 4 * i);
    }
  }
  const uint32_t at = op + (blk << 14) + cg * (16 * 128);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    uint32_t v[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = look<B>(w[p], 2 * B * k, lut);
    sts128(at + k * 128 + ((uint32_t)(c8 ^ (k & 7)) << 4), v[0], v[1], v[2], v[3]);
  }
}

template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) tree_attend_kernel(const TreeParams p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  if (smem_u32(smem) != kBase) {  // the layout below is absolute
    if (threadIdx.x == 0) atomicOr(p.status, 1);
    return;
  }
  Bars& bar = *reinterpret_cast<Bars*>(smem + (kBars - kBase));
  volatile int* abort_flag = &bar.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t lim = p.wait_limit;
  const uint32_t lut_k = p.same_lut ? kLutV : kLutV - lut_bytes(p.kb);
  const uint32_t stage = raw_bytes(p.kb, p.vb);
  const int RS = min(3, (int)((lut_k - kRaw) / stage));  // raw stages that fit below the tables
  auto norm_slot = [&](uint32_t i) -> uint32_t {
    const uint32_t s = i % kNormSlots;
    return s == 3 ? kBase : kNorms + s * 1024u;
  };

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bar.raw_full[i], 1);
      mbar_init(&bar.raw_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.kh_full[i], 4);
      mbar_init(&bar.kh_empty[i], 1);
      mbar_init(&bar.vh_full[i], 4);
      mbar_init(&bar.vh_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.pv_done[i], 1);
    }
    for (int i = 0; i < kNormSlots; ++i) {
      mbar_init(&bar.n_full[i], 1);
      mbar_init(&bar.n_empty[i], 4);
    }
    mbar_init(&bar.q_full, 4);
    mbar_init(&bar.drain, 1);
    bar.abort = 0;
    fence_mbar_init();
  }
  {
    uint32_t* lv = reinterpret_cast<uint32_t*>(smem + (kLutV - kBase));
    for (int i = tid; i < (32 << (2 * p.vb)); i += kThreads) lv[i] = __ldg(p.vlut + (i >> 5));
    if (!p.same_lut) {
      uint32_t* lk = reinterpret_cast<uint32_t*>(smem + (lut_k - kBase));
      for (int i = tid; i < (32 << (2 * p.kb)); i += kThreads) lk[i] = __ldg(p.klut + (i >> 5));
    }
  }
  if (warp == 12) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  griddep_wait();
  griddep_launch();

  const int64_t units = p.seq[p.B].unit;
  int64_t u = tree_cut(blockIdx.x, units, p.ctas);
  const int64_t u_end = tree_cut(blockIdx.x + 1, units, p.ctas);
  int b = u < u_end ? p.cta_seq[blockIdx.x] : 0;

  if (warp < 4) {
    // ---------------- softmax: thread = row
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    const uint32_t tO = tmem + lane_base + kColO, tQ = tmem + lane_base + kColQ;
    uint32_t i = 0;
    bool ok = true;
    while (ok && u < u_end) {
      const TreeSeg g = tree_seg(p, u, u_end, b);
      b = g.b;
      const int r = 32 * warp + lane, rho = g.row0 + r;
      const bool live = r < g.nrow, active = 32 * warp < g.nrow;
      const int ti = live ? rho / p.G : 0;
      const int64_t vec = live ? (int64_t)(g.s.start + ti) * p.Hq + g.kvh * p.G + (rho - ti * p.G) : 0;
      // Q̂ into tensor memory (every product of the last segment with the old
      // one has completed: its last S was read here)
      if (active) {
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __half*>(p.qrot) + vec * 256);
#pragma unroll
        for (int c = 0; c < (SPLIT ? 8 : 4); ++c) {
          uint32_t v[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 x = live ? src[4 * c + e] : make_uint4(0u, 0u, 0u, 0u);
            v[4 * e] = x.x;
            v[4 * e + 1] = x.y;
            v[4 * e + 2] = x.z;
            v[4 * e + 3] = x.w;
          }
          tmem_st16(tQ + 16 * c, v);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full);
      const float rs = live ? p.qfac[vec] * p.zfold : 0.f;
      float M = -INFINITY, l = 0.f;
      for (int t = g.first; ok && t < g.last; ++t, ++i) {
        const uint32_t sb = i & 1u, ns = i % kNormSlots;
        ok = __all_sync(kFull, bar_wait(&bar.s_full[sb], (i >> 1) & 1u, abort_flag, p.status, lim) &&
                                   bar_wait(&bar.n_full[ns], (i / kNormSlots) & 1u, abort_flag, p.status, lim));
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const uint32_t tS = tmem + lane_base + kColS + sb * 128;
          const uint32_t kn = norm_slot(i), vn = kn + 512;
          // Tokens of the tile that this row sees: all of them (whole), or the
          // bits of see(c) for tokens 32c..
          const bool draft = t >= g.ctiles;
          const int t0 = draft ? (t - g.ctiles) * kTreeTok : t * kTreeTok;
          const int nt = min(kTreeTok, (draft ? g.s.T : g.s.len) - t0);
          const uint32_t chunks = bar.valid[ns];
          const bool whole = nt == kTreeTok && chunks == 0xFFu && !draft;
          auto see = [&](int c) -> uint32_t {
            const int n = nt - 32 * c;
            const uint32_t m = n >= 32 ? 0xFFFFFFFFu : (n > 0 ? (1u << n) - 1u : 0u);
            if (!draft)
              return m & (((chunks >> (2 * c)) & 1u ? 0xFFFFu : 0u) | ((chunks >> (2 * c + 1)) & 1u ? 0xFFFF0000u : 0u));
            if (p.mask) {
              const int at = (t0 >> 5) + c;
              return m & (live && at < p.mask_words ? p.mask[(int64_t)(g.s.start + ti) * p.mask_words + at] : 0u);
            }
            const int k = ti - t0 - 32 * c + 1;  // a chain: tokens 0..ti
            return m & (k >= 32 ? 0xFFFFFFFFu : (k > 0 ? (1u << k) - 1u : 0u));
          };
          // largest s_v of the tile (of the tokens that are there), as a power
          // of two's exponent
          float vmax = 0.f;
          {
            const uint4 x = lds128(vn + 16 * lane);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            const uint32_t here = whole ? 0xFu : (nt > 4 * lane ? 0xFu >> max(0, 4 * lane + 4 - nt) : 0u) *
                                                     (draft ? 1u : ((chunks >> (lane >> 2)) & 1u));
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((here >> e) & 1u) vmax = fmaxf(vmax, __uint_as_float(w[e]));
#pragma unroll
            for (int o = 16; o; o >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(kFull, vmax, o));
          }
          // 2^lv >= vmax, kept within 2^±100
          const float lv = fminf(fmaxf((float)((int)(__float_as_uint(vmax) >> 23) - 126), -100.f), 100.f);
          // pass 1: the row's largest S·s_k
          float mx = -INFINITY;
          if (whole) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t s[32];
              tmem_ld32_nw(tS + 32 * c, s);
              wait_ld(s);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint4 k4 = lds128(kn + 128 * c + 16 * e);
                float a0, a1, a2, a3;
                up2(mul2(pk2(__uint_as_float(s[4 * e]), __uint_as_float(s[4 * e + 1])),
                         pk2(__uint_as_float(k4.x), __uint_as_float(k4.y))), a0, a1);
                up2(mul2(pk2(__uint_as_float(s[4 * e + 2]), __uint_as_float(s[4 * e + 3])),
                         pk2(__uint_as_float(k4.z), __uint_as_float(k4.w))), a2, a3);
                mx = fmaxf(fmaxf(mx, fmaxf(a0, a1)), fmaxf(a2, a3));
              }
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t sw = see(c);
              uint32_t s[32];
              tmem_ld32_nw(tS + 32 * c, s);
              wait_ld(s);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if ((sw >> e) & 1u) mx = fmaxf(mx, __uint_as_float(s[e]) * __uint_as_float(lds32(kn + 128 * c + 4 * e)));
            }
          }
          // a weight is 2^(z - M)·s_v <= 2^(cand - M): raise M before one passes 2^14
          const float cand = mx == -INFINITY ? -INFINITY : fmaf(mx, rs, lv);
          const bool raise = live && cand > M + kLazyUp;
          if (__any_sync(kFull, raise)) {
            const float nm = raise ? cand - kShift : M;
            const float f = raise ? (M == -INFINITY ? 0.f : ex2(M - nm)) : 1.f;
            if (t > g.first) {  // the sums so far, once the last product into them is done
              ok = __all_sync(kFull, bar_wait(&bar.pv_done[(i - 1) & 1u], ((i - 1) >> 1) & 1u, abort_flag, p.status, lim));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                tmem_ld16_nw(tO + 16 * c, o);
                wait_ld(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(tO + 16 * c, o);
              }
            }
            l *= f;
            M = nm;
          }
          const float use = M == -INFINITY ? 0.f : M;
          // pass 2: weights and their sum; the weights of 32 tokens over the 32
          // columns their scores were in (16 of leading parts, 16 of remainders)
          if (whole) {
            const uint64_t rs2 = pk2(rs, rs), nm2 = pk2(-use, -use);
            uint64_t l2 = pk2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t s[32];
              tmem_ld32_nw(tS + 32 * c, s);
              wait_ld(s);
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint4 k4 = lds128(kn + 128 * c + 16 * e), v4 = lds128(vn + 128 * c + 16 * e);
                const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w}, vw[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  float a, d, w0, w1;
                  const uint64_t z = mul2(pk2(__uint_as_float(s[4 * e + 2 * q]), __uint_as_float(s[4 * e + 2 * q + 1])),
                                          pk2(__uint_as_float(kw[2 * q]), __uint_as_float(kw[2 * q + 1])));
                  up2(fma2(z, rs2, nm2), a, d);
                  const uint64_t pp = pk2(ex2(a), ex2(d));
                  l2 = add2(l2, pp);
                  up2(mul2(pp, pk2(__uint_as_float(vw[2 * q]), __uint_as_float(vw[2 * q + 1]))), w0, w1);
                  const __half2 h = __floats2half2_rn(w0, w1);
                  hi[2 * e + q] = h2_bits(h);
                  if constexpr (SPLIT)
                    lo[2 * e + q] = h2_bits(__floats2half2_rn(w0 - __low2float(h), w1 - __high2float(h)));
                }
              }
              tmem_st16(tS + 32 * c, hi);
              if constexpr (SPLIT) tmem_st16(tS + 32 * c + 16, lo);
            }
            float la, lb;
            up2(l2, la, lb);
            l += la + lb;
          } else {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t sw = see(c);
              uint32_t s[32];
              tmem_ld32_nw(tS + 32 * c, s);
              wait_ld(s);
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float w[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const uint32_t at = 128 * c + 8 * e + 4 * q;
                  const bool on = (sw >> (2 * e + q)) & 1u;
                  const float z = __uint_as_float(s[2 * e + q]) * __uint_as_float(lds32(kn + at));
                  const float pr = on ? ex2(fmaf(z, rs, -use)) : 0.f;
                  l += pr;
                  w[q] = on ? pr * __uint_as_float(lds32(vn + at)) : 0.f;
                }
                const __half2 h = __floats2half2_rn(w[0], w[1]);
                hi[e] = h2_bits(h);
                if constexpr (SPLIT) lo[e] = h2_bits(__floats2half2_rn(w[0] - __low2float(h), w[1] - __high2float(h)));
              }
              tmem_st16(tS + 32 * c, hi);
              if constexpr (SPLIT) tmem_st16(tS + 32 * c + 16, lo);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.p_full[sb]);
          mbar_arrive(&bar.n_empty[ns]);
        }
      }
      // the segment's sums, once its last product is done
      if (!ok) break;
      ok = __all_sync(kFull, bar_wait(&bar.pv_done[(i - 1) & 1u], ((i - 1) >> 1) & 1u, abort_flag, p.status, lim));
      if (!ok) break;
      tc_fence_after();
      if (active) {
        float* rec = g.first == 0 ? p.rec + vec * kTreeRec : p.crec + ((int64_t)blockIdx.x * 128 + r) * kTreeRec;
        if (live) *reinterpret_cast<float2*>(rec) = make_float2(M, l);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32_nw(tO + 32 * c, o);
          wait_ld(o);
          if (live)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(rec + 4 + 32 * c + 4 * e) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      tc_fence_before();
      u += g.last - g.first;
    }
  } else if (warp < 12) {
    // ---------------- K̂ (warps 4-7) and V̂ᵀ (8-11) operands
    const bool is_v = warp >= 8;
    const int v = tid - (is_v ? 256 : 128);  // thread of the role
    uint64_t* full = is_v ? bar.vh_full : bar.kh_full;
    uint64_t* empty = is_v ? bar.vh_empty : bar.kh_empty;
    const uint32_t ops = kOps + (is_v ? 2u * kOp : 0u);
    const uint32_t lut = (is_v ? kLutV : lut_k) | (uint32_t)(lane * 4);
    const int c8 = v & 7, cg = (v >> 3) & 7, blk = v >> 6;  // V̂ᵀ: tokens 64·blk + 8·c8.., coordinates 16·cg..
    uint32_t i = 0, rc = 0;
    bool ok = true;
    while (ok && u < u_end) {
      const TreeSeg g = tree_seg(p, u, u_end, b);
      b = g.b;
      for (int t = g.first; t < g.last; ++t, ++i) {
        const uint32_t sb = i & 1u, op = ops + sb * kOp;
        const bool draft = t >= g.ctiles;
        const uint32_t st = rc % RS;
        ok = bar_wait(&empty[sb], ((i >> 1) & 1u) ^ 1u, abort_flag, p.status, lim) &&
             (draft || bar_wait(&bar.raw_full[st], (rc / RS) & 1u, abort_flag, p.status, lim));
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        if (!draft) {
          const uint32_t raw = kRaw + st * stage;
          if (!is_v) {
            switch (p.kb) {
              case 1: dequant_k<1>(raw, op, lut, v); break;
              case 2: dequant_k<2>(raw, op, lut, v); break;
              case 3: dequant_k<3>(raw, op, lut, v); break;
              default: dequant_k<4>(raw, op, lut, v); break;
            }
          } else {
            const uint32_t rv = raw + raw_v_off(p.kb);
            switch (p.vb) {
              case 1: dequant_v<1>(rv, op, lut, c8, cg, blk); break;
              case 2: dequant_v<2>(rv, op, lut, c8, cg, blk); break;
              case 3: dequant_v<3>(rv, op, lut, c8, cg, blk); break;
              default: dequant_v<4>(rv, op, lut, c8, cg, blk); break;
            }
          }
        } else {
          // drafted rows, rotated and rounded already; zeros past the last one
          const int t0 = (t - g.ctiles) * kTreeTok, nt = p.kn ? g.s.T - t0 : 0;
          const int64_t tok = g.s.start + t0;
          if (!is_v) {
            const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __half*>(p.krot) +
                                                              ((tok + v) * p.Hkv + g.kvh) * 128);
#pragma unroll 4
            for (int c = 0; c < 16; ++c) {
              const uint4 x = v < nt ? src[c] : make_uint4(0u, 0u, 0u, 0u);
              sts128(op + ((c >> 3) << 14) + v * 128 + ((uint32_t)((c & 7) ^ (v & 7)) << 4), x.x, x.y, x.z, x.w);
            }
          } else {
            const int first = 64 * blk + 8 * c8;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {  // 8 coordinates of 8 tokens
              uint32_t w[8][4];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint4 x = first + k < nt
                                    ? *(reinterpret_cast<const uint4*>(reinterpret_cast<const __half*>(p.vrot) +
                                                                       ((tok + first + k) * p.Hkv + g.kvh) * 128 + 16 * cg) + half)
                                    : make_uint4(0u, 0u, 0u, 0u);
                w[k][0] = x.x;
                w[k][1] = x.y;
                w[k][2] = x.z;
                w[k][3] = x.w;
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) {  // coordinate 16·cg + 8·half + k
                uint32_t q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  q[e] = __byte_perm(w[2 * e][k >> 1], w[2 * e + 1][k >> 1], (k & 1) ? 0x7632 : 0x5410);
                sts128(op + (blk << 14) + (16 * cg + 8 * half + k) * 128 + ((uint32_t)(c8 ^ k) << 4), q[0], q[1], q[2], q[3]);
              }
            }
          }
        }
        fence_proxy_async();  // generic-proxy stores, read next by the tensor cores
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[sb]);
          if (!draft) mbar_arrive(&bar.raw_empty[st]);
        }
        if (!draft) ++rc;
      }
      u += g.last - g.first;
    }
  } else if (warp == 12) {
    // ---------------- the products: S of tile j goes before P·V̂ of tile j - 1,
    // except where a new group's Q̂ has to wait for the last group's end
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_f16(128, 128);
      const int64_t n = u_end - u;
      int left = 0;
      uint32_t qn = 0;
      bool ok = true, fresh = false, fresh_prev = false;
      auto product = [&](int64_t j, bool first) -> bool {  // P·V̂ of tile j
        const uint32_t sb = (uint32_t)j & 1u, ph = (uint32_t)(j >> 1) & 1u;
        if (!bar_wait(&bar.p_full[sb], ph, abort_flag, p.status, lim) ||
            !bar_wait(&bar.vh_full[sb], ph, abort_flag, p.status, lim))
          return false;
        tc_fence_after();
        const uint32_t a = tmem + kColS + sb * 128, op = kOps + (2 + sb) * kOp;
#pragma unroll
        for (int pass = SPLIT ? 0 : 1; pass < 2; ++pass)  // remainders first: not truncated against a large sum
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma_f16_ts(tmem + kColO, a + 32 * (ks >> 1) + 8 * (ks & 1) + (pass == 0 ? 16 : 0),
                        umma_desc_sw128(op + (ks >> 2) * 16384 + (ks & 3) * 32), idesc,
                        (first && ks == 0 && pass == (SPLIT ? 0 : 1)) ? 0u : 1u);
        umma_commit(&bar.vh_empty[sb]);
        umma_commit(&bar.pv_done[sb]);
        return true;
      };
      for (int64_t j = 0; ok && j <= n; ++j) {
        if (j < n) {
          fresh_prev = fresh;
          fresh = left == 0;
          if (left == 0) {
            const TreeSeg g = tree_seg(p, u + j, u_end, b);
            b = g.b;
            left = g.last - g.first;
          }
          --left;
          if (fresh && j > 0 && !(ok = product(j - 1, fresh_prev))) break;
          if (fresh && !(ok = bar_wait(&bar.q_full, qn++ & 1u, abort_flag, p.status, lim))) break;
          const uint32_t sb = (uint32_t)j & 1u;
          if (!(ok = bar_wait(&bar.kh_full[sb], (uint32_t)(j >> 1) & 1u, abort_flag, p.status, lim))) break;
          tc_fence_after();
          const uint32_t op = kOps + sb * kOp;
#pragma unroll
          for (int pass = SPLIT ? 0 : 1; pass < 2; ++pass)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_f16_ts(tmem + kColS + sb * 128, tmem + kColQ + 8 * ks + (pass == 0 ? 64 : 0),
                          umma_desc_sw128(op + (ks >> 2) * 16384 + (ks & 3) * 32), idesc,
                          (ks == 0 && pass == (SPLIT ? 0 : 1)) ? 0u : 1u);
          umma_commit(&bar.kh_empty[sb]);
          umma_commit(&bar.s_full[sb]);
          if (!fresh && !(ok = product(j - 1, fresh_prev))) break;
        } else if (j > 0 && !(ok = product(j - 1, fresh))) {
          break;
        }
      }
      umma_commit(&bar.drain);  // every product issued completes before tensor memory is released
      for (uint32_t k = 0; k < kSpinLimitDev && !mbar_try_wait(&bar.drain, 0u); ++k) {
      }
    }
  } else {
    // ---------------- copies of the packed tiles: lane = (16-token chunk, part)
    const int c = lane >> 2, part = lane & 3;
    uint32_t i = 0, rc = 0;
    bool ok = true;
    while (ok && u < u_end) {
      const TreeSeg g = tree_seg(p, u, u_end, b);
      b = g.b;
      for (int t = g.first; t < g.last; ++t, ++i) {
        const uint32_t ns = i % kNormSlots, nb = norm_slot(i);
        const bool draft = t >= g.ctiles;
        const uint32_t st = rc % RS;
        ok = bar_wait(&bar.n_empty[ns], ((i / kNormSlots) & 1u) ^ 1u, abort_flag, p.status, lim) &&
             (draft || bar_wait(&bar.raw_empty[st], ((rc / RS) & 1u) ^ 1u, abort_flag, p.status, lim));
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        if (draft) {
          const int t0 = (t - g.ctiles) * kTreeTok, nt = p.kn ? g.s.T - t0 : 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 4 * lane + e;
            const int64_t at = (int64_t)g.kvh * p.R + g.s.start + t0 + k;
            const float fk = k < nt ? p.kfac[at] : 0.f, fv = k < nt ? p.vfac[at] : 0.f;
            asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(nb + 4 * k), "f"(fk) : "memory");
            asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(nb + 512 + 4 * k), "f"(fv) : "memory");
          }
          if (lane == 0) bar.valid[ns] = 0xFFu;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.n_full[ns]);
          continue;
        }
        const int tok = t * kTreeTok + 16 * c;
        int64_t vec = -1;
        if (tok < g.s.len) {
          const int j = tok / p.block;
          const int64_t page = p.table ? (int64_t)__ldg(p.table + (int64_t)g.b * p.max_blocks + j) : g.b;
          if (page >= 0 && page < p.pages)
            vec = (page * p.Hkv + g.kvh) * p.block + (tok - j * p.block);
          else if (part == 0)
            atomicOr(p.status, 2);
        }
        const uint32_t there = __ballot_sync(kFull, vec >= 0 && part == 0);
        const uint32_t n = __popc(there);
        const uint32_t raw = kRaw + st * stage;
        if (lane == 0) {
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) m |= ((there >> (4 * k)) & 1u) << k;
          bar.valid[ns] = m;
          mbar_arrive_expect_tx(&bar.raw_full[st], n * 256u * (uint32_t)(p.kb + p.vb));
          mbar_arrive_expect_tx(&bar.n_full[ns], n * 128u);
        }
        __syncwarp();
        if (vec >= 0) {
          unsigned char* base = smem + (raw - kBase);
          if (part == 0) {
            bulk_g2s(base + c * 256 * p.kb, p.kcodes + vec * (4 * p.kb), 256 * p.kb, &bar.raw_full[st]);
          } else if (part < 3) {  // 8 tokens, four PAIR blocks
            const int h = part - 1;
            bulk_g2s(base + raw_v_off(p.kb) + (2 * c + h) * (128 * p.vb + 16),
                     p.vcodes + ((vec >> 1) + 4 * h) * (8 * p.vb), 128 * p.vb, &bar.raw_full[st]);
          } else {
            unsigned char* nd = smem + (nb - kBase) + 64 * c;
            bulk_g2s(nd, p.knorm + vec, 64, &bar.n_full[ns]);
            bulk_g2s(nd + 512, p.vnorm + vec, 64, &bar.n_full[ns]);
          }
        }
        ++rc;
      }
      u += g.last - g.first;
    }
    if (lane == 0) {
      // every copy issued lands before the CTA may exit (bounded)
      for (uint32_t j = rc > (uint32_t)RS ? rc - RS : 0u; j < rc; ++j)
        for (uint32_t k = 0; k < kSpinLimitDev && !mbar_try_wait(&bar.raw_full[j % RS], (j / RS) & 1u); ++k) {
        }
      for (uint32_t j = i > kNormSlots ? i - kNormSlots : 0u; j < i; ++j)
        for (uint32_t k = 0; k < kSpinLimitDev && !mbar_try_wait(&bar.n_full[j % kNormSlots], (j / kNormSlots) & 1u); ++k) {
        }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool SPLIT>
cudaError_t run(const TreeParams& p, cudaStream_t st) {
  static PerDeviceValue attr;
  constexpr int bytes = (int)(kBars + sizeof(Bars) - kBase);
  const cudaError_t e = smem_attr_once(attr, (const void*)tree_attend_kernel<SPLIT>, bytes);
  if (e != cudaSuccess) return e;
  return tree_launch(tree_attend_kernel<SPLIT>, p.ctas, kThreads, bytes, p, st);
}

}  // namespace

cudaError_t tree_attend_umma(const TreeParams& p, cudaStream_t st) {
  return p.dtype == TQ_F16 ? run<true>(p, st) : run<false>(p, st);
}

}  // namespace tq
