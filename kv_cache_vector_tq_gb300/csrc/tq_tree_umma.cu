// Attention of drafted tokens over a packed cache on the fifth-generation
// tensor cores (fp16 and bf16 inputs).  tq_tree.cuh has the mathematics and
// the division of the work into units of 128 tokens.
//
// A persistent CTA per SM; per unit, with the 128 tokens on the lanes of
// tensor memory and N rows (drafted token x query head) on its columns:
//     Sᵀ[token][row] = K̂·Q̂ᵀ        A = K̂ (tensor memory), B = Q̂ (shared memory)
//     P[token][row]  = 2^(Sᵀ·s_k·c - M)·s_v   in fp16, shared memory
//     Oᵀ[coord][row] += V̂ᵀ·P       A = V̂ᵀ (tensor memory), B = P (row-contiguous)
// Tokens on the lanes make the work on scores proportional to the rows there
// are (a single token has four or eight of them), and a token's norms one
// register each.  K̂ and V̂ᵀ are the codebook's fp16 pairs (α·c), written to
// tensor memory by the threads that look them up: TOKEN rows hold pairs of
// coordinates of a token, PAIR blocks pairs of tokens of a coordinate, which are
// the pairs along K of the two products.  The norms act on scores and weights
// in fp32, so no rounding depends on them.  M (per row) is a running maximum of
// log2 of weight times s_v, raised only before a weight passes 2^14 (the sums
// are then rescaled, which is rare); with s_v inside it, weights stay inside fp16
// for norms from 2^-80 to the end of fp32's range.  The weights without s_v, of
// which the sum is taken, are then between 2^-104 and 2^104 where they matter.
// Rounding of the operands: for fp16 outputs Q̂ and P are split into two fp16
// terms each (two products), since one rounding of either costs as much as the
// output's own; bf16 outputs round eight times coarser and take one term.  The
// drafted rows of fp16 calls are in two terms as well (in one, the error was up to
// 1.9 times the output's own where they carry the weight): a unit is 64 of them,
// the leading parts on lanes and columns 0-63, the remainders on 64-127.  The two
// scores of a token are added before the softmax; its weight stands in both places
// and is summed in the first.
//
// Warps: 0-7 softmax (thread = token, half of the rows), 8-15 K̂ (thread = token,
// half of the coordinates: 32 lookups of two codes), 16-23 V̂ᵀ (thread =
// coordinate, half of the tokens: 32 lookups, one per PAIR block), 24 issues the
// products, 25 and 26 the bulk copies of the packed tiles (K and V, one per run of
// 16-token chunks inside a page, so pages may end anywhere on a multiple of 16;
// one warp for both kept the others waiting).  Lookup tables are replicated
// per lane (one bank each) and aligned to their size, so an address is a shift
// and an and-or.  Four roles run on each quarter of the SM, each through its own
// code once per unit, so every role is a short rolled loop: unrolled over the
// unit, instruction fetch bounded all of them (7000-11000 clocks a unit).
// A long cache is bound by the lookups' and the softmax's instructions: about 8000
// a unit of 64 rows, 0.73 a clock and quarter; a batch, at 0.50, by the pipeline's
// beginnings and ends as well.  Whole calls, three kernels: 24 us for one
// token of 32 heads over 16384 cached (b = 4, 0.11 of the copy bandwidth); 75 us
// for 8 requests of up to 16 drafted over 8191 (42.9 MB, 9.7 GFLOP); 339 us for 32
// drafted of 64 heads over 131072 (b = 3, 137 GFLOP, 404 TFLOP/s).
#include "tq_tree.cuh"

namespace tq {

namespace {

constexpr int kSoft = 8;                    // softmax warps: two per 32 tokens, half of the rows each
constexpr int kMma = kSoft + 16, kCopy = kMma + 1;
constexpr int kThreads = (kSoft + 20) * 32;  // 28 warps of 72 registers; one fills the last warpgroup
constexpr int kRegSoft = 96, kRegOps = 64, kRegRest = 56;  // 8·96 + 16·64 + 4·56 = 28·72
static_assert(8 * kRegSoft + 16 * kRegOps + 4 * kRegRest <= 28 * 72, "registers that the launch does not have would be waited for");
constexpr int kRS = 5;                     // packed tiles in flight (3 where K and V have tables of their own)
constexpr int kNormSlots = 8;
template <bool SPLIT>
constexpr int kDraft = SPLIT ? kTreeTok / 2 : kTreeTok;  // drafted tokens of a unit
constexpr uint32_t kLandPolls = 1u << 14;  // a millisecond or more for copies under way
// Tensor memory columns: Sᵀ x 2, Oᵀ, the rows' sums of weights per token lane, K̂ x 2, V̂ᵀ x 2
constexpr uint32_t kColO = 128, kColL = 192, kColK = 256, kColV = 384;
constexpr float kLazyUp = 14.f;            // raise M before a weight passes 2^14
constexpr float kLogLo = -90.f, kLogHi = 110.f;  // log2 of s_v·2^-20 as M takes it
constexpr float kShift = 6.f;              // a fresh maximum sits at weight 2^6: small weights keep their bits longer

// Shared memory
constexpr int kLutV = 0, kLutK = 32768;    // (one table for both: kLutV)
constexpr int kQ = 65536;                  // Q̂: leading parts, remainders; 64 rows x 256 bytes each
constexpr int kQPart = 64 * 256;
constexpr int kP = kQ + 2 * kQPart;        // P x 2: leading parts, remainders; 128 tokens x 128 bytes each
constexpr int kPPart = 128 * 128;
constexpr int kRaw = kP + 4 * kPPart;      // packed tiles: K codes, V codes
constexpr int kRawStage = 2 * 128 * 64;
// packed tile s: three stages of their own, two in the place of the second table
__device__ __forceinline__ int raw_at(uint32_t s) { return s < 3 ? kRaw + (int)s * kRawStage : kLutK + (int)(s - 3) * kRawStage; }
static_assert(kLutK + 2 * kRawStage <= kQ, "shared memory");
constexpr int kNorms = kRaw + 3 * kRawStage;  // [slot][K | V][128] fp32
constexpr int kMisc = kNorms + kNormSlots * 1024;

struct Misc {
  float c[64];       // factors of the rows' scores
  float nm[64];      // -M
  float f[64];       // rescale factors of a raise
  float red[4][64];
  int vec[64];       // record of a row; -1: no such row
  int ti[64];        // its drafted token
  uint64_t raw_full[kRS], raw_empty[kRS];
  uint64_t kh_full[2], kh_empty[2], vh_full[2], vh_empty[2];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t n_full[kNormSlots], n_empty[kNormSlots];
  uint64_t q_full, drain;
  uint32_t valid[kNormSlots];  // bit c: the tile's 16-token chunk c is there
  uint32_t sent[2][2];  // cached tiles and tiles that the copy warps have issued
  uint32_t tmem;
  int abort;
};
constexpr int kSmem = kMisc + (int)sizeof(Misc);
static_assert(kSmem <= 227 * 1024, "shared memory");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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
__device__ __forceinline__ void tmem_st_n(uint32_t at, const uint32_t (&v)[32]) {
  uint32_t a[16], b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = v[i];
    b[i] = v[16 + i];
  }
  tmem_st16(at, a);
  tmem_st16(at + 16, b);
}
__device__ __forceinline__ void tmem_ld_n(uint32_t at, uint32_t (&v)[32]) { tmem_ld32_nw(at, v); }
__device__ __forceinline__ void tmem_ld_n(uint32_t at, uint32_t (&v)[16]) { tmem_ld16_nw(at, v); }
__device__ __forceinline__ void tmem_ld_n(uint32_t at, uint32_t (&v)[8]) { tmem_ld8_nw(at, v); }
__device__ __forceinline__ void tmem_st_n(uint32_t at, const uint32_t (&v)[16]) { tmem_st16(at, v); }
__device__ __forceinline__ void tmem_st_n(uint32_t at, const uint32_t (&v)[8]) { tmem_st8(at, v); }
// One poll of a phase, suspended for up to a few microseconds: 25 warps that poll
// as fast as they can take issue slots from those that work.
__device__ __forceinline__ bool poll_rest(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(4000u)
      : "memory");
  return ok != 0;
}
// bar_wait with such polls; the first one, which mostly does, takes five
// instructions (a third of all instructions here once were waits).
__device__ __forceinline__ bool bar_rest(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                         uint32_t limit) {
  if (limit != 0u && poll_rest(bar, parity)) return true;
#pragma unroll 1
  for (uint32_t n = 1;; ++n) {
    if (n >= limit) {
      *abort_flag = 1;
      atomicOr(status, 1);
      return false;
    }
    if (poll_rest(bar, parity)) return true;
    if ((n & 15u) == 15u && *abort_flag) return false;
  }
}
// One lane of a converged warp, by the instruction made for it: the products
// inside a branch on it issue every 31 clocks (N = 64, the tensor cores' rate),
// on `lane == 0` every 54, predicated every 70 (descriptors are then moved to
// uniform registers for each of them).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 256;\n" ::: "memory"); }
// Barrier of the softmax warps that tells whether any thread asked.
__device__ __forceinline__ bool bar_any(bool ask) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)ask)
      : "memory");
  return r != 0;
}

// Lane l gets the result of column l over the warp's lanes (v: a lane's 32 columns).
template <bool SUM>
__device__ __forceinline__ float reduce_columns(float (&v)[32], int lane) {
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) {
    const bool up = (lane & w) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
      const float got = __shfl_xor_sync(kFull, send, w);
      v[i] = SUM ? keep + got : fmaxf(keep, got);
    }
  }
  return v[0];
}

__device__ __forceinline__ uint32_t lds_u32(const unsigned char* p) { return *reinterpret_cast<const uint32_t*>(p); }

// Half of the K̂ row of token t (tensor-memory lane t): 32 columns of coordinate
// pairs, 16 at a time: 32 coordinates are B whole words of the row.
template <int B>
__device__ __forceinline__ void dequant_k(const unsigned char* smem, int raw, uint32_t tmem, uint32_t lut, int t, int half) {
  constexpr uint32_t m = ((1u << (2 * B)) - 1u) << 7;
  const unsigned char* row = smem + raw + t * (16 * B) + half * (8 * B);
  uint32_t all[2 * B];
  if constexpr (B == 4) {
    // rows of 64 bytes: eight lanes reading the same 16-byte piece would meet in
    // two of eight bank groups; lanes in two orders meet in four
    const bool r = (t >> 1) & 1;
    const uint4 x = *reinterpret_cast<const uint4*>(row + (r ? 16 : 0)), y = *reinterpret_cast<const uint4*>(row + (r ? 0 : 16));
    all[0] = r ? y.x : x.x;
    all[1] = r ? y.y : x.y;
    all[2] = r ? y.z : x.z;
    all[3] = r ? y.w : x.w;
    all[4] = r ? x.x : y.x;
    all[5] = r ? x.y : y.y;
    all[6] = r ? x.z : y.z;
    all[7] = r ? x.w : y.w;
  } else if constexpr (B == 2) {
    const uint4 x = *reinterpret_cast<const uint4*>(row);
    all[0] = x.x;
    all[1] = x.y;
    all[2] = x.z;
    all[3] = x.w;
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const uint2 x = *reinterpret_cast<const uint2*>(row + 8 * i);
      all[2 * i] = x.x;
      all[2 * i + 1] = x.y;
    }
  }
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int i = (2 * B * e) >> 5, s = (2 * B * e) & 31;
      uint32_t x;  // the field to bits 7..
      if (s + 2 * B > 32)
        x = __funnelshift_r(all[i], all[i + 1 < B ? i + 1 : i], s - 7);
      else
        x = s >= 7 ? all[i] >> (s - 7) : all[i] << (7 - s);
      v[e] = lds_u32(smem + ((x & m) | lut));
    }
    tmem_st16(tmem + 16 * c, v);
#pragma unroll
    for (int i = 0; i < B; ++i) all[i] = all[i + B];
  }
}

// Coordinate of lane l of V̂ᵀ and Oᵀ.  With 3-bit codes a pair field is six bits,
// and those of coordinates 5 and 10 of every 16 cross a 32-bit word: they are
// gathered in the last lanes, so that the other warps take one load per field
// instead of two bytes (349 -> 332 us for 32 tokens of 64 heads over 131072; with
// split operands, whose other roles are longer, two bytes are the faster way, 295
// against 310 us for 252 rows over 48K: there lanes keep their coordinates).
template <bool WORDS>
__device__ __forceinline__ int lane_coord(int l, int vb) {
  if (!WORDS || vb != 3) return l;
  const int q = l < 112 ? l / 14 : (l - 112) >> 1, r = l - 14 * q;
  return 16 * q + (l < 112 ? r + (r >= 5) + (r >= 9) : ((l & 1) ? 10 : 5));
}

// Half of the V̂ᵀ row of coordinate d (tensor-memory lane l): column i holds PAIR
// block i's two tokens, the 2B bits at bit 2B·d of the block.
template <int B, bool WORDS>
__device__ __forceinline__ void dequant_v(const unsigned char* smem, int raw, uint32_t tmem, uint32_t lut, int d, int l, int half) {
  constexpr uint32_t m = ((1u << (2 * B)) - 1u) << 7;
  if constexpr (B == 3 && WORDS) {
    const unsigned char* src = smem + raw + half * (32 * 32 * B) + ((6 * d) >> 5) * 4;
    const uint32_t s = (6 * d) & 31;
    if (l < 96) {  // whole warps: the field inside one word, turned to bits 7..
      const uint32_t turn = (39u - s) & 31u;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = lds_u32(src + e * 96);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = lds_u32(smem + ((__funnelshift_l(v[e], v[e], turn) & m) | lut));
        tmem_st16(tmem + 16 * c, v);
        src += 16 * 96;
      }
    } else {  // the field across this word and the next (one word past the last block stays in the tile's buffer)
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          v[e] = __funnelshift_r(lds_u32(src + e * 96), lds_u32(src + e * 96 + 4), s);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = lds_u32(smem + (((v[e] << 7) & m) | lut));
        tmem_st16(tmem + 16 * c, v);
        src += 16 * 96;
      }
    }
  } else {
    const unsigned char* src = smem + raw + half * (32 * 32 * B) + ((2 * B * d) >> 3);
    const int up = B == 4 ? 7 : 7 - ((2 * B * d) & 7);  // the field to bits 7..
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      uint32_t v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        v[e] = src[e * (32 * B)];
        if constexpr (B == 3) v[e] |= (uint32_t)src[e * (32 * B) + 1] << 8;  // six bits may end in the next byte
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = lds_u32(smem + (B == 4 ? lut + v[e] * 128u : (((v[e] << up) & m) | lut)));
      tmem_st16(tmem + 16 * c, v);
      src += 16 * 32 * B;
    }
  }
}

// Adds the scores of the lane `to` bytes away, through a place [row][token] of
// shared memory.  A call: inside the loop over tiles, most of which never come here,
// it cost 2% (252 rows over 48K: 310 -> 303 us).
template <int HN, int PC>
__device__ __noinline__ void join_terms(uint32_t tS, unsigned char* at, int to) {
#pragma unroll 1
  for (int c = 0; c < HN / PC; ++c) {
    uint32_t s[PC];
    tmem_ld_n(tS + PC * c, s);
    wait_ld(s);
#pragma unroll
    for (int e = 0; e < PC; ++e) *reinterpret_cast<uint32_t*>(at + (PC * c + e) * (4 * kTreeTok)) = s[e];
  }
  bar_softmax();
  at += to;
#pragma unroll 1
  for (int c = 0; c < HN / PC; ++c) {
    uint32_t s[PC];
    tmem_ld_n(tS + PC * c, s);
    wait_ld(s);
#pragma unroll
    for (int e = 0; e < PC; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) + *reinterpret_cast<const float*>(at + (PC * c + e) * (4 * kTreeTok)));
    tmem_st_n(tS + PC * c, s);
  }
  tmem_wait_st();
}

// Scores times their rows' factors, in place: a call for the same reason.
template <int HN, int PC>
__device__ __noinline__ void scale_scores(uint32_t tS, const float* c) {
#pragma unroll 1
  for (int i = 0; i < HN; i += PC) {
    uint32_t s[PC];
    tmem_ld_n(tS + i, s);
    wait_ld(s);
#pragma unroll
    for (int e = 0; e < PC; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) * c[i + e]);
    tmem_st_n(tS + i, s);
  }
  tmem_wait_st();
}

template <int N, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) tree_attend_kernel(const TreeParams p) {
  static_assert(N == 16 || N == 32 || N == 64, "rows per tile");
  constexpr int PC = N < 32 ? N / 2 : 16;  // columns of a piece
  extern __shared__ __align__(1024) unsigned char smem[];
  Misc& ms = *reinterpret_cast<Misc*>(smem + kMisc);
  if ((smem_u32(smem) & 1023u) != 0u) {  // the swizzled operands need it
    griddep_wait();  // as every CTA, before it ends: the join is let in by that
    if (threadIdx.x == 0) atomicOr(p.status, 1);
    return;
  }
  volatile int* abort_flag = &ms.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t lim = p.wait_limit;
  const int lut_k = p.same_lut ? kLutV : kLutK;
  const uint32_t RS = p.same_lut ? kRS : 3;

  if (tid == 0) {
    for (int i = 0; i < kRS; ++i) {
      mbar_init(&ms.raw_full[i], 2);  // K and V
      mbar_init(&ms.raw_empty[i], 16);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.kh_full[i], 8);
      mbar_init(&ms.kh_empty[i], 1);
      mbar_init(&ms.vh_full[i], 8);
      mbar_init(&ms.vh_empty[i], 1);
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.p_full[i], kSoft);
      mbar_init(&ms.pv_done[i], 1);
    }
    for (int i = 0; i < kNormSlots; ++i) {
      mbar_init(&ms.n_full[i], 2);
      mbar_init(&ms.n_empty[i], kSoft);
    }
    mbar_init(&ms.q_full, kSoft);
    mbar_init(&ms.drain, 1);
    ms.abort = 0;
    fence_mbar_init();
  }
  {
    uint4* lv = reinterpret_cast<uint4*>(smem + kLutV);
    for (int i = tid; i < (8 << (2 * p.vb)); i += kThreads) {
      const uint32_t x = __ldg(p.vlut + (i >> 3));
      lv[i] = make_uint4(x, x, x, x);
    }
    if (!p.same_lut) {
      uint4* lk = reinterpret_cast<uint4*>(smem + kLutK);
      for (int i = tid; i < (8 << (2 * p.kb)); i += kThreads) {
        const uint32_t x = __ldg(p.klut + (i >> 3));
        lk[i] = make_uint4(x, x, x, x);
      }
    }
  }
  if (warp == kMma) tmem_alloc(&ms.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // 512 columns are all there are: they start at 0
  griddep_wait();
  griddep_launch();

  const TreeCta& share = p.cta[blockIdx.x];
  int64_t u = share.u;
  const int64_t u_end = share.end;
  int b = share.b;

  if (warp < kSoft) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegSoft));
    // ---------------- softmax: thread = token tok (its tensor-memory lane) and
    // rows n0 .. n0 + HN - 1; in the epilogue coordinate `coord`
    constexpr int HN = N / 2;  // rows of a thread
    const int n0 = (warp >> 2) * HN, quad = warp & 3, tok = tid & 127, coord = lane_coord<!SPLIT>(tok, p.vb);
    const uint32_t lane_base = ((uint32_t)(32 * quad) << 16) + n0;
    const uint32_t tO = tmem + lane_base + kColO, tL = tmem + lane_base + kColL;
    const int sw = tok & 7;
    uint32_t i = 0;
    bool ok = true;
    while (ok && u < u_end) {
      const TreeSeg g = tree_seg(p, u, u_end, b);
      // the rows: Q̂ into shared memory (every product with the last segment's
      // has completed: its last Sᵀ was read here), their factors and records
      if (tid < N) {
        int vec = -1, ti = 0;
        float c = 0.f, m = INFINITY;  // no such row: weights 0 (M = inf)
        if (tid < g.nrow) {
          const int rho = g.row0 + tid;
          ti = rho / p.G;
          vec = (g.s.start + ti) * p.Hq + g.kvh * p.G + (rho - ti * p.G);
          c = p.qfac[vec] * p.zfold;
          m = -INFINITY;
        }
        // a row that is not a number: every weight that it has is none either
        ms.c[tid] = c == c ? c : 0.f;
        ms.nm[tid] = c == c ? -m : c;
        ms.vec[tid] = vec;
        ms.ti[tid] = ti;
      }
      bar_softmax();
      // Rows within 2^13 of the tile's largest factor are scaled down to it by powers
      // of two and share it: what fp16 drops is below 2^-22 of a row's largest
      // entry.  Where one is further below (another row is huge, it is tiny), every
      // row keeps its own and the scores are multiplied in tensor memory first (in
      // the softmax it cost all calls 4%).  Factor 0: no row, a row of zeros or
      // one that is not a number.
      const float c0 = ms.c[lane & (N - 1)], c1 = ms.c[(lane + 32) & (N - 1)];
      float ct = fmaxf(c0, c1);
#pragma unroll
      for (int o = 16; o; o >>= 1) ct = fmaxf(ct, __shfl_xor_sync(kFull, ct, o));
      const float least = ct * 1.220703125e-4f;  // 2^-13
      // (a factor whose inverse is no number scales nothing)
      const bool shared_c = __all_sync(kFull, ct >= 1e-30f && (c0 == 0.f || c0 >= least) && (c1 == 0.f || c1 >= least));
      const float inv_ct = shared_c ? 1.f / ct : 0.f;
      // 16-byte pieces: 16 of the leading part and 16 of the remainder per row
#pragma unroll 4
      for (int e = tid; e < N * (SPLIT ? 32 : 16); e += 32 * kSoft) {
        const int n = SPLIT ? e >> 5 : e >> 4, k = SPLIT ? e & 31 : e & 15, c = k & 15, part = k >> 4;
        const int vec = ms.vec[n];
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (vec >= 0) x = *(reinterpret_cast<const uint4*>(reinterpret_cast<const __half*>(p.qrot) + (int64_t)vec * 256) + k);
        if (shared_c) {
          const __half2 sc = __float2half2_rn(ms.c[n] * inv_ct);  // a power of two up to rounding: made one by fp16's
          __half2* h = reinterpret_cast<__half2*>(&x);
#pragma unroll
          for (int q = 0; q < 4; ++q) h[q] = __hmul2(h[q], sc);
        }
        *reinterpret_cast<uint4*>(smem + kQ + part * kQPart + (c >> 3) * (N * 128) + n * 128 + (((c & 7) ^ (n & 7)) << 4)) = x;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.q_full);
      {
        const uint32_t zero[PC] = {};
#pragma unroll 1
        for (int c = 0; c < HN / PC; ++c) tmem_st_n(tL + PC * c, zero);
        tmem_wait_st();
      }

      for (int t = g.first; t < g.last; ++t, ++i) {
        const uint32_t sb = i & 1u, ns = i % kNormSlots;
        ok = __all_sync(kFull, bar_rest(&ms.s_full[sb], (i >> 1) & 1u, abort_flag, p.status, lim) &&
                                   bar_rest(&ms.n_full[ns], (i / kNormSlots) & 1u, abort_flag, p.status, lim));
        tc_fence_after();  // (a wait that gave up: what follows is garbage and dropped below)
        const uint32_t tS = tmem + lane_base + sb * 64;
        const float* nrm = reinterpret_cast<const float*>(smem + kNorms + ns * 1024);
        const bool draft = t >= g.ctiles;
        const int t0 = draft ? (t - g.ctiles) * kDraft<SPLIT> : t * kTreeTok;
        const int nt = min(kTreeTok, (draft ? g.s.T : g.s.len) - t0);
        const uint32_t chunks = ms.valid[ns];
        const bool here = (tok & (SPLIT && draft ? 63 : 127)) < nt && ((chunks >> (tok >> 4)) & 1u);  // this token is there
        const bool whole = nt == kTreeTok && chunks == 0xFFu && !draft;
        const float kn = nrm[tok], vn = draft ? nrm[128 + tok] : nrm[128 + tok] * kTreeVDown;
        // 2^lv > vn.  The upper end is past every finite value; below the lower one
        // a weight is smaller than it might be, and the sum of weights has 2^23 tokens' room
        const float lv = fminf(fmaxf((float)((int)((__float_as_uint(vn) >> 23) & 255u) - 126), kLogLo), kLogHi);
        const float ck = shared_c ? ct * kn : kn;
        // drafted tokens: bit `lane` of a row's mask word for this warp's 32
        // tokens; lane n holds the word of row n0 + n
        uint32_t mw = 0u;
        if (draft && lane < HN && ms.vec[n0 + lane] >= 0) {
          const int ti = ms.ti[n0 + lane], at = (t0 >> 5) + (SPLIT ? quad & 1 : quad);
          if (p.mask) {
            if (at < p.mask_words) mw = __ldg(p.mask + (int64_t)(g.s.start + ti) * p.mask_words + at);
          } else {  // a chain: tokens 0..ti
            const int k = ti - 32 * at + 1;
            mw = k >= 32 ? 0xFFFFFFFFu : (k > 0 ? (1u << k) - 1u : 0u);
          }
        }
        auto sees = [&](int n) -> bool {  // this token is seen by row n0 + n
          const bool named = !draft || ((__shfl_sync(kFull, mw, n) >> lane) & 1u);
          return here && named;
        };
        if (SPLIT && draft) {  // a drafted token's two scores: each of its lanes gets the sum
          // (where this tile's P will be, which is written behind the barrier that follows)
          join_terms<HN, PC>(tS, smem + kP + sb * (2 * kPPart) + (n0 * kTreeTok + tok) * 4, quad >= 2 ? -256 : 256);
        }
        if (!shared_c) scale_scores<HN, PC>(tS, ms.c + n0);
        // weights with the M there is; should one pass the limit (M = -inf, a
        // row's first token, does), M is raised and they are computed again
        float pr[HN];
        for (int tries = 0;; ++tries) {
          float top = -INFINITY;
          {
            uint32_t s[HN];
            tmem_ld_n(tS, s);
            wait_ld(s);
#pragma unroll
            for (int e = 0; e < HN; e += 4) {
              const float4 m4 = *reinterpret_cast<const float4*>(ms.nm + n0 + e);
              pr[e] = fmaf(__uint_as_float(s[e]), ck, m4.x);
              pr[e + 1] = fmaf(__uint_as_float(s[e + 1]), ck, m4.y);
              pr[e + 2] = fmaf(__uint_as_float(s[e + 2]), ck, m4.z);
              pr[e + 3] = fmaf(__uint_as_float(s[e + 3]), ck, m4.w);
            }
          }
          if (!whole) {
#pragma unroll
            for (int e = 0; e < HN; ++e)
              if (!sees(e)) pr[e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < HN; e += 2) top = max3(top, pr[e], pr[e + 1]);
#pragma unroll
          for (int e = 0; e < HN; ++e) pr[e] = ex2(pr[e]);
          if (!bar_any(!ok || (top + lv > kLazyUp && tries < 2))) break;
          if (bar_any(!ok)) {  // the eight warps stop together
            ok = false;
            break;
          }
          // the rows' maxima over the tile, then new M where one is passed
          {
            uint32_t s[HN];
            tmem_ld_n(tS, s);
            wait_ld(s);
            float v[32];
#pragma unroll
            for (int n = 0; n < 32; ++n) {
              v[n] = -INFINITY;
              if (n < HN) {
                const bool on = sees(n);
                if (on) v[n] = fmaf(__uint_as_float(s[n < HN ? n : 0]), ck, lv);
              }
            }
            const float r = reduce_columns<false>(v, lane);
            if (lane < HN) ms.red[quad][n0 + lane] = r;
          }
          bar_softmax();
          if (tid < N) {
            const float m = fmaxf(fmaxf(ms.red[0][tid], ms.red[1][tid]), fmaxf(ms.red[2][tid], ms.red[3][tid]));
            const float old = -ms.nm[tid];
            const bool up = m > old + kShift;
            ms.f[tid] = up ? (old == -INFINITY ? 0.f : ex2(old - (m - kShift))) : 1.f;
            if (up) ms.nm[tid] = kShift - m;
          }
          if (t > g.first)  // the sums so far, once the last product into them is done
            ok = __all_sync(kFull, bar_rest(&ms.pv_done[(i - 1) & 1u], ((i - 1) >> 1) & 1u, abort_flag, p.status, lim));
          if (bar_any(!ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (t > g.first) {
#pragma unroll 1
            for (int c = 0; c < 2 * (HN / PC); ++c) {  // Oᵀ, then the sums
              const uint32_t at = (c & 1 ? tL : tO) + PC * (c >> 1);
              uint32_t o[PC];
              tmem_ld_n(at, o);
              wait_ld(o);
#pragma unroll
              for (int e = 0; e < PC; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * ms.f[n0 + PC * (c >> 1) + e]);
              tmem_st_n(at, o);
            }
            tmem_wait_st();
          }
        }
        if (!ok) break;
        // the rows' sums; P of a token: N values, 16-byte pieces in the 128-byte swizzle
        unsigned char* prow = smem + kP + sb * (2 * kPPart) + tok * 128;
        float vs = here ? vn : 0.f;  // the factors of a token that is not there may be anything
        if (draft && vs != vs) {  // a drafted row that is not a number: neither are the rows that see it
          vs = 0.f;
#pragma unroll
          for (int e = 0; e < HN; ++e) pr[e] = pr[e] == 0.f ? 0.f : NAN;
        }
        uint32_t l[HN];
        tmem_ld_n(tL, l);
        wait_ld(l);
#pragma unroll
        for (int c = 0; c < HN / 8; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = 8 * c + 2 * e;
            l[n] = __float_as_uint(__uint_as_float(l[n]) + pr[n]);
            l[n + 1] = __float_as_uint(__uint_as_float(l[n + 1]) + pr[n + 1]);
            const float w0 = pr[n] * vs, w1 = pr[n + 1] * vs;
            const __half2 h = __floats2half2_rn(w0, w1);
            hi[e] = h2_bits(h);
            if constexpr (SPLIT) lo[e] = h2_bits(__floats2half2_rn(w0 - __low2float(h), w1 - __high2float(h)));
          }
          unsigned char* at = prow + (((n0 / 8 + c) ^ sw) << 4);
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if constexpr (SPLIT) *reinterpret_cast<uint4*>(at + kPPart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (!(SPLIT && draft && quad >= 2)) tmem_st_n(tL, l);  // (lanes of remainders leave the sums)
        tmem_wait_st();
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ms.p_full[sb]);
          mbar_arrive(&ms.n_empty[ns]);
        }
      }
      if (!ok) break;
      // the rows' records, once the segment's last product is done
      {
        float v[32];
#pragma unroll
        for (int c = 0; c < 32 / PC; ++c) {
          uint32_t x[PC];
          if (c < HN / PC) {
            tmem_ld_n(tL + PC * c, x);
            wait_ld(x);
          }
#pragma unroll
          for (int e = 0; e < PC; ++e) v[PC * c + e] = PC * c + e < HN ? __uint_as_float(x[e]) : 0.f;
        }
        const float r = reduce_columns<true>(v, lane);
        if (lane < HN) ms.red[quad][n0 + lane] = r;
      }
      ok = __all_sync(kFull, bar_rest(&ms.pv_done[(i - 1) & 1u], ((i - 1) >> 1) & 1u, abort_flag, p.status, lim));
      if (bar_any(!ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float* base = g.first == 0 ? p.rec : p.crec + (int64_t)blockIdx.x * N * kTreeRec;
      if (tid < g.nrow)
        *reinterpret_cast<float2*>(base + (int64_t)(g.first == 0 ? ms.vec[tid] : tid) * kTreeRec) =
            make_float2(-ms.nm[tid], (ms.red[0][tid] + ms.red[1][tid]) + (ms.red[2][tid] + ms.red[3][tid]));
#pragma unroll 1
      for (int c = 0; c < HN / PC; ++c) {
        if (n0 + PC * c >= g.nrow) break;
        uint32_t o[PC];
        tmem_ld_n(tO + PC * c, o);
        wait_ld(o);
#pragma unroll
        for (int e = 0; e < PC; ++e) {
          const int n = n0 + PC * c + e;
          if (n < g.nrow) base[(int64_t)(g.first == 0 ? ms.vec[n] : n) * kTreeRec + 4 + coord] = __uint_as_float(o[e]);
        }
      }
      tc_fence_before();
      bar_softmax();  // the rows' tables are rewritten next
      u += g.last - g.first;
      if (u < u_end) b = tree_next(p, u, b);
    }
  } else if (warp < kSoft + 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegOps));
    // ---------------- K̂ (thread = token v) and V̂ᵀ (thread = coordinate v), half of the columns each
    const bool is_v = warp >= kSoft + 8;
    const int v = tid & 127, half = (warp >> 2) & 1, vd = lane_coord<!SPLIT>(v, p.vb);
    uint64_t* full = is_v ? ms.vh_full : ms.kh_full;
    uint64_t* empty = is_v ? ms.vh_empty : ms.kh_empty;
    const uint32_t dst = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (is_v ? kColV : kColK) + 32 * half;
    const uint32_t lut = (uint32_t)((is_v ? kLutV : lut_k) + lane * 4);
    uint32_t i = 0, st = 0, rph = 0;  // tile, raw stage and its phase
    bool ok = true;
    while (ok && u < u_end) {
      const TreeSeg g = tree_seg(p, u, u_end, b);
      for (int t = g.first; t < g.last; ++t, ++i) {
        const uint32_t sb = i & 1u, op = dst + sb * 64;
        const bool draft = t >= g.ctiles;
        ok = bar_rest(&empty[sb], ((i >> 1) & 1u) ^ 1u, abort_flag, p.status, lim) &&
             (draft || bar_rest(&ms.raw_full[st], rph, abort_flag, p.status, lim));
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        tc_fence_after();
        if (!draft) {
          const int raw = raw_at(st);
          if (!is_v) {
            switch (p.kb) {
              case 1: dequant_k<1>(smem, raw, op, lut, v, half); break;
              case 2: dequant_k<2>(smem, raw, op, lut, v, half); break;
              case 3: dequant_k<3>(smem, raw, op, lut, v, half); break;
              default: dequant_k<4>(smem, raw, op, lut, v, half); break;
            }
          } else {
            const int rv = raw + 2048 * p.kb;
            switch (p.vb) {
              case 1: dequant_v<1, !SPLIT>(smem, rv, op, lut, vd, v, half); break;
              case 2: dequant_v<2, !SPLIT>(smem, rv, op, lut, vd, v, half); break;
              case 3: dequant_v<3, !SPLIT>(smem, rv, op, lut, vd, v, half); break;
              default: dequant_v<4, !SPLIT>(smem, rv, op, lut, vd, v, half); break;
            }
          }
        } else {
          // drafted rows, rotated and rounded already; zeros past the last one
          const int t0 = (t - g.ctiles) * kDraft<SPLIT>, nt = p.kn ? g.s.T - t0 : 0;
          const int64_t tok = g.s.start + t0;
          constexpr int kRow = SPLIT ? 256 : 128;  // halves of a row
          if (!is_v) {
            const int vt = SPLIT ? v & 63 : v;
            const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __half*>(p.krot) +
                                                              ((tok + vt) * p.Hkv + g.kvh) * kRow + 128 * (SPLIT ? v >> 6 : 0)) + 8 * half;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint4 x = vt < nt ? src[4 * c + e] : make_uint4(0u, 0u, 0u, 0u);
                w[4 * e] = x.x;
                w[4 * e + 1] = x.y;
                w[4 * e + 2] = x.z;
                w[4 * e + 3] = x.w;
              }
              tmem_st16(op + 16 * c, w);
            }
          } else {
            const uint16_t* src = reinterpret_cast<const uint16_t*>(p.vrot) + (tok * p.Hkv + g.kvh) * kRow + vd + 128 * (SPLIT ? half : 0);
            const int64_t step = (int64_t)p.Hkv * kRow;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int k = (SPLIT ? 0 : 64 * half) + 32 * c + 2 * e;
                const uint32_t x = k < nt ? src[k * step] : 0u, y = k + 1 < nt ? src[(k + 1) * step] : 0u;
                w[e] = x | (y << 16);
              }
              tmem_st16(op + 16 * c, w);
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[sb]);
          if (!draft) mbar_arrive(&ms.raw_empty[st]);
        }
        if (!draft && ++st == RS) {
          st = 0;
          rph ^= 1u;
        }
      }
      u += g.last - g.first;
      if (u < u_end) b = tree_next(p, u, b);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegRest));
    if (warp == kMma) {
      // ---------------- the products: Sᵀ of tile j goes before V̂ᵀ·P of tile j - 1,
      // except where a new group's Q̂ has to wait for the last group's end.  The
      // whole warp walks through it, an elected lane issues
      constexpr uint32_t idesc = umma_idesc_f16(128, N);
      constexpr uint32_t idesc_p = idesc | (1u << 16);  // B contiguous along N
      const uint64_t dq = umma_desc_sw128(smem_u32(smem + kQ));
      // P: 64 rows of a token in 128 bytes, swizzled; 8-token groups 1024 bytes apart
      constexpr uint64_t kPDesc = ((uint64_t)(1024 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
                                  ((uint64_t)2 << 61);
      const uint64_t dp = kPDesc | (uint64_t)((smem_u32(smem + kP) >> 4) & 0x3FFF);
      const int n = (int)(u_end - u);  // a CTA's share: fewer than 2^31
      int left = 0;
      uint32_t qn = 0;
      bool ok = true, fresh = false, fresh_prev = false;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(kFull, bar_rest(bar, parity, abort_flag, p.status, lim));
      };
      auto product = [&](int j, bool first) -> bool {  // V̂ᵀ·P of tile j
        const uint32_t sb = (uint32_t)j & 1u, ph = (uint32_t)(j >> 1) & 1u;
        if (!wait(&ms.p_full[sb], ph) || !wait(&ms.vh_full[sb], ph)) return false;
        tc_fence_after();
        const uint64_t bd = dp + (uint64_t)(sb * (2 * kPPart / 16));
        const uint32_t a = tmem + kColV + sb * 64;
        if (elect_one()) {
          if constexpr (SPLIT) {  // remainders first: not truncated against a large sum
            umma_f16_ts(tmem + kColO, a, bd + kPPart / 16, idesc_p, first ? 0u : 1u);
#pragma unroll
            for (int ks = 1; ks < 8; ++ks) umma_f16_ts(tmem + kColO, a + 8 * ks, bd + kPPart / 16 + ks * 128, idesc_p, 1u);
          }
          umma_f16_ts(tmem + kColO, a, bd, idesc_p, SPLIT || !first ? 1u : 0u);
#pragma unroll
          for (int ks = 1; ks < 8; ++ks) umma_f16_ts(tmem + kColO, a + 8 * ks, bd + ks * 128, idesc_p, 1u);
          umma_commit(&ms.vh_empty[sb]);
          umma_commit(&ms.pv_done[sb]);
        }
        __syncwarp();
        return true;
      };
      for (int j = 0; ok && j <= n; ++j) {
        if (j < n) {
          fresh_prev = fresh;
          fresh = left == 0;
          if (left == 0) {
            if (j > 0) b = tree_next(p, u + j, b);
            const TreeSeg g = tree_seg(p, u + j, u_end, b);
            left = __shfl_sync(kFull, g.last - g.first, 0);
          }
          --left;
          if (fresh && j > 0 && !(ok = product(j - 1, fresh_prev))) break;
          if (fresh && !(ok = wait(&ms.q_full, qn++ & 1u))) break;
          const uint32_t sb = (uint32_t)j & 1u;
          if (!(ok = wait(&ms.kh_full[sb], (uint32_t)(j >> 1) & 1u))) break;
          tc_fence_after();
          const uint32_t d = tmem + sb * 64, a = tmem + kColK + sb * 64;
          if (elect_one()) {
#pragma unroll
            for (int pass = SPLIT ? 0 : 1; pass < 2; ++pass)
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                umma_f16_ts(d, a + 8 * ks, dq + ((pass == 0 ? kQPart : 0) + (ks >> 2) * (N * 128) + (ks & 3) * 32) / 16, idesc,
                            (ks == 0 && pass == (SPLIT ? 0 : 1)) ? 0u : 1u);
            umma_commit(&ms.kh_empty[sb]);
            umma_commit(&ms.s_full[sb]);
          }
          __syncwarp();
          if (!fresh && !(ok = product(j - 1, fresh_prev))) break;
        } else if (j > 0 && !(ok = product(j - 1, fresh))) {
          break;
        }
      }
      if (elect_one()) umma_commit(&ms.drain);  // every product issued completes before tensor memory is released
      for (uint32_t k = 0; k < kSpinLimitDev && !mbar_try_wait(&ms.drain, 0u); ++k) {
      }
    } else if (warp <= kCopy + 1) {
      // ---------------- copies of the packed tiles, K by one warp and V by the
      // other: lane = 16-token chunk (codes: lanes 0-7, norms: 8-15); the first
      // chunk of a run inside one page copies the run
      const bool is_v = warp != kCopy;
      const int c = lane & 7, bits = is_v ? p.vb : p.kb;
      const unsigned char* codes = reinterpret_cast<const unsigned char*>(is_v ? p.vcodes : p.kcodes);
      const float* norms = is_v ? p.vnorm : p.knorm;
      const float* fac = is_v ? p.vfac : p.kfac;
      const int raw_off = is_v ? 2048 * p.kb : 0, norm_off = is_v ? 512 : 0;
      uint32_t i = 0, rc = 0, st = 0, rph = 1;  // tile, cached tile, its stage and phase
      bool ok = true;
      // pages and places advance by a tile without a division
      const int jt = kTreeTok / p.block, ot = kTreeTok - jt * p.block;
      while (ok && u < u_end) {
        const TreeSeg g = tree_seg(p, u, u_end, b);
        // this lane's chunk of tile t: token, page number within the sequence and
        // place in the page
        int at = g.first * kTreeTok + 16 * c, j = at / p.block, o = at - j * p.block;
        const int32_t* pages = p.table ? p.table + (int64_t)g.b * p.max_blocks : nullptr;
        auto page_here = [&](int t) -> int { return t < g.ctiles && at < g.s.len ? (pages ? __ldg(pages + j) : g.b) : 0; };
        int page = page_here(g.first);
        for (int t = g.first; t < g.last; ++t, ++i) {
          const uint32_t ns = i % kNormSlots;
          unsigned char* nb = smem + kNorms + ns * 1024 + norm_off;
          const bool draft = t >= g.ctiles;
          // the vector of the chunk (-1: no such token, -2: no such page)
          const int64_t vec = draft || at >= g.s.len ? -1
                              : page >= 0 && page < p.pages ? ((int64_t)page * p.Hkv + g.kvh) * p.block + o : -2;
          at += kTreeTok;
          j += jt;
          o += ot;
          if (o >= p.block) {
            o -= p.block;
            ++j;
          }
          page = page_here(t + 1);  // read while this tile waits for room, used with the next
          ok = bar_rest(&ms.n_empty[ns], ((i / kNormSlots) & 1u) ^ 1u, abort_flag, p.status, lim) &&
               (draft || bar_rest(&ms.raw_empty[st], rph, abort_flag, p.status, lim));
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          if (draft) {
            const int t0 = (t - g.ctiles) * kDraft<SPLIT>, nt = p.kn ? g.s.T - t0 : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = (32 * e) % kDraft<SPLIT> + lane;
              reinterpret_cast<float*>(nb)[32 * e + lane] = k < nt ? fac[(int64_t)g.kvh * p.R + g.s.start + t0 + k] : 0.f;
            }
            if (lane == 0 && !is_v) ms.valid[ns] = 0xFFu;
            fence_proxy_async();  // before the bulk copy that writes the slot next
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.n_full[ns]);
            continue;
          }
          const uint32_t there = __ballot_sync(kFull, vec >= 0) & 0xFFu;
          const int64_t before = __shfl_up_sync(kFull, vec, 1);
          const bool leads = vec >= 0 && (c == 0 || before < 0 || vec != before + 16);
          const uint32_t starts = __ballot_sync(kFull, leads || vec < 0) & 0xFFu;
          if (lane == 0) {
            if (!is_v) ms.valid[ns] = there;
            const uint32_t n = __popc(there);
            mbar_arrive_expect_tx(&ms.raw_full[st], n * 256u * (uint32_t)bits);
            mbar_arrive_expect_tx(&ms.n_full[ns], n * 64u);
          }
          if (vec == -2 && lane < 8 && !is_v) atomicOr(p.status, 2);
          __syncwarp();
          if (leads && lane < 16) {
            const uint32_t later = starts >> (c + 1);  // up to the next start (or the tile's end)
            const uint32_t run = later ? (uint32_t)__ffs(later) : (uint32_t)(8 - c);
            const bool nrm = lane >= 8;
            bulk_g2s(nrm ? nb + 64 * c : smem + raw_at(st) + raw_off + c * 256 * bits,
                     nrm ? (const void*)(norms + vec) : (const void*)(codes + vec * (16 * bits)),
                     run * (nrm ? 64u : 256u * bits), nrm ? &ms.n_full[ns] : &ms.raw_full[st]);
          }
          ++rc;
          if (++st == RS) {
            st = 0;
            rph ^= 1u;
          }
        }
        u += g.last - g.first;
        if (u < u_end) b = tree_next(p, u, b);
      }
      if (lane == 0) {
        ms.sent[warp - kCopy][0] = rc;
        ms.sent[warp - kCopy][1] = i;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // Every copy issued lands before the CTA exits.  A walk to the end has had all
    // of them consumed; one that a wait cut short, in whichever warp, leaves some
    // under way: each stage's and slot's last phase (bounded, and short: a barrier
    // that only one of the two warps armed stays as it is).
    if ((warp == kCopy || warp == kCopy + 1) && lane == 0) {
      const uint32_t rc = ms.sent[warp - kCopy][0], i = ms.sent[warp - kCopy][1];
      for (uint32_t q = rc > RS ? rc - RS : 0u; q < rc; ++q)
        for (uint32_t k = 0; k < kLandPolls && !mbar_try_wait(&ms.raw_full[q % RS], (q / RS) & 1u); ++k) {
        }
      for (uint32_t q = i > kNormSlots ? i - kNormSlots : 0u; q < i; ++q)
        for (uint32_t k = 0; k < kLandPolls && !mbar_try_wait(&ms.n_full[q % kNormSlots], (q / kNormSlots) & 1u); ++k) {
        }
    }
    __syncthreads();
  }
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(ms.tmem, 512);
  }
}

template <int N, bool SPLIT>
cudaError_t run(const TreeParams& p, cudaStream_t st) {
  static PerDeviceValue attr;
  const cudaError_t e = smem_attr_once(attr, (const void*)tree_attend_kernel<N, SPLIT>, kSmem);
  if (e != cudaSuccess) return e;
  return tree_launch(tree_attend_kernel<N, SPLIT>, p.ctas, kThreads, kSmem, st, p);
}

template <bool SPLIT>
cudaError_t run_n(const TreeParams& p, cudaStream_t st) {
  switch (p.rows) {
    case 16: return run<16, SPLIT>(p, st);
    case 32: return run<32, SPLIT>(p, st);
    case 64: return run<64, SPLIT>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// Rows of a tile: enough for the mean sequence (its drafted tokens times the
// query heads of a KV head), at most 64.  A longer one takes several tiles.
int tree_umma_rows(int64_t rows, int B, int G) {
  const int64_t mean = (rows + B - 1) / B * G;
  return mean <= 16 ? 16 : mean <= 32 ? 32 : 64;
}

cudaError_t tree_attend_umma(const TreeParams& p, cudaStream_t st) {
  return p.dtype == TQ_F16 ? run_n<true>(p, st) : run_n<false>(p, st);
}

}  // namespace tq
