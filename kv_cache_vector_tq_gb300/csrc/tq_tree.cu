// Attention of drafted tokens over a packed cache: rotation of the rows, the
// fp32 attention kernel, the join of the CTAs' partial states, and the host
// side.  tq_tree.cuh has the mathematics and the division of the work.
#include <algorithm>

#include "tq_tree.cuh"

namespace tq {

namespace {

// ------------------------------------------------------------------ rotation of q, k, v
// y = Π·x for groups of kPrepV vectors.  Warp w of a CTA keeps columns
// [16w, 16w + 16) of the matrix in registers (loaded once, before the wait for
// the kernel ahead: the matrix is constant), every lane four rows of them, and
// multiplies group after group; the eight partial sums meet in shared memory.
// fp32 sums.  CTA 0 also lays out the units of the sequences.  Bound by latency
// for few rows (4.5 us for one token of 32 heads), by the FMA rate and its shared
// reads for many (about 1.5 us for each eight rows that every CTA takes).
// A drafted row that holds an infinity or a NaN is stored as zeros with the
// factor NaN: rows that see it become NaN through the factor, and rows that do
// not see it are not touched by a product 0 · NaN.
constexpr int kPrepV = 8;

// part[w][v][j]: warp w's share of coordinate j of vector v.
struct RotSmem {
  float x[kPrepV][128];
  float part[8][kPrepV][128];
};

// TC: rows for the tensor cores, scaled by a power of two into fp16's range,
// the leading part and (q, and the drafted rows of an fp16 call) the remainder;
// else fp32.
template <bool TC>
__global__ void __launch_bounds__(256, 2) tree_prep_kernel(const TreeParams p, const int per, const int nbq, const int nbk) {
  __shared__ __align__(16) RotSmem sm;
  __shared__ float wmax[kPrepV][4];
  __shared__ int64_t wsum[8], first_unit[256];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0) {
    griddep_wait();
    griddep_launch();
    int64_t base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 256) {
      const int b = b0 + tid;
      TreeSeq s;
      int64_t n = 0;
      if (b < p.B) {
        s = tree_seq(p, b);
        n = (int64_t)s.rt * p.Hkv * s.per;
      }
      int64_t inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += a;
      }
      __syncthreads();
      if (lane == 31) wsum[warp] = inc;
      __syncthreads();
      int64_t before = 0, tot = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w < warp) before += wsum[w];
        tot += wsum[w];
      }
      if (b < p.B) {
        s.unit = base + before + inc - n;
        p.seq[b] = s;
        if (p.B <= 256) first_unit[b] = s.unit;
      }
      base += tot;
    }
    if (tid == 0) p.seq[p.B].unit = base;
    __syncthreads();
    for (int c = tid; c < p.ctas; c += 256) {
      TreeCta share;
      share.u = tree_cut(c, base, p.ctas);
      share.end = tree_cut(c + 1, base, p.ctas);
      int lo = 0, hi = p.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((p.B <= 256 ? first_unit[mid] : p.seq[mid].unit) <= share.u)
          lo = mid;
        else
          hi = mid - 1;
      }
      share.b = ~lo;
      share.s = p.seq[lo];
      p.cta[c] = share;
    }
    return;
  }
  // this CTA's rows: q, drafted k or drafted v, `per` groups of kPrepV
  int c = blockIdx.x - 1, kind = 0, heads = p.Hq;
  const void* src = p.q;
  float *dst = p.qrot, *fac = p.qfac;
  const float4* mat = p.kslices;
  int64_t stride = p.qs;
  float one = 1.f;
  if (c >= nbq) {
    c -= nbq;
    heads = p.Hkv;
    kind = 1;
    if (c >= nbk) {
      c -= nbk;
      src = p.vn;
      dst = p.vrot;
      mat = p.vslices;
      stride = p.vs;
      fac = p.vfac;
      one = p.vone;
    } else {
      src = p.kn;
      dst = p.krot;
      stride = p.ks;
      fac = p.kfac;
      one = p.kone;
    }
  }
  float4 w[4][4];  // Π[32b + lane][16·warp + 4a ..]
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) w[a][b] = __ldg(mat + (4 * warp + a) * 128 + 32 * b + lane);
  griddep_wait();
  griddep_launch();
  const int64_t live = (int64_t)min(max((int64_t)p.row_start[p.B], (int64_t)0), p.R) * heads;
  for (int gi = 0; gi < per; ++gi) {
    const int64_t v0 = ((int64_t)c * per + gi) * kPrepV;
    if (v0 >= live) return;
    {  // a warp per row, four elements a lane (rows of all kinds: fewer than 2^31)
      const uint32_t v = (uint32_t)v0 + warp;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (v < (uint32_t)live) {
        const uint32_t r = v / (uint32_t)heads;
        x = tree_load4(src, (int64_t)r * stride + (v - r * heads) * 128 + 4 * lane, p.dtype);
      }
      *reinterpret_cast<float4*>(&sm.x[warp][4 * lane]) = x;
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kPrepV; ++v) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.x[v][16 * warp + 4 * a]);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          acc[b] = fmaf(w[a][b].x, x.x, fmaf(w[a][b].y, x.y, fmaf(w[a][b].z, x.z, fmaf(w[a][b].w, x.w, acc[b]))));
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) sm.part[warp][v][32 * b + lane] = acc[b];
    }
    __syncthreads();
    const int j = tid & 127, h = tid >> 7;
    float y[kPrepV / 2];
#pragma unroll
    for (int v = 0; v < kPrepV / 2; ++v) {
      const int vi = h * (kPrepV / 2) + v;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += sm.part[k][vi][j];
      y[v] = s;
      // the row's largest magnitude (+inf where one is not a number)
      float m = fabsf(s) <= 3.4e38f ? fabsf(s) : INFINITY;
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      if (lane == 0) wmax[vi][warp & 3] = m;
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kPrepV / 2; ++v) {
      const int vi = h * (kPrepV / 2) + v;
      const int64_t at = v0 + vi;
      const float m = fmaxf(fmaxf(wmax[vi][0], wmax[vi][1]), fmaxf(wmax[vi][2], wmax[vi][3]));
      if (at >= live) continue;
      const bool bad = m == INFINITY && (TC || kind != 0);  // fp32 rows of q are used as they are
      float sc = 1.f;
      if (TC && m > 0.f && !bad) {  // largest magnitude to [2^11, 2^12) for q, [8, 16) for drafted rows
        const int ex = (int)(__float_as_uint(m) >> 23) - 127, up = (kind == 0 ? 11 : 3) - ex;
        sc = __uint_as_float((uint32_t)(127 + min(max(up, -120), 120)) << 23);
      }
      const float z = bad ? 0.f : y[v] * sc;
      if (j == 0) {
        const uint32_t r = (uint32_t)at / (uint32_t)heads;
        fac[kind == 0 ? at : (int64_t)((uint32_t)at - r * heads) * p.R + r] =
            bad ? NAN : TC && m == 0.f ? 0.f : one / sc;  // zeros have no say in anyone's scaling
      }
      if constexpr (TC) {
        const bool two = kind == 0 || p.dtok < kTreeTok;
        __half* d = reinterpret_cast<__half*>(dst) + at * (two ? 256 : 128) + j;
        const __half hi = __float2half_rn(z);
        d[0] = hi;
        if (two) d[128] = __float2half_rn(z - __half2float(hi));
      } else {
        dst[at * 128 + j] = z;
      }
    }
  }
}

// ------------------------------------------------------------------ attention, fp32
// 16·RT rows against 64 tokens at a time on the CUDA cores, products and sums in
// fp32 throughout.  For few shared reads a product, a thread's tiles are as square
// as its registers allow and the long axis of either product is split over
// threads (one token of 32 heads over 16384: 101 -> 69 us):
//   S = Q·K̂ᵀ  a warp takes 2·RT rows, a thread all of them by 8 tokens over a
//              quarter of the coordinates; four lanes join (2·RT x 2 scores each);
//   O += P·V̂  a thread takes kOR rows by 8 coordinates over a share of the tokens;
//              the shares are joined once, at the segment's end.
// The next tile's packed words are loaded into registers before this one's
// products; a thread unpacks 32 coordinates of a token, whole words in both
// layouts, against 16 centroids in 16 banks.  16, 32 or 64 rows (RT = 1, 2, 4) by
// the mean sequence, the smaller two with two CTAs an SM (32 rows for the 256
// of a long group: 4.76 ms against 4.26, every tile being unpacked twice as often).
// Calls: one token of 32 heads over 16384 cached (b = 4) 69 us; 8 requests of up to
// 16 drafted over 8191 438 us; 32 drafted of 64 heads over 131072 (b = 3) 4.10 ms,
// 34 TFLOP/s.  Bound by no one thing: issue 0.58 a clock and quarter, shared memory
// two thirds busy; half the shared reads or twice the warps gained under 3%, pairs
// of products in one instruction for O (fma2) 4%.
// Runs of 32 coordinates lie 40 words apart and rows of Q, K̂, V̂ 164, so that the
// eight lanes of a 16-byte access meet no bank twice.
constexpr int kFTok = 64, kFStride = 164, kFPStride = 68, kFRun = 40;
template <int RT>
constexpr int kFSmem = (16 * RT * kFStride + 2 * kFTok * kFStride + 16 * RT * kFPStride + 3 * kFTok + 3 * 16 * RT + 32) * 4;

// 32 fields of B bits, S bits apart, of the words w: centroids as floats.
template <int B, int S>
__device__ __forceinline__ void tree_unpack(const uint32_t* w, const float* cen, float4* dst) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int bit = (4 * k + e) * S, i = bit >> 5, s = bit & 31;
      const uint32_t x = s + B > 32 ? __funnelshift_r(w[i], w[i + 1], s) : w[i] >> s;
      v[e] = cen[x & ((1u << B) - 1u)];
    }
    dst[k] = make_float4(v[0], v[1], v[2], v[3]);
  }
}
template <int B>
__device__ __forceinline__ void tree_unpack_pair(uint32_t* w, int slot, const float* cen, float4* dst) {
#pragma unroll
  for (int i = 0; i < 2 * B; ++i) w[i] = __funnelshift_r(w[i], i + 1 < 2 * B ? w[i + 1] : 0u, slot * B);
  tree_unpack<B, 2 * B>(w, cen, dst);
}

// Two fp32 products and sums in one instruction.
__device__ __forceinline__ void fma2(float2& d, const float2& a, const float2& b) {
  uint64_t x = *reinterpret_cast<uint64_t*>(&d);
  asm("fma.rn.f32x2 %0, %1, %2, %0;\n" : "+l"(x) : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  d = *reinterpret_cast<float2*>(&x);
}

template <int RT>
__global__ void __launch_bounds__(256, RT == 4 ? 1 : 2) tree_attend_f32_kernel(const TreeParams p) {
  constexpr int kFRows = 16 * RT, kSR = 2 * RT, kOR = RT == 4 ? 8 : 4, kGroups = kFRows / kOR, kShares = 16 / kGroups;
  extern __shared__ __align__(16) float fsm[];
  float* Qs = fsm;                              // [rows][164]
  float* Ks = Qs + kFRows * kFStride;           // [64][164]
  float* Vs = Ks + kFTok * kFStride;            // [64][164]
  float* Ps = Vs + kFTok * kFStride;            // [rows][68]
  float* kn = Ps + kFRows * kFPStride;          // [64] K norm / √d
  float* vn = kn + kFTok;                       // [64] V norm / √d
  float* ok = vn + kFTok;                       // [64] 1: a token of the sequence
  float* rm = ok + kFTok;                       // [64] row maximum
  float* rl = rm + kFRows;                      // [64] row sum
  float* rf = rl + kFRows;                      // [64] rescale factor of the tile
  float* cen = rf + kFRows;                     // [2][16]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ds = lane & 3, tg = lane >> 2;  // S: quarter of the coordinates, tokens tg + 8k
  const int cg = tid & 15, rg = (tid >> 4) % kGroups, sh = (tid >> 4) / kGroups;  // O: coordinates, rows, share of the tokens
  const float inv_sd = 0.08838834764831845f;  // 1/√128
  if (tid < 16) {
    cen[tid] = p.kcen[tid];
    cen[16 + tid] = p.vcen[tid];
  }
  griddep_wait();
  griddep_launch();
  const TreeCta& share = p.cta[blockIdx.x];
  int64_t u = share.u;
  const int64_t u_end = share.end;
  int b = share.b;
  while (u < u_end) {
    const TreeSeg g = tree_seg(p, u, u_end, b);
    const TreeSeq& s = g.s;
    const int kvh = g.kvh, row0 = g.row0, nrow = g.nrow, first = g.first, last = g.last, ctiles = g.ctiles;
    __syncthreads();
    for (int e = tid; e < kFRows * 128; e += 256) {
      const int r = e >> 7, rho = row0 + r;
      Qs[r * kFStride + (e & 127) + (kFRun - 32) * ((e & 127) >> 5)] =
          r < nrow ? p.qrot[((int64_t)(s.start + rho / p.G) * p.Hq + kvh * p.G + rho % p.G) * 128 + (e & 127)] : 0.f;
    }
    if (tid < kFRows) {
      rm[tid] = -INFINITY;
      rl[tid] = 0.f;
    }
    float2 o[kOR][4];
#pragma unroll
    for (int i = 0; i < kOR; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = make_float2(0.f, 0.f);

    // this thread's token of a tile and 32 of its coordinates: packed words and norms
    const int tok0 = tid >> 2, quarter = tid & 3;
    uint32_t kw[4], vw[8];
    float skn = 0.f, svn = 0.f;
    bool good = false;
    int slot = 0;
    auto fetch = [&](int t2) {
      const int t = t2 * kFTok + tok0;
      good = t < s.len;
      skn = svn = 0.f;
      slot = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) kw[i] = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) vw[i] = 0u;
      if (!good) return;
      const int j = t / p.block;
      const int64_t page = p.table ? (int64_t)p.table[(int64_t)g.b * p.max_blocks + j] : g.b;
      good = page >= 0 && page < p.pages;
      if (!good) {
        atomicOr(p.status, 2);
        return;
      }
      const int64_t vec = (page * p.Hkv + kvh) * p.block + (t - j * p.block);
      const uint32_t* ks = p.kcodes + vec * (4 * p.kb) + quarter * p.kb;
      const uint2* vs = reinterpret_cast<const uint2*>(p.vcodes + (vec >> 1) * (8 * p.vb)) + quarter * p.vb;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < p.kb) kw[i] = __ldg(ks + i);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < p.vb) {
          const uint2 x = __ldg(vs + i);
          vw[2 * i] = x.x;
          vw[2 * i + 1] = x.y;
        }
      slot = (int)(vec & 1);
      skn = p.knorm[vec];
      svn = p.vnorm[vec];
    };
    const int cend = min(2 * last, (s.len + kFTok - 1) / kFTok);  // cached tiles of the segment end here
    if (2 * first < cend) fetch(2 * first);
    for (int t2 = 2 * first; t2 < 2 * last; ++t2) {
      const bool draft = (t2 >> 1) >= ctiles;
      const int t0 = draft ? (t2 - 2 * ctiles) * kFTok : t2 * kFTok;  // first token of the tile
      const int nt = min(kFTok, (draft ? (p.kn ? s.T : 0) : s.len) - t0);
      if (nt <= 0) continue;
      __syncthreads();  // the last tile's operands have been read
      {
        float4* kd = reinterpret_cast<float4*>(Ks + tok0 * kFStride + kFRun * quarter);
        float4* vd = reinterpret_cast<float4*>(Vs + tok0 * kFStride + kFRun * quarter);
        if (draft) {
          good = tok0 < nt;
          skn = svn = 0.f;
          const int64_t row = s.start + t0 + tok0, at = (row * p.Hkv + kvh) * 128 + 32 * quarter;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            kd[k] = good ? *reinterpret_cast<const float4*>(p.krot + at + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
            vd[k] = good ? *reinterpret_cast<const float4*>(p.vrot + at + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          if (good) {
            skn = p.kfac[(int64_t)kvh * p.R + row];
            svn = p.vfac[(int64_t)kvh * p.R + row];
          }
        } else {
          switch (p.kb) {
            case 1: tree_unpack<1, 1>(kw, cen, kd); break;
            case 2: tree_unpack<2, 2>(kw, cen, kd); break;
            case 3: tree_unpack<3, 3>(kw, cen, kd); break;
            default: tree_unpack<4, 4>(kw, cen, kd); break;
          }
          switch (p.vb) {
            case 1: tree_unpack_pair<1>(vw, slot, cen + 16, vd); break;
            case 2: tree_unpack_pair<2>(vw, slot, cen + 16, vd); break;
            case 3: tree_unpack_pair<3>(vw, slot, cen + 16, vd); break;
            default: tree_unpack_pair<4>(vw, slot, cen + 16, vd); break;
          }
          skn *= inv_sd;
          svn *= inv_sd;
        }
        if (quarter == 0) {
          kn[tok0] = skn;
          vn[tok0] = svn;
          ok[tok0] = good ? 1.f : 0.f;
        }
      }
      if (t2 + 1 < cend) fetch(t2 + 1);
      __syncthreads();
      float sc[kSR][2];  // the thread's scores: tokens tg + 8·(2·ds + e)
      {
        float acc[kSR][8];
#pragma unroll
        for (int i = 0; i < kSR; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;
        const float* qrow = Qs + kSR * warp * kFStride + kFRun * ds;
        const float* krow = Ks + tg * kFStride + kFRun * ds;
#pragma unroll 2
        for (int d = 0; d < 32; d += 4) {
          float4 a[kSR];
#pragma unroll
          for (int i = 0; i < kSR; ++i) a[i] = *reinterpret_cast<const float4*>(qrow + i * kFStride + d);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 c = *reinterpret_cast<const float4*>(krow + 8 * k * kFStride + d);
#pragma unroll
            for (int i = 0; i < kSR; ++i)
              acc[i][k] = fmaf(a[i].x, c.x, fmaf(a[i].y, c.y, fmaf(a[i].z, c.z, fmaf(a[i].w, c.w, acc[i][k]))));
          }
        }
        const bool up2 = (ds & 2) != 0, up1 = (ds & 1) != 0;
#pragma unroll
        for (int i = 0; i < kSR; ++i) {
          float h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            h[k] = (up2 ? acc[i][k + 4] : acc[i][k]) + __shfl_xor_sync(kFull, up2 ? acc[i][k] : acc[i][k + 4], 2);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            sc[i][k] = (up1 ? h[k + 2] : h[k]) + __shfl_xor_sync(kFull, up1 ? h[k] : h[k + 2], 1);
        }
      }
      // scores in base-2 units, masks, the tile's row maxima and sums (a warp has all of a row)
      const int tk = tg + 16 * ds;
      const float k0 = kn[tk] * p.zscale, k1 = kn[tk + 8] * p.zscale, w0 = vn[tk], w1 = vn[tk + 8];
      const bool on0 = ok[tk] != 0.f, on1 = ok[tk + 8] != 0.f;
#pragma unroll
      for (int i = 0; i < kSR; ++i) {
        const int r = kSR * warp + i;
        bool s0 = on0 && r < nrow, s1 = on1 && r < nrow;
        if (draft && r < nrow) {
          const int ti = (row0 + r) / p.G, j0 = t0 + tk, j1 = j0 + 8;
          if (p.mask) {
            const uint32_t* m = p.mask + (int64_t)(s.start + ti) * p.mask_words;
            s0 = s0 && (j0 >> 5) < p.mask_words && ((m[j0 >> 5] >> (j0 & 31)) & 1u) != 0u;
            s1 = s1 && (j1 >> 5) < p.mask_words && ((m[j1 >> 5] >> (j1 & 31)) & 1u) != 0u;
          } else {
            s0 = s0 && j0 <= ti;
            s1 = s1 && j1 <= ti;
          }
        }
        const float z0 = s0 ? sc[i][0] * k0 : -INFINITY, z1 = s1 ? sc[i][1] * k1 : -INFINITY;
        float m = fmaxf(z0, z1);
#pragma unroll
        for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
        const float old = rm[r];
        __syncwarp();
        const float nm = fmaxf(old, m), use = nm == -INFINITY ? 0.f : nm;
        const float f = old == -INFINITY ? 0.f : exp2f(old - use);
        const float p0 = exp2f(z0 - use), p1 = exp2f(z1 - use);
        Ps[r * kFPStride + tk] = p0 == 0.f ? 0.f : p0 * w0;
        Ps[r * kFPStride + tk + 8] = p1 == 0.f ? 0.f : p1 * w1;
        float l = p0 + p1;
#pragma unroll
        for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(kFull, l, off);
        if (lane == 0) {
          rm[r] = nm;
          rl[r] = rl[r] * f + l;
          rf[r] = f;
        }
      }
      __syncthreads();
      // O: rows kOR·rg.., coordinates 4·cg.. and 64 + 4·cg.., a share of the tokens
      const float* vrow = Vs + kFRun * (cg >> 3) + 4 * (cg & 7);
#pragma unroll
      for (int i = 0; i < kOR; ++i) {
        const float f = rf[kOR * rg + i];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[i][k].x *= f;
          o[i][k].y *= f;
        }
      }
#pragma unroll 1
      for (int t4 = sh * (kFTok / kShares); t4 < (sh + 1) * (kFTok / kShares); t4 += 4) {
        float4 pr[kOR];
#pragma unroll
        for (int i = 0; i < kOR; ++i) pr[i] = *reinterpret_cast<const float4*>(Ps + (kOR * rg + i) * kFPStride + t4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v0 = *reinterpret_cast<const float4*>(vrow + (t4 + e) * kFStride);
          const float4 v1 = *reinterpret_cast<const float4*>(vrow + (t4 + e) * kFStride + 2 * kFRun);
#pragma unroll
          for (int i = 0; i < kOR; ++i) {
            const float x = e == 0 ? pr[i].x : (e == 1 ? pr[i].y : (e == 2 ? pr[i].z : pr[i].w));
            const float2 xx = make_float2(x, x);
            fma2(o[i][0], xx, make_float2(v0.x, v0.y));
            fma2(o[i][1], xx, make_float2(v0.z, v0.w));
            fma2(o[i][2], xx, make_float2(v1.x, v1.y));
            fma2(o[i][3], xx, make_float2(v1.z, v1.w));
          }
        }
      }
    }
    // the shares of the tokens meet in the place of K̂ and V̂, then the records
    __syncthreads();
    float4* red = reinterpret_cast<float4*>(Ks);  // [shares - 1][rows][coordinates]
    if (sh > 0) {
#pragma unroll
      for (int i = 0; i < kOR; ++i) {
        float4* at = red + ((sh - 1) * kFRows + kOR * rg + i) * 32 + cg;
        at[0] = make_float4(o[i][0].x, o[i][0].y, o[i][1].x, o[i][1].y);
        at[16] = make_float4(o[i][2].x, o[i][2].y, o[i][3].x, o[i][3].y);
      }
    }
    __syncthreads();
    if (sh == 0) {
#pragma unroll
      for (int i = 0; i < kOR; ++i) {
        const int r = kOR * rg + i, rho = row0 + r;
        if (r < nrow) {
          float4 x = make_float4(o[i][0].x, o[i][0].y, o[i][1].x, o[i][1].y), y = make_float4(o[i][2].x, o[i][2].y, o[i][3].x, o[i][3].y);
#pragma unroll
          for (int h = 1; h < kShares; ++h) {
            const float4* at = red + ((h - 1) * kFRows + r) * 32 + cg;
            const float4 u = at[0], v = at[16];
            x.x += u.x;
            x.y += u.y;
            x.z += u.z;
            x.w += u.w;
            y.x += v.x;
            y.y += v.y;
            y.z += v.z;
            y.w += v.w;
          }
          float* rec = first == 0 ? p.rec + ((int64_t)(s.start + rho / p.G) * p.Hq + kvh * p.G + rho % p.G) * kTreeRec
                                  : p.crec + ((int64_t)blockIdx.x * p.rows + r) * kTreeRec;
          if (cg == 0) {
            rec[0] = rm[r];
            rec[1] = rl[r];
          }
          *reinterpret_cast<float4*>(rec + 4 + 4 * cg) = x;
          *reinterpret_cast<float4*>(rec + 68 + 4 * cg) = y;
        }
      }
    }
    u += last - first;
    if (u < u_end) b = tree_next(p, u, b);
  }
}

// ------------------------------------------------------------------ join and rotation back
// A warp per row: its records (its own and those of the CTAs that continued its
// group) under their common maximum, divided by the sum of weights; then
// out = Πᵀ·o for the CTA's kPrepV rows, the matrix in registers as in the
// rotation.  A row that saw nothing is zero.  Bound by latency, a record's two
// reads after the attention kernel's end; where the records are is found before
// it (25.4 -> 23.9 us for the three kernels on one token over 16384).
__global__ void __launch_bounds__(256, 2) tree_join_kernel(const TreeParams p, const int per) {
  __shared__ __align__(16) RotSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float4 w[16];  // Π[16·warp + k][4·lane ..]
#pragma unroll
  for (int k = 0; k < 16; ++k) w[k] = __ldg(reinterpret_cast<const float4*>(p.vpi + (16 * warp + k) * 128) + lane);
  // Where a row's records are, from what was laid out before the attention kernel
  // could begin: found before the wait for it.  (All its CTAs had waited for the
  // rotation's end when this kernel was let in.)
  const int64_t live = (int64_t)min(max((int64_t)__ldcg(p.row_start + p.B), (int64_t)0), p.R) * p.Hq;
  const int64_t units = __ldcg(&p.seq[p.B].unit);
  const int64_t step = (int64_t)p.rows * kTreeRec;
  struct Row {
    const float *own, *more;
    int c0, c1;  // CTAs that have records of it (c1 < c0: none)
  };
  auto row_at = [&](int64_t at) -> Row {
    Row w{nullptr, nullptr, 0, -1};
    if (at >= live) return w;
    const int r = (int)((uint32_t)at / (uint32_t)p.Hq), head = (int)at - r * p.Hq, kvh = head / p.G;
    const int4* sp = reinterpret_cast<const int4*>(p.seq + tree_find(p.row_start, p.B, r));  // the last sequence that starts at or before r
    const int4 s0 = __ldcg(sp), s1 = __ldcg(sp + 1);
    TreeSeq s;
    s.start = s0.x;
    s.T = s0.y;
    s.rt = s0.w;
    s.per = s1.x;
    s.unit = (int64_t)((uint64_t)(uint32_t)s1.z | ((uint64_t)(uint32_t)s1.w << 32));
    if (r < s.start || r >= s.start + s.T) return w;
    const int rho = (r - s.start) * p.G + head - kvh * p.G;
    const int rt = rho / p.rows;
    const int64_t gs = s.unit + (int64_t)(kvh * s.rt + rt) * s.per, ge = gs + s.per;
    const int64_t n0 = (gs + 1) * p.ctas - 1, n1 = ge * p.ctas - 1;  // 32-bit division where it will do
    const bool small = n1 <= 0xFFFFFFFFll;
    w.c0 = small ? (int)((uint32_t)n0 / (uint32_t)units) : (int)(n0 / units);
    w.c1 = small ? (int)((uint32_t)n1 / (uint32_t)units) : (int)(n1 / units);
    w.own = p.rec + at * kTreeRec;
    w.more = p.crec + (int64_t)(rho - rt * p.rows) * kTreeRec;
    return w;
  };
  Row row = row_at((int64_t)blockIdx.x * per * kPrepV + warp);
  griddep_wait();
  griddep_launch();
  for (int gi = 0; gi < per; ++gi) {
    const int64_t v0 = ((int64_t)blockIdx.x * per + gi) * kPrepV;
    if (v0 >= live) return;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    {
      if (row.c1 >= row.c0) {
        const int c0 = row.c0, c1 = row.c1;
        const float *own = row.own, *more = row.more;
        // records 0 (own) .. c1 - c0, 32 at a time; with fewer units than CTAs
        // some of the CTAs between have none
        float M = -INFINITY, L = 0.f;
        for (int k0 = 0; k0 <= c1 - c0; k0 += 32) {
          const int k = k0 + lane;
          bool on = k <= c1 - c0;
          if (on && k > 0 && units < p.ctas)
            on = tree_cut(c0 + k + 1, units, p.ctas) != tree_cut(c0 + k, units, p.ctas);
          float m = -INFINITY, l = 0.f;
          if (on) {
            const float2 ml = *reinterpret_cast<const float2*>(k == 0 ? own : more + (c0 + k) * step);
            m = ml.x;
            l = ml.y;
          }
          on = on && l != 0.f;  // saw nothing (a NaN sum goes on)
          float top = on ? m : -INFINITY;
#pragma unroll
          for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
          const float nm = fmaxf(M, top), use = nm == -INFINITY ? 0.f : nm;
          const float fa = M == -INFINITY ? 0.f : exp2f(M - use);
          const float f = on ? exp2f(m - use) : 0.f;
          float ls = on ? l * f : 0.f;
#pragma unroll
          for (int i = 16; i; i >>= 1) ls += __shfl_xor_sync(kFull, ls, i);
          L = L * fa + ls;
          o.x *= fa;
          o.y *= fa;
          o.z *= fa;
          o.w *= fa;
          uint32_t todo = __ballot_sync(kFull, on);
          while (todo) {  // eight records at a time, all their loads in flight
            float4 a[8];
            float fk[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              fk[q] = 0.f;
              a[q] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (todo) {
                const int kk = __ffs(todo) - 1;
                todo &= todo - 1;
                fk[q] = __shfl_sync(kFull, f, kk);
                a[q] = *(reinterpret_cast<const float4*>((k0 + kk == 0 ? own : more + (c0 + k0 + kk) * step) + 4) + lane);
              }
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              o.x = fmaf(a[q].x, fk[q], o.x);
              o.y = fmaf(a[q].y, fk[q], o.y);
              o.z = fmaf(a[q].z, fk[q], o.z);
              o.w = fmaf(a[q].w, fk[q], o.w);
            }
          }
          M = nm;
        }
        const float inv = L == 0.f ? 0.f : p.ofold / L;  // a NaN stays one
        o.x *= inv;
        o.y *= inv;
        o.z *= inv;
        o.w *= inv;
      }
    }
    *reinterpret_cast<float4*>(&sm.x[warp][4 * lane]) = o;
    if (gi + 1 < per) row = row_at(v0 + kPrepV + warp);
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kPrepV; ++v) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k4 = 0; k4 < 4; ++k4) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.x[v][16 * warp + 4 * k4]);
        const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc.x = fmaf(w[4 * k4 + e].x, xs[e], acc.x);
          acc.y = fmaf(w[4 * k4 + e].y, xs[e], acc.y);
          acc.z = fmaf(w[4 * k4 + e].z, xs[e], acc.z);
          acc.w = fmaf(w[4 * k4 + e].w, xs[e], acc.w);
        }
      }
      *reinterpret_cast<float4*>(&sm.part[warp][v][4 * lane]) = acc;
    }
    __syncthreads();
    const int j = tid & 127, h = tid >> 7;
#pragma unroll
    for (int v = 0; v < kPrepV / 2; ++v) {
      const int vi = h * (kPrepV / 2) + v;
      if (v0 + vi >= live) continue;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += sm.part[k][vi][j];
      const int64_t to = (v0 + vi) * 128 + j;
      if (p.dtype == TQ_F32)
        static_cast<float*>(p.out)[to] = s;
      else if (p.dtype == TQ_F16)
        static_cast<__half*>(p.out)[to] = __float2half_rn(s);
      else
        static_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(s);
    }
  }
}

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

struct TreeWs {
  size_t seq, cta, q, k, v, qf, kf, vf, rec, crec, total;
};
TreeWs tree_ws(int B, int Hq, int Hkv, int64_t R) {
  TreeWs w;
  const size_t rq = (size_t)R * Hq, rk = (size_t)R * Hkv;
  w.seq = 0;
  w.cta = w.seq + al256((size_t)(B + 1) * sizeof(TreeSeq));
  w.q = w.cta + al256((size_t)num_sms() * 2 * sizeof(TreeCta));
  w.k = w.q + al256(rq * 512);
  w.v = w.k + al256(rk * 512);
  w.qf = w.v + al256(rk * 512);
  w.kf = w.qf + al256(rq * 4);
  w.vf = w.kf + al256(rk * 4);
  w.rec = w.vf + al256(rk * 4);
  w.crec = w.rec + al256(rq * kTreeRec * 4);
  w.total = w.crec + al256((size_t)num_sms() * 64 * kTreeRec * 4);
  return w;
}

}  // namespace

template <int RT>
static cudaError_t attend_f32(const TreeParams& p, cudaStream_t st) {
  static PerDeviceValue attr;
  const cudaError_t e = smem_attr_once(attr, (const void*)tree_attend_f32_kernel<RT>, kFSmem<RT>);
  if (e != cudaSuccess) return e;
  return tree_launch(tree_attend_f32_kernel<RT>, p.ctas, 256, kFSmem<RT>, st, p);
}
cudaError_t tree_attend_f32(const TreeParams& p, cudaStream_t st) {
  return p.rows == 16 ? attend_f32<1>(p, st) : p.rows == 32 ? attend_f32<2>(p, st) : attend_f32<4>(p, st);
}

size_t tree_ws_bytes(int B, int Hq, int Hkv, int64_t R) { return tree_ws(B, Hq, Hkv, R).total; }

tq_status launch_tree(const DevCtx& kc, const DevCtx& vc, const TreeArgs& a, cudaStream_t stream) {
  TreeParams p;
  p.q = a.q;
  p.kn = a.k_new;
  p.vn = a.v_new;
  p.qs = a.q_stride;
  p.ks = a.k_stride;
  p.vs = a.v_stride;
  p.dtype = a.dtype;
  p.row_start = a.row_start;
  p.len = a.len;
  p.table = a.table;
  p.mask = a.mask;
  p.mask_words = a.mask_words;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.max_blocks = a.table ? a.max_blocks : 1;
  p.block = a.block;
  p.R = a.R;
  p.pages = std::min(a.K->n, a.V->n) / ((int64_t)a.Hkv * a.block);
  p.kcodes = a.K->d_codes;
  p.vcodes = a.V->d_codes;
  p.knorm = a.K->d_norm;
  p.vnorm = a.V->d_norm;
  p.kb = kc.b_mse;
  p.vb = vc.b_mse;
  p.kslices = kc.pi_slices;
  p.vslices = vc.pi_slices;
  p.vpi = vc.pi;
  for (int k = 0; k < 16; ++k) {
    p.kcen[k] = kc.cen[k];
    p.vcen[k] = vc.cen[k];
  }
  p.zscale = a.scale * kTreeLog2e;
  p.out = a.out;
  p.status = kc.status;
  const TreeWs w = tree_ws(a.B, a.Hq, a.Hkv, a.R);
  unsigned char* base = static_cast<unsigned char*>(a.ws);
  p.seq = reinterpret_cast<TreeSeq*>(base + w.seq);
  p.cta = reinterpret_cast<TreeCta*>(base + w.cta);
  p.qrot = reinterpret_cast<float*>(base + w.q);
  p.krot = reinterpret_cast<float*>(base + w.k);
  p.vrot = reinterpret_cast<float*>(base + w.v);
  p.qfac = reinterpret_cast<float*>(base + w.qf);
  p.kfac = reinterpret_cast<float*>(base + w.kf);
  p.vfac = reinterpret_cast<float*>(base + w.vf);
  p.rec = reinterpret_cast<float*>(base + w.rec);
  p.crec = reinterpret_cast<float*>(base + w.crec);
  // fp32 rows are computed in fp32; 16-bit types round coarser than the
  // tensor-core kernel does
  const bool tc = a.dtype != TQ_F32;
  p.rows = tree_umma_rows(a.R, a.B, p.G);
  p.dtok = a.dtype == TQ_F16 ? kTreeTok / 2 : kTreeTok;
  p.ctas = num_sms() * (tc || p.rows == 64 ? 1 : 2);  // as many as fit at once
  p.klut = kc.lut;
  p.vlut = vc.lut;
  bool same = kc.b_mse == vc.b_mse && kc.alpha == vc.alpha;
  for (int k = 0; same && k < (1 << kc.b_mse); ++k) same = kc.cen[k] == vc.cen[k];
  p.same_lut = same;
  p.kone = tc ? kc.sqrt_d * kc.alpha : 1.f;
  p.vone = tc ? vc.sqrt_d * vc.alpha * kTreeVDown : 1.f;
  p.zfold = p.zscale / p.kone;
  p.ofold = 1.f / p.vone;
  p.wait_limit = kc.wait_limit;
  // the units of a sequence, whatever it turns out to be, are counted in 32 bits
  const int64_t most_rt = (a.R * p.G + p.rows - 1) / p.rows;
  const int64_t most_per = (int64_t)p.max_blocks * p.block / kTreeTok + a.R / p.dtok + 2;
  if (most_rt > 0 && most_per > (int64_t)INT32_MAX / (most_rt * a.Hkv)) return TQ_ERR_UNSUPPORTED;
  // groups of kPrepV rows, as many to a CTA as leave two CTAs on every SM
  const int64_t nq = (a.R * a.Hq + kPrepV - 1) / kPrepV, nk = a.k_new ? (a.R * a.Hkv + kPrepV - 1) / kPrepV : 0;
  const int64_t fill = 2 * (int64_t)num_sms();
  const int per = (int)((nq + 2 * nk + fill - 1) / fill), perj = (int)((nq + fill - 1) / fill);
  const int nbq = (int)((nq + per - 1) / per), nbk = (int)((nk + per - 1) / per);
  const int grid = 1 + nbq + 2 * nbk;
  cudaError_t e = tc ? tree_launch(tree_prep_kernel<true>, grid, 256, 0, stream, p, per, nbq, nbk)
                     : tree_launch(tree_prep_kernel<false>, grid, 256, 0, stream, p, per, nbq, nbk);
  if (e == cudaSuccess) e = tc ? tree_attend_umma(p, stream) : tree_attend_f32(p, stream);
  if (e == cudaSuccess) e = tree_launch(tree_join_kernel, (int)((nq + perj - 1) / perj), 256, 0, stream, p, perj);
  return e == cudaSuccess ? TQ_OK : set_cuda_error(e);
}

}  // namespace tq
