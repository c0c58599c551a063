// Attention of drafted tokens over a packed cache: rotation of the rows, the
// fp32 attention kernel, the join of the CTAs' partial states, and the host
// side.  tq_tree.cuh has the mathematics and the division of the work.
#include <algorithm>

#include "tq_tree.cuh"

namespace tq {

namespace {

// ------------------------------------------------------------------ rotation of q, k, v
// y = Π·x for kPrepV vectors per CTA: thread (coordinate, half of the vectors),
// the matrix in column slices (coalesced, L2-resident), x broadcast from
// shared memory, fp32 sums.  CTA 0 also lays out the units of the sequences.
// A drafted row that holds an infinity or a NaN is stored as zeros with the
// factor NaN: rows that see it become NaN through the factor, and rows that do
// not see it are not touched by a product 0 · NaN.
constexpr int kPrepV = 8;

// TC: rows for the tensor cores, scaled by a power of two into fp16's range,
// the leading part and (q) the remainder; else fp32.
template <bool TC>
__global__ void __launch_bounds__(256) tree_prep_kernel(const TreeParams p) {
  __shared__ __align__(16) float xs[kPrepV][128];
  __shared__ float wmax[kPrepV][4];
  __shared__ int64_t wsum[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch();
  const int64_t nq = p.R * p.Hq, nk = p.kn ? p.R * p.Hkv : 0;
  const int64_t cq = (nq + kPrepV - 1) / kPrepV, ck = (nk + kPrepV - 1) / kPrepV;
  if (blockIdx.x == 0) {
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
      }
      base += tot;
    }
    if (tid == 0) p.seq[p.B].unit = base;
    __syncthreads();
    for (int c = tid; c < p.ctas; c += 256) {
      const int64_t u = tree_cut(c, base, p.ctas);
      int lo = 0, hi = p.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.seq[mid].unit <= u)
          lo = mid;
        else
          hi = mid - 1;
      }
      p.cta_seq[c] = lo;
    }
    return;
  }
  int64_t c = blockIdx.x - 1;
  const void* src = p.q;
  float *dst = p.qrot, *fac = p.qfac;
  const float4* mat = p.kslices;
  int64_t stride = p.qs, n = nq;
  int heads = p.Hq, kind = 0;
  float one = 1.f;
  if (c >= cq) {
    c -= cq;
    n = nk;
    heads = p.Hkv;
    kind = 1;
    if (c >= ck) {
      c -= ck;
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
  const int64_t v0 = c * kPrepV;
  const int64_t live = (int64_t)min(max((int64_t)p.row_start[p.B], (int64_t)0), p.R) * heads;
  if (v0 >= live) return;
  for (int e = tid; e < kPrepV * 128; e += 256) {
    const int64_t v = v0 + (e >> 7);
    xs[e >> 7][e & 127] = v < live ? tree_load(src, (v / heads) * stride + (v % heads) * 128 + (e & 127), p.dtype) : 0.f;
  }
  __syncthreads();
  const int j = tid & 127, h = tid >> 7;
  float acc[kPrepV / 2];
#pragma unroll
  for (int v = 0; v < kPrepV / 2; ++v) acc[v] = 0.f;
#pragma unroll 8
  for (int i4 = 0; i4 < 32; ++i4) {
    const float4 w = __ldg(mat + i4 * 128 + j);
#pragma unroll
    for (int v = 0; v < kPrepV / 2; ++v) {
      const float4 x = *reinterpret_cast<const float4*>(&xs[h * (kPrepV / 2) + v][4 * i4]);
      acc[v] = fmaf(w.x, x.x, fmaf(w.y, x.y, fmaf(w.z, x.z, fmaf(w.w, x.w, acc[v]))));
    }
  }
  if (!TC && kind == 0) {  // fp32 rows of q are used as they are
#pragma unroll
    for (int v = 0; v < kPrepV / 2; ++v) {
      const int64_t at = v0 + h * (kPrepV / 2) + v;
      if (at < n) dst[at * 128 + j] = acc[v];
    }
    return;
  }
  // the largest magnitude of every row (+inf where one is not a number)
#pragma unroll
  for (int v = 0; v < kPrepV / 2; ++v) {
    float m = fabsf(acc[v]) <= 3.4e38f ? fabsf(acc[v]) : INFINITY;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (lane == 0) wmax[h * (kPrepV / 2) + v][warp & 3] = m;
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kPrepV / 2; ++v) {
    const int vi = h * (kPrepV / 2) + v;
    const int64_t at = v0 + vi;
    const float m = fmaxf(fmaxf(wmax[vi][0], wmax[vi][1]), fmaxf(wmax[vi][2], wmax[vi][3]));
    if (at >= n) continue;
    const bool bad = m == INFINITY;
    float sc = 1.f;
    if (TC && m > 0.f && !bad) {  // largest magnitude to [2^11, 2^12) for q, [8, 16) for drafted rows
      const int ex = (int)(__float_as_uint(m) >> 23) - 127, up = (kind == 0 ? 11 : 3) - ex;
      sc = __uint_as_float((uint32_t)(127 + min(max(up, -120), 120)) << 23);
    }
    const float y = bad ? 0.f : acc[v] * sc;
    if (j == 0) {
      const float f = bad ? NAN : one / sc;
      fac[kind == 0 ? at : (at % heads) * p.R + at / heads] = f;
    }
    if constexpr (TC) {
      __half* d = reinterpret_cast<__half*>(dst) + at * (kind == 0 ? 256 : 128) + j;
      const __half hi = __float2half_rn(y);
      d[0] = hi;
      if (kind == 0) d[128] = __float2half_rn(y - __half2float(hi));
    } else {
      dst[at * 128 + j] = y;
    }
  }
}

// ------------------------------------------------------------------ attention, fp32
// 64 rows against 64 tokens at a time on the CUDA cores: S = Q·K̂ᵀ with 4 x 4
// values per thread, running maximum and sum per row, O += P·V̂ with 4 x 8.
// Products and sums in fp32 throughout; bound by the FMA rate.
constexpr int kFRows = 64, kFTok = 64, kFStride = 132, kFPStride = 68;
constexpr int kFSmem = (2 * kFRows * kFStride + kFTok * 128 + kFRows * kFPStride + 3 * kFTok + 3 * kFRows + 32) * 4;

// Code j of a vector: b bits at bit j·b of its own stream, or (PAIR) at bit
// (2j + slot)·b of the block it shares.
__device__ __forceinline__ uint32_t tree_code(const uint32_t* w, int j, int b, bool pair, int slot) {
  const int bit = pair ? (2 * j + slot) * b : j * b;
  const int i = bit >> 5, sh = bit & 31;
  uint32_t v = __ldg(w + i) >> sh;
  if (sh + b > 32) v |= __ldg(w + i + 1) << (32 - sh);
  return v & ((1u << b) - 1u);
}

__global__ void __launch_bounds__(256) tree_attend_f32_kernel(const TreeParams p) {
  extern __shared__ __align__(16) float fsm[];
  float* Qs = fsm;                              // [64][132]
  float* Ks = Qs + kFRows * kFStride;           // [64][132]
  float* Vs = Ks + kFTok * kFStride;            // [64][128]
  float* Ps = Vs + kFTok * 128;                 // [64][68]
  float* kn = Ps + kFRows * kFPStride;          // [64] K norm / √d
  float* vn = kn + kFTok;                       // [64] V norm / √d
  float* ok = vn + kFTok;                       // [64] 1: a token of the sequence
  float* rm = ok + kFTok;                       // [64] row maximum
  float* rl = rm + kFRows;                      // [64] row sum
  float* rf = rl + kFRows;                      // [64] rescale factor of the tile
  float* cen = rf + kFRows;                     // [2][16]
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const float inv_sd = 0.08838834764831845f;  // 1/√128
  if (tid < 16) {
    cen[tid] = p.kcen[tid];
    cen[16 + tid] = p.vcen[tid];
  }
  griddep_wait();
  griddep_launch();
  const int64_t units = p.seq[p.B].unit;
  int64_t u = tree_cut(blockIdx.x, units, p.ctas);
  const int64_t u_end = tree_cut(blockIdx.x + 1, units, p.ctas);
  int sb = u < u_end ? p.cta_seq[blockIdx.x] : 0;
  while (u < u_end) {
    const TreeSeg g = tree_seg(p, u, u_end, sb);
    sb = g.b;
    const TreeSeq& s = g.s;
    const int b = g.b, kvh = g.kvh, row0 = g.row0, nrow = g.nrow, first = g.first, last = g.last, ctiles = g.ctiles;
    __syncthreads();
    for (int e = tid; e < kFRows * 128; e += 256) {
      const int r = e >> 7, rho = row0 + r;
      Qs[r * kFStride + (e & 127)] =
          r < nrow ? p.qrot[((int64_t)(s.start + rho / p.G) * p.Hq + kvh * p.G + rho % p.G) * 128 + (e & 127)] : 0.f;
    }
    if (tid < kFRows) {
      rm[tid] = -INFINITY;
      rl[tid] = 0.f;
    }
    float o[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) o[i][k] = 0.f;

    for (int t2 = 2 * first; t2 < 2 * last; ++t2) {
      const bool draft = (t2 >> 1) >= ctiles;
      const int t0 = draft ? (t2 - 2 * ctiles) * kFTok : t2 * kFTok;  // first token of the tile
      const int nt = min(kFTok, (draft ? (p.kn ? s.T : 0) : s.len) - t0);
      if (nt <= 0) continue;
      __syncthreads();  // the last tile's operands have been read
      {
        const int tok = tid >> 2, c0 = (tid & 3) * 32;  // token and 32 coordinates of this thread
        bool good = tok < nt;
        float4* kd = reinterpret_cast<float4*>(Ks + tok * kFStride + c0);
        float4* vd = reinterpret_cast<float4*>(Vs + tok * 128 + c0);
        float skn = 0.f, svn = 0.f;
        if (draft) {
          const int64_t at = ((int64_t)(s.start + t0 + tok) * p.Hkv + kvh) * 128 + c0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            kd[k] = good ? *reinterpret_cast<const float4*>(p.krot + at + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
            vd[k] = good ? *reinterpret_cast<const float4*>(p.vrot + at + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          if (good) {
            skn = p.kfac[(int64_t)kvh * p.R + s.start + t0 + tok];
            svn = p.vfac[(int64_t)kvh * p.R + s.start + t0 + tok];
          }
        } else {
          int64_t vec = 0;
          if (good) {
            const int t = t0 + tok, j = t / p.block;
            const int64_t page = p.table ? (int64_t)p.table[(int64_t)b * p.max_blocks + j] : b;
            good = page >= 0 && page < p.pages;
            if (!good) atomicOr(p.status, 2);
            vec = good ? (page * p.Hkv + kvh) * p.block + (t - j * p.block) : 0;
          }
          const uint32_t* kw = p.kcodes + vec * (4 * p.kb);
          const uint32_t* vw = p.vcodes + (vec >> 1) * (8 * p.vb);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
            if (good) {
              const int j = c0 + 4 * k, sl = (int)(vec & 1);
              kv = make_float4(cen[tree_code(kw, j, p.kb, false, 0)], cen[tree_code(kw, j + 1, p.kb, false, 0)],
                               cen[tree_code(kw, j + 2, p.kb, false, 0)], cen[tree_code(kw, j + 3, p.kb, false, 0)]);
              vv = make_float4(cen[16 + tree_code(vw, j, p.vb, true, sl)], cen[16 + tree_code(vw, j + 1, p.vb, true, sl)],
                               cen[16 + tree_code(vw, j + 2, p.vb, true, sl)],
                               cen[16 + tree_code(vw, j + 3, p.vb, true, sl)]);
            }
            kd[k] = kv;
            vd[k] = vv;
          }
          if (good) {
            skn = p.knorm[vec] * inv_sd;
            svn = p.vnorm[vec] * inv_sd;
          }
        }
        if ((tid & 3) == 0) {
          kn[tok] = skn;
          vn[tok] = svn;
          ok[tok] = good ? 1.f : 0.f;
        }
      }
      __syncthreads();
      // S: rows 4·ty.., tokens tx + 16·k
      float acc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] = 0.f;
#pragma unroll 4
      for (int d4 = 0; d4 < 32; ++d4) {
        float4 a[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(Qs + (4 * ty + i) * kFStride + 4 * d4);
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * k) * kFStride + 4 * d4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc[i][k] = fmaf(a[i].x, c[k].x, fmaf(a[i].y, c[k].y, fmaf(a[i].z, c[k].z, fmaf(a[i].w, c[k].w, acc[i][k]))));
      }
      // scores in base-2 units, masks, the tile's row maxima (16 threads share a row)
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i, rho = row0 + r, ti = rho / p.G;
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tok = tx + 16 * k;
          bool on = r < nrow && ok[tok] != 0.f;
          if (draft && on) {
            const int j = t0 + tok;
            if (p.mask)
              on = (j >> 5) < p.mask_words &&
                   ((p.mask[(int64_t)(s.start + ti) * p.mask_words + (j >> 5)] >> (j & 31)) & 1u) != 0u;
            else
              on = j <= ti;
          }
          acc[i][k] = on ? acc[i][k] * kn[tok] * p.zscale : -INFINITY;
          m = fmaxf(m, acc[i][k]);
        }
#pragma unroll
        for (int off = 8; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
        const float old = rm[r];
        __syncwarp();
        const float nm = fmaxf(old, m), use = nm == -INFINITY ? 0.f : nm;
        f[i] = old == -INFINITY ? 0.f : exp2f(old - use);
        float l = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float pr = exp2f(acc[i][k] - use);
          l += pr;
          const int tok = tx + 16 * k;
          Ps[r * kFPStride + tok] = pr == 0.f ? 0.f : pr * vn[tok];
        }
#pragma unroll
        for (int off = 8; off; off >>= 1) l += __shfl_xor_sync(kFull, l, off);
        if (tx == 0) {
          rm[r] = nm;
          rl[r] = rl[r] * f[i] + l;
        }
      }
      __syncthreads();
      // O: rows 4·ty.., coordinates 8·tx..
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) o[i][k] *= f[i];
      for (int t4 = 0; t4 < kFTok / 4; ++t4) {
        float4 pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4*>(Ps + (4 * ty + i) * kFPStride + 4 * t4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v0 = *reinterpret_cast<const float4*>(Vs + (4 * t4 + e) * 128 + 8 * tx);
          const float4 v1 = *reinterpret_cast<const float4*>(Vs + (4 * t4 + e) * 128 + 8 * tx + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = e == 0 ? pr[i].x : (e == 1 ? pr[i].y : (e == 2 ? pr[i].z : pr[i].w));
            o[i][0] = fmaf(x, v0.x, o[i][0]);
            o[i][1] = fmaf(x, v0.y, o[i][1]);
            o[i][2] = fmaf(x, v0.z, o[i][2]);
            o[i][3] = fmaf(x, v0.w, o[i][3]);
            o[i][4] = fmaf(x, v1.x, o[i][4]);
            o[i][5] = fmaf(x, v1.y, o[i][5]);
            o[i][6] = fmaf(x, v1.z, o[i][6]);
            o[i][7] = fmaf(x, v1.w, o[i][7]);
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i, rho = row0 + r;
      if (r < nrow) {
        float* rec = first == 0 ? p.rec + ((int64_t)(s.start + rho / p.G) * p.Hq + kvh * p.G + rho % p.G) * kTreeRec
                                : p.crec + ((int64_t)blockIdx.x * p.rows + r) * kTreeRec;
        if (tx == 0) {
          rec[0] = rm[r];
          rec[1] = rl[r];
        }
        *reinterpret_cast<float4*>(rec + 4 + 8 * tx) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        *reinterpret_cast<float4*>(rec + 8 + 8 * tx) = make_float4(o[i][4], o[i][5], o[i][6], o[i][7]);
      }
    }
    u += last - first;
  }
}

// ------------------------------------------------------------------ join and rotation back
// kPrepV rows per CTA: each row's records (its own and those of the CTAs that
// continued its group) under their common maximum, divided by the sum, then
// out = Πᵀ·o.  A row that saw nothing is zero.
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p) {
  __shared__ __align__(16) float os[kPrepV][128];
  const int tid = threadIdx.x, j = tid & 127, h = tid >> 7;
  griddep_wait();
  griddep_launch();
  const int64_t v0 = (int64_t)blockIdx.x * kPrepV;
  const int64_t live = (int64_t)min(max((int64_t)p.row_start[p.B], (int64_t)0), p.R) * p.Hq;
  if (v0 >= live) return;
  const int64_t units = p.seq[p.B].unit;
  for (int v = h; v < kPrepV; v += 2) {
    const int64_t at = v0 + v;
    float val = 0.f;
    if (at < live) {
      const int r = (int)(at / p.Hq), head = (int)(at % p.Hq), kvh = head / p.G;
      const int b = tree_find(p.row_start, p.B, r);  // the last sequence that starts at or before r
      const TreeSeq s = p.seq[b];
      const int rho = (r - s.start) * p.G + head % p.G;
      if (r >= s.start && r < s.start + s.T) {
        const int64_t gs = s.unit + (int64_t)(kvh * s.rt + rho / p.rows) * s.per, ge = gs + s.per;
        const int64_t c0 = ((gs + 1) * p.ctas - 1) / units, c1 = (ge * p.ctas - 1) / units;
        const float* own = p.rec + at * kTreeRec;
        float M = own[0], L = own[1], A = own[4 + j];
        for (int64_t c = c0 + 1; c <= c1; ++c) {
          if (tree_cut(c + 1, units, p.ctas) == tree_cut(c, units, p.ctas)) continue;  // no unit of its own
          const float* rec = p.crec + (c * p.rows + rho % p.rows) * kTreeRec;
          const float m = rec[0];
          if (rec[1] == 0.f) continue;  // saw nothing (a NaN sum goes on)
          const float nm = fmaxf(M, m), fa = M == -INFINITY ? 0.f : exp2f(M - nm), fb = exp2f(m - nm);
          L = L * fa + rec[1] * fb;
          A = A * fa + rec[4 + j] * fb;
          M = nm;
        }
        val = L > 0.f ? A / L : (L == 0.f ? 0.f : A + L);  // a NaN stays one
      }
    }
    os[v][j] = val * p.ofold;
  }
  __syncthreads();
  float acc[kPrepV / 2];
#pragma unroll
  for (int v = 0; v < kPrepV / 2; ++v) acc[v] = 0.f;
#pragma unroll 4
  for (int k4 = 0; k4 < 32; ++k4) {
    const float w0 = __ldg(p.vpi + (4 * k4 + 0) * 128 + j), w1 = __ldg(p.vpi + (4 * k4 + 1) * 128 + j);
    const float w2 = __ldg(p.vpi + (4 * k4 + 2) * 128 + j), w3 = __ldg(p.vpi + (4 * k4 + 3) * 128 + j);
#pragma unroll
    for (int v = 0; v < kPrepV / 2; ++v) {
      const float4 x = *reinterpret_cast<const float4*>(&os[h * (kPrepV / 2) + v][4 * k4]);
      acc[v] = fmaf(w0, x.x, fmaf(w1, x.y, fmaf(w2, x.z, fmaf(w3, x.w, acc[v]))));
    }
  }
#pragma unroll
  for (int v = 0; v < kPrepV / 2; ++v) {
    const int64_t at = v0 + h * (kPrepV / 2) + v;
    if (at >= live) continue;
    if (p.dtype == TQ_F32)
      static_cast<float*>(p.out)[at * 128 + j] = acc[v];
    else if (p.dtype == TQ_F16)
      static_cast<__half*>(p.out)[at * 128 + j] = __float2half_rn(acc[v]);
    else
      static_cast<__nv_bfloat16*>(p.out)[at * 128 + j] = __float2bfloat16_rn(acc[v]);
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
  w.q = w.cta + al256((size_t)num_sms() * 4);
  w.k = w.q + al256(rq * 512);
  w.v = w.k + al256(rk * 512);
  w.qf = w.v + al256(rk * 512);
  w.kf = w.qf + al256(rq * 4);
  w.vf = w.kf + al256(rk * 4);
  w.rec = w.vf + al256(rk * 4);
  w.crec = w.rec + al256(rq * kTreeRec * 4);
  w.total = w.crec + al256((size_t)num_sms() * 128 * kTreeRec * 4);
  return w;
}

}  // namespace

cudaError_t tree_attend_f32(const TreeParams& p, cudaStream_t st) {
  static PerDeviceValue attr;
  const cudaError_t e = smem_attr_once(attr, (const void*)tree_attend_f32_kernel, kFSmem);
  if (e != cudaSuccess) return e;
  return tree_launch(tree_attend_f32_kernel, p.ctas, 256, kFSmem, p, st);
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
  p.cta_seq = reinterpret_cast<int*>(base + w.cta);
  p.qrot = reinterpret_cast<float*>(base + w.q);
  p.krot = reinterpret_cast<float*>(base + w.k);
  p.vrot = reinterpret_cast<float*>(base + w.v);
  p.qfac = reinterpret_cast<float*>(base + w.qf);
  p.kfac = reinterpret_cast<float*>(base + w.kf);
  p.vfac = reinterpret_cast<float*>(base + w.vf);
  p.rec = reinterpret_cast<float*>(base + w.rec);
  p.crec = reinterpret_cast<float*>(base + w.crec);
  p.ctas = num_sms();
  // fp32 rows are computed in fp32; 16-bit types round coarser than the
  // tensor-core kernel does
  const bool tc = a.dtype != TQ_F32;
  p.rows = tc ? 128 : kFRows;
  p.klut = kc.lut;
  p.vlut = vc.lut;
  bool same = kc.b_mse == vc.b_mse && kc.alpha == vc.alpha;
  for (int k = 0; same && k < (1 << kc.b_mse); ++k) same = kc.cen[k] == vc.cen[k];
  p.same_lut = same;
  p.kone = tc ? kc.sqrt_d * kc.alpha : 1.f;
  p.vone = tc ? vc.sqrt_d * vc.alpha : 1.f;
  p.zfold = p.zscale / p.kone;
  p.ofold = 1.f / p.vone;
  p.wait_limit = kc.wait_limit;
  const int64_t nq = (a.R * a.Hq + kPrepV - 1) / kPrepV, nk = a.k_new ? (a.R * a.Hkv + kPrepV - 1) / kPrepV : 0;
  if (1 + nq + 2 * nk > INT32_MAX) return TQ_ERR_UNSUPPORTED;
  const int grid = (int)(1 + nq + 2 * nk);
  cudaError_t e = tc ? tree_launch(tree_prep_kernel<true>, grid, 256, 0, p, stream)
                     : tree_launch(tree_prep_kernel<false>, grid, 256, 0, p, stream);
  if (e == cudaSuccess) e = tc ? tree_attend_umma(p, stream) : tree_attend_f32(p, stream);
  if (e == cudaSuccess) e = tree_launch(tree_join_kernel, (int)nq, 256, 0, p, stream);
  return e == cudaSuccess ? TQ_OK : set_cuda_error(e);
}

}  // namespace tq
