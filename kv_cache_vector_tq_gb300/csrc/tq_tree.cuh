#pragma once
// Attention of drafted tokens over a packed cache: what the kernels share.
//
//   out_i = (Σ_t p_it v̂_t + Σ_j p_ij v_j) / (Σ_t p_it + Σ_j p_ij),
//   p = exp(scale·⟨q_i, k⟩), t over the cached tokens of the row's sequence,
//   j over the drafted tokens that the row's mask names.
//
// Everything runs in the rotated domain: q, the drafted k and the drafted v
// are rotated once (⟨q, k⟩ = ⟨Πq, Πk⟩), the cached k̂ = s·ŷ/√d needs no rotation
// there, and the sum of values is rotated back once per row.
//
// Work: a group is (sequence, KV head, tile of kRows rows), a row being one
// (drafted token, query head of the KV head) pair; its units are 128 cached
// tokens each, then 128 drafted tokens each (fp16 rows: 64, in two terms).  The units of all groups, laid
// end to end, are shared evenly among the CTAs of a grid that fits the GPU
// once, whatever the lengths are: lengths live on the device, so a captured
// call serves every later length.  A CTA that starts a group leaves the rows'
// state (m, l, acc) in their own records, one that continues a group in the
// CTA's; a last kernel joins them.
#include <cuda_bf16.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

constexpr int kTreeTok = 128;       // tokens per unit
constexpr int kTreeRec = 132;       // floats per record: m, l, 2 pad, acc[128]
constexpr float kTreeLog2e = 1.4426950408889634f;
// Tensor-core path: values are taken 2^20 smaller, so that weights, which hold the
// inverse of a value's magnitude, leave fp32's range at neither end of it.
constexpr float kTreeVDown = 9.5367431640625e-07f;

// A sequence as the kernels see it: bad offsets and lengths are cut to what
// the buffers hold.  unit: its first unit.
struct TreeSeq {
  int start, T, len, rt, per;  // first row, drafted tokens, cached tokens, row tiles, units per group
  int pad;
  int64_t unit;
};

// A CTA's share of the units, and the sequence of its first unit: all that it
// needs to begin, in one read.
struct __align__(16) TreeCta {
  TreeSeq s;
  int64_t u, end;
  int b, pad[3];  // b: ~ of its number
};

struct TreeParams {
  const void *q, *kn, *vn;
  int64_t qs, ks, vs;  // strides between tokens in elements
  int dtype;
  const int32_t *row_start, *len, *table;
  const uint32_t* mask;
  int mask_words;
  int B, Hq, Hkv, G, max_blocks, block;
  int64_t R, pages;
  const uint32_t *kcodes, *vcodes;
  const float *knorm, *vnorm;
  int kb, vb;           // bits of a code
  const float4 *kslices, *vslices;  // Π of the K and V contexts in column slices
  const float* vpi;     // Π of the V context, row-major
  float kcen[16], vcen[16];
  float zscale;         // scale·log2(e)
  // tensor-core path
  const uint32_t *klut, *vlut;  // pair tables α·c
  int same_lut;
  float zfold;          // scale·log2(e)/(√d·α_K)
  float kone, vone;     // factor of a drafted row of scale 1: √d·α, v's times kTreeVDown (fp32 path: 1)
  float ofold;          // 1/vone
  uint32_t wait_limit;
  void* out;
  int* status;
  // workspace
  TreeSeq* seq;         // [B + 1]; seq[B].unit: the number of units
  TreeCta* cta;         // [ctas]
  float *qrot, *krot, *vrot;  // rotated rows: fp32, or fp16 (q, and all of an fp16 call: 128 leading parts, 128 remainders)
  float* qfac;          // [R·Hq] power of two that was divided out of a row of q (tensor-core path)
  float *kfac, *vfac;   // [Hkv][R] the same of the drafted rows, times kone / vone
  float* rec;           // [R·Hq] records of the rows
  float* crec;          // [ctas][rows] records of continued groups
  int ctas, rows;       // CTAs of the grid, rows per tile
  int dtok;             // drafted tokens per unit
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  const int64_t lo = min(max((int64_t)p.row_start[b], (int64_t)0), p.R);
  const int64_t hi = min(max((int64_t)p.row_start[b + 1], lo), p.R);
  s.start = (int)lo;
  s.T = (int)(hi - lo);
  s.len = (int)min((int64_t)max(p.len[b], 0), (int64_t)p.max_blocks * p.block);
  s.rt = (int)(((int64_t)s.T * p.G + p.rows - 1) / p.rows);
  s.per = (s.len + kTreeTok - 1) / kTreeTok + (p.kn ? (s.T + p.dtok - 1) / p.dtok : 0);
  if (s.per < 1) s.per = 1;
  s.pad = 0;
  s.unit = 0;
  return s;
}
// First unit of CTA c of n.
__device__ __forceinline__ int64_t tree_cut(int64_t c, int64_t units, int64_t n) { return c * units / n; }

// Largest index i in [0, n) with a[i] <= x (a ascending, a[0] <= x).  Past L1:
// the join asks before it has waited for the kernel ahead.
template <typename T>
__device__ __forceinline__ int tree_find(const T* a, int n, T x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldcg(a + mid) <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// A run of units of one group: units [first, last) of it, rows row0.. of the group.
struct TreeSeg {
  int b, kvh, row0, nrow, first, last, ctiles;
  TreeSeq s;
};
// The segment that starts at unit u of sequence b (~b: the CTA's first).
__device__ __forceinline__ TreeSeg tree_seg(const TreeParams& p, int64_t u, int64_t u_end, int b) {
  TreeSeg g;
  g.b = b < 0 ? ~b : b;
  g.s = *(b < 0 ? &p.cta[blockIdx.x].s : p.seq + b);
  const TreeSeq& s = g.s;
  const int w = (int)(u - s.unit);  // fewer than 2^31 units in a sequence: rows and lengths are
  const int grp = w / s.per;
  g.first = w - grp * s.per;
  g.kvh = grp / s.rt;
  g.row0 = (grp - g.kvh * s.rt) * p.rows;
  g.nrow = min(p.rows, s.T * p.G - g.row0);
  g.last = (int)min((int64_t)s.per, g.first + (u_end - u));
  g.ctiles = (s.len + kTreeTok - 1) / kTreeTok;
  return g;
}
// The sequence of unit u, b being it or one before it.
__device__ __forceinline__ int tree_next(const TreeParams& p, int64_t u, int b) {
  if (b < 0) b = ~b;
  while (b + 1 < p.B && p.seq[b + 1].unit <= u) ++b;
  return b;
}

// Four elements from element i on (a multiple of four) as fp32.
__device__ __forceinline__ float4 tree_load4(const void* p, int64_t i, int dtype) {
  if (dtype == TQ_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  float2 a, b;
  if (dtype == TQ_F16) {
    a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
  } else {
    a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
  }
  return make_float4(a.x, a.y, b.x, b.y);
}

cudaError_t tree_attend_f32(const TreeParams& p, cudaStream_t st);
cudaError_t tree_attend_umma(const TreeParams& p, cudaStream_t st);
int tree_umma_rows(int64_t rows, int B, int G);

// A launch that may begin while the kernel before it in the stream ends; every
// kernel here waits for that one (griddep_wait) before it touches its data.
template <typename... P, typename... A>
inline cudaError_t tree_launch(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
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

}  // namespace tq
