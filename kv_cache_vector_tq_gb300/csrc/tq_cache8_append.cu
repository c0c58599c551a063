// New tokens into the 8-bit paged cache (tq_cache8_append): norms and position
// rotation of q and k on the way, one launch.
//
//   q_out = turn(norm(q));  per page, KV head and side, with a the largest
//   magnitude among the new rows of the block:
//   s' = 2^e, the least with a <= 448·2^e, and no less than the block's scale s
//   where it holds earlier tokens; codes of those: e4m3(code·s / s'), new ones:
//   e4m3(x / s').
//
// A job is the new rows of one block, one KV head and side.  Its rows come by
// asynchronous copies, a slot of shared memory for every lane and pass (no
// barrier), are normed and turned in place there as fp32, and read again once
// the job's warps have agreed on the scale.  A job has a warp for every two rows
// of a pass, four passes a block, so that a block of any size has as many bytes
// in flight for each warp; more passes than kApPass slots are read twice (from
// L2).  Jobs need no sum over the requests: request b's are numbered from
// row_start[b] / block + 2b on.
// The CTAs behind the jobs turn q as tq_qk_norm_rope does.
#include <algorithm>
#include <cmath>

#include "tq_cache8.cuh"
#include "tq_rows.cuh"

namespace tq {

namespace {

constexpr int kApPass = 4;  // passes whose rows stay in shared memory

struct AppendParams {
  NormRopeParams q;  // the rows of q (Hkv = 0)
  const void *k, *v, *wk;
  int64_t ks, vs;
  const int32_t *row_start, *len, *table;
  int rows, B, Hkv, max_blocks, block, d;
  int64_t pages;
  uint8_t *k8, *v8;
  float *kscale, *vscale;
  int32_t* status;
  int jobs, warps;  // jobs in all, warps of a job
  int kv_ctas;
};

__device__ __forceinline__ uint32_t pack8(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// Four codes times f, rounded again.
__device__ __forceinline__ uint32_t again8(uint32_t w, float f) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
    const float2 x = __half22float2(__half2(r));
    v[2 * i] = x.x * f;
    v[2 * i + 1] = x.y * f;
  }
  return pack8(v[0], v[1], v[2], v[3]);
}
// The least power of two s with a <= 448·s, within the scales there are.
__device__ __forceinline__ float scale_of(float a) {
  const int bits = __float_as_int(a);
  const int e = (bits >> 23) - 127;  // a subnormal a: far below the least scale
  const int up = (bits & 0x7FFFFF) > 0x600000 ? 1 : 0;  // 448 = 1.75·2^8
  return __int_as_float((min(max(e - 8 + up, -60), 40) + 127) << 23);
}

template <typename TI, int LPR, bool HALF, bool NORM>
__device__ __forceinline__ void append_job(const AppendParams& p, int job, int w, int bar, unsigned char* smem, float* red) {
  constexpr int RPW = 32 / LPR;
  using Raw = Raw4<TI>;
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const bool is_v = (job & 1) != 0;
  const int slot = (job >> 1) / p.Hkv, h = (job >> 1) - slot * p.Hkv;
  const int b = c8_find(p.row_start, p.B, p.rows, 1, p.block, 2, slot);
  const int j = slot - c8_key(p.row_start, b, p.rows, 1, p.block, 2);
  const C8Seq s = c8_seq(p.row_start, p.len, b, p.rows);
  if (j < 0) return;  // offsets that do not ascend
  const int64_t pg = (int64_t)(s.len / p.block) + j;
  const int o0 = j == 0 ? s.len % p.block : 0;
  const int64_t done = pg * p.block + o0 - s.len;  // the request's new rows before this block's
  if (done >= s.T) return;
  const int r0 = s.start + (int)done, m = min(p.block - o0, s.T - (int)done);
  int page = -1;
  if (pg < p.max_blocks) page = p.table[(int64_t)b * p.max_blocks + pg];
  if (page < 0 || page >= p.pages) {
    if (p.status && lane == 0 && w == 0) atomicOr(p.status, 1);
    return;
  }
  const int64_t blk = (int64_t)page * p.Hkv + h;
  float* scale = (is_v ? p.vscale : p.kscale) + blk;
  uint8_t* codes = (is_v ? p.v8 : p.k8) + blk * p.block * p.d;
  const bool turns = !is_v && 8 * l < p.q.rot;
  const int ja = HALF && turns ? 4 * l : 8 * l, jb = HALF && turns ? (p.q.rot >> 1) + 4 * l : 8 * l + 4;
  const TI* src = static_cast<const TI*>(is_v ? p.v : p.k) + (int64_t)r0 * (is_v ? p.vs : p.ks) + (int64_t)h * p.d;
  const int64_t step = is_v ? p.vs : p.ks;
  const int per = p.warps * RPW, passes = (m + per - 1) / per;  // rows of a pass
  const int first = w * RPW + sub;
  // this lane's slots: 32 bytes a pass, the row as it comes and then as fp32
  unsigned char* mine = smem + threadIdx.x * 16;
  auto at = [&](int pass, int half) { return reinterpret_cast<float4*>(mine + (pass * 2 + half) * (kNrThreads * 16)); };
#pragma unroll
  for (int i = 0; i < kApPass; ++i) {
    const int r = i * per + first;
    if (r < m) {
      nr_copy<(int)sizeof(Raw)>(at(i, 0), src + r * step + ja);
      nr_copy<(int)sizeof(Raw)>(at(i, 1), src + r * step + jb);
    }
  }
  asm volatile("cp.async.commit_group;\n" ::: "memory");
  const float old = o0 > 0 ? *scale : 0.f;
  const float inv_d = 1.f / (float)p.d;
  auto row = [&](int i, float (&z)[8]) {  // row of pass i; zeros past the last
    const int r = i * per + first;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < m) {
      Raw a, c;
      if (i < kApPass) {
        a = *reinterpret_cast<const Raw*>(at(i, 0));
        c = *reinterpret_cast<const Raw*>(at(i, 1));
      } else {
        a = *reinterpret_cast<const Raw*>(src + r * step + ja);
        c = *reinterpret_cast<const Raw*>(src + r * step + jb);
      }
      widen4<TI>(a, x);
      widen4<TI>(c, x + 4);
    }
    if (is_v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = x[e];
    } else {
      float cs[4], sn[4];
      turn_angles(r < m ? (uint64_t)(int64_t)p.q.pos[r0 + r] : 0, p.q.freq, l, turns, cs, sn);
      const TurnFactors f = turn_factors<TI, HALF>(static_cast<const TI*>(p.wk), true, ja, jb, cs, sn);
      turn_row<LPR, HALF, NORM>(x, f, turns, inv_d, p.q.eps, z);
    }
  };
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  float top = 0.f;  // infinite where a value is not finite
#pragma unroll 1
  for (int i = 0; i < passes; ++i) {
    float z[8];
    row(i, z);
    if (i < kApPass) {
      *at(i, 0) = make_float4(z[0], z[1], z[2], z[3]);
      *at(i, 1) = make_float4(z[4], z[5], z[6], z[7]);
    }
    if (i * per + first < m) {
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(z[e]) <= 3.4028234e38f ? fabsf(z[e]) : INFINITY);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  if (p.warps > 1) {
    if (lane == 0) red[w] = top;
    asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "r"(32 * p.warps) : "memory");
    for (int i = 0; i < p.warps; ++i) top = fmaxf(top, red[i]);
  }
  float now = scale_of(top);
  if (o0 > 0 && old > now) now = old;
  const bool bad = top == INFINITY || old != old;
  if (o0 > 0 && !bad && now > old) {  // the tokens that are there, rounded again
    uint4* held = reinterpret_cast<uint4*>(codes);
    const float f = old / now;
    for (int i = w * 32 + lane; i < o0 * p.d / 16; i += 32 * p.warps) {
      uint4 c = held[i];
      c.x = again8(c.x, f);
      c.y = again8(c.y, f);
      c.z = again8(c.z, f);
      c.w = again8(c.w, f);
      held[i] = c;
    }
  }
  if (w == 0 && lane == 0) *scale = bad ? __int_as_float(0x7FC00000) : now;
  const float inv = 1.f / now;
#pragma unroll 1
  for (int i = 0; i < passes; ++i) {
    float z[8];
    if (i < kApPass) {
      *reinterpret_cast<float4*>(z) = *at(i, 0);
      *reinterpret_cast<float4*>(z + 4) = *at(i, 1);
    } else {
      row(i, z);
    }
    const int r = i * per + first;
    if (r < m) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = z[e] == z[e] ? z[e] * inv : 0.f;  // codes are numbers whatever comes
      uint8_t* to = codes + (int64_t)(o0 + r) * p.d;
      *reinterpret_cast<uint32_t*>(to + ja) = pack8(z[0], z[1], z[2], z[3]);
      *reinterpret_cast<uint32_t*>(to + jb) = pack8(z[4], z[5], z[6], z[7]);
    }
  }
}

template <typename TI, int LPR, bool HALF, bool NORM>
__global__ void __launch_bounds__(kNrThreads, 3) append_kernel(const AppendParams p) {
  __shared__ __align__(16) unsigned char smem[kApPass * 32 * kNrThreads];
  __shared__ float red[kNrThreads / 32];
  static_assert(kNrAhead<TI> * kNrThreads * sizeof(NrSlot<TI>) <= sizeof(smem), "the rows of q use the same place");
  if ((int)blockIdx.x < p.kv_ctas) {
    const int warp = threadIdx.x >> 5, group = warp / p.warps;
    const int job = blockIdx.x * (kNrThreads / 32 / p.warps) + group;
    if (job < p.jobs) append_job<TI, LPR, HALF, NORM>(p, job, warp - group * p.warps, 1 + group, smem, red + group * p.warps);
  } else {
    const int64_t live = c8_row(p.row_start, p.B, p.rows);
    norm_rope_rows<TI, TI, LPR, HALF, NORM>(p.q, (int64_t)blockIdx.x - p.kv_ctas, live,
                                            reinterpret_cast<NrSlot<TI>(*)[kNrThreads]>(smem));
  }
}

template <typename TI, int LPR>
cudaError_t run_append(const AppendParams& p, int grid, bool norm, cudaStream_t st) {
  const bool half = p.q.style == TQ_ROPE_HALF;
  if (half && norm)
    append_kernel<TI, LPR, true, true><<<grid, kNrThreads, 0, st>>>(p);
  else if (half)
    append_kernel<TI, LPR, true, false><<<grid, kNrThreads, 0, st>>>(p);
  else if (norm)
    append_kernel<TI, LPR, false, true><<<grid, kNrThreads, 0, st>>>(p);
  else
    append_kernel<TI, LPR, false, false><<<grid, kNrThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename TI>
cudaError_t run_append_d(const AppendParams& p, int grid, bool norm, cudaStream_t st) {
  return p.d == 64 ? run_append<TI, 8>(p, grid, norm, st) : run_append<TI, 16>(p, grid, norm, st);
}

}  // namespace

tq_status launch_cache8_append(const Cache8AppendArgs& a, cudaStream_t stream) {
  const tq_cache8& c = *a.cache;
  AppendParams p{};
  p.q.q = a.q;
  p.q.wq = a.wq;
  p.q.qo = a.q_out;
  p.q.freq = a.freq;
  p.q.pos = a.pos;
  p.q.N = a.rows;
  p.q.qs = a.q_stride;
  p.q.qos = a.q_out_stride;
  p.q.Hq = a.Hq;
  p.q.d = c.d;
  p.q.rot = a.rot;
  p.q.style = a.style;
  p.q.eps = a.eps;
  p.k = a.k;
  p.v = a.v;
  p.wk = a.wk;
  p.ks = a.k_stride;
  p.vs = a.v_stride;
  p.row_start = a.row_start;
  p.len = a.len;
  p.table = a.table;
  p.rows = (int)a.rows;
  p.B = a.B;
  p.Hkv = c.Hkv;
  p.max_blocks = a.max_blocks;
  p.block = c.block;
  p.d = c.d;
  p.pages = c.pages;
  p.k8 = c.d_k;
  p.v8 = c.d_v;
  p.kscale = c.d_kscale;
  p.vscale = c.d_vscale;
  p.status = c.d_status;
  const int rpw = c.d == 64 ? 4 : 2;  // rows of a warp's pass
  // four passes a block: one warp for blocks of 16 tokens of 64, eight from 64 of 128 on
  p.warps = 1;
  while (p.warps < kNrThreads / 32 && p.warps * rpw * kApPass < c.block) p.warps <<= 1;
  const int64_t jobs = (a.rows / c.block + 2 * (int64_t)a.B) * c.Hkv * 2, per = kNrThreads / 32 / p.warps;
  // q: a whole token per warp once the tokens alone fill the GPU, else as many
  // warps per token as there are trips
  int64_t qctas = 0;
  if (a.Hq > 0) {
    const int64_t fill = (int64_t)num_sms() * 32;
    const int trips = (a.Hq + rpw - 1) / rpw;
    const int64_t n = std::max<int64_t>(1, std::min<int64_t>((fill + a.rows - 1) / a.rows, trips));
    p.q.chunk = (int)((trips + n - 1) / n) * rpw;
    p.q.chunks = (a.Hq + p.q.chunk - 1) / p.q.chunk;
    qctas = (a.rows * p.q.chunks + kNrThreads / 32 - 1) / (kNrThreads / 32);
  }
  const int64_t kv = (jobs + per - 1) / per;
  if (kv * per + qctas > INT32_MAX) return TQ_ERR_UNSUPPORTED;
  p.jobs = (int)jobs;
  p.kv_ctas = (int)kv;
  const int grid = (int)(kv + qctas);
  const bool norm = a.eps > 0.f;
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.dtype) {
    case TQ_F32: e = run_append_d<float>(p, grid, norm, stream); break;
    case TQ_F16: e = run_append_d<__half>(p, grid, norm, stream); break;
    case TQ_BF16: e = run_append_d<__nv_bfloat16>(p, grid, norm, stream); break;
  }
  return e == cudaSuccess ? TQ_OK : set_cuda_error(e);
}

}  // namespace tq
