// New tokens into the 8-bit paged cache (tq_cache8_append): norms and position
// rotation of q and k on the way, one launch.
//
//   q_out = turn(norm(q));  per page, KV head and side, with a the largest
//   magnitude among the new rows of the block:
//   s' = 2^e, the least with a <= 448·2^e, and no less than the block's scale s
//   where it holds earlier tokens; codes of those: e4m3(code·s / s'), new ones:
//   e4m3(x / s').
//
// A job is the new rows of one block, one side and some KV heads, one after the
// other: angles, once for a token, stay in shared memory for all of them.  Rows come
// by asynchronous copies, a slot of shared memory for every lane and pass (no barrier),
// the next head's while this one's are scaled and stored; normed and turned they wait
// in registers until the job's warps have agreed on the scale.  A job has a warp for
// every two rows of a pass, four passes a block, so that a block of any size has as
// many bytes in flight for each warp; further passes read their rows twice (from L2).
// Jobs need no sum over the requests: request b's are numbered from row_start[b] /
// block + 2b on.
// The CTAs behind the jobs turn q as tq_qk_norm_rope does.
// Measured: prompt of 16384, 32 + 8 heads of 128, bf16, norms: 85 us, 4.3 TB/s (k and v
// 45 us, bound by the issue of 34 M warp instructions; q 40 us, by its 268 MB); 32
// requests of up to 5 tokens 5.9 us, one token 4.0 us (latency).  80 registers a thread for
// three CTAs an SM; with norms 44 to 72 bytes of them spill.
#include <algorithm>
#include <cmath>

#include "tq_cache8.cuh"
#include "tq_rows.cuh"

namespace tq {

namespace {

constexpr int kApPass = 4;  // passes whose rows stay in registers

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
  int jobs, warps, heads, groups;  // jobs in all, warps of a job, its heads, jobs of a block and side
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

// Shared memory of a CTA: the rows as they come, the angles (float4 cosines, sines).
template <typename TI>
constexpr int kApRaw = kApPass * kNrThreads * (int)sizeof(NrSlot<TI>);
constexpr int kApTrig = kApPass * kNrThreads * 32;

template <typename TI, int LPR, bool HALF, bool NORM, bool V>
__device__ __forceinline__ void append_job(const AppendParams& p, int slot, int h0, int h1, int w, int bar, unsigned char* smem,
                                           uint32_t (*red)[kNrThreads / 32], int red0) {
  constexpr int RPW = 32 / LPR;
  using Raw = Raw4<TI>;
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
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
  const bool turns = !V && 8 * l < p.q.rot;
  const int ja = HALF && turns ? 4 * l : 8 * l, jb = HALF && turns ? (p.q.rot >> 1) + 4 * l : 8 * l + 4;
  const int64_t step = V ? p.vs : p.ks;
  const TI* src = static_cast<const TI*>(V ? p.v : p.k) + (int64_t)r0 * step;
  const int per = p.warps * RPW, first = w * RPW + sub;  // rows of a pass, this lane's of the first
  NrSlot<TI>* mine = reinterpret_cast<NrSlot<TI>*>(smem) + threadIdx.x;
  float4* trig = reinterpret_cast<float4*>(smem + kApRaw<TI>) + threadIdx.x;
  auto fetch = [&](int h) {
    const TI* from = src + (int64_t)h * p.d;
#pragma unroll
    for (int i = 0; i < kApPass; ++i) {
      const int r = i * per + first;
      if (r < m) {
        nr_copy<(int)sizeof(Raw)>(&mine[i * kNrThreads].a, from + r * step + ja);
        nr_copy<(int)sizeof(Raw)>(&mine[i * kNrThreads].b, from + r * step + jb);
      }
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  fetch(h0);
  if (!V) {
#pragma unroll 1
    for (int i = 0; i < kApPass && i * per < m; ++i) {
      const int r = i * per + first;
      float cs[4], sn[4];
      turn_angles(r < m ? (uint64_t)(int64_t)p.q.pos[r0 + r] : 0, p.q.freq, l, turns, cs, sn);
      trig[2 * i * kNrThreads] = make_float4(cs[0], cs[1], cs[2], cs[3]);
      trig[(2 * i + 1) * kNrThreads] = make_float4(sn[0], sn[1], sn[2], sn[3]);
    }
  }
  const float inv_d = 1.f / (float)p.d;
  // one row: x as it came, z as it is stored but for the scale
  auto row = [&](float (&x)[8], const float (&cs)[4], const float (&sn)[4], float (&z)[8]) {
    const TurnFactors f = turn_factors<TI, HALF>(static_cast<const TI*>(p.wk), true, ja, jb, cs, sn);
    turn_row<LPR, HALF, NORM>(x, f, turns, inv_d, p.q.eps, z);
  };
  auto far_row = [&](int h, int i, float (&z)[8]) {  // of a pass whose rows are not kept
    const int r = i * per + first;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < m) {
      widen4<TI>(*reinterpret_cast<const Raw*>(src + (int64_t)h * p.d + r * step + ja), x);
      widen4<TI>(*reinterpret_cast<const Raw*>(src + (int64_t)h * p.d + r * step + jb), x + 4);
    }
    if constexpr (V) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = x[e];
    } else {
      float cs[4], sn[4];
      turn_angles(r < m ? (uint64_t)(int64_t)p.q.pos[r0 + r] : 0, p.q.freq, l, turns, cs, sn);
      row(x, cs, sn, z);
    }
  };
  auto top_of = [](uint32_t top, const float (&z)[8]) -> uint32_t {  // magnitudes' bits in order, what is not finite above all
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(z[e]) & 0x7FFFFFFFu);
    return top;
  };
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const int64_t blk = (int64_t)page * p.Hkv + h;
    float* scale = (V ? p.vscale : p.kscale) + blk;
    uint8_t* codes = (V ? p.v8 : p.k8) + blk * p.block * p.d;
    const float old = o0 > 0 ? *scale : 0.f;
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    float z[kApPass][8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kApPass; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] = 0.f;
      if (i * per < m) {
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (i * per + first < m) {
          const NrSlot<TI> raw = mine[i * kNrThreads];
          widen4<TI>(raw.a, x);
          widen4<TI>(raw.b, x + 4);
        }
        if constexpr (V) {
#pragma unroll
          for (int e = 0; e < 8; ++e) z[i][e] = x[e];
        } else {
          const float4 c = trig[2 * i * kNrThreads], n = trig[(2 * i + 1) * kNrThreads];
          const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {n.x, n.y, n.z, n.w};
          row(x, cs, sn, z[i]);
        }
        if (i * per + first < m) top = top_of(top, z[i]);
      }
    }
#pragma unroll 1
    for (int i = kApPass; i * per < m; ++i) {
      float y[8];
      far_row(h, i, y);
      if (i * per + first < m) top = top_of(top, y);
    }
    if (h + 1 < h1) fetch(h + 1);  // the slots have been read
#pragma unroll
    for (int o = 16; o; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    if (p.warps > 1) {
      uint32_t* mx = red[h & 1] + red0;  // (the other half while a slow warp still reads the head before)
      if (lane == 0) mx[w] = top;
      asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "r"(32 * p.warps) : "memory");
      for (int i = 0; i < p.warps; ++i) top = max(top, mx[i]);
    } else {
      __syncwarp();  // every lane has the scale as it was
    }
    float now = scale_of(__uint_as_float(top));
    if (o0 > 0 && old > now) now = old;
    const bool bad = top >= 0x7F800000u || old != old;
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
    uint8_t* to = codes + (o0 + first) * p.d;
    auto store = [&](int i, float (&y)[8]) {
      if (bad) {  // codes are numbers whatever comes
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] == y[e] ? y[e] : 0.f;
      }
      const uint32_t ca = pack8(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
      const uint32_t cb = pack8(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
      if (i * per + first < m) {
        if (V || !HALF) {
          *reinterpret_cast<uint2*>(to + i * per * p.d + ja) = make_uint2(ca, cb);
        } else {
          *reinterpret_cast<uint32_t*>(to + i * per * p.d + ja) = ca;
          *reinterpret_cast<uint32_t*>(to + i * per * p.d + jb) = cb;
        }
      }
    };
#pragma unroll
    for (int i = 0; i < kApPass; ++i)
      if (i * per < m) store(i, z[i]);
#pragma unroll 1
    for (int i = kApPass; i * per < m; ++i) {
      float y[8];
      far_row(h, i, y);
      store(i, y);
    }
  }
}

template <typename TI, int LPR, bool HALF, bool NORM>
__global__ void __launch_bounds__(kNrThreads, 3) append_kernel(const AppendParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint32_t red[2][kNrThreads / 32];
  static_assert(kNrAhead<TI> * kNrThreads * sizeof(NrSlot<TI>) <= kApRaw<TI> + kApTrig, "the rows of q use the same place");
  if ((int)blockIdx.x < p.kv_ctas) {
    const int warp = threadIdx.x >> 5, group = warp / p.warps, w = warp - group * p.warps;
    const int job = blockIdx.x * (kNrThreads / 32 / p.warps) + group;
    if (job >= p.jobs) return;
    // K and V in turn
    const int slot = (job >> 1) / p.groups, h0 = ((job >> 1) - slot * p.groups) * p.heads, h1 = min(h0 + p.heads, p.Hkv);
    if (job & 1)
      append_job<TI, LPR, HALF, NORM, true>(p, slot, h0, h1, w, 1 + group, smem, red, group * p.warps);
    else
      append_job<TI, LPR, HALF, NORM, false>(p, slot, h0, h1, w, 1 + group, smem, red, group * p.warps);
  } else {
    const int64_t live = c8_row(p.row_start, p.B, p.rows);
    norm_rope_rows<TI, TI, LPR, HALF, NORM>(p.q, (int64_t)blockIdx.x - p.kv_ctas, live,
                                            reinterpret_cast<NrSlot<TI>(*)[kNrThreads]>(smem));
  }
}

template <typename TI, int LPR, bool HALF, bool NORM>
cudaError_t run_append_k(const AppendParams& p, int grid, cudaStream_t st) {
  static PerDeviceValue attr;
  constexpr int bytes = kApRaw<TI> + kApTrig;
  const cudaError_t e = smem_attr_once(attr, (const void*)append_kernel<TI, LPR, HALF, NORM>, bytes);
  if (e != cudaSuccess) return e;
  append_kernel<TI, LPR, HALF, NORM><<<grid, kNrThreads, bytes, st>>>(p);
  return cudaGetLastError();
}

template <typename TI, int LPR>
cudaError_t run_append(const AppendParams& p, int grid, bool norm, cudaStream_t st) {
  const bool half = p.q.style == TQ_ROPE_HALF;
  if (half) return norm ? run_append_k<TI, LPR, true, true>(p, grid, st) : run_append_k<TI, LPR, true, false>(p, grid, st);
  return norm ? run_append_k<TI, LPR, false, true>(p, grid, st) : run_append_k<TI, LPR, false, false>(p, grid, st);
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
  const int64_t slots = a.rows / c.block + 2 * (int64_t)a.B, per = kNrThreads / 32 / p.warps;
  // all heads of a block to a job while there are two CTAs an SM of such jobs with work
  // (half of the slots of many short requests have none), else fewer
  p.heads = c.Hkv;
  while (p.heads > 1 && (a.rows + c.block - 1) / c.block * ((c.Hkv + p.heads - 1) / p.heads) * 2 < 2 * num_sms() * per)
    p.heads = (p.heads + 1) / 2;
  p.groups = (c.Hkv + p.heads - 1) / p.heads;
  const int64_t jobs = slots * p.groups * 2;
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
