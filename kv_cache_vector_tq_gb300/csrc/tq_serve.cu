// What a serving loop does around the packed cache, beside encode and
// attention: pages for the tokens of a step (tq_block_tables) and the norms
// and position rotation of queries and keys (tq_qk_norm_rope).
#include <algorithm>

#include <type_traits>

#include <cuda_bf16.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

// ------------------------------------------------------------------ block tables
//   need_b = ceil((len_b + new_b) / P), take_b = max(need_b - held_b, 0),
//   give_b = max(held_b - need_b, 0); request b is served iff take_b = 0 or
//   take_0 + ... + take_b <= tail - head.
// Three prefix sums over the requests (takes, gives, served tokens) place every
// page and every token row, so no CTA depends on another: each one computes the
// sums for itself (B <= 4096 entries of L2-resident input) and fills its share
// of the rows.  Rows read pages they hold from the table and new pages from the
// ring, never what another CTA writes.  Bound by launch latency and a chain of
// four dependent reads at a step's sizes (32 requests: 5.4 us a call in a graph),
// by the rows' lookups at a prompt's, which are spread over the grid (131K rows
// of 257 requests, 1.6 MB written: 7.5 us).
constexpr int kBtThreads = 512;
constexpr int kBtMaxB = 4096;
constexpr int kBtRowsPerCta = 512;  // a row a thread while two CTAs fit every SM (four rows: 8.9 us for 131K rows)

struct BlockTableParams {
  const int32_t *len, *nnew, *held, *ring_in;
  const int64_t* state;
  int32_t *ring, *table, *held_out, *row_start, *pos;
  int64_t *state_out, *slots;
  int64_t ring_size, rows;
  int B, block, max_blocks;
};

// Inclusive sums of x and y over the CTA's threads, in place; returns the totals.
__device__ __forceinline__ int2 cta_scan2(int& x, int& y, int2* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(kFull, x, o), b = __shfl_up_sync(kFull, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  __syncthreads();  // the sums of the last call have been read
  if (lane == 31) warp_sums[warp] = make_int2(x, y);
  __syncthreads();
  int2 base = make_int2(0, 0), tot = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kBtThreads / 32; ++w) {
    const int2 s = warp_sums[w];
    if (w < warp) {
      base.x += s.x;
      base.y += s.y;
    }
    tot.x += s.x;
    tot.y += s.y;
  }
  x += base.x;
  y += base.y;
  return tot;
}

__global__ void __launch_bounds__(kBtThreads) block_tables_kernel(const BlockTableParams p) {
  extern __shared__ int bt_smem[];
  int* s_start = bt_smem;             // [B] first row of request b
  int* s_first = bt_smem + p.B;       // [B] its first new page, counted from the ring's head
  __shared__ int2 warp_sums[kBtThreads / 32];
  __shared__ int s_taken, s_many;
  __shared__ int4 many[kBtThreads];  // request, pages held and needed, its first new page
  __shared__ int many_back[kBtThreads];  // its first page given back
  const int tid = threadIdx.x;
  const int64_t head = p.state[0], tail = p.state[1];
  const int64_t avail = tail > head ? tail - head : 0;
  // places in the ring: one remainder each, then offsets below the ring's size
  const int64_t head_at = head % p.ring_size, tail_at = tail % p.ring_size;
  auto place = [&](int64_t base, int64_t k) -> int64_t {  // k: fewer than the ring holds, but for broken states
    int64_t at = base + k;
    if (at >= p.ring_size) at -= p.ring_size;
    return at < p.ring_size && at >= 0 ? at : ((at % p.ring_size) + p.ring_size) % p.ring_size;
  };
  if (tid == 0) s_taken = s_many = 0;
  int take0 = 0, give0 = 0, row0 = 0;
  for (int b0 = 0; b0 < p.B; b0 += kBtThreads) {
    const int b = b0 + tid;
    int len = 0, nn = 0, held = 0, need = 0, take = 0, give = 0;
    bool ok = false;
    if (b < p.B) {
      len = p.len[b];
      nn = p.nnew[b];
      held = p.held[b];
      const int64_t all = (int64_t)len + nn, want = (all + p.block - 1) / p.block;
      ok = len >= 0 && nn >= 0 && held >= 0 && held <= p.max_blocks && want <= p.max_blocks && all <= INT32_MAX;
      need = ok ? (int)want : held;
      take = max(need - held, 0);
      give = max(held - need, 0);
    }
    int it = take, ig = give;
    const int2 tg = cta_scan2(it, ig, warp_sums);
    it += take0;
    ig += give0;
    const bool served = ok && (take == 0 || it <= avail);
    int rows = served ? nn : 0, dummy = 0;
    const int mine = rows;
    const int2 rr = cta_scan2(rows, dummy, warp_sums);
    if (b < p.B) {
      s_start[b] = row0 + rows - mine;
      s_first[b] = it - take;
      if (served && take > 0) atomicMax(&s_taken, it);
      if (blockIdx.x == 0) {
        p.held_out[b] = served ? need : held;
        p.row_start[b] = row0 + rows - mine;
      }
      if (blockIdx.x == b % gridDim.x) {
        int32_t* row = p.table + (int64_t)b * p.max_blocks;
        // few pages a request: its own thread moves them (a prompt's many are moved below)
        if (served && take <= 32)
          for (int j = 0; j < take; ++j)
            row[held + j] = p.ring_in[place(head_at, it - take + j)];
        if (served && give <= 32)
          for (int j = 0; j < give; ++j) {
            const int64_t k = (int64_t)(ig - give) + j;
            if (tail + k < head + p.ring_size) p.ring[place(tail_at, k)] = row[need + j];
          }
      }
    }
    // requests that take or give many pages (a prompt comes, a request ends): the
    // whole CTA moves them, one after the other
    if (b < p.B && served && (take > 32 || give > 32) && blockIdx.x == b % gridDim.x) {
      const int k = atomicAdd(&s_many, 1);
      many[k] = make_int4(b, held, need, it - take);
      many_back[k] = ig - give;
    }
    __syncthreads();
    for (int k = 0; k < s_many; ++k) {
      const int4 m = many[k];
      int32_t* row = p.table + (int64_t)m.x * p.max_blocks;
      for (int j = tid; j < m.z - m.y; j += kBtThreads) row[m.y + j] = p.ring_in[place(head_at, m.w + j)];
      for (int j = tid; j < m.y - m.z; j += kBtThreads) {
        const int64_t g = (int64_t)many_back[k] + j;
        if (tail + g < head + p.ring_size) p.ring[place(tail_at, g)] = row[m.z + j];
      }
    }
    __syncthreads();
    if (tid == 0) s_many = 0;
    take0 += tg.x;
    give0 += tg.y;
    row0 += rr.x;
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    p.row_start[p.B] = row0;
    p.state_out[0] = head + s_taken;
    p.state_out[1] = tail + give0;
  }
  for (int64_t r = (int64_t)blockIdx.x * kBtThreads + tid; r < p.rows; r += (int64_t)gridDim.x * kBtThreads) {
    int64_t slot = -1;
    int pos = 0;
    if (r < row0) {
      int lo = 0, hi = p.B - 1;  // last request whose first row is <= r (requests without rows come before it)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_start[mid] <= r)
          lo = mid;
        else
          hi = mid - 1;
      }
      pos = p.len[lo] + (int)(r - s_start[lo]);
      const int j = pos / p.block, held = p.held[lo];
      const int32_t page = j < held ? p.table[(int64_t)lo * p.max_blocks + j]
                                          : p.ring_in[place(head_at, s_first[lo] + (j - held))];
      slot = page >= 0 ? (int64_t)page * p.block + pos % p.block : -1;
    }
    p.slots[r] = slot;
    p.pos[r] = pos;
  }
}

// ------------------------------------------------------------------ norms and rotation
//   y = x · w / sqrt(mean(x²) + eps);  pairs (a, b) of y turn by the angle
//   pos·f_j:  (a cos - b sin, b cos + a sin).
// Angles: f_j as a 64-bit fraction of a turn, so that pos·f_j modulo one turn
// is one 64-bit integer product, right to 2^-64 of a turn per position (a
// 32-bit angle is off by whole degrees past 10^6 positions), so to 2^-32 half
// turns at any int32 position.  The fraction's leading 32 bits, as a signed
// multiple of half a turn, go to sincospif; the rest is below 2^-31 half turns and
// their rounding to fp32 at most 2^-25.
// One pass: a row is d/8 lanes of 8 elements, its sum of squares a shuffle tree in
// fp32.  With the half-split pairing a lane holds 4 elements and their 4 partners,
// so no value changes lanes; cosines and sines are multiplied by the weights once
// per token, so that a lane's 8 elements take 32 multiply-adds in all.
// Prompts are bound by HBM (16384 tokens of 40 heads of 128, bf16 to fp16,
// 335.6 MB: 62 us, 5.4 TB/s, 80% of the measured copy; with partners exchanged by
// shuffles it was instructions, 76 us); a token (3.0 us) or a tree of 509 (6.8 us)
// is one launch's latency.
constexpr int kNrThreads = 256;

struct NormRopeParams {
  const void *q, *k, *wq, *wk;
  void *qo, *ko;
  const uint64_t* freq;
  const int32_t* pos;
  int64_t N, qs, ks, qos, kos;  // strides between tokens in elements
  int Hq, Hkv, d, rot, style;
  int chunk, chunks;  // heads per warp, warps per token
  float eps;
};

// Four elements as they lie in memory, and as fp32.
template <typename T>
using Raw4 = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;

template <typename T>
__device__ __forceinline__ void widen4(const Raw4<T>& r, float* v) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  } else {
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 f;
      if constexpr (std::is_same<T, __half>::value)
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else
        f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        w[i] = h2_bits(__floats2half2_rn(v[2 * i], v[2 * i + 1]));
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// LPR lanes per row (the power of two at or above d/8).  Rows come by asynchronous
// copies into slots of shared memory that are each lane's own (no barrier),
// kNrAhead lane groups of rows ahead of the one in use: 32 warps with eight times
// 512 bytes each cover the memory's latency several times over.
template <typename TI>
constexpr int kNrAhead = sizeof(TI) == 4 ? 4 : 8;

template <int BYTES>
__device__ __forceinline__ void nr_copy(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}

template <typename TI, typename TO, int LPR, bool HALF>
__global__ void __launch_bounds__(kNrThreads, 4) norm_rope_kernel(const NormRopeParams p) {
  constexpr int RPW = 32 / LPR, A = kNrAhead<TI>;
  using Raw = Raw4<TI>;
  struct Slot {
    Raw a, b;
  };
  __shared__ __align__(16) Slot ring[A][kNrThreads];
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const int64_t job = (int64_t)blockIdx.x * (kNrThreads / 32) + (threadIdx.x >> 5);
  if (job >= p.N * p.chunks) return;  // whole warps
  int64_t n = job;
  int h0 = 0;
  if (p.chunks > 1) {
    n = job <= 0xFFFFFFFFll ? (int64_t)((uint32_t)job / (uint32_t)p.chunks) : job / p.chunks;
    h0 = (int)(job - n * p.chunks) * p.chunk;
  }
  const int h1 = min(h0 + p.chunk, p.Hq + p.Hkv);
  const bool in = 8 * l < p.d, turns = 8 * l < p.rot;
  // this lane's elements: ja.., jb.. (four each); half-split: partners of one another
  const int ja = HALF && turns ? 4 * l : 8 * l, jb = HALF && turns ? (p.rot >> 1) + 4 * l : 8 * l + 4;
  const TI* qrow = static_cast<const TI*>(p.q) + n * p.qs;
  const TI* krow = static_cast<const TI*>(p.k) + n * p.ks;
  auto fetch = [&](int h, int slot) {  // this lane's piece of head h
    if (in && h < h1) {
      const TI* src = h < p.Hq ? qrow + (int64_t)h * p.d : krow + (int64_t)(h - p.Hq) * p.d;
      Slot& s = ring[slot][threadIdx.x];
      nr_copy<(int)sizeof(Raw)>(&s.a, src + ja);
      nr_copy<(int)sizeof(Raw)>(&s.b, src + jb);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");  // always, so that the groups count the heads
  };
#pragma unroll
  for (int a = 0; a < A; ++a) fetch(h0 + a * RPW + sub, a);
  // cosines and sines of the lane's four pairs
  float cs[4], sn[4];
  const uint64_t pos = (uint64_t)(int64_t)p.pos[n];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (turns) {
      const uint64_t t = pos * p.freq[4 * l + e];
      sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f /* 2^-31 */, &sn[e], &cs[e]);
    }
  }
  const float inv_d = 1.f / (float)p.d;
  // z_a = r·(x_a·ca - x_b·sb), z_b = r·(x_b·cb + x_a·sa) with the weights inside
  float ca[4], sa[4], cb[4], sb[4];
  int of = -1;  // whose weights they hold: 1 q, 0 k

  int slot = 0;
#pragma unroll 1
  for (int hb = h0; hb < h1; hb += RPW) {
    const int h = hb + sub;
    const bool isq = h < p.Hq;
    if (of != (int)isq) {
      of = isq;
      const TI* w = static_cast<const TI*>(isq ? p.wq : p.wk);
      float wv[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (in && w) {
        widen4<TI>(*reinterpret_cast<const Raw*>(w + ja), wv);
        widen4<TI>(*reinterpret_cast<const Raw*>(w + jb), wv + 4);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float wa = HALF ? wv[e] : wv[2 * e], wb = HALF ? wv[4 + e] : wv[2 * e + 1];
        ca[e] = wa * cs[e];
        sa[e] = wa * sn[e];
        cb[e] = wb * cs[e];
        sb[e] = wb * sn[e];
      }
    }
    asm volatile("cp.async.wait_group %0;\n" ::"n"(A - 1) : "memory");
    float x[8];
    {
      Slot s{};
      if (in && h < h1) s = ring[slot][threadIdx.x];
      widen4<TI>(s.a, x);
      widen4<TI>(s.b, x + 4);
    }
    fetch(h + A * RPW, slot);  // the slot's words are in registers
    if (++slot == A) slot = 0;
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    float r = rsqrtf(fmaf(ss, inv_d, p.eps));
    if (__any_sync(kFull, !(ss < 1e36f))) {
      // squares past the fp32 range (or not numbers): once more with the row
      // scaled by the power of two that brings its largest magnitude to [1, 2)
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
      for (int o = LPR / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      int ex = 1;
      if (m > 0.f && m < INFINITY) frexpf(m, &ex);
      const float sc = ldexpf(1.f, 1 - ex);
      float s2 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s2 = fmaf(x[e] * sc, x[e] * sc, s2);
#pragma unroll
      for (int o = LPR / 2; o; o >>= 1) s2 += __shfl_xor_sync(kFull, s2, o);
      if (!(ss < 1e36f)) {  // x·r without the large x meeting the weights first
        r = rsqrtf(fmaf(s2, inv_d, p.eps * sc * sc)) * sc;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= r;
        r = 1.f;
      }
    }
    float z[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = HALF ? e : 2 * e, k = HALF ? 4 + e : 2 * e + 1;
      // a lane past `rot` has sines 0, and no product with them
      const float a = turns ? fmaf(x[i], ca[e], -x[k] * sb[e]) : x[i] * ca[e];
      const float b = turns ? fmaf(x[k], cb[e], x[i] * sa[e]) : x[k] * cb[e];
      z[i] = a * r;
      z[k] = b * r;
    }
    if (in && h < h1) {
      TO* dst = isq ? static_cast<TO*>(p.qo) + n * p.qos + (int64_t)h * p.d
                    : static_cast<TO*>(p.ko) + n * p.kos + (int64_t)(h - p.Hq) * p.d;
      store4(dst + ja, z);
      store4(dst + jb, z + 4);
    }
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");
}

template <typename TI, typename TO>
cudaError_t run_norm_rope(NormRopeParams p, cudaStream_t st) {
  int lpr = 4;
  while (8 * lpr < p.d) lpr <<= 1;
  const int heads = p.Hq + p.Hkv, rows_per_trip = 32 / lpr;
  // a whole token per warp once the tokens alone fill the GPU (its sines are
  // then computed once); else as many warps per token as there are trips
  const int64_t fill = (int64_t)num_sms() * 32;
  int64_t per = (fill + p.N - 1) / p.N;
  const int trips = (heads + rows_per_trip - 1) / rows_per_trip;
  per = std::max<int64_t>(1, std::min<int64_t>(per, trips));
  p.chunk = (int)((trips + per - 1) / per) * rows_per_trip;
  p.chunks = (heads + p.chunk - 1) / p.chunk;
  const int64_t jobs = p.N * p.chunks, grid = (jobs + kNrThreads / 32 - 1) / (kNrThreads / 32);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  switch (lpr) {
    case 4:
      if (p.style == TQ_ROPE_HALF)
        norm_rope_kernel<TI, TO, 4, true><<<(int)grid, kNrThreads, 0, st>>>(p);
      else
        norm_rope_kernel<TI, TO, 4, false><<<(int)grid, kNrThreads, 0, st>>>(p);
      break;
    case 8:
      if (p.style == TQ_ROPE_HALF)
        norm_rope_kernel<TI, TO, 8, true><<<(int)grid, kNrThreads, 0, st>>>(p);
      else
        norm_rope_kernel<TI, TO, 8, false><<<(int)grid, kNrThreads, 0, st>>>(p);
      break;
    case 16:
      if (p.style == TQ_ROPE_HALF)
        norm_rope_kernel<TI, TO, 16, true><<<(int)grid, kNrThreads, 0, st>>>(p);
      else
        norm_rope_kernel<TI, TO, 16, false><<<(int)grid, kNrThreads, 0, st>>>(p);
      break;
    case 32:
      if (p.style == TQ_ROPE_HALF)
        norm_rope_kernel<TI, TO, 32, true><<<(int)grid, kNrThreads, 0, st>>>(p);
      else
        norm_rope_kernel<TI, TO, 32, false><<<(int)grid, kNrThreads, 0, st>>>(p);
      break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <typename TI>
cudaError_t run_norm_rope_o(const NormRopeParams& p, int out_dtype, cudaStream_t st) {
  switch (out_dtype) {
    case TQ_F32: return run_norm_rope<TI, float>(p, st);
    case TQ_F16: return run_norm_rope<TI, __half>(p, st);
    case TQ_BF16: return run_norm_rope<TI, __nv_bfloat16>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int block_tables_max_batch() { return kBtMaxB; }

tq_status launch_block_tables(const int32_t* len, const int32_t* nnew, const int32_t* held, int B, int block,
                              int32_t* ring, int64_t ring_size, const int64_t* state, int32_t* table, int max_blocks,
                              int32_t* held_out, int64_t* state_out, int32_t* row_start, int64_t* slots, int32_t* pos,
                              int64_t rows, cudaStream_t stream) {
  BlockTableParams p;
  p.len = len;
  p.nnew = nnew;
  p.held = held;
  p.ring_in = ring;
  p.ring = ring;
  p.state = state;
  p.table = table;
  p.held_out = held_out;
  p.row_start = row_start;
  p.pos = pos;
  p.state_out = state_out;
  p.slots = slots;
  p.ring_size = ring_size;
  p.rows = rows;
  p.B = B;
  p.block = block;
  p.max_blocks = max_blocks;
  const int64_t ctas = std::max<int64_t>((rows + kBtRowsPerCta - 1) / kBtRowsPerCta, (B + 63) / 64);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(ctas, 2 * (int64_t)num_sms()));
  block_tables_kernel<<<grid, kBtThreads, 2 * B * (int)sizeof(int), stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TQ_OK : set_cuda_error(e);
}

tq_status launch_norm_rope(const void* q, const void* k, int in_dtype, int64_t N, int Hq, int Hkv, int d, int64_t qs,
                           int64_t ks, const void* wq, const void* wk, float eps, const uint64_t* freq, int rot,
                           int style, const int32_t* pos, void* qo, void* ko, int out_dtype, int64_t qos, int64_t kos,
                           cudaStream_t stream) {
  NormRopeParams p;
  p.q = q;
  p.k = k;
  p.wq = wq;
  p.wk = wk;
  p.qo = qo;
  p.ko = ko;
  p.freq = freq;
  p.pos = pos;
  p.N = N;
  p.qs = qs;
  p.ks = ks;
  p.qos = qos;
  p.kos = kos;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  p.rot = rot;
  p.style = style;
  p.eps = eps;
  cudaError_t e = cudaErrorInvalidValue;
  switch (in_dtype) {
    case TQ_F32: e = run_norm_rope_o<float>(p, out_dtype, stream); break;
    case TQ_F16: e = run_norm_rope_o<__half>(p, out_dtype, stream); break;
    case TQ_BF16: e = run_norm_rope_o<__nv_bfloat16>(p, out_dtype, stream); break;
  }
  return e == cudaSuccess ? TQ_OK : set_cuda_error(e);
}

}  // namespace tq
