// What a serving loop does around the packed cache, beside encode and
// attention: pages for the tokens of a step (tq_block_tables) and the norms
// and position rotation of queries and keys (tq_qk_norm_rope).
#include <algorithm>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_rows.cuh"

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
template <typename TI, typename TO, int LPR, bool HALF>
__global__ void __launch_bounds__(kNrThreads, 4) norm_rope_kernel(const NormRopeParams p) {
  __shared__ __align__(16) NrSlot<TI> ring[kNrAhead<TI>][kNrThreads];
  norm_rope_rows<TI, TO, LPR, HALF, true>(p, blockIdx.x, p.N, ring);
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
