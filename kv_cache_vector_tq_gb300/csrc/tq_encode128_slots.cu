// The d = 128 encoder through a slot map (tq_encode_slots): the same kernel with
// another destination rule, instantiated apart so that the plain encoder's
// instances stay what they are.  Tokens of one head sit hkv rows apart, so the
// two vectors of a PAIR block meet in one warp while hkv <= 16 and are then
// written as whole words; the others are merged with atomics.  16384 tokens of 8
// heads, fp16, b = 3, K and V: 49.8 us for 80.7 MB (1.6 TB/s, 5.3 G rows/s); 3 tokens
// of 32 requests: 15 us for both.  tq_encode takes 21.5 us for as many rows of one of
// them (24.9 here) and 114 us for a million (179 here, slots in random order): what
// is more is the way to a row's destination, which each of a row's four epilogue
// warps finds, with a load that a 64-bit division and the stores wait for (0.49
// instructions a clock and quarter against 0.56).
#include "tq_encode128_kernel.cuh"

namespace tq {

tq_status launch_encode_slots(const DevCtx& c, const void* x, int x_dtype, int64_t N, int Hkv, const int64_t* slots,
                              int block, const tq_codes* out, cudaStream_t stream) {
  if (!enc128_supported(c) || N > INT32_MAX / Hkv) return TQ_ERR_UNSUPPORTED;  // TMA row coordinates are 32-bit
  Enc128Params p = enc128_params(c, x, N * Hkv, out);
  p.slots = slots;
  p.hkv = Hkv;
  p.block = block;
  p.pages = out->n / ((int64_t)Hkv * block);
  CUtensorMap xmap;
  const tq_status ms = rows_tensor_map(&xmap, x, N * Hkv, c.d, x_dtype == TQ_F16);
  if (ms != TQ_OK) return ms;
  const bool mix = c.mode == TQ_MIXED, prod = c.mode == TQ_PROD;
  const cudaError_t e = x_dtype == TQ_F16 ? launch_mode<true, true>(p, xmap, c.b_mse, prod, mix, stream)
                                          : launch_mode<true, false>(p, xmap, c.b_mse, prod, mix, stream);
  return e == cudaSuccess ? TQ_OK : set_cuda_error(e);
}

}  // namespace tq
