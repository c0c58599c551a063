// The d = 128 encoder into consecutive vectors (tq_encode).
#include "tq_encode128_kernel.cuh"

namespace tq {

bool enc128_supported(const DevCtx& c) {
  // symmetric codebooks only (tq_codebook_build makes them; the bucketize
  // compares |v| with the positive thresholds); others take the general encoder
  return c.d == kDim && c.enc_tab != nullptr && (c.mode != TQ_PROD || c.enc_tab_m != nullptr) &&
         c.b_mse >= 1 && c.b_mse <= (c.mode == TQ_MSE ? 4 : 3) && c.sym_thr != 0;
}

tq_status launch_encode128(const DevCtx& c, const void* x, int x_dtype, int64_t N, const tq_codes* out,
                           int64_t offset, int64_t group_rows, int64_t group_stride, cudaStream_t stream) {
  if (!enc128_supported(c)) return TQ_ERR_UNSUPPORTED;
  if (N > INT32_MAX) return TQ_ERR_UNSUPPORTED;  // TMA row coordinates are 32-bit
  Enc128Params p = enc128_params(c, x, N, out);
  const bool mix = c.mode == TQ_MIXED;
  p.offset = offset;
  p.group_rows = group_rows;
  p.group_stride = group_stride;
  p.pair_aligned = (offset % 2 == 0) && (group_rows % 2 == 0 || group_rows >= N) && (group_stride % 2 == 0);
  CUtensorMap xmap;
  const tq_status ms = rows_tensor_map(&xmap, x, N, c.d, x_dtype == TQ_F16);
  if (ms != TQ_OK) return ms;
  const cudaError_t e = x_dtype == TQ_F16 ? launch_mode<false, true>(p, xmap, c.b_mse, c.mode == TQ_PROD, mix, stream)
                                          : launch_mode<false, false>(p, xmap, c.b_mse, c.mode == TQ_PROD, mix, stream);
  return e == cudaSuccess ? TQ_OK : set_cuda_error(e);
}

}  // namespace tq
