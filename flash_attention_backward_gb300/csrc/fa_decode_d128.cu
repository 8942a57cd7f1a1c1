// Single-token attention for D = 128 (every Dv): its own translation unit, so that the kernel
// instantiations compile in parallel.
#include "fa_decode.cuh"

namespace fap {
cudaError_t run_decode_d128(const DecodeArgs& a, const DecodeMaps& m, int nw, size_t smem, cudaStream_t s) {
  return pick_decode<128>(a, m, nw, smem, s);
}
}  // namespace fap
