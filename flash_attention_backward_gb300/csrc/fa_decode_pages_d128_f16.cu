// Single-token attention over selected pages, D = 128, f16 keys: every Dv and value type.
#include "fa_decode.cuh"

namespace fap {
FAP_INSTANTIATE_DECODE(128, FA_F16, true)
}  // namespace fap
