// Single-token attention, D = 64, f32 keys: every Dv and value type.
#include "fa_decode.cuh"

namespace fap {
FAP_INSTANTIATE_DECODE(64, FA_F32)
}  // namespace fap
