// Single-token attention, D = 128, f32 keys: every Dv and value type.
#include "fa_decode.cuh"

namespace fap {
FAP_INSTANTIATE_DECODE(128, FA_F32)
}  // namespace fap
