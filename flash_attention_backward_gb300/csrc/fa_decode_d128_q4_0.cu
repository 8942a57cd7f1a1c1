// Single-token attention, D = 128, q4_0 keys: every Dv and value type.
#include "fa_decode.cuh"

namespace fap {
FAP_INSTANTIATE_DECODE(128, FA_Q4_0)
}  // namespace fap
