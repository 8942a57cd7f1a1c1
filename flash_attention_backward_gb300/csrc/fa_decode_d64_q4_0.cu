// Single-token attention, D = 64, q4_0 keys: every Dv and value type.
#include "fa_decode.cuh"

namespace fap {
FAP_INSTANTIATE_DECODE(64, FA_Q4_0)
}  // namespace fap
