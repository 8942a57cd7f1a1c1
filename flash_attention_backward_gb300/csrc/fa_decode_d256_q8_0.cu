// Single-token attention, D = 256, q8_0 keys: every Dv and value type.
#include "fa_decode.cuh"

namespace fap {
FAP_INSTANTIATE_DECODE(256, FA_Q8_0)
}  // namespace fap
