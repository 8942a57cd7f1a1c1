// The gradient of the norm with rotation by positions of several axes for every head size and pair of types: its own translation unit, so
// that the kernel instantiations compile in parallel.
#include "fa_norm_rope.cuh"

namespace fap {

FAP_PICK_NORM(BackKernel, pick_norm_back, norm_back_style, true)

}  // namespace fap
