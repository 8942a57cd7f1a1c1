// The forward of the norm with rotation by positions of several axes for every head size and pair of types: its own translation unit, so
// that the kernel instantiations compile in parallel.
#include "fa_norm_rope.cuh"

namespace fap {

FAP_PICK_NORM(NormKernel, pick_norm_fwd, norm_fwd_style, true)

}  // namespace fap
