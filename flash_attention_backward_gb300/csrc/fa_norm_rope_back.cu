// The gradient of the norm with rotation for every head size and pair of types: its own translation unit, so
// that the kernel instantiations compile in parallel.
#include "fa_norm_rope.cuh"

namespace fap {

template <int D, typename TX, typename TY>
static BackKernel pick_style(bool vec, int style) {
  constexpr int heads = kBackHeads<D, TX, TY>, ring = kBackWarps * kBackSlots<TX, TY> * heads * D * (int)(sizeof(TX) + sizeof(TY));
  const bool pairs = style == FA_ROPE_PAIRS;
  static std::atomic<uint64_t> ready[2];
  if (!vec)
    return BackKernel{pairs ? k_norm_rope_back_any<D, TX, TY, FA_ROPE_PAIRS> : k_norm_rope_back_any<D, TX, TY, FA_ROPE_HALVES>, heads, 0,
                      nullptr};
  return BackKernel{pairs ? k_norm_rope_back<D, TX, TY, FA_ROPE_PAIRS> : k_norm_rope_back<D, TX, TY, FA_ROPE_HALVES>, heads, ring,
                    &ready[pairs]};
}
template <int D, typename TX>
static BackKernel pick_y(int ty, bool vec, int style) {
  switch (ty) {
    case FA_ACT_F32: return pick_style<D, TX, float>(vec, style);
    case FA_ACT_F16: return pick_style<D, TX, __half>(vec, style);
  }
  return pick_style<D, TX, __nv_bfloat16>(vec, style);
}
template <int D>
static BackKernel pick_x(int tx, int ty, bool vec, int style) {
  switch (tx) {
    case FA_ACT_F32: return pick_y<D, float>(ty, vec, style);
    case FA_ACT_F16: return pick_y<D, __half>(ty, vec, style);
  }
  return pick_y<D, __nv_bfloat16>(ty, vec, style);
}
BackKernel pick_norm_back(int D, int tx, int ty, bool vec, int style) {
  return D == 64    ? pick_x<64>(tx, ty, vec, style)
         : D == 128 ? pick_x<128>(tx, ty, vec, style)
                    : pick_x<256>(tx, ty, vec, style);
}

}  // namespace fap
