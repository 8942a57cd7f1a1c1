// The entry points of single-token attention on the host, up to their launches.  "D Dv kt vt B Hkv H num_pages page_size
// max_pages K SMs" a line in; out: the workspace that is asked for, and the status that the call over all pages (K 0) or over
// selected ones ends with when it is given just that.
#include <cstdio>
#include <iostream>

#include "../flash_attention_backward_gb300/csrc/fa_paged_decode.cu"

static int g_sms;

extern "C" fa_status fab_device(int* nsm, int** err) {
  static int word;
  *nsm = g_sms;
  if (err) *err = &word;
  return FA_OK;
}
extern "C" unsigned long long fab_take_wait_ns(void) { return 1; }

namespace fap {

fa_status check_cache(const fa_paged_cache* c, Cache* out) {
  *out = Cache{};
  out->k_type = c->k_type, out->v_type = c->v_type, out->num_pages = c->num_pages, out->page_size = c->page_size;
  out->B = c->B, out->max_pages = c->max_pages, out->Hkv = c->Hkv, out->D = c->D, out->Dv = c->Dv;
  out->rbk = out->rbv = 34;  // rows are copied one by one: no tensor maps, which need a driver
  return FA_OK;
}
static cudaError_t launched(DecodeArgs, const DecodeMaps&, cudaStream_t) { return cudaSuccess; }
#define STUB(D, SEL)                                                                  \
  template <> DecodeFn pick_decode<D, FA_F32, SEL>(int, int) { return launched; }     \
  template <> DecodeFn pick_decode<D, FA_F16, SEL>(int, int) { return launched; }     \
  template <> DecodeFn pick_decode<D, FA_Q8_0, SEL>(int, int) { return launched; }    \
  template <> DecodeFn pick_decode<D, FA_Q4_0, SEL>(int, int) { return launched; }
STUB(64, false)
STUB(64, true)
STUB(128, false)
STUB(128, true)
STUB(256, false)
STUB(256, true)

}  // namespace fap

int main() {
  fa_paged_cache c = {};
  int H, K;
  while (std::cin >> c.D >> c.Dv >> c.k_type >> c.v_type >> c.B >> c.Hkv >> H >> c.num_pages >> c.page_size >> c.max_pages >> K >> g_sms) {
    c.page_size |= 1;  // (no boxes of rows either)
    void* at = reinterpret_cast<void*>(0x100000);
    const int32_t* ints = static_cast<const int32_t*>(at);
    const size_t need = fa_paged_decode_workspace_size(&c, H);
    const int rc = K ? fa_paged_decode_pages(at, FA_ACT_F32, 0, 0, &c, ints, ints, K, H, 1.f, nullptr, 0.f, nullptr, at, nullptr, at, need, nullptr)
                     : fa_paged_decode(at, FA_ACT_F32, 0, 0, &c, ints, H, 1.f, nullptr, 0.f, nullptr, at, nullptr, at, need, nullptr);
    std::printf("%zu %d\n", need, rc);
  }
}
