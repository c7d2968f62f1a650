// Stand-in launchers of the e4m3 and grouped products for the host-only build
// of their argument checks (fp8_api.cpp, no HIP runtime): each counts the call
// and keeps its arguments.
#include "../../gguf_block_quantized_qmv_amd/csrc/fp8_internal.h"

namespace stub {
int launches = 0;
qmv::ProductArgs last{};
int last_m = 0, last_k = 0;
}  // namespace stub

namespace qmv {

static int note(const ProductArgs &a) {
  ++stub::launches;
  stub::last = a;
  return 0;
}

int launch_fp8_quant(const void *, bool, bool, uint8_t *, float *, int m, int k, void *) {
  ++stub::launches;
  stub::last_m = m;
  stub::last_k = k;
  return 0;
}
int launch_fp8_dense(const ProductArgs &a, void *) { return note(a); }
int launch_fp8_grouped(const ProductArgs &a, void *) { return note(a); }
int launch_bf16_grouped(const ProductArgs &a, void *) { return note(a); }

}  // namespace qmv
