// Down projection of the feed-forward block.
#include "ffn_tile.h"

using namespace fp8z1;

extern "C" int fp8z1_ffn_down(const fp8z1_ffn* f, const void* a, const uint8_t* down_codes, const float* down_scales,
                              const int32_t* offsets, void* y, void* stream) {
  const char* what = "ffn_down";
  int rc = check_cfg(f, offsets, what);
  if (!rc && f->T) rc = check_rows({a, y}, what);
  if (!rc) rc = check_weights(down_codes, down_scales, what);
  if (rc) return rc;
  FfnArgs p = base_args(f, offsets, false);
  p.x0 = bytes(a);
  p.w0 = down_codes;
  p.s0 = down_scales;
  p.o0 = static_cast<uint16_t*>(y);
  return launch<kFfnDown>(p, f->dtype, static_cast<hipStream_t>(stream), what);
}
