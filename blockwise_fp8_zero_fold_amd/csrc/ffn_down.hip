// Down projection of the feed-forward block.
#include "ffn_tile.h"

using namespace fp8z1;

extern "C" int fp8z1_ffn_down(const fp8z1_ffn* f, const void* a, const uint8_t* down_codes, const float* down_scales,
                              const int32_t* offsets, void* y, void* d_workspace, size_t workspace_bytes, void* stream) {
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
  return launch<kFfnDown>(p, f->dtype, d_workspace, workspace_bytes, static_cast<hipStream_t>(stream),
                       what);
}

extern "C" int fp8z1_ffn_workspace_bytes(const fp8z1_ffn* f, size_t* bytes) {
  if (!f || !bytes) return refuse(FP8Z1_EINVAL, "ffn_workspace_bytes", "NULL argument");
  static const int32_t some_offsets = 0;
  const int rc = check_cfg(f, &some_offsets, "ffn_workspace_bytes");
  if (rc) return rc;
  const int64_t most = f->D > 2 * f->F ? f->D : 2 * f->F;  // longest sum of the four calls
  *bytes = f->T && most > 2 * kB ? part_bytes(4) : 0;
  return FP8Z1_OK;
}
