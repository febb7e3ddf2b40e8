// Backward of the down projection with the activation's backward in its epilogue.
#include "ffn_tile.h"

using namespace fp8z1;

extern "C" int fp8z1_ffn_down_bwd(const fp8z1_ffn* f, const void* dy, const uint8_t* down_codes,
                                  const float* down_scales, const void* h, const void* u, const int32_t* offsets,
                                  void* dh, void* du, void* a, void* d_workspace, size_t workspace_bytes, void* stream) {
  const char* what = "ffn_down_bwd";
  int rc = check_cfg(f, offsets, what);
  if (!rc && f->T) rc = check_rows({dy, h, u, dh, du}, what);
  if (!rc && misaligned(a, 2)) rc = refuse(FP8Z1_EINVAL, "ffn_down_bwd", "misaligned rows");
  if (!rc) rc = check_weights(down_codes, down_scales, what);
  if (rc) return rc;
  FfnArgs p = base_args(f, offsets, true);
  p.x0 = bytes(dy);
  p.w0 = down_codes;
  p.s0 = down_scales;
  p.h = static_cast<const uint16_t*>(h);
  p.u = static_cast<const uint16_t*>(u);
  p.o0 = static_cast<uint16_t*>(dh);
  p.o1 = static_cast<uint16_t*>(du);
  p.o2 = static_cast<uint16_t*>(a);
  return launch<kFfnDownBwd>(p, f->dtype, d_workspace, workspace_bytes, static_cast<hipStream_t>(stream),
                       what);
}
