// Gradient at the block's input: both products in one sum.
#include "ffn_tile.h"

using namespace fp8z1;

extern "C" int fp8z1_ffn_up_bwd(const fp8z1_ffn* f, const void* dh, const void* du, const uint8_t* gate_codes,
                                const float* gate_scales, const uint8_t* up_codes, const float* up_scales,
                                const int32_t* offsets, void* dx, void* d_workspace, size_t workspace_bytes, void* stream) {
  const char* what = "ffn_up_bwd";
  int rc = check_cfg(f, offsets, what);
  if (!rc && f->T) rc = check_rows({dh, du, dx}, what);
  if (!rc) rc = check_weights(gate_codes, gate_scales, what);
  if (!rc) rc = check_weights(up_codes, up_scales, what);
  if (rc) return rc;
  FfnArgs p = base_args(f, offsets, false);
  p.x0 = bytes(dh);
  p.x1 = bytes(du);
  p.w0 = gate_codes;
  p.w1 = up_codes;
  p.s0 = gate_scales;
  p.s1 = up_scales;
  p.o0 = static_cast<uint16_t*>(dx);
  return launch<kFfnUpBwd>(p, f->dtype, d_workspace, workspace_bytes, static_cast<hipStream_t>(stream),
                       what);
}
