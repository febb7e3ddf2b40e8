// Both projections of the feed-forward block with the gated activation, in one kernel.
#include "ffn_tile.h"

using namespace fp8z1;

extern "C" int fp8z1_ffn_up(const fp8z1_ffn* f, const void* x, const uint8_t* gate_codes, const float* gate_scales,
                            const uint8_t* up_codes, const float* up_scales, const int32_t* offsets, void* h, void* u,
                            void* a, void* d_workspace, size_t workspace_bytes, void* stream) {
  const char* what = "ffn_up";
  int rc = check_cfg(f, offsets, what);
  if (!rc && f->T) rc = check_rows({x, a}, what);
  if (!rc && f->T && (h || u)) rc = check_rows({h, u}, what);
  if (!rc) rc = check_weights(gate_codes, gate_scales, what);
  if (!rc) rc = check_weights(up_codes, up_scales, what);
  if (rc) return rc;
  FfnArgs p = base_args(f, offsets, true);
  p.x0 = bytes(x);
  p.w0 = gate_codes;
  p.w1 = up_codes;
  p.s0 = gate_scales;
  p.s1 = up_scales;
  p.o0 = static_cast<uint16_t*>(a);
  p.o1 = static_cast<uint16_t*>(h);
  p.o2 = static_cast<uint16_t*>(u);
  return launch<kFfnUp>(p, f->dtype, d_workspace, workspace_bytes, static_cast<hipStream_t>(stream),
                       what);
}
