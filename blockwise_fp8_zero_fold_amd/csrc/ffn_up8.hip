// Both projections of rows in 8 bits with the gated activation, its result in 8 bits.
#include "linear8.h"

using namespace fp8z1;

extern "C" int fp8z1_ffn_up8_workspace_bytes(const fp8z1_ffn* f, size_t* bytes) {
  const char* what = "ffn_up8_workspace_bytes";
  if (!f || !bytes) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  static const int32_t some_offsets = 0;
  const int rc = check_cfg(f, &some_offsets, what);
  if (rc) return rc;
  *bytes = !f->T ? 0 : few_rows8(f->T, f->E, f->F, f->D, 2) ? rows8_bytes(f->T, f->F) : tiles8_bytes(f->T, 2 * f->E * f->F, f->D);
  return FP8Z1_OK;
}

extern "C" int fp8z1_ffn_up8(const fp8z1_ffn* f, const uint8_t* x, const float* x_scales, const uint8_t* gate_codes,
                             const float* gate_scales, const uint8_t* up_codes, const float* up_scales,
                             const int32_t* offsets, void* h, void* u, uint8_t* a, float* a_scales, int32_t scale_rule,
                             void* d_workspace, size_t workspace_bytes, void* stream) {
  const char* what = "ffn_up8";
  int rc = check_cfg(f, offsets, what);
  if (rc) return rc;
  if (f->T && (!x || !x_scales || !a || !a_scales)) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  if (misaligned(x_scales, 4) || misaligned(a_scales, 4)) return refuse(FP8Z1_EINVAL, what, "misaligned scales");
  if ((h == nullptr) != (u == nullptr)) return refuse(FP8Z1_EINVAL, what, "h and u are kept both or not at all");
  if (f->T && h) rc = check_rows({h, u}, what);
  if (!rc) rc = check_weights(gate_codes, gate_scales, what);
  if (!rc) rc = check_weights(up_codes, up_scales, what);
  if (rc) return rc;
  if (scale_rule != FP8Z1_SCALE_AMAX && scale_rule != FP8Z1_SCALE_POW2)
    return refuse(FP8Z1_EINVAL, what, "scale_rule must be FP8Z1_SCALE_AMAX or FP8Z1_SCALE_POW2");
  FfnArgs p = base_args(f, offsets, true);
  p.x0 = x;
  p.xs = x_scales;
  p.w0 = gate_codes;
  p.w1 = up_codes;
  p.s0 = gate_scales;
  p.s1 = up_scales;
  p.o1 = static_cast<uint16_t*>(h);
  p.o2 = static_cast<uint16_t*>(u);
  p.codes = a;
  p.code_scales = a_scales;
  p.pow2 = scale_rule == FP8Z1_SCALE_POW2;
  return launch8<kFfnUp>(p, f->dtype, d_workspace, workspace_bytes, static_cast<hipStream_t>(stream), what);
}
