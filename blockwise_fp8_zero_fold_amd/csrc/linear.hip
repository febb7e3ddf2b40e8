// A product with one weight, its epilogue y = res + act(x W^T + bias) where the sums are; x in 16 bits on the tile and
// row kernels of the feed-forward block, x in 8 bits on those of linear8.h.  One token of width 7168 by 2048 columns,
// bias and residual, 8-bit rows: 7.8 to 8.2 us in a graph (15 MB of codes, 1.9 TB/s), 10.2 eager.  Latency bounds it:
// the launch, each wave's 3 or 4 blocks of codes, the sums of 16 waves, and then bias and residual, which are loaded
// only behind the sums though they do not depend on them (0.4 us).  Rows in 16 bits: one token 8.4 us in a graph; 8192
// tokens, 8 experts, 7168 of width 2048 266 us (0.91 PFLOP/s), 4096^3 129 to 132 (1.04 to 1.07), on the tiles of
// ffn_tile.h.
#include "ffn_tile.h"

using namespace fp8z1;

extern "C" int fp8z1_linear_workspace_bytes(const fp8z1_product* f, size_t* bytes) {
  const char* what = "linear_workspace_bytes";
  if (!f || !bytes) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  static const int32_t some_offsets = 0;
  const int rc = check_product(f, &some_offsets, what);
  if (rc) return rc;
  const bool eight = f->x_dtype == FP8Z1_E4M3;
  *bytes = !f->T ? 0 : eight ? linear8_workspace(f->T, f->E, f->N, f->K) : f->K > 2 * kB ? part_bytes(4) : 0;
  return FP8Z1_OK;
}

extern "C" int fp8z1_linear(const fp8z1_product* f, const void* x, const float* x_scales, const uint8_t* codes,
                            const float* scales, const int32_t* offsets, const float* bias, const void* res, void* y,
                            void* p, void* d_workspace, size_t workspace_bytes, void* stream) {
  const char* what = "linear";
  int rc = check_product(f, offsets, what);
  if (rc) return rc;
  const bool eight = f->x_dtype == FP8Z1_E4M3;
  if (f->T) rc = eight ? check_rows({y}, what) : check_rows({x, y}, what);
  if (rc) return rc;
  if (f->T && eight && (!x || !x_scales)) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  if (!eight && x_scales) return refuse(FP8Z1_EINVAL, what, "scales belong to FP8Z1_E4M3 rows");
  if (misaligned(x_scales, 4) || misaligned(bias, 4) || misaligned(res, 2) || misaligned(p, 2))
    return refuse(FP8Z1_EINVAL, what, "misaligned argument");
  rc = check_weights(codes, scales, what);
  if (rc) return rc;
  FfnArgs a{};
  a.offsets = offsets;
  a.T = static_cast<int32_t>(f->T);
  a.E = static_cast<int32_t>(f->E);
  a.N = static_cast<int32_t>(f->N);
  a.K = static_cast<int32_t>(f->K);
  a.act = f->act;
  a.x0 = bytes(x);
  a.w0 = codes;
  a.s0 = scales;
  a.bias = bias;
  a.res = static_cast<const uint16_t*>(res);
  a.o0 = static_cast<uint16_t*>(y);
  a.o1 = static_cast<uint16_t*>(p);
  if (!eight)
    return launch<kLinear>(a, f->dtype, d_workspace, workspace_bytes, static_cast<hipStream_t>(stream), what);
  a.xs = x_scales;
  return linear8(a, f->dtype, d_workspace, workspace_bytes, static_cast<hipStream_t>(stream), what);
}
