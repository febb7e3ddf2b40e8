// Gradients of y = res + act(x W^T + bias): dp = dy act'(p) with its sums over an expert's rows (the
// bias's gradient) in one pass over dy and p, and dx = dp W on the tile kernel of the feed-forward block.
//
// The pass reads dy and p and writes dp; its arithmetic (the activation's slope, about 30 instructions an element)
// takes as long as half of the transfers, and runs under other waves'.  A workgroup takes 8 rows (of many elements
// more, see sum_rows) of one expert by up to 2048 columns, 8 of them per thread, and writes their float32 column sums
// to the workspace; a second kernel adds an expert's groups in order.  4096 x 4096, GELU: 24 us (4.2 TB/s) and 5.7 for
// the sums; groups of 16 rows 27 and 4.9, and with the next rows' loads ahead of the arithmetic 29.
#include "ffn_tile.h"
#include "rows.h"

namespace fp8z1 {
namespace {

// Rows of a group: 8 while there are fewer than 10^8 elements, 64 up to 2^31, then 512, so that the groups' sums take
// 50 MB, 134 MB or 1/256 of dy (and a row for each expert) at most.  8 and 64 rows, GELU: 8192 x 7168 90 and 105 us,
// 32,768 x 2048 103 and 115, 16,384 x 7168 177 and 172, 65,536 x 2048 212 and 182, 262,144 x 1024 510 and 377, 65,536 x
// 7168 658 and 608; 64 and 512: 524,288 x 2048 1323 and 1312, 262,144 x 7168 2321 and 2422, 65,536 x 2048 182 and 527.
int32_t sum_rows(int64_t T, int64_t N) { return T * N < 100000000 ? 8 : T * N < (1ll << 31) ? 64 : 512; }

struct DpArgs {
  const uint16_t *dy, *p;
  uint16_t* dp;
  float* sums;  // [groups][N], or NULL
  const int32_t* offsets;
  int32_t T, E, N, act;
};

template <class H, int ROWS>
__global__ __launch_bounds__(kThreads) void linear_dp_kernel(DpArgs a) {
  int32_t e, lo, hi, t0;
  const int32_t group = static_cast<int32_t>(blockIdx.z * gridDim.y + blockIdx.y);
  if (!find_group<ROWS>(a.offsets, a.T, a.E, group, e, lo, hi, t0)) return;
  const int32_t n = static_cast<int32_t>(blockIdx.x * blockDim.x + threadIdx.x) * 8, rows = min(hi - t0, ROWS);
  if (n >= a.N) return;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  for (int32_t r0 = 0; r0 < rows; r0 += 4) {
    Raw8<H> d[4], p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r0 + k < rows) {
        d[k] = fetch8<H>(row_of<H>(static_cast<const void*>(a.dy), t0 + r0 + k, a.N), a.N, n);
        if (a.p) p[k] = fetch8<H>(row_of<H>(static_cast<const void*>(a.p), t0 + r0 + k, a.N), a.N, n);
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r0 + k < rows) {
        float dy[8], h[8];
        widen8f<H>(d[k], dy);
        if (a.p) {
          widen8f<H>(p[k], h);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float value, slope;
            act_both(a.act, h[i], value, slope);
            dy[i] *= slope;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += dy[i];
        if (a.dp) store8<H>(row_of<H>(static_cast<void*>(a.dp), t0 + r0 + k, a.N), a.N, n, dy);
      }
  }
  if (a.sums) store8<F32>(a.sums + static_cast<int64_t>(group) * a.N, a.N, n, sum);
}

// dbias[e][n]: the sums of expert e's groups, numbered as find_group numbers them.  64 columns a workgroup, each
// of its 16 waves adds every 16th group; the waves' sums are added in order.
constexpr int kBiasWaves = 16, kBiasCols = 64;
__global__ __launch_bounds__(64 * kBiasWaves) void linear_dbias_kernel(const float* sums, const int32_t* offsets, int32_t T,
                                                                       int32_t E, int32_t N, int32_t rows, float* dbias) {
  __shared__ float parts[kBiasWaves][kBiasCols];
  const int32_t strips = (N + kBiasCols - 1) / kBiasCols;
  const int32_t e = static_cast<int32_t>(blockIdx.x) / strips;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int32_t n = min((static_cast<int32_t>(blockIdx.x) - e * strips) * kBiasCols + lane, N - 1);
  int32_t lo, hi;
  expert_rows(offsets, T, e, lo, hi);
  float sum = 0.0f;
  if (lo < hi) {
    if (w == 0) sum = sums[static_cast<int64_t>(e) * N + n];
    const float* const from = sums + (static_cast<int64_t>(E) + lo / rows) * N + n;
    const int32_t more = (hi - lo - 1) / rows;  // groups behind the first
#pragma unroll 8
    for (int32_t k = w; k < more; k += kBiasWaves) sum += from[static_cast<int64_t>(k) * N];
  }
  parts[w][lane] = sum;
  __syncthreads();
  if (w != 0 || (static_cast<int32_t>(blockIdx.x) - e * strips) * kBiasCols + lane >= N) return;
#pragma unroll
  for (int k = 1; k < kBiasWaves; ++k) sum += parts[k][lane];
  dbias[static_cast<int64_t>(e) * N + n] = sum;
}

int64_t sum_groups(int64_t T, int64_t E, int64_t N) { return E + T / sum_rows(T, N); }

template <class H>
void launch_dp(const DpArgs& a, int32_t rows, dim3 g, dim3 b, hipStream_t s) {
  if (rows == 8)
    hipLaunchKernelGGL((linear_dp_kernel<H, 8>), g, b, 0, s, a);
  else if (rows == 64)
    hipLaunchKernelGGL((linear_dp_kernel<H, 64>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((linear_dp_kernel<H, 512>), g, b, 0, s, a);
}

}  // namespace
}  // namespace fp8z1

using namespace fp8z1;

extern "C" int fp8z1_linear_bwd_workspace_bytes(const fp8z1_product* f, size_t* bytes) {
  const char* what = "linear_bwd_workspace_bytes";
  if (!f || !bytes) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  static const int32_t some_offsets = 0;
  const int rc = check_product(f, &some_offsets, what);
  if (rc) return rc;
  // the bias's sums are joined before the tiles are split: both use the same memory
  const size_t sums = sizeof(float) * static_cast<size_t>(sum_groups(f->T, f->E, f->N)) * static_cast<size_t>(f->N);
  const size_t parts = f->N > 2 * kB ? part_bytes(4) : 0;
  *bytes = !f->T ? 0 : ((sums > parts ? sums : parts) + 15) / 16 * 16;
  return FP8Z1_OK;
}

extern "C" int fp8z1_linear_bwd(const fp8z1_product* f, const void* dy, const void* p, const uint8_t* codes,
                                const float* scales, const int32_t* offsets, void* dp, float* dbias, void* dx,
                                void* d_workspace, size_t workspace_bytes, void* stream) {
  const char* what = "linear_bwd";
  int rc = check_product(f, offsets, what);
  if (rc) return rc;
  const bool act = f->act != FP8Z1_ACT_NONE;
  if (!dp && !dbias && !dx) return refuse(FP8Z1_EINVAL, what, "no gradient is wanted");
  if (f->T) rc = check_rows({dy}, what);
  if (f->T && !rc && act) rc = check_rows({p}, what);
  if (rc) return rc;
  if (f->T && dx && act && !dp) return refuse(FP8Z1_EINVAL, what, "dx needs dp behind an activation");
  if (misaligned(dp, 2) || misaligned(dx, 2) || misaligned(dbias, 4))
    return refuse(FP8Z1_EINVAL, what, "misaligned argument");
  if (dx) rc = check_weights(codes, scales, what);
  if (rc) return rc;
  if (misaligned(d_workspace, 16)) return refuse(FP8Z1_EINVAL, what, "misaligned workspace");
  hipStream_t s = static_cast<hipStream_t>(stream);
  DpArgs a{};
  a.dy = static_cast<const uint16_t*>(dy);
  a.p = act ? static_cast<const uint16_t*>(p) : nullptr;
  a.dp = static_cast<uint16_t*>(dp);
  a.offsets = offsets;
  a.T = static_cast<int32_t>(f->T);
  a.E = static_cast<int32_t>(f->E);
  a.N = static_cast<int32_t>(f->N);
  a.act = f->act;
  const int64_t groups = sum_groups(f->T, f->E, f->N);
  if (dbias && f->T) {
    if (!d_workspace || workspace_bytes < sizeof(float) * static_cast<size_t>(groups) * static_cast<size_t>(f->N))
      return refuse(FP8Z1_EINVAL, what, "workspace too small");
    a.sums = static_cast<float*>(d_workspace);
  }
  const int64_t strips = f->E * ((f->N + kBiasCols - 1) / kBiasCols);
  if (dbias && strips > 0x7fffffff / (64 * kBiasWaves)) return refuse(FP8Z1_ESHAPE, what, "too many gradients of biases");
  if (f->T && (dp || dbias)) {
    const int64_t chunks = (f->N + 7) / 8, threads = chunks < kThreads ? (chunks + 63) / 64 * 64 : kThreads;
    const int64_t turns = (groups + 65534) / 65535;  // (a grid's y ends at 65,535)
    const dim3 g(static_cast<unsigned>((chunks + threads - 1) / threads),
                 static_cast<unsigned>((groups + turns - 1) / turns), static_cast<unsigned>(turns));
    const dim3 b(static_cast<unsigned>(threads));
    if (f->dtype == FP8Z1_BF16)
      launch_dp<Bf16>(a, sum_rows(f->T, f->N), g, b, s);
    else
      launch_dp<F16>(a, sum_rows(f->T, f->N), g, b, s);
    rc = launched(what);
    if (rc) return rc;
  }
  if (dbias) {
    hipLaunchKernelGGL(linear_dbias_kernel, dim3(static_cast<unsigned>(strips)), dim3(64 * kBiasWaves), 0, s, a.sums, offsets, a.T,
                       a.E, a.N, sum_rows(f->T, f->N), dbias);
    rc = launched(what);
    if (rc) return rc;
  }
  if (!dx) return FP8Z1_OK;
  FfnArgs q{};
  q.offsets = offsets;
  q.T = a.T;
  q.E = a.E;
  q.N = static_cast<int32_t>(f->K);
  q.K = static_cast<int32_t>(f->N);
  q.x0 = bytes(act ? dp : dy);
  q.w0 = codes;
  q.s0 = scales;
  q.o0 = static_cast<uint16_t*>(dx);
  return launch<kLinearBwd>(q, f->dtype, d_workspace, workspace_bytes, s, what);
}
