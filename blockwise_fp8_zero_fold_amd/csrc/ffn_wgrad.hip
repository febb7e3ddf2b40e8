// Weight gradients of the feed-forward block: per expert dW[m][n] = sum over its
// tokens t of p[t][m] q[t][n], written as the row-major [E, M, N] gradient that the
// shard step reads.
//
// A workgroup of 4 waves computes 128 x 128 of one expert's dW, each wave 64 x 64 as
// 2 x 2 matrix tiles of 32 x 32.  Both operands run along the columns while the sum
// runs down the rows, so a stage of 64 tokens is kept in LDS as it lies in memory and
// the matrix operands are gathered by the transposing LDS reads.
#include <hip/hip_runtime.h>

#include "ffn.h"

namespace fp8z1 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;  // rows and columns of a tile
constexpr int kStep = 64;   // tokens per stage
constexpr int kBytes = kTile * kStep * 2;

struct WgradArgs {
  const uint8_t *p, *q;  // [T, M], [T, N]
  const int32_t* offsets;
  float* part;  // [splits, E, M, N] partial sums, or NULL
  void* dw;
  int32_t T, E, M, N, mt, nt, splits, accumulate;
};

template <class H, bool F32OUT>
__global__ __launch_bounds__(kThreads, 2) void ffn_wgrad_kernel(WgradArgs g) {
  typedef typename H::v8 v8;
  __shared__ __attribute__((aligned(16))) uint8_t sp[2][kBytes];
  __shared__ __attribute__((aligned(16))) uint8_t sq[2][kBytes];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, wm = w >> 1, wn = w & 1;

  // tiles in contiguous runs per XCD, in groups of 8 tile rows by all tile columns
  const int32_t all = static_cast<int32_t>(gridDim.x), x = blockIdx.x % kXcds;
  int32_t id = x * (all / kXcds) + min(x, all % kXcds) + static_cast<int32_t>(blockIdx.x) / kXcds;
  const int32_t per = g.mt * g.nt, split = id / (per * g.E);
  id -= split * per * g.E;
  const int32_t e = id / per;
  id -= e * per;
  const int32_t gr = id / (kGroup * g.nt), in = id - gr * kGroup * g.nt, rows = min(kGroup, g.mt - gr * kGroup);
  const int32_t m0 = (gr * kGroup + in % rows) * kTile, n0 = in / rows * kTile;

  int32_t lo, hi;
  expert_rows(g.offsets, g.T, e, lo, hi);
  const int32_t stages = (hi - lo + kStep - 1) / kStep;
  const int32_t s0 = static_cast<int32_t>(static_cast<int64_t>(stages) * split / g.splits);
  const int32_t s1 = static_cast<int32_t>(static_cast<int64_t>(stages) * (split + 1) / g.splits);

  int64_t poff[4], qoff[4];
  int32_t pn[4], qn[4], row[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int ch = t + kThreads * j, r = ch >> 4, c = ((ch & 15) ^ ((r & 3) << 2)) * 8;
    row[j] = r;
    poff[j] = (static_cast<int64_t>(lo + r) * g.M + m0 + c) * 2;
    qoff[j] = (static_cast<int64_t>(lo + r) * g.N + n0 + c) * 2;
    pn[j] = (g.M - m0 - c) * 2;
    qn[j] = (g.N - n0 - c) * 2;
  }
  uint4 rp[4], rq[4];
  auto load = [&](int32_t s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in_run = lo + s * kStep + row[j] < hi;
      rp[j] = ld16_part(g.p + poff[j] + static_cast<int64_t>(s) * kStep * g.M * 2, in_run ? pn[j] : 0);
      rq[j] = ld16_part(g.q + qoff[j] + static_cast<int64_t>(s) * kStep * g.N * 2, in_run ? qn[j] : 0);
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      *reinterpret_cast<uint4*>(&sp[buf][(t + kThreads * j) * 16]) = rp[j];
      *reinterpret_cast<uint4*>(&sq[buf][(t + kThreads * j) * 16]) = rq[j];
    }
  };
  const int l16 = lane & 15, grp = lane >> 4;
  // 8 tokens of one column per lane: two reads of 4
  auto operand = [&](const uint8_t* s, int col0, int ks) {
    const int r = ks * 16 + (grp >> 1) * 8 + (l16 >> 2);
    const int c = col0 / 8 + (grp & 1) * 2 + ((l16 & 3) >> 1);
    const uint8_t* at = s + r * 256 + ((c ^ ((r & 3) << 2)) << 4) + (l16 & 1) * 8;
    const i32x2 a = read_tr16(at), b = read_tr16(at + 4 * 256);
    return as_v8<H>(make_uint4(a.x, a.y, b.x, b.y));
  };

  f32x16 acc[2][2];
  const f32x16 zero = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = zero;

  if (s0 < s1) {
    load(s0);
    store(0);
  }
  __syncthreads();
  for (int32_t s = s0; s < s1; ++s) {
    const int buf = (s - s0) & 1;
    if (s + 1 < s1) load(s + 1);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      v8 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = operand(sp[buf], wm * 64 + i * 32, ks);
        b[i] = operand(sq[buf], wn * 64 + i * 32, ks);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = H::mma32(a[i], b[j], acc[i][j]);
    }
    if (s + 1 < s1) store(buf ^ 1);
    __syncthreads();
  }

  const int64_t size = static_cast<int64_t>(g.E) * g.M * g.N;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int32_t m = m0 + wm * 64 + i * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
      if (m >= g.M) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int32_t n = n0 + wn * 64 + j * 32 + (lane & 31);
        if (n >= g.N) continue;
        const int64_t at = (static_cast<int64_t>(e) * g.M + m) * g.N + n;
        if (g.part)
          g.part[split * size + at] = acc[i][j][r];
        else if (F32OUT)
          static_cast<float*>(g.dw)[at] = g.accumulate ? static_cast<float*>(g.dw)[at] + acc[i][j][r] : acc[i][j][r];
        else
          static_cast<uint16_t*>(g.dw)[at] = Bf16::from_f32(acc[i][j][r]);
      }
    }
}

// The splits' partial sums added in order, one element per thread.
template <bool F32OUT>
__global__ __launch_bounds__(256) void ffn_wgrad_join_kernel(const float* __restrict__ part, int32_t splits,
                                                             int64_t size, void* dw, int32_t accumulate) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < size;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    float v = part[i];
    for (int32_t s = 1; s < splits; ++s) v += part[s * size + i];
    if (F32OUT)
      static_cast<float*>(dw)[i] = accumulate ? static_cast<float*>(dw)[i] + v : v;
    else
      static_cast<uint16_t*>(dw)[i] = Bf16::from_f32(v);
  }
}

// Splits of the tokens: where the output has fewer tiles than the card runs at once
// (two workgroups on each of 256 compute units), the tokens are cut so that about that
// many run, each with at least 4 stages of an even share.
int32_t wgrad_splits(int64_t T, int64_t E, int64_t M, int64_t N) {
  const int64_t tiles = E * ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  const int64_t want = 512 / (tiles < 1 ? 1 : tiles), most = T / E / (4 * kStep);
  const int64_t s = want < most ? want : most;
  return static_cast<int32_t>(s < 1 ? 1 : s);
}

int check_wgrad(int64_t T, int64_t E, int64_t M, int64_t N) {
  if (T < 0 || T > FP8Z1_FFN_MAX_ROWS) return set_error(FP8Z1_ESHAPE, "ffn_wgrad: T outside 0 .. 2^30");
  if (E < 1 || E > FP8Z1_FFN_MAX_EXPERTS) return set_error(FP8Z1_ESHAPE, "ffn_wgrad: E outside 1 .. 65535");
  if (M < 1 || M > FP8Z1_FFN_MAX_WIDTH || N < 1 || N > FP8Z1_FFN_MAX_WIDTH)
    return set_error(FP8Z1_ESHAPE, "ffn_wgrad: M and N must be 1 .. 2^20");
  const int64_t tiles = E * ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  if (tiles > 0x7fffffff) return set_error(FP8Z1_ESHAPE, "ffn_wgrad: too many tiles");
  return FP8Z1_OK;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

}  // namespace
}  // namespace fp8z1

using namespace fp8z1;

extern "C" int fp8z1_ffn_wgrad_workspace_bytes(int64_t T, int64_t E, int64_t M, int64_t N, size_t* bytes) {
  if (!bytes) return set_error(FP8Z1_EINVAL, "ffn_wgrad_workspace_bytes: NULL argument");
  const int rc = check_wgrad(T, E, M, N);
  if (rc) return rc;
  const int32_t s = wgrad_splits(T, E, M, N);
  *bytes = s > 1 ? sizeof(float) * static_cast<size_t>(s) * E * M * N : 0;
  return FP8Z1_OK;
}

extern "C" int fp8z1_ffn_wgrad(int64_t T, int64_t E, int64_t M, int64_t N, int32_t dtype, const void* p, const void* q,
                               const int32_t* offsets, int32_t dw_dtype, void* dw, int32_t accumulate, void* workspace,
                               size_t workspace_bytes, void* stream) {
  int rc = check_wgrad(T, E, M, N);
  if (rc) return rc;
  if (dtype != FP8Z1_BF16 && dtype != FP8Z1_F16)
    return set_error(FP8Z1_EINVAL, "ffn_wgrad: dtype must be FP8Z1_BF16 or FP8Z1_F16");
  if (dw_dtype != FP8Z1_F32 && dw_dtype != FP8Z1_BF16)
    return set_error(FP8Z1_EINVAL, "ffn_wgrad: dw_dtype must be FP8Z1_F32 or FP8Z1_BF16");
  if (accumulate && dw_dtype != FP8Z1_F32)
    return set_error(FP8Z1_EINVAL, "ffn_wgrad: only FP8Z1_F32 gradients can be accumulated");
  if (!dw || (T && (!p || !q))) return set_error(FP8Z1_EINVAL, "ffn_wgrad: NULL argument");
  if (!offsets && E != 1) return set_error(FP8Z1_EINVAL, "ffn_wgrad: offsets may be NULL for one expert only");
  if (misaligned(p, 2) || misaligned(q, 2) || misaligned(offsets, 4) || misaligned(workspace, 4) ||
      misaligned(dw, dw_dtype == FP8Z1_F32 ? 4 : 2))
    return set_error(FP8Z1_EINVAL, "ffn_wgrad: misaligned argument");
  WgradArgs g{};
  g.p = static_cast<const uint8_t*>(p);
  g.q = static_cast<const uint8_t*>(q);
  g.offsets = offsets;
  g.dw = dw;
  g.T = static_cast<int32_t>(T);
  g.E = static_cast<int32_t>(E);
  g.M = static_cast<int32_t>(M);
  g.N = static_cast<int32_t>(N);
  g.mt = static_cast<int32_t>((M + kTile - 1) / kTile);
  g.nt = static_cast<int32_t>((N + kTile - 1) / kTile);
  g.accumulate = accumulate;
  g.splits = 1;
  const int32_t splits = wgrad_splits(T, E, M, N);
  const int64_t size = E * M * N;
  if (splits > 1 && workspace && workspace_bytes >= sizeof(float) * static_cast<size_t>(splits) * size) {
    g.splits = splits;
    g.part = static_cast<float*>(workspace);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(g.E * g.mt * g.nt * g.splits)), block(kThreads);
  if (dtype == FP8Z1_BF16 && dw_dtype == FP8Z1_F32)
    hipLaunchKernelGGL((ffn_wgrad_kernel<Bf16, true>), grid, block, 0, s, g);
  else if (dtype == FP8Z1_BF16)
    hipLaunchKernelGGL((ffn_wgrad_kernel<Bf16, false>), grid, block, 0, s, g);
  else if (dw_dtype == FP8Z1_F32)
    hipLaunchKernelGGL((ffn_wgrad_kernel<F16, true>), grid, block, 0, s, g);
  else
    hipLaunchKernelGGL((ffn_wgrad_kernel<F16, false>), grid, block, 0, s, g);
  rc = check_hip(hipGetLastError(), "ffn_wgrad: launch");
  if (rc || !g.part) return rc;
  const int64_t want = (size + 255) / 256;
  const dim3 jgrid(static_cast<unsigned>(want < 4096 ? want : 4096));
  if (dw_dtype == FP8Z1_F32)
    hipLaunchKernelGGL(ffn_wgrad_join_kernel<true>, jgrid, dim3(256), 0, s, g.part, g.splits, size, dw, accumulate);
  else
    hipLaunchKernelGGL(ffn_wgrad_join_kernel<false>, jgrid, dim3(256), 0, s, g.part, g.splits, size, dw, accumulate);
  return check_hip(hipGetLastError(), "ffn_wgrad: join launch");
}
