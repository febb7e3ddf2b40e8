// Weight gradients of the feed-forward block: per expert dW[m][n] = sum over its
// tokens t of p[t][m] q[t][n], written as the row-major [E, M, N] gradient that the
// shard step reads.
//
// A workgroup of 4 waves computes 128 x 64 NT of one expert's dW, each wave 64 x 32 NT as
// 2 x NT matrix tiles of 32 x 32.  Both operands run along the columns while the sum
// runs down the rows, so a stage of 32 tokens is kept in LDS as it lies in memory and
// the matrix operands are gathered by the transposing LDS reads.
#include <hip/hip_runtime.h>

#include "ffn.h"

namespace fp8z1 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;  // tile rows
constexpr int kStep = 32;   // tokens per stage
constexpr int kPBytes = kTile * kStep * 2;

struct WgradArgs {
  const uint8_t *p, *q;  // [T, M], [T, N]
  const int32_t* offsets;
  float* part;  // [splits, E, M, N] partial sums, or NULL
  void* dw;
  int32_t T, E, M, N, mt, nt, splits, accumulate;
};

// Chunk c (16 bytes) of row r of a stage sits at position c ^ swizzle(r): a transposing read
// takes 4 rows of 4 neighbouring chunks at a time, which then lie in 16 different places.
__device__ __forceinline__ int swizzle(int r) { return (r & 3) << 2; }

// DIRECT: rows are 4-byte aligned, so a stage goes from memory to LDS by direct copies;
// otherwise through registers, with the bytes outside a row left out.
template <class H, bool F32OUT, int NT, bool DIRECT>
__global__ __launch_bounds__(kThreads, 2) void ffn_wgrad_kernel(WgradArgs g) {
  typedef typename H::v8 v8;
  constexpr int kCols = NT * 64, kQBytes = kCols * kStep * 2, kStage = kPBytes + kQBytes;
  constexpr int kPC = kPBytes / 16 / kThreads, kQC = kQBytes / 16 / kThreads;  // chunks per thread
  __shared__ __attribute__((aligned(16))) uint8_t lds[3 * kStage];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6), wm = w >> 1, wn = w & 1;

  // tiles in contiguous runs per XCD, in groups of kGroup tile rows by all tile columns
  int32_t id = xcd_run(static_cast<int32_t>(blockIdx.x), static_cast<int32_t>(gridDim.x));
  const int32_t per = g.mt * g.nt, split = id / (per * g.E);
  id -= split * per * g.E;
  const int32_t e = id / per;
  id -= e * per;
  const int32_t gr = id / (kGroup * g.nt), in = id - gr * kGroup * g.nt, rows = min(kGroup, g.mt - gr * kGroup);
  const int32_t m0 = (gr * kGroup + in % rows) * kTile, n0 = in / rows * kCols;

  int32_t lo, hi;
  expert_rows(g.offsets, g.T, e, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  const int32_t stages = (hi - lo + kStep - 1) / kStep;
  const int32_t s0 = static_cast<int32_t>(static_cast<int64_t>(stages) * split / g.splits);
  const int32_t s1 = static_cast<int32_t>(static_cast<int64_t>(stages) * (split + 1) / g.splits);

  uint32_t poff[kPC], qoff[kQC];
  int32_t pc[kPC], qc[kQC];  // byte column of the chunk
#pragma unroll
  for (int j = 0; j < kPC; ++j) {
    const int ch = t + kThreads * j, r = ch / (kTile / 8);
    pc[j] = ((ch % (kTile / 8)) ^ swizzle(r)) * 16;
    poff[j] = static_cast<uint32_t>(r) * static_cast<uint32_t>(g.M) * 2 + pc[j];
  }
#pragma unroll
  for (int j = 0; j < kQC; ++j) {
    const int ch = t + kThreads * j, r = ch / (kCols / 8);
    qc[j] = ((ch % (kCols / 8)) ^ swizzle(r)) * 16;
    qoff[j] = static_cast<uint32_t>(r) * static_cast<uint32_t>(g.N) * 2 + qc[j];
  }
  uint4 rp[kPC], rq[kQC];
  auto fetch = [&](int32_t s, uint8_t* to) {
    const int32_t t0 = lo + s * kStep;
    const uint8_t* const pb = g.p + (static_cast<int64_t>(t0) * g.M + m0) * 2;
    const uint8_t* const qb = g.q + (static_cast<int64_t>(t0) * g.N + n0) * 2;
    if (DIRECT) {
      // The buffers end with the run: chunks of later rows are not read.  A chunk past the
      // end of a row is the next row's; its columns are not stored.
      const buffer_t ba = make_buffer(pb, (static_cast<int64_t>(hi - t0) * g.M - m0) * 2);
      const buffer_t bb = make_buffer(qb, (static_cast<int64_t>(hi - t0) * g.N - n0) * 2);
#pragma unroll
      for (int j = 0; j < kPC; ++j) copy16_to_lds(ba, poff[j], to + (w * 64 + kThreads * j) * 16);
#pragma unroll
      for (int j = 0; j < kQC; ++j) copy16_to_lds(bb, qoff[j], to + kPBytes + (w * 64 + kThreads * j) * 16);
      return;
    }
#pragma unroll
    for (int j = 0; j < kPC; ++j) {
      const int r = (t + kThreads * j) / (kTile / 8);
      rp[j] = ld16_part(pb + poff[j], t0 + r < hi ? (g.M - m0) * 2 - pc[j] : 0, m0 * 2 + pc[j]);
    }
#pragma unroll
    for (int j = 0; j < kQC; ++j) {
      const int r = (t + kThreads * j) / (kCols / 8);
      rq[j] = ld16_part(qb + qoff[j], t0 + r < hi ? (g.N - n0) * 2 - qc[j] : 0, n0 * 2 + qc[j]);
    }
  };
  auto put = [&](uint8_t* to) {
    if (DIRECT) return;
#pragma unroll
    for (int j = 0; j < kPC; ++j) *reinterpret_cast<uint4*>(to + (t + kThreads * j) * 16) = rp[j];
#pragma unroll
    for (int j = 0; j < kQC; ++j) *reinterpret_cast<uint4*>(to + kPBytes + (t + kThreads * j) * 16) = rq[j];
  };
  const int l16 = lane & 15, grp = lane >> 4;
  // 8 tokens of one column per lane: two reads of 4
  auto operand = [&](const uint8_t* s, int stride, int col0, int ks) {
    const int r = ks * 16 + (grp >> 1) * 8 + (l16 >> 2);
    const int c = col0 / 8 + (grp & 1) * 2 + ((l16 & 3) >> 1);
    const uint8_t* at = s + r * stride + ((c ^ swizzle(r)) << 4) + (l16 & 1) * 8;
    const i32x2 a = read_tr16(at), b = read_tr16(at + 4 * stride);
    return as_v8<H>(make_uint4(a.x, a.y, b.x, b.y));
  };

  f32x16 acc[2][NT];
  const f32x16 zero = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = zero;

  // Three stages: direct copies run two stages ahead (one stage's matrix instructions take
  // less time than a copy), loads through registers one.
  int at = 0;  // stage in use
  if (s0 < s1) {
    fetch(s0, lds);
    put(lds);
    if (DIRECT && s0 + 1 < s1) fetch(s0 + 1, lds + kStage);
  }
  for (int32_t s = s0; s < s1; ++s) {
    uint8_t* const here = lds + at * kStage;
    const int32_t ahead = s + (DIRECT ? 2 : 1);
    uint8_t* const there = lds + (at + (DIRECT ? 2 : 1)) % 3 * kStage;
    at = at == 2 ? 0 : at + 1;
    if (DIRECT) {
      if (s + 1 < s1)
        wait_copies<kPC + kQC>();
      else
        wait_copies<0>();
    }
    __syncthreads();
    const int32_t left = hi - lo - s * kStep;
    if (DIRECT && left < kStep) {  // the run ends inside the stage: rows past it count nothing
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      for (int c = left * (kTile / 8) + t; c < kStep * (kTile / 8); c += kThreads)
        *reinterpret_cast<uint4*>(here + c * 16) = z;
      for (int c = left * (kCols / 8) + t; c < kStep * (kCols / 8); c += kThreads)
        *reinterpret_cast<uint4*>(here + kPBytes + c * 16) = z;
      __syncthreads();
    }
    v8 a[2][2], b[2][NT];
    auto read = [&](int ks) {
#pragma unroll
      for (int i = 0; i < 2; ++i) a[ks][i] = operand(here, kTile * 2, wm * 64 + i * 32, ks);
#pragma unroll
      for (int j = 0; j < NT; ++j) b[ks][j] = operand(here + kPBytes, kCols * 2, (wn * NT + j) * 32, ks);
    };
    read(0);
    if (ahead < s1) fetch(ahead, there);
    read(1);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[i][j] = H::mma32(a[ks][i], b[ks][j], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
    if (ahead < s1) put(there);
  }

  const int64_t size = static_cast<int64_t>(g.E) * g.M * g.N;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int32_t m = m0 + wm * 64 + i * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
      if (m >= g.M) continue;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int32_t n = n0 + (wn * NT + j) * 32 + (lane & 31);
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

// Columns of a tile: 256 where such tiles fill the card twice over (as many workgroups as run
// at once, two on each of 256 compute units), else 128.
int wgrad_nt(int64_t E, int64_t M, int64_t N, bool direct) {
  return direct && E * ((M + kTile - 1) / kTile) * ((N + 255) / 256) >= 2 * kSlots ? 4 : 2;
}

// Splits of the tokens: where the output has fewer tiles (of 128 columns) than the card runs at
// once, the tokens are cut so that about that many run, each with at least 8 stages of
// an even share.
int32_t wgrad_splits(int64_t T, int64_t E, int64_t M, int64_t N) {
  const int64_t tiles = E * ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  const int64_t want = kSlots / (tiles < 1 ? 1 : tiles), most = T / E / (8 * kStep);
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

template <class H, bool F32OUT>
void launch_wgrad_as(const WgradArgs& g, int nt, bool direct, dim3 grid, hipStream_t s) {
  if (nt == 4)
    hipLaunchKernelGGL((ffn_wgrad_kernel<H, F32OUT, 4, true>), grid, dim3(kThreads), 0, s, g);
  else if (direct)
    hipLaunchKernelGGL((ffn_wgrad_kernel<H, F32OUT, 2, true>), grid, dim3(kThreads), 0, s, g);
  else
    hipLaunchKernelGGL((ffn_wgrad_kernel<H, F32OUT, 2, false>), grid, dim3(kThreads), 0, s, g);
}

template <class H>
void launch_wgrad(const WgradArgs& g, bool f32out, int nt, bool direct, dim3 grid, hipStream_t s) {
  if (f32out)
    launch_wgrad_as<H, true>(g, nt, direct, grid, s);
  else
    launch_wgrad_as<H, false>(g, nt, direct, grid, s);
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
  const bool direct = M % 2 == 0 && N % 2 == 0 && !misaligned(p, 4) && !misaligned(q, 4);
  const int nt = wgrad_nt(E, M, N, direct);
  g.mt = static_cast<int32_t>((M + kTile - 1) / kTile);
  g.nt = static_cast<int32_t>((N + nt * 64 - 1) / (nt * 64));
  g.accumulate = accumulate;
  g.splits = 1;
  const int32_t splits = wgrad_splits(T, E, M, N);
  const int64_t size = E * M * N;
  if (splits > 1 && workspace && workspace_bytes >= sizeof(float) * static_cast<size_t>(splits) * size) {
    g.splits = splits;
    g.part = static_cast<float*>(workspace);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(g.E * g.mt * g.nt * g.splits));
  if (dtype == FP8Z1_BF16)
    launch_wgrad<Bf16>(g, dw_dtype == FP8Z1_F32, nt, direct, grid, s);
  else
    launch_wgrad<F16>(g, dw_dtype == FP8Z1_F32, nt, direct, grid, s);
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
