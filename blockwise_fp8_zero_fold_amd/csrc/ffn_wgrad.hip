// Weight gradients of the feed-forward block: per expert dW[m][n] = sum over its
// tokens t of p[t][m] q[t][n], written as the row-major [E, M, N] gradient that the
// shard step reads.
//
// A workgroup of 4 waves computes 128 x 64 NT of one expert's dW, each wave 64 x 32 NT as
// 2 x NT matrix tiles of 32 x 32.  Both operands run along the columns while the sum
// runs down the rows, so a stage of 32 tokens is kept in LDS as it lies in memory and
// the matrix operands are gathered by the transposing LDS reads.
//
// 8192 tokens of 8 experts, widths 7168 and 2048, float32 gradients: 390 us for one gradient, 1.10 to 1.16
// ms for the three (620 to 660 TFLOP/s).  A gradient's 470 MB of output take 100 us by themselves (4.6
// TB/s), which 32 stages of a tile do not hide; with four times the tokens it runs at 810 TFLOP/s, 940
// for the tokens added.  The matrix cores are busy for 27 % of the cycles, at 2.2 GHz of 2.4 (power is not
// what ends), the waves wait for 28 % of theirs on data and barriers (16 matrix instructions a wave between
// two) and for 37 % until an instruction can issue.  Added to what is there (`accumulate`) the three take
// 2.0 ms, 1.7 where 2048 tokens' take 0.57: each result's load waits behind the loop.
// 20,000 tokens on widths 520 and 300 (few tiles, 11 parts each): 51 us; matrix cores 22 %, waves on data 27
// %, at issue 31 %; 98 MB of HBM read, 5.7 million L2 requests of which 84 % hit: neither memory ends it.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "ffn.h"

namespace fp8z1 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;  // tile rows
constexpr int kStep = 32;   // tokens per stage
constexpr int kPBytes = kTile * kStep * 2;

// One gradient dw [E, M, N] of rows p [T, M] and q [T, N]
struct Wgrad {
  const uint8_t *p, *q;
  void* dw;
  int64_t part;  // of its partial sums within a split's
  int32_t M, N, mt, nt;
};

// Up to three gradients over the same tokens in one launch (the block's own three: each alone
// may have too few tiles to fill the card, and a launch takes as long as a small gradient)
constexpr int kMost = 3;
struct WgradArgs {
  Wgrad g[kMost];
  const int32_t* offsets;
  float* part;  // partial sums of each split: all gradients [E, M, N] in turn; or NULL
  int64_t size;  // elements of all gradients
  int32_t T, E, count, tiles, splits, accumulate;
};

// Chunk c (16 bytes) of row r of a stage sits at position c ^ swizzle(r): a transposing read
// takes 4 rows of 4 neighbouring chunks at a time, which then lie in 16 different places.
__device__ __forceinline__ int swizzle(int r) { return (r & 3) << 2; }

// DIRECT: rows are 4-byte aligned, so a stage goes from memory to LDS by direct copies;
// otherwise through registers, with the bytes outside a row left out.
template <class H, bool F32OUT, int NT, bool DIRECT>
__global__ __launch_bounds__(kThreads, NT == 2 ? 3 : 2) void ffn_wgrad_kernel(WgradArgs all) {
  typedef typename H::v8 v8;
  constexpr int kCols = NT * 64, kQBytes = kCols * kStep * 2, kStage = kPBytes + kQBytes;
  constexpr int kPC = kPBytes / 16 / kThreads, kQC = kQBytes / 16 / kThreads;  // chunks per thread
  __shared__ __attribute__((aligned(16))) uint8_t lds[3 * kStage];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6), wm = w >> 1, wn = w & 1;

  // tiles in contiguous runs per XCD, in groups of kGroup tile rows by all tile columns
  int32_t id = xcd_run(static_cast<int32_t>(blockIdx.x), static_cast<int32_t>(gridDim.x));
  const int32_t split = id / all.tiles;
  id -= split * all.tiles;
  int which = 0;
  for (; which + 1 < all.count; ++which) {
    const int32_t n = all.E * all.g[which].mt * all.g[which].nt;
    if (id < n) break;
    id -= n;
  }
  const Wgrad g = all.g[which];
  const int32_t per = g.mt * g.nt, e = id / per;
  id -= e * per;
  const int32_t gr = id / (kGroup * g.nt), in = id - gr * kGroup * g.nt, rows = min(kGroup, g.mt - gr * kGroup);
  const int32_t m0 = (gr * kGroup + in % rows) * kTile, n0 = in / rows * kCols;

  int32_t lo, hi;
  expert_rows(all.offsets, all.T, e, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  const int32_t stages = (hi - lo + kStep - 1) / kStep;
  const int32_t s0 = static_cast<int32_t>(static_cast<int64_t>(stages) * split / all.splits);
  const int32_t s1 = static_cast<int32_t>(static_cast<int64_t>(stages) * (split + 1) / all.splits);

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

  float* const part = all.part ? all.part + split * all.size + g.part : nullptr;
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
        if (part)
          part[at] = acc[i][j][r];
        else if (F32OUT)
          static_cast<float*>(g.dw)[at] = all.accumulate ? static_cast<float*>(g.dw)[at] + acc[i][j][r] : acc[i][j][r];
        else
          static_cast<uint16_t*>(g.dw)[at] = Bf16::from_f32(acc[i][j][r]);
      }
    }
}

// The splits' partial sums added in order, one element per thread and turn (blockIdx.y: which
// gradient), four splits' loads on their way at a time.
template <bool F32OUT>
__global__ __launch_bounds__(256) void ffn_wgrad_join_kernel(WgradArgs all) {
  const Wgrad g = all.g[blockIdx.y];
  const int64_t size = static_cast<int64_t>(all.E) * g.M * g.N;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < size;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const float* from = all.part + g.part + i;
    float v = 0.0f;
    int32_t s = 0;
    for (; s + 4 <= all.splits; s += 4, from += 4 * all.size) {
      const float x0 = from[0], x1 = from[all.size], x2 = from[2 * all.size], x3 = from[3 * all.size];
      v = (((v + x0) + x1) + x2) + x3;
    }
    for (; s < all.splits; ++s, from += all.size) v += *from;
    if (F32OUT)
      static_cast<float*>(g.dw)[i] = all.accumulate ? static_cast<float*>(g.dw)[i] + v : v;
    else
      static_cast<uint16_t*>(g.dw)[i] = Bf16::from_f32(v);
  }
}

int64_t tiles_of(int64_t E, int64_t M, int64_t N, int64_t cols) {
  return E * ((M + kTile - 1) / kTile) * ((N + cols - 1) / cols);
}

// Splits of the tokens: where the outputs have fewer tiles (of 128 columns) than the card runs at
// once (three workgroups on each of 256 compute units), the tokens are cut so that more run, each
// with at least 8 stages of an even share.  A part writes and reads 64 KB, about 1/12 of a stage's
// time for each tile, so s parts of each of n tiles are least dear at s = sqrt(12 stages / n); no
// more are made, and up to a quarter less where that leaves the compute units more evenly filled.
// (Three weight gradients, against two workgroups a unit and no such bound: 8192 tokens, 1024 x 1024
// 106 -> 85 us; 1024 tokens, 1024 x 1024 34 -> 26; 65,536 tokens, 512 x 512 179 -> 165.)
constexpr int64_t kUnits = 256, kParts = 3 * kUnits;
int32_t wgrad_splits(int64_t T, int64_t E, int64_t tiles) {
  if (tiles < 1) tiles = 1;
  const int64_t stages = T / E / kStep;
  int64_t s = kParts / tiles;
  if (s > stages / 8) s = stages / 8;
  while (s > 1 && s * s * tiles > 12 * stages) --s;
  auto filled = [&](int64_t n) { return n * tiles * 100 / ((n * tiles + kUnits - 1) / kUnits * kUnits); };  // %
  int64_t best = s;
  for (int64_t n = s - 1; n >= 1 && 4 * n >= 3 * s; --n)
    if (filled(n) > filled(best)) best = n;
  return static_cast<int32_t>(best < 1 ? 1 : best);
}

struct Shape {
  int64_t M, N;
};

int check_wgrad(int64_t T, int64_t E, std::initializer_list<Shape> shapes, const char* what) {
  if (T < 0 || T > FP8Z1_FFN_MAX_ROWS) return refuse(FP8Z1_ESHAPE, what, "T outside 0 .. 2^30");
  if (E < 1 || E > FP8Z1_FFN_MAX_EXPERTS) return refuse(FP8Z1_ESHAPE, what, "E outside 1 .. 65535");
  int64_t tiles = 0;
  for (const Shape& s : shapes) {
    if (s.M < 1 || s.M > FP8Z1_FFN_MAX_WIDTH || s.N < 1 || s.N > FP8Z1_FFN_MAX_WIDTH)
      return refuse(FP8Z1_ESHAPE, what, "widths must be 1 .. 2^20");
    tiles += tiles_of(E, s.M, s.N, kTile);
  }
  if (tiles > 0x7fffffff) return refuse(FP8Z1_ESHAPE, what, "too many tiles");
  return FP8Z1_OK;
}

size_t workspace_for(int64_t T, int64_t E, std::initializer_list<Shape> shapes) {
  int64_t tiles = 0, size = 0;
  for (const Shape& s : shapes) {
    tiles += tiles_of(E, s.M, s.N, kTile);
    size += E * s.M * s.N;
  }
  const int32_t s = wgrad_splits(T, E, tiles);
  return s > 1 ? sizeof(float) * static_cast<size_t>(s) * size : 0;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

template <class H, bool F32OUT>
void launch_kernels(const WgradArgs& w, int nt, bool direct, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(w.tiles * w.splits)), block(kThreads);
  if (nt == 4)
    hipLaunchKernelGGL((ffn_wgrad_kernel<H, F32OUT, 4, true>), grid, block, 0, s, w);
  else if (direct)
    hipLaunchKernelGGL((ffn_wgrad_kernel<H, F32OUT, 2, true>), grid, block, 0, s, w);
  else
    hipLaunchKernelGGL((ffn_wgrad_kernel<H, F32OUT, 2, false>), grid, block, 0, s, w);
  if (!w.part) return;
  int64_t most = 0;
  for (int i = 0; i < w.count; ++i) {
    const int64_t n = static_cast<int64_t>(w.E) * w.g[i].M * w.g[i].N;
    most = most > n ? most : n;
  }
  const int64_t want = (most + 255) / 256;
  hipLaunchKernelGGL(ffn_wgrad_join_kernel<F32OUT>,
                     dim3(static_cast<unsigned>(want < 4096 ? want : 4096), static_cast<unsigned>(w.count)), block, 0, s,
                     w);
}

int launch_wgrad(int64_t T, int64_t E, int32_t dtype, const int32_t* offsets, int32_t dw_dtype, int32_t accumulate,
                 std::initializer_list<Wgrad> gs, void* workspace, size_t workspace_bytes, void* stream,
                 const char* what) {
  if (dtype != FP8Z1_BF16 && dtype != FP8Z1_F16)
    return refuse(FP8Z1_EINVAL, what, "dtype must be FP8Z1_BF16 or FP8Z1_F16");
  if (dw_dtype != FP8Z1_F32 && dw_dtype != FP8Z1_BF16)
    return refuse(FP8Z1_EINVAL, what, "dw_dtype must be FP8Z1_F32 or FP8Z1_BF16");
  if (accumulate && dw_dtype != FP8Z1_F32)
    return refuse(FP8Z1_EINVAL, what, "only FP8Z1_F32 gradients can be accumulated");
  if (!offsets && E != 1) return refuse(FP8Z1_EINVAL, what, "offsets may be NULL for one expert only");
  if (misaligned(offsets, 4) || misaligned(workspace, 4))
    return refuse(FP8Z1_EINVAL, what, "misaligned argument");
  bool direct = true;
  int64_t wide = 0, narrow = 0, size = 0;
  for (const Wgrad& g : gs) {
    if (!g.dw || (T && (!g.p || !g.q))) return refuse(FP8Z1_EINVAL, what, "NULL argument");
    if (misaligned(g.p, 2) || misaligned(g.q, 2) || misaligned(g.dw, dw_dtype == FP8Z1_F32 ? 4 : 2))
      return refuse(FP8Z1_EINVAL, what, "misaligned argument");
    direct = direct && g.M % 2 == 0 && g.N % 2 == 0 && !misaligned(g.p, 4) && !misaligned(g.q, 4);
    wide += tiles_of(E, g.M, g.N, 256);
    narrow += tiles_of(E, g.M, g.N, kTile);
    size += E * g.M * g.N;
  }
  // Columns of a tile: 256 where such tiles fill the card twice over (twice as many as the workgroups that
  // run at once, two on each of 256 compute units), else 128.  Rows of odd width go through registers, in
  // tiles of 128 (wider ones have not been tried).
  const int nt = direct && wide >= 2 * kSlots ? 4 : 2;
  WgradArgs w{};
  for (const Wgrad& g : gs) {
    Wgrad& to = w.g[w.count++];
    to = g;
    to.mt = (g.M + kTile - 1) / kTile;
    to.nt = (g.N + nt * 64 - 1) / (nt * 64);
    to.part = w.size;
    w.size += E * g.M * g.N;
  }
  w.offsets = offsets;
  w.T = static_cast<int32_t>(T);
  w.E = static_cast<int32_t>(E);
  w.tiles = static_cast<int32_t>(nt == 4 ? wide : narrow);
  w.accumulate = accumulate;
  w.splits = 1;
  const int32_t splits = wgrad_splits(T, E, narrow);
  if (splits > 1 && workspace && workspace_bytes >= sizeof(float) * static_cast<size_t>(splits) * size) {
    w.splits = splits;
    w.part = static_cast<float*>(workspace);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == FP8Z1_BF16 && dw_dtype == FP8Z1_F32)
    launch_kernels<Bf16, true>(w, nt, direct, s);
  else if (dtype == FP8Z1_BF16)
    launch_kernels<Bf16, false>(w, nt, direct, s);
  else if (dw_dtype == FP8Z1_F32)
    launch_kernels<F16, true>(w, nt, direct, s);
  else
    launch_kernels<F16, false>(w, nt, direct, s);
  return launched(what);
}

Wgrad gradient(const void* p, const void* q, void* dw, int64_t M, int64_t N) {
  Wgrad g{};
  g.p = static_cast<const uint8_t*>(p);
  g.q = static_cast<const uint8_t*>(q);
  g.dw = dw;
  g.M = static_cast<int32_t>(M);
  g.N = static_cast<int32_t>(N);
  return g;
}

}  // namespace
}  // namespace fp8z1

using namespace fp8z1;

extern "C" int fp8z1_ffn_wgrad_workspace_bytes(int64_t T, int64_t E, int64_t M, int64_t N, size_t* bytes) {
  if (!bytes) return refuse(FP8Z1_EINVAL, "ffn_wgrad_workspace_bytes", "NULL argument");
  const int rc = check_wgrad(T, E, {{M, N}}, "ffn_wgrad_workspace_bytes");
  if (rc) return rc;
  *bytes = workspace_for(T, E, {{M, N}});
  return FP8Z1_OK;
}

extern "C" int fp8z1_ffn_wgrad(int64_t T, int64_t E, int64_t M, int64_t N, int32_t dtype, const void* p, const void* q,
                               const int32_t* offsets, int32_t dw_dtype, void* dw, int32_t accumulate,
                               void* d_workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_wgrad(T, E, {{M, N}}, "ffn_wgrad");
  if (rc) return rc;
  return launch_wgrad(T, E, dtype, offsets, dw_dtype, accumulate, {gradient(p, q, dw, M, N)}, d_workspace,
                      workspace_bytes, stream, "ffn_wgrad");
}

extern "C" int fp8z1_ffn_bwd_weights_workspace_bytes(const fp8z1_ffn* f, size_t* bytes) {
  if (!f || !bytes) return refuse(FP8Z1_EINVAL, "ffn_bwd_weights_workspace_bytes", "NULL argument");
  const int rc = check_wgrad(f->T, f->E, {{f->F, f->D}, {f->F, f->D}, {f->D, f->F}}, "ffn_bwd_weights_workspace_bytes");
  if (rc) return rc;
  *bytes = workspace_for(f->T, f->E, {{f->F, f->D}, {f->F, f->D}, {f->D, f->F}});
  return FP8Z1_OK;
}

extern "C" int fp8z1_ffn_bwd_weights(const fp8z1_ffn* f, const void* x, const void* a, const void* dy, const void* dh,
                                     const void* du, const int32_t* offsets, int32_t dw_dtype, void* dw_gate,
                                     void* dw_up, void* dw_down, int32_t accumulate, void* d_workspace,
                                     size_t workspace_bytes, void* stream) {
  if (!f) return refuse(FP8Z1_EINVAL, "ffn_bwd_weights", "NULL description");
  const int rc = check_wgrad(f->T, f->E, {{f->F, f->D}, {f->F, f->D}, {f->D, f->F}}, "ffn_bwd_weights");
  if (rc) return rc;
  return launch_wgrad(f->T, f->E, f->dtype, offsets, dw_dtype, accumulate,
                      {gradient(dh, x, dw_gate, f->F, f->D), gradient(du, x, dw_up, f->F, f->D),
                       gradient(dy, a, dw_down, f->D, f->F)},
                      d_workspace, workspace_bytes, stream, "ffn_bwd_weights");
}
