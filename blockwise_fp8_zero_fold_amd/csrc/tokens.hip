// Tokens sorted by expert and back: the plan (each expert's first row, each choice's row), the rows copied
// to their places, and the rows weighted and summed in the tokens' order, with the gradients.
//   row_of[t][j] = offsets[e] + choices before (t, j) with the same expert e = experts[t][j]
//   rows[row_of[t][j]] = x[t]
//   y[t] = base[t] + sum_j w[t][j] rows[row_of[t][j]]                 (without w: the copy's gradient)
//   drows[row_of[t][j]] = w[t][j] dy[t],  dw[t][j] = sum_c dy[t][c] rows[row_of[t][j]][c]
// All but the plan are bound by HBM: each token's row is read once and its k rows are written (or read)
// once, by the token's own workgroup, so nothing is added to by two workgroups and no atomics are needed.
//
// 8192 tokens of 7168 in bfloat16 with 8 choices of 64 experts (a copy of 0.94 GB moves 4.9 to 5.75 TB/s here):
//   plan           9 us    two launches: 128 workgroups' counts, then the places (5 + 4)
//   dispatch     200 us    1.06 GB, 5.2 TB/s; rows in 8 bits with their scales 117 us, 0.55 GB, 4.7 TB/s
//   combine      217 us    1.06 GB, 4.9 TB/s
//   its gradient 387 us    2.0 GB, 5.15 TB/s
// Copying in the rows' order instead (each row looks its token up, and reads it again) took 217 to 290 us.
#include <hip/hip_runtime.h>

#include "device_util.h"
#include "ffn_refuse.h"
#include "rows.h"

namespace fp8z1 {
namespace {

// ---------------------------------------------------------------------------------------------- plan

// A stable counting sort.  A wave takes 64 choices at a time: the lanes with the same expert find each other
// by a ballot per bit of the expert's number, so a choice's rank among the wave's is a count of lower lanes,
// and the wave's counts so far are one LDS entry per expert, written by one of those lanes.  Waves and
// workgroups own consecutive choices; their counts are added in order.
constexpr int kSortWaves = 16, kSortThreads = 64 * kSortWaves;
constexpr int64_t kSortGroups = 256;  // most workgroups of a plan

struct SortArgs {
  const int32_t* experts;
  int32_t *offsets, *row_of, *counts;  // counts: [gridDim.x][E], or NULL with one workgroup
  int32_t n, E, bits, per;             // choices; per: of a wave
};

// The choices of this wave: ranks among the workgroup's choices of the same expert to row_of (-1: no expert),
// the workgroup's counts to `total` (LDS, [E]); `base` is LDS, [kSortWaves][E].
__device__ __forceinline__ void rank_choices(const SortArgs& a, int32_t* base, int32_t* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int32_t i = threadIdx.x; i < kSortWaves * a.E; i += kSortThreads) base[i] = 0;
  __syncthreads();
  const int32_t begin = static_cast<int32_t>(blockIdx.x * kSortWaves + w) * a.per;
  int32_t* const count = base + w * a.E;
  for (int32_t i0 = 0; i0 < a.per; i0 += 64) {
    const int32_t i = begin + i0 + lane;
    int32_t e = i < a.n ? a.experts[i] : -1;
    if (e < 0 || e >= a.E) e = -1;
    uint64_t same = __ballot(e >= 0);
    for (int32_t b = 0; b < a.bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    int32_t rank = -1;
    if (e >= 0) {
      const int before = __popcll(same & ((1ull << lane) - 1));
      rank = count[e] + before;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (before == 0) count[e] = rank + __popcll(same);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (i < a.n) a.row_of[i] = rank;
  }
  __syncthreads();
  // counts of the waves before
  for (int32_t e = threadIdx.x; e < a.E; e += kSortThreads) {
    int32_t sum = 0;
    for (int k = 0; k < kSortWaves; ++k) {
      const int32_t c = base[k * a.E + e];
      base[k * a.E + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
  __syncthreads();
}

// total[e] -> sum of those before e (all threads of the workgroup); E <= kSortThreads.  Returns the whole sum.
__device__ __forceinline__ int32_t before_each(int32_t* total, int32_t E, int32_t* lds) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int32_t mine = static_cast<int32_t>(threadIdx.x) < E ? total[threadIdx.x] : 0;
  int32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t v = __shfl_up(upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 63) lds[w] = upto;
  __syncthreads();
  int32_t before = 0, sum = 0;
  for (int k = 0; k < kSortWaves; ++k) {
    if (k < w) before += lds[k];
    sum += lds[k];
  }
  if (static_cast<int32_t>(threadIdx.x) < E) total[threadIdx.x] = before + upto - mine;
  __syncthreads();
  return sum;
}

// rank among the workgroup -> row: the expert's first row, and the choices of the workgroups and waves before
__device__ __forceinline__ void place_choices(const SortArgs& a, const int32_t* base, const int32_t* first) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int32_t begin = static_cast<int32_t>(blockIdx.x * kSortWaves + w) * a.per;
  for (int32_t i0 = 0; i0 < a.per; i0 += 64) {
    const int32_t i = begin + i0 + lane;
    if (i >= a.n) break;
    const int32_t rank = a.row_of[i];
    if (rank >= 0) {
      const int32_t e = a.experts[i];
      a.row_of[i] = rank + first[e] + base[w * a.E + e];
    }
  }
}

// One workgroup: the whole plan.  Several: their counts, and ranks within a workgroup.
__global__ __launch_bounds__(kSortThreads) void sort_kernel(SortArgs a) {
  extern __shared__ int32_t lds[];
  int32_t *const base = lds, *const total = lds + kSortWaves * a.E, *const sums = total + a.E;
  rank_choices(a, base, total);
  if (a.counts) {
    // (ranks within the workgroup: the waves before are added here, the rest by the second launch)
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int32_t begin = static_cast<int32_t>(blockIdx.x * kSortWaves + w) * a.per;
    for (int32_t i0 = 0; i0 < a.per; i0 += 64) {
      const int32_t i = begin + i0 + lane;
      if (i >= a.n) break;
      const int32_t rank = a.row_of[i];
      if (rank >= 0) a.row_of[i] = rank + base[w * a.E + a.experts[i]];
    }
    for (int32_t e = threadIdx.x; e < a.E; e += kSortThreads)
      a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = total[e];
    return;
  }
  const int32_t all = before_each(total, a.E, sums);
  for (int32_t e = threadIdx.x; e <= a.E; e += kSortThreads) a.offsets[e] = e < a.E ? total[e] : all;
  place_choices(a, base, total);
}

// The workgroups' counts added up: before this one to `first`, and over all
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  extern __shared__ int32_t lds[];
  int32_t *const first = lds, *const sums = lds + a.E;
  const int32_t groups = gridDim.x;
  int32_t before = 0, sum = 0;
  const int32_t e = threadIdx.x;
  if (e < a.E) {
#pragma unroll 8
    for (int32_t g = 0; g < groups; ++g) {
      const int32_t c = a.counts[static_cast<int64_t>(g) * a.E + e];
      before += g < static_cast<int32_t>(blockIdx.x) ? c : 0;
      sum += c;
    }
    first[e] = sum;
  }
  __syncthreads();
  const int32_t all = before_each(first, a.E, sums);
  if (blockIdx.x == 0)
    for (int32_t i = threadIdx.x; i <= a.E; i += kSortThreads) a.offsets[i] = i < a.E ? first[i] : all;
  __syncthreads();
  if (e < a.E) first[e] += before;
  __syncthreads();
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * kSortWaves * a.per;
  const int64_t end = min(begin + static_cast<int64_t>(kSortWaves) * a.per, static_cast<int64_t>(a.n));
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const int32_t rank = a.row_of[i];
    if (rank >= 0) a.row_of[i] = rank + first[a.experts[i]];
  }
}

// Choices of a wave, and workgroups.  A workgroup's 16 waves take 64 choices each while that gives no more
// than kSortGroups workgroups.
int64_t sort_per_wave(int64_t n) {
  const int64_t per = (n + kSortGroups * kSortWaves - 1) / (kSortGroups * kSortWaves);
  return (per + 63) / 64 * 64;
}
constexpr int64_t kSortOneGroup = 4096;  // most choices that one workgroup places by itself
int64_t sort_groups(int64_t n) {
  if (n <= kSortOneGroup) return 1;
  const int64_t per = sort_per_wave(n) * kSortWaves;
  return (n + per - 1) / per;
}

// ---------------------------------------------------------------------------------------------- rows

struct RowsArgs {
  const int32_t* row_of;
  const void *x, *dy, *base;
  const float *scales, *weights;
  void *rows, *y;
  float *row_scales, *dweights;
  int64_t D, R;
  int32_t T, k;
  int32_t blocks;  // workgroups of a token (dispatch, combine)
  int32_t chunks;  // 16-byte chunks of a thread (dispatch)
  int64_t items;   // workgroups that all tokens need; where a launch has fewer, they take several each
};

// The row of choice j of token t, -1 where it has none among the R there are
__device__ __forceinline__ int64_t row_at(const RowsArgs& a, int32_t t, int32_t j) {
  const int32_t r = a.row_of[static_cast<int64_t>(t) * a.k + j];
  return r >= 0 && r < a.R ? r : -1;
}

typedef uint32_t v4u_a1_rw_global_t __attribute__((ext_vector_type(4), aligned(1), address_space(1)));

// A token's row of `bytes` to its k places: up to 4 chunks of 16 bytes per thread at any alignment, all loads before
// the stores; the last chunk overlaps the one before it (the same bytes twice).  Rows of less than 16 go byte by byte.
// Stores carry no hint: what follows reads the rows.
constexpr int kCopyThreads = 256, kCopyChunks = 4;
__device__ __forceinline__ void copy_rows(const RowsArgs& a, int32_t t, const uint8_t* x, uint8_t* rows, int64_t bytes,
                                          int64_t first, int64_t step) {
  const uint8_t* const from = x + t * bytes;
  if (bytes < 16) {
    if (first >= 16 * bytes) return;
    for (int32_t j = 0; j < a.k; ++j) {
      const int64_t r = row_at(a, t, j);
      if (r >= 0) rows[r * bytes + first / 16] = from[first / 16];
    }
    return;
  }
  uint4 v[kCopyChunks];
  int64_t at[kCopyChunks];
#pragma unroll
  for (int i = 0; i < kCopyChunks; ++i) {
    const int64_t c = first + i * step;
    at[i] = c < bytes ? min(c, bytes - 16) : -1;
    if (at[i] >= 0) v[i] = ld16(from + at[i]);
  }
  for (int32_t j = 0; j < a.k; ++j) {
    const int64_t r = row_at(a, t, j);
    if (r < 0) continue;
#pragma unroll
    for (int i = 0; i < kCopyChunks; ++i)
      if (at[i] >= 0) *(v4u_a1_rw_global_t*)(rows + r * bytes + at[i]) = v4u_v_t{v[i].x, v[i].y, v[i].z, v[i].w};
  }
}

// ELEM: bytes of an element.  EIGHT: the scales' rows too, by the last workgroup of a token.
template <int ELEM, bool EIGHT>
__global__ __launch_bounds__(kCopyThreads) void dispatch_kernel(RowsArgs a) {
  constexpr int64_t kTurn = kCopyThreads * 16;
  for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int32_t t = static_cast<int32_t>(item / a.blocks), b = static_cast<int32_t>(item % a.blocks);
    copy_rows(a, t, static_cast<const uint8_t*>(a.x), static_cast<uint8_t*>(a.rows), a.D * ELEM,
              b * a.chunks * kTurn + threadIdx.x * 16, a.chunks > 1 ? kTurn : kTurn << 32);
    if (EIGHT && b == a.blocks - 1) {
      const int64_t n = (a.D + kB - 1) / kB * 4;
      for (int64_t i = threadIdx.x * 16; i < max(n, static_cast<int64_t>(256)); i += kCopyChunks * kTurn)
        copy_rows(a, t, reinterpret_cast<const uint8_t*>(a.scales), reinterpret_cast<uint8_t*>(a.row_scales), n, i, kTurn);
    }
  }
}

// 8 columns per thread; the rows of up to kAhead choices are on their way at once
constexpr int kAhead = 8;
// KNOWN: the workgroup's threads are all of one token, and rows are whole chunks of 8 columns: nothing stands between
// the loads.
template <class H>
__device__ __forceinline__ Raw8<H> fetch_whole8(const void* row, int32_t c) {
  typedef typename Elem<H>::type E;
  Raw8<H> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(E)) * 8 / 16; ++i)
    r.x[i] = ((const v4u_a2_global_t*)(static_cast<const E*>(row) + c))[i];
  return r;
}
template <class H, bool WEIGHTED, bool KNOWN>
__device__ __forceinline__ void combine_chunk(const RowsArgs& a, int32_t t, int32_t C, int32_t c) {
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  if (a.base) load8<H>(row_of<H>(a.base, t, C), C, c, sum);
  for (int32_t j0 = 0; j0 < a.k; j0 += kAhead) {
    Raw8<H> v[kAhead];
    float w[kAhead];
    int32_t r[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      r[j] = j0 + j < a.k ? static_cast<int32_t>(row_at(a, t, j0 + j)) : -1;
      w[j] = WEIGHTED && r[j] >= 0 ? a.weights[static_cast<int64_t>(t) * a.k + j0 + j] : 1.0f;
      if (KNOWN) {
        r[j] = __builtin_amdgcn_readfirstlane(r[j]);
        w[j] = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(w[j])));
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (r[j] >= 0) {
        const void* const row = row_of<H>(static_cast<const void*>(a.rows), r[j], C);
        v[j] = KNOWN ? fetch_whole8<H>(row, c) : fetch8<H>(row, C, c);
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (r[j] < 0) continue;
      float x[8];
      widen8f<H>(v[j], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = WEIGHTED ? fmaf(w[j], x[i], sum[i]) : sum[i] + x[i];
    }
  }
  store8<H>(row_of<H>(a.y, t, C), C, c, sum);
}

template <class H, bool WEIGHTED, bool KNOWN>
__global__ __launch_bounds__(512) void combine_kernel(RowsArgs a, int32_t per) {
  // `per` threads take a token's (part of a) row, so several short rows share a workgroup
  const int32_t sub = KNOWN ? 0 : static_cast<int32_t>(threadIdx.x) / per;
  const int32_t in = static_cast<int32_t>(threadIdx.x) - sub * per, tokens = KNOWN ? 1 : blockDim.x / per;
  const int32_t C = static_cast<int32_t>(a.D);
  if (sub >= tokens) return;
  for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int64_t t = item / a.blocks * tokens + sub;
    const int32_t c = (static_cast<int32_t>(item % a.blocks) * per + in) * 8;
    if (t < a.T && c < C) combine_chunk<H, WEIGHTED, KNOWN>(a, static_cast<int32_t>(t), C, c);
  }
}

// A workgroup (of as many waves as a row fills, at most 16) per token; dw's sums over the row by wave, then
// over the waves in order.
template <class H>
__global__ __launch_bounds__(1024) void combine_bwd_kernel(RowsArgs a) {
  __shared__ float lds[16][kAhead];
  const int32_t C = static_cast<int32_t>(a.D), parts = (a.k + kAhead - 1) / kAhead;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int32_t t = static_cast<int32_t>(item / parts), j0 = static_cast<int32_t>(item % parts) * kAhead;
    int64_t r[kAhead];
    float wt[kAhead], dot[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      dot[j] = 0.0f;
      r[j] = j0 + j < a.k ? row_at(a, t, j0 + j) : -1;
      wt[j] = r[j] >= 0 ? a.weights[static_cast<int64_t>(t) * a.k + j0 + j] : 0.0f;
    }
    for (int32_t c = threadIdx.x * 8; c < C; c += blockDim.x * 8) {
      float dy[8];
      load8<H>(row_of<H>(a.dy, t, C), C, c, dy);
      Raw8<H> v[kAhead];
      if (a.dweights) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (r[j] >= 0) v[j] = fetch8<H>(row_of<H>(a.x, r[j], C), C, c);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (r[j] < 0) continue;
        if (a.rows) {
          float d[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = wt[j] * dy[i];
          store8<H>(row_of<H>(a.rows, r[j], C), C, c, d);
        }
        if (a.dweights) {
          float x[8];
          widen8f<H>(v[j], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[j] = fmaf(dy[i], x[i], dot[j]);
        }
      }
    }
    if (!a.dweights) continue;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) dot[j] = wave_fsum(dot[j]);
    if (lane == 0)
#pragma unroll
      for (int j = 0; j < kAhead; ++j) lds[w][j] = dot[j];
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < kAhead && j0 + static_cast<int>(threadIdx.x) < a.k) {
      float sum = 0.0f;
      for (int k = 0; k < waves; ++k) sum += lds[k][threadIdx.x];
      a.dweights[static_cast<int64_t>(t) * a.k + j0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

int elem_size(int32_t dtype) { return dtype == FP8Z1_F32 ? 4 : dtype == FP8Z1_E4M3 ? 1 : 2; }

int check_routed(const fp8z1_routed* f, const int32_t* row_of, bool eight, const char* what) {
  if (!f) return refuse(FP8Z1_EINVAL, what, "NULL description");
  if (f->dtype != FP8Z1_F32 && f->dtype != FP8Z1_BF16 && f->dtype != FP8Z1_F16 && !(eight && f->dtype == FP8Z1_E4M3))
    return refuse(FP8Z1_EINVAL, what, eight ? "dtype must be FP8Z1_BF16, FP8Z1_F16, FP8Z1_F32 or FP8Z1_E4M3"
                                            : "dtype must be FP8Z1_BF16, FP8Z1_F16 or FP8Z1_F32");
  if (f->T < 0 || f->T > FP8Z1_FFN_MAX_ROWS) return refuse(FP8Z1_ESHAPE, what, "T outside 0 .. 2^30");
  if (f->k < 1 || f->k > FP8Z1_ROUTE_MAX_CHOICES) return refuse(FP8Z1_ESHAPE, what, "k outside 1 .. 32");
  if (f->D < 1 || f->D > FP8Z1_FFN_MAX_WIDTH) return refuse(FP8Z1_ESHAPE, what, "D must be 1 .. 2^20");
  if (f->R < 0 || f->R > FP8Z1_FFN_MAX_ROWS) return refuse(FP8Z1_ESHAPE, what, "R outside 0 .. 2^30");
  if (f->T && !row_of) return refuse(FP8Z1_EINVAL, what, "NULL row_of");
  if (misaligned(row_of, 4)) return refuse(FP8Z1_EINVAL, what, "misaligned row_of");
  return FP8Z1_OK;
}

RowsArgs base_args(const fp8z1_routed* f, const int32_t* row_of) {
  RowsArgs a{};
  a.row_of = row_of;
  a.D = f->D;
  a.R = f->R;
  a.T = static_cast<int32_t>(f->T);
  a.k = f->k;
  return a;
}

// most workgroups of a launch (of up to 1024 threads, whose number has 32 bits)
constexpr int64_t kMostGroups = 1 << 21;
dim3 groups_of(const RowsArgs& a) { return dim3(static_cast<unsigned>(a.items < kMostGroups ? a.items : kMostGroups)); }

}  // namespace
}  // namespace fp8z1

using namespace fp8z1;

extern "C" int fp8z1_sort_tokens_workspace_bytes(int64_t T, int32_t k, int32_t E, size_t* bytes) {
  const char* what = "sort_tokens_workspace_bytes";
  if (!bytes) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  if (T < 0 || T > FP8Z1_FFN_MAX_ROWS) return refuse(FP8Z1_ESHAPE, what, "T outside 0 .. 2^30");
  if (k < 1 || k > FP8Z1_ROUTE_MAX_CHOICES || T * k > FP8Z1_FFN_MAX_ROWS)
    return refuse(FP8Z1_ESHAPE, what, "k outside 1 .. 32, or more than 2^30 choices");
  if (E < 1 || E > FP8Z1_ROUTE_MAX_EXPERTS) return refuse(FP8Z1_ESHAPE, what, "E outside 1 .. 1024");
  const int64_t groups = sort_groups(T * k);
  *bytes = groups > 1 ? sizeof(int32_t) * static_cast<size_t>(groups) * static_cast<size_t>(E) : 0;
  return FP8Z1_OK;
}

extern "C" int fp8z1_sort_tokens(int64_t T, int32_t k, int32_t E, const int32_t* experts, int32_t* offsets,
                                 int32_t* row_of, void* d_workspace, size_t workspace_bytes, void* stream) {
  const char* what = "sort_tokens";
  size_t need = 0;
  const int rc = fp8z1_sort_tokens_workspace_bytes(T, k, E, &need);
  if (rc) return rc;
  if (!offsets || (T && (!experts || !row_of))) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  if (misaligned(experts, 4) || misaligned(offsets, 4) || misaligned(row_of, 4))
    return refuse(FP8Z1_EINVAL, what, "misaligned argument");
  if (need && (!d_workspace || workspace_bytes < need)) return refuse(FP8Z1_EINVAL, what, "workspace too small");
  if (need && misaligned(d_workspace, 16)) return refuse(FP8Z1_EINVAL, what, "misaligned workspace");
  SortArgs a{};
  a.experts = experts;
  a.offsets = offsets;
  a.row_of = row_of;
  a.n = static_cast<int32_t>(T * k);
  a.E = E;
  while ((1 << a.bits) < E) ++a.bits;
  const int64_t groups = sort_groups(a.n);
  a.per = static_cast<int32_t>(groups > 1 ? sort_per_wave(a.n) : (a.n + kSortThreads - 1) / kSortThreads * 64);
  a.counts = groups > 1 ? static_cast<int32_t*>(d_workspace) : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 g(static_cast<unsigned>(groups)), b(kSortThreads);
  hipLaunchKernelGGL(sort_kernel, g, b, sizeof(int32_t) * ((kSortWaves + 1) * E + kSortWaves), s, a);
  if (groups > 1) hipLaunchKernelGGL(sort_place_kernel, g, b, sizeof(int32_t) * (E + kSortWaves), s, a);
  return launched(what);
}

extern "C" int fp8z1_dispatch(const fp8z1_routed* f, const int32_t* row_of, const void* x, const float* scales, void* rows,
                              float* row_scales, void* stream) {
  const char* what = "dispatch";
  const int rc = check_routed(f, row_of, true, what);
  if (rc) return rc;
  const bool eight = f->dtype == FP8Z1_E4M3;
  if (!eight && (scales || row_scales)) return refuse(FP8Z1_EINVAL, what, "scales belong to FP8Z1_E4M3 rows");
  if (f->T == 0 || f->R == 0) return FP8Z1_OK;
  if (!x || !rows || (eight && (!scales || !row_scales))) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  if (misaligned(x, elem_size(f->dtype)) || misaligned(rows, elem_size(f->dtype)) || misaligned(scales, 4) ||
      misaligned(row_scales, 4))
    return refuse(FP8Z1_EINVAL, what, "misaligned argument");
  RowsArgs a = base_args(f, row_of);
  a.x = x;
  a.scales = scales;
  a.rows = rows;
  a.row_scales = row_scales;
  // many tokens: 4 chunks a thread (8192 tokens of 7168, 8 choices: 200 us, 221 with one); few: a chunk each, on more
  // compute units
  a.chunks = f->T >= 512 ? kCopyChunks : 1;
  const int64_t per = kCopyThreads * 16 * a.chunks;
  a.blocks = static_cast<int32_t>((f->D * elem_size(f->dtype) + per - 1) / per);
  a.items = f->T * a.blocks;
  const dim3 g = groups_of(a), b(kCopyThreads);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (eight)
    hipLaunchKernelGGL((dispatch_kernel<1, true>), g, b, 0, s, a);
  else if (f->dtype == FP8Z1_F32)
    hipLaunchKernelGGL((dispatch_kernel<4, false>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((dispatch_kernel<2, false>), g, b, 0, s, a);
  return launched(what);
}

namespace fp8z1 {
namespace {

template <class H, bool WEIGHTED>
void launch_combine_as(const RowsArgs& a, dim3 g, dim3 b, int32_t per, hipStream_t s) {
  if (static_cast<int32_t>(b.x) == per && a.D % 8 == 0)
    hipLaunchKernelGGL((combine_kernel<H, WEIGHTED, true>), g, b, 0, s, a, per);
  else
    hipLaunchKernelGGL((combine_kernel<H, WEIGHTED, false>), g, b, 0, s, a, per);
}
template <class H>
void launch_combine(const RowsArgs& a, dim3 g, dim3 b, int32_t per, hipStream_t s) {
  if (a.weights)
    launch_combine_as<H, true>(a, g, b, per, s);
  else
    launch_combine_as<H, false>(a, g, b, per, s);
}

}  // namespace
}  // namespace fp8z1

extern "C" int fp8z1_combine(const fp8z1_routed* f, const int32_t* row_of, const void* rows, const float* weights,
                             const void* base, void* y, void* stream) {
  const char* what = "combine";
  const int rc = check_routed(f, row_of, false, what);
  if (rc) return rc;
  if (f->T == 0) return FP8Z1_OK;
  if ((f->R && !rows) || !y) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  const size_t el = elem_size(f->dtype);
  if (misaligned(rows, el) || misaligned(y, el) || misaligned(base, el) || misaligned(weights, 4))
    return refuse(FP8Z1_EINVAL, what, "misaligned argument");
  RowsArgs a = base_args(f, row_of);
  a.rows = const_cast<void*>(rows);
  a.weights = weights;
  a.base = base;
  a.y = y;
  // the chunks of 8 columns of a row, in workgroups of as many waves each; short rows share one
  const int64_t chunks = (f->D + 7) / 8;
  a.blocks = static_cast<int32_t>((chunks + 511) / 512);
  int64_t per = (chunks + a.blocks - 1) / a.blocks, threads = (per + 63) / 64 * 64, tokens = 1;
  if (per < 64) {
    tokens = 256 / per;
    threads = 256;
  } else {
    per = threads;
  }
  a.items = (f->T + tokens - 1) / tokens * a.blocks;
  const dim3 g = groups_of(a), b(static_cast<unsigned>(threads));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int32_t p = static_cast<int32_t>(per);
  if (f->dtype == FP8Z1_F32)
    launch_combine<F32>(a, g, b, p, s);
  else if (f->dtype == FP8Z1_BF16)
    launch_combine<Bf16>(a, g, b, p, s);
  else
    launch_combine<F16>(a, g, b, p, s);
  return launched(what);
}

extern "C" int fp8z1_combine_bwd(const fp8z1_routed* f, const int32_t* row_of, const void* dy, const void* rows,
                                 const float* weights, void* drows, float* dweights, void* stream) {
  const char* what = "combine_bwd";
  const int rc = check_routed(f, row_of, false, what);
  if (rc) return rc;
  if (!drows && !dweights) return refuse(FP8Z1_EINVAL, what, "no gradient is wanted");
  if (f->T == 0) return FP8Z1_OK;
  if (!dy || !weights || (f->R && dweights && !rows)) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  const size_t el = elem_size(f->dtype);
  if (misaligned(rows, el) || misaligned(dy, el) || misaligned(drows, el) || misaligned(weights, 4) ||
      misaligned(dweights, 4))
    return refuse(FP8Z1_EINVAL, what, "misaligned argument");
  RowsArgs a = base_args(f, row_of);
  a.dy = dy;
  a.x = rows;
  a.weights = weights;
  a.rows = drows;
  a.dweights = dweights;
  const int64_t waves = (f->D + 511) / 512, threads = 64 * (waves < 16 ? waves : 16);
  a.items = f->T * ((f->k + kAhead - 1) / kAhead);
  const dim3 g = groups_of(a), b(static_cast<unsigned>(threads));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (f->dtype == FP8Z1_F32)
    hipLaunchKernelGGL((combine_bwd_kernel<F32>), g, b, 0, s, a);
  else if (f->dtype == FP8Z1_BF16)
    hipLaunchKernelGGL((combine_bwd_kernel<Bf16>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((combine_bwd_kernel<F16>), g, b, 0, s, a);
  return launched(what);
}
