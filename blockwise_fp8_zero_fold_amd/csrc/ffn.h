// Shared by the feed-forward kernels: arguments, expert ranges, the gated activation.
#pragma once

#include "device_util.h"
#include "ffn_refuse.h"
#include "mfma.h"

namespace fp8z1 {

template <int N>
struct Int {
  static constexpr int value = N;
};

enum FfnKind {
  kFfnUp = 0,       // a = act(x Wg^T) * (x Wu^T)
  kFfnDown = 1,     // y = a Wd^T
  kFfnDownBwd = 2,  // da = dy Wd, then dh, du (and a) from da, h, u
  kFfnUpBwd = 3,    // dx = dh Wg + du Wu
  kLinear = 4,      // y = res + act(x W^T + bias)
  kLinearBwd = 5    // dx = dp W
};

struct FfnArgs {
  const uint8_t *x0, *x1;  // 16-bit rows [T, K] (x1: du of kFfnUpBwd)
  const uint8_t *w0, *w1;  // codes: [E, N, K] (forward) or [E, K, N]
  const float *s0, *s1;    // their block scales
  const int32_t* offsets;  // [E + 1], or NULL: one expert, all rows
  const uint16_t *h, *u;   // [T, N] inputs of kFfnDownBwd
  uint16_t *o0, *o1, *o2;  // outputs [T, N]
  const float* bias;       // [E, N] (kLinear; NULL: 0)
  const uint16_t* res;     // [T, N] (kLinear; NULL: 0)
  const float* xs;         // x0 in 8 bits: its scales [T, blocks of K]
  uint8_t* codes;          // kFfnUp of 8-bit rows: a in 8 bits [T, N]
  float* code_scales;      // [T, blocks of N]
  int32_t pow2;            // their rule
  float* part;             // partial sums of split tiles, or NULL: no tile is split
  int32_t T, E, N, K, act;
  int32_t split_from;  // sums of at least so many scale blocks may be split
};

// y = res + act(x W^T + bias) of rows in 8 bits (checked arguments), and the workspace that it can use
int linear8(const FfnArgs& p, int32_t dtype, void* workspace, size_t workspace_bytes, hipStream_t s, const char* what);
size_t linear8_workspace(int64_t T, int64_t E, int64_t N, int64_t K);

// Rows of expert e, kept inside [0, T] whatever the offsets hold, so a wrong
// offset gives wrong rows but no access out of bounds.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int32_t T, int32_t e, int32_t& lo, int32_t& hi) {
  lo = 0;
  hi = T;
  if (offsets) {
    lo = min(max(offsets[e], 0), T);
    hi = min(max(offsets[e + 1], lo), T);
  }
}

// Rows in groups of ROWS for launches that give each group a workgroup of its own.  Group e < E is the
// first of expert e, as one would number them if no expert had more.  The others follow: expert e
// has the numbers E + rows_before / ROWS and on, as many as its rows can need (one may be over), so that a
// group's expert is the last whose first number is not above it, and E + T / ROWS groups are enough.
// A wave looks for it 64 experts at a time (a step per power of 64).  False: the group has no rows;
// also for offsets out of order, which give wrong rows but no access out of bounds.
template <int ROWS>
__device__ __forceinline__ bool find_group(const int32_t* offsets, int32_t T, int32_t E, int32_t group, int32_t& e,
                                           int32_t& lo, int32_t& hi, int32_t& t0) {
  if (group < E) {
    e = group;
    expert_rows(offsets, T, e, lo, hi);
    t0 = lo;
    return t0 < hi;
  }
  group -= E;
  e = 0;
  lo = 0;
  hi = T;
  if (offsets) {
    const int lane = threadIdx.x & 63;
    int32_t stride = 1;
    while (static_cast<int64_t>(stride) * 64 < E) stride *= 64;
    for (; stride > 0; stride /= 64) {
      const int32_t at = min(e + lane * stride, E - 1);
      int32_t from, to;
      expert_rows(offsets, T, at, from, to);
      const uint64_t upto = __ballot(e + lane * stride < E && from / ROWS <= group);
      const int last = upto ? 63 - __builtin_clzll(upto) : 0;
      e = __builtin_amdgcn_readfirstlane(e + last * stride);
      lo = __builtin_amdgcn_readlane(from, last);  // (of expert e once the stride is 1)
      hi = __builtin_amdgcn_readlane(to, last);
    }
  }
  const int32_t past = group - lo / ROWS + 1;  // groups of this expert before it
  t0 = lo + past * ROWS;
  return past >= 1 && past <= (hi - lo) / ROWS && t0 < hi;
}

// Sums over this lane and those before it, by lane moves within rows of 16 and from a row's last
// lane on (through LDS, as shuffles go, the sum's six steps take 0.3 us of a launch)
__device__ __forceinline__ int32_t wave_upto(int32_t v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // 1, 2, 4, 8 lanes up the row
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 of rows 0 and 2 to the next row
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2 and 3
  return v;
}

// Work items of a launch.  The tiles (row tiles of all experts by tile columns) are counted on
// the device, which alone knows the offsets; the grid holds the most there can be.
// The card runs kSlots workgroups at once (two on each compute unit).  Where the tiles
// past the last full round would leave most of it idle, they are split along k instead into
// `splits` parts each, the parts' float32 sums go to the workspace and a second kernel
// (some 5 us) adds them in order and finishes the tiles.  A part is at least 8 scale
// blocks of k behind full rounds, and 2 where there is no full round; sums of less than
// split_from blocks are not split: 8 with direct copies (a block takes about 1 us), 4
// through registers (twice that).  A part also writes and reads 64 KB, so that s parts of each
// of n tiles cost about blocks / s + n s / 80 us: with direct copies no more than the s where
// that is least, sqrt(80 blocks / n).  (512 tokens, 1024 x 4096, forward: 48 us without this
// bound, 36 with it; 1024 tokens on 8 experts, 2048 x 1024: 52 and 48; 1024 tokens, 7168 x 2048:
// 129 and 126; through registers, where a block takes longer, it cost up to 9 %.)
constexpr int32_t kSlots = 512;
constexpr int32_t kDirectFrom = 8, kRegisterFrom = 4;  // split_from

__host__ __device__ __forceinline__ int32_t tile_splits(int64_t tiles, int32_t blocks, int32_t from) {
  const int32_t rest = static_cast<int32_t>(tiles % kSlots);
  if (!rest || !from || blocks < from) return 1;
  int32_t s = kSlots / rest, most = blocks / (tiles < kSlots ? 2 : 8);
  if (tiles < kSlots && from == kDirectFrom) {
    const int32_t least = static_cast<int32_t>(sqrtf(80.0f * static_cast<float>(blocks) / static_cast<float>(rest)));
    most = least < most ? least : most;
  }
  if (s > most) s = most;
  return s > 1 ? s : 1;
}

struct Plan {
  int32_t tiles;   // all tiles
  int32_t whole;   // tiles done by one workgroup; the others by `splits`
  int32_t splits;
  __device__ int64_t items() const { return whole + static_cast<int64_t>(tiles - whole) * splits; }
};

// Rows and row tiles of an expert, and the tiles of the 64 that lanes hold up to and with its own
struct Run {
  int32_t lo, hi, tiles, upto;
};
template <int ROWS>
__device__ __forceinline__ Run run_of(const int32_t* offsets, int32_t T, int32_t E, int32_t e) {
  Run r = {0, 0, 0, 0};
  if (e < E) {
    expert_rows(offsets, T, e, r.lo, r.hi);
    r.tiles = (r.hi - r.lo + ROWS - 1) / ROWS;
  }
  r.upto = wave_upto(r.tiles);
  return r;
}

// `first`: the run of expert `lane`, for find_tile
template <int ROWS>
__device__ __forceinline__ Plan plan_tiles(const int32_t* offsets, int32_t T, int32_t E, int32_t ncols, int32_t blocks,
                                           int32_t split_from, int32_t& rowtiles, Run& first) {
  const int lane = threadIdx.x & 63;
  first = run_of<ROWS>(offsets, T, E, lane);
  int32_t total;
  if (offsets) {
    total = __builtin_amdgcn_readlane(first.upto, 63);
    for (int32_t e0 = 64; e0 < E; e0 += 64)
      total += __builtin_amdgcn_readlane(run_of<ROWS>(offsets, T, E, e0 + lane).upto, 63);
  } else {
    total = (T + ROWS - 1) / ROWS;
  }
  rowtiles = __builtin_amdgcn_readfirstlane(total);
  Plan p;
  // (offsets out of order can count rows twice: no more tiles than an int can number)
  p.tiles = static_cast<int32_t>(min(static_cast<int64_t>(rowtiles) * ncols, static_cast<int64_t>(0x7fffffff)));
  p.whole = p.tiles;
  p.splits = 1;
  const int32_t rest = p.tiles % kSlots;
  const int32_t s = tile_splits(p.tiles, blocks, split_from);
  if (s > 1) {
    p.whole = p.tiles - rest;
    p.splits = s;
  }
  return p;
}

// Consecutive workgroups go to the XCDs in turn; item b of n becomes a tile so that each
// XCD gets a contiguous run of them.
__device__ __forceinline__ int32_t xcd_run(int32_t b, int32_t n) {
  const int32_t x = b % kXcds;
  return x * (n / kXcds) + min(x, n % kXcds) + b / kXcds;
}

// Tile id -> expert, its rows lo..hi, first row m0 and tile column.  Tiles are ordered in
// groups of kGroup row tiles by all columns, so that the tiles running on one XCD at a
// time share rows and weights in its L2.
constexpr int kGroup = 8;
template <int ROWS>
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int32_t T, int32_t E, int32_t ncols, int32_t rowtiles,
                                          const Run& first, int32_t id, int32_t& e, int32_t& lo, int32_t& hi, int32_t& m0,
                                          int32_t& col) {
  const int lane = threadIdx.x & 63;
  const int32_t grp = id / (kGroup * ncols), in = id - grp * kGroup * ncols;
  const int32_t rows = min(kGroup, rowtiles - grp * kGroup);
  col = in / rows;
  int32_t mt = grp * kGroup + in - col * rows;
  e = 0;
  lo = 0;
  hi = T;
  if (offsets) {
    for (int32_t e0 = 0; e0 < E; e0 += 64) {
      const Run run = e0 == 0 ? first : run_of<ROWS>(offsets, T, E, e0 + lane);
      const int32_t upto = run.upto;
      const uint64_t past = __ballot(upto > mt);
      if (past) {
        const int at = __builtin_ctzll(past);
        e = e0 + at;
        mt -= __builtin_amdgcn_readlane(upto - run.tiles, at);
        lo = __builtin_amdgcn_readlane(run.lo, at);
        hi = __builtin_amdgcn_readlane(run.hi, at);
        break;
      }
      mt -= __builtin_amdgcn_readlane(upto, 63);
    }
  }
  e = __builtin_amdgcn_readfirstlane(e);
  mt = __builtin_amdgcn_readfirstlane(mt);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  m0 = lo + mt * ROWS;
  return m0 < hi;
}

// act(h) and its derivative.  SiLU: h s(h).  GELU (tanh form): 0.5 h (1 + tanh(v)) = h s(2 v)
// with v = sqrt(2/pi) (h + 0.044715 h^3); s is the logistic function, so one exponential
// serves both.  Beyond |h| = 10^4, where s(1 - s) is 0 in float32, the derivative's second
// term is taken at the border, which keeps h^3 from overflowing against that zero.
// Where the exponential overflows, below -88.7, the logistic is 0 (it is less than 3e-39 there).
// (the hardware's exponential and reciprocal, 1 ulp each, a third of the instructions of the
// exact division; a reciprocal that would be subnormal is taken of a scaled argument)
__device__ __forceinline__ float logistic(float x) {
  const float t = 1.0f + __expf(-x);
  const bool big = t > 0x1p100f;
  return __builtin_amdgcn_rcpf(big ? t * 0x1p-64f : t) * (big ? 0x1p-64f : 1.0f);
}

__device__ __forceinline__ float gelu_arg(float h) { return 1.5957691216057308f * (h + 0.044715f * h * h * h); }

__device__ __forceinline__ float act_value(int act, float h) {
  return h * logistic(act == FP8Z1_ACT_SILU ? h : gelu_arg(h));
}
// with FP8Z1_ACT_NONE too
__device__ __forceinline__ float linear_act(int act, float h) { return act == FP8Z1_ACT_NONE ? h : act_value(act, h); }

__device__ __forceinline__ void act_both(int act, float h, float& value, float& slope) {
  const float c = fminf(fmaxf(h, -1e4f), 1e4f);
  float s, dv;
  if (act == FP8Z1_ACT_SILU) {
    s = logistic(h);
    dv = 1.0f;
  } else {
    s = logistic(gelu_arg(h));
    dv = 1.5957691216057308f * (1.0f + 0.134145f * c * c);
  }
  value = h * s;
  slope = s + c * dv * s * (1.0f - s);
}

}  // namespace fp8z1
