// Shared by the feed-forward kernels: arguments, expert ranges, the gated activation.
#pragma once

#include "device_util.h"
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
  kFfnUpBwd = 3     // dx = dh Wg + du Wu
};

struct FfnArgs {
  const uint8_t *x0, *x1;  // 16-bit rows [T, K] (x1: du of kFfnUpBwd)
  const uint8_t *w0, *w1;  // codes: [E, N, K] (kFfnUp, kFfnDown) or [E, K, N]
  const float *s0, *s1;    // their block scales
  const int32_t* offsets;  // [E + 1], or NULL: one expert, all rows
  const uint16_t *h, *u;   // [T, N] inputs of kFfnDownBwd
  uint16_t *o0, *o1, *o2;  // outputs [T, N]
  int32_t T, E, N, K, act;
};

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

__device__ __forceinline__ int32_t wave_isum(int32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// The tile (expert, its rows lo..hi, first row m0, tile column) of workgroup b, or
// false if there is none: the number of row tiles depends on the offsets, which only
// the device knows, so the grid holds the most there can be.  Consecutive workgroups
// go to the XCDs in turn; each XCD gets a contiguous run of tiles, ordered in groups
// of kGroup row tiles by all columns, so that the tiles running on one XCD at a time
// share rows and weights in its L2.
constexpr int kGroup = 8;
template <int ROWS>
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int32_t T, int32_t E, int32_t ncols, int32_t b,
                                          int32_t& e, int32_t& lo, int32_t& hi, int32_t& m0, int32_t& col) {
  const int lane = threadIdx.x & 63;
  int32_t total = 0;
  if (offsets) {
    for (int32_t e0 = 0; e0 < E; e0 += 64) {
      int32_t n = 0;
      if (e0 + lane < E) {
        int32_t l, h;
        expert_rows(offsets, T, e0 + lane, l, h);
        n = (h - l + ROWS - 1) / ROWS;
      }
      total += wave_isum(n);
    }
  } else {
    total = (T + ROWS - 1) / ROWS;
  }
  total = __builtin_amdgcn_readfirstlane(total);
  const int64_t all = static_cast<int64_t>(total) * ncols;
  if (b >= all) return false;
  const int32_t g = static_cast<int32_t>(all), x = b % kXcds, per = g / kXcds, rem = g % kXcds;
  const int32_t id = x * per + min(x, rem) + b / kXcds;
  const int32_t grp = id / (kGroup * ncols), in = id - grp * kGroup * ncols;
  const int32_t rows = min(kGroup, total - grp * kGroup);
  col = in / rows;
  int32_t mt = grp * kGroup + in - col * rows;
  e = 0;
  if (offsets) {
    for (int32_t e0 = 0; e0 < E; e0 += 64) {
      int32_t n = 0;
      if (e0 + lane < E) {
        int32_t l, h;
        expert_rows(offsets, T, e0 + lane, l, h);
        n = (h - l + ROWS - 1) / ROWS;
      }
      int32_t upto = n;  // tiles of this chunk's experts up to and with this lane's
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int32_t v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
      }
      const uint64_t past = __ballot(upto > mt);
      if (past) {
        const int at = __builtin_ctzll(past);
        e = e0 + at;
        mt -= __shfl(upto - n, at);
        break;
      }
      mt -= __shfl(upto, 63);
    }
  }
  e = __builtin_amdgcn_readfirstlane(e);
  mt = __builtin_amdgcn_readfirstlane(mt);
  expert_rows(offsets, T, e, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  m0 = lo + mt * ROWS;
  return m0 < hi;
}

// act(h) and its derivative.  SiLU: h s(h).  GELU (tanh form): 0.5 h (1 + tanh(v)) = h s(2 v)
// with v = sqrt(2/pi) (h + 0.044715 h^3); s is the logistic function, so one exponential
// serves both.  Beyond |h| = 10^4, where s(1 - s) is 0 in float32, the derivative's second
// term is taken at the border, which keeps h^3 from overflowing against that zero.
__device__ __forceinline__ float logistic(float x) { return 1.0f / (1.0f + __expf(-x)); }

__device__ __forceinline__ float gelu_arg(float h) { return 1.5957691216057308f * (h + 0.044715f * h * h * h); }

__device__ __forceinline__ float act_value(int act, float h) {
  return h * logistic(act == FP8Z1_ACT_SILU ? h : gelu_arg(h));
}

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
