// Forward products for few rows per expert (serving): bound by the read of the weights.
//
// A workgroup takes 16 weight rows (of gate and up, or of down) of one expert and 16 TT of the expert's
// rows of x, and its WAVES waves share k among them, a block of 128 (one scale) at a time in turn.  A
// wave reads each of its weight rows' 128 bytes straight into registers, 32 bytes per lane, widens
// them and multiplies by the rows of x on the matrix cores; the next block's bytes are
// on their way meanwhile.  The waves' sums are added in order through LDS.
//
// The groups of an expert's rows run side by side, whatever its load (find_group).  One workgroup that
// walked over all of them took, forward, with all rows on one expert, 1730 us for 8192 rows and 256 experts of 510 x
// 510 (188 now; spread evenly 244, 188 now), 900 for 768 and 64 of 7168 x 2048 (429; evenly 798, 818 now) and 187
// for 1500 and 64 of 512 x 384 (24; evenly 24 both); 256 rows evenly on 32 of 7168 x 2048 lose 3 % by it.
//
// 128 tokens, evenly on 32 experts of widths 7168 and 2048: up 158 us (6.0 TB/s), down 97 us (4.9 TB/s; 2048 is 4
// blocks for each wave, little to have on its way); with 1, 2 or 8 waves a workgroup up takes
// 183, 175 or 188 us.  One token on one expert: 9.4 and 5.4 us, the latency of a few reads
// after one another.
#pragma once

#include "ffn.h"

namespace fp8z1 {
namespace {

//
// PAIR (kFfnUp where workgroups are few): the 16 rows of the matrix tile are 8 of gate and the
// same 8 of up, which makes twice as many workgroups.
template <class H, int KIND, int WAVES, int TT, bool ALIGNED, bool PAIR>
__global__ __launch_bounds__(WAVES * 64) void ffn_rows_kernel(FfnArgs p) {
  constexpr bool kUp = KIND == kFfnUp;
  constexpr int kM = kUp && !PAIR ? 2 : 1;  // matrix tiles
  constexpr int kRowsN = PAIR ? 8 : 16;     // columns of the result per workgroup
  typedef typename H::v8 v8;
  __shared__ f32x4 sums[WAVES][kM * TT][64];
  int32_t e, lo, hi, t0;
  const int32_t group = static_cast<int32_t>(blockIdx.z * gridDim.y + blockIdx.y);
  if (!find_group<16 * TT>(p.offsets, p.T, p.E, group, e, lo, hi, t0)) return;
  const int32_t N = p.N, K = p.K, n0 = static_cast<int32_t>(blockIdx.x) * kRowsN;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int32_t kb = (K + kB - 1) / kB, nb = (N + kB - 1) / kB;
  const int64_t row = (static_cast<int64_t>(e) * N + min(n0 + r % kRowsN, N - 1)) * K + g * 32;
  const uint8_t* const wt[2] = {(PAIR && r >= 8 ? p.w1 : p.w0) + row, kM == 2 ? p.w1 + row : nullptr};
  const int64_t sat = (static_cast<int64_t>(e) * nb + n0 / kB) * kb;
  const float* const sc[2] = {(PAIR && g >= 2 ? p.s1 : p.s0) + sat, kM == 2 ? p.s1 + sat : nullptr};  // of this lane's results

  struct Block {
    uint4 c[kM][2];
    uint4 x[TT][4];
    float s[kM];
  };
  const uint8_t* xr[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) xr[i] = p.x0 + (static_cast<int64_t>(min(t0 + 16 * i + r, hi - 1)) * K + g * 32) * 2;
  auto load = [&](int32_t q, Block& b) {
    const int32_t left = K - q * kB - g * 32;  // of this lane's 32 k
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      b.s[m] = sc[m][q];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* src = wt[m] + q * kB + 16 * i;
        if (ALIGNED)
          b.c[m][i] = 16 * i < left ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
        else
          b.c[m][i] = ld16_part(src, left - 16 * i, K - left + 16 * i);
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* src = xr[t] + q * kB * 2 + 16 * i;
        if (ALIGNED)
          b.x[t][i] = 8 * i < left ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
        else
          b.x[t][i] = ld16_part(src, 2 * left - 16 * i, 2 * (K - left) + 16 * i);
      }
  };
  f32x4 acc[kM][TT];
  const f32x4 zero = {};
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[m][t] = zero;
  auto add = [&](const Block& b) {
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      f32x4 part[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) part[t] = zero;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 c = b.c[m][i / 2];
        const v8 wv = i % 2 ? widen8<H>(c.z, c.w) : widen8<H>(c.x, c.y);
#pragma unroll
        for (int t = 0; t < TT; ++t) part[t] = H::mma16(wv, as_v8<H>(b.x[t][i]), part[t]);
      }
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][t][i] = fmaf(b.s[m], part[t][i], acc[m][t][i]);
    }
  };
  Block b0, b1;
  if (w < kb) load(w, b0);
  if (w + WAVES < kb) load(w + WAVES, b1);
  for (int32_t q = w; q < kb; q += 2 * WAVES) {
    add(b0);
    if (q + 2 * WAVES < kb) load(q + 2 * WAVES, b0);
    if (q + WAVES < kb) {
      add(b1);
      if (q + 3 * WAVES < kb) load(q + 3 * WAVES, b1);
    }
  }
#pragma unroll
  for (int m = 0; m < kM; ++m)
#pragma unroll
    for (int t = 0; t < TT; ++t) sums[w][m * TT + t][lane] = acc[m][t];
  __syncthreads();
  if (w < TT) {
    f32x4 v[2];
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      v[m] = sums[0][m * TT + w][lane];
      for (int k = 1; k < WAVES; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[m][i] += sums[k][m * TT + w][lane][i];
    }
    if (PAIR)  // the up results of a column are in the upper lanes
#pragma unroll
      for (int i = 0; i < 4; ++i) v[1][i] = __shfl_xor(v[0][i], 32);
    const int32_t t = t0 + 16 * w + r;
    if (t < hi && (!PAIR || g < 2)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t n = n0 + 4 * g + i;
        if (n >= N) continue;
        const int64_t at = static_cast<int64_t>(t) * N + n;
        if (kUp) {
          p.o0[at] = H::from_f32(act_value(p.act, v[0][i]) * v[1][i]);
          if (p.o1) {
            p.o1[at] = H::from_f32(v[0][i]);
            p.o2[at] = H::from_f32(v[1][i]);
          }
        } else {
          p.o0[at] = H::from_f32(v[0][i]);
        }
      }
    }
  }
}

template <class H, int KIND, int WAVES, int TT, bool PAIR>
void launch_rows_as(const FfnArgs& p, bool aligned, hipStream_t s) {
  constexpr int kRowsN = PAIR ? 8 : 16;
  const int64_t groups = static_cast<int64_t>(p.E) + p.T / (16 * TT);
  const int64_t turns = (groups + 65534) / 65535;  // (a grid's y ends at 65,535)
  const dim3 g(static_cast<unsigned>((p.N + kRowsN - 1) / kRowsN), static_cast<unsigned>((groups + turns - 1) / turns),
               static_cast<unsigned>(turns));
  if (aligned)
    hipLaunchKernelGGL((ffn_rows_kernel<H, KIND, WAVES, TT, true, PAIR>), g, dim3(WAVES * 64), 0, s, p);
  else
    hipLaunchKernelGGL((ffn_rows_kernel<H, KIND, WAVES, TT, false, PAIR>), g, dim3(WAVES * 64), 0, s, p);
}

// Workgroups that do not fill the card twice: 8 waves each (and gate and up in one tile);
// else 4.  Up to 8 rows per expert on average: one matrix tile of rows at a time; else two.
template <class H, int KIND>
void launch_rows(const FfnArgs& p, bool aligned, hipStream_t s) {
  constexpr bool kUp = KIND == kFfnUp;
  const bool deep = static_cast<int64_t>((p.N + 15) / 16) * p.E < 512, two = static_cast<int64_t>(p.T) > 8ll * p.E;
  if (deep && two)
    launch_rows_as<H, KIND, 8, 2, kUp>(p, aligned, s);
  else if (deep)
    launch_rows_as<H, KIND, 8, 1, kUp>(p, aligned, s);
  else if (two)
    launch_rows_as<H, KIND, 4, 2, false>(p, aligned, s);
  else
    launch_rows_as<H, KIND, 4, 1, false>(p, aligned, s);
}

}  // namespace
}  // namespace fp8z1
