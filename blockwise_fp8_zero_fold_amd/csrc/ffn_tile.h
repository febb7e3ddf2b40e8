// The feed-forward block over blockwise-FP8 weights, tokens sorted by expert: both
// projections with the gated activation, the down projection, and the backward pass
// with respect to the activations.
//
// One tile kernel serves all four calls.  A workgroup of 4 waves computes 128 rows
// (tokens of one expert) x 256 weight columns (kFfnUp: 128 of gate and 128 of up), each wave 64 x 128
// as 2 x 4 matrix tiles of 32 x 32; or half as many columns where the wide tiles would not
// fill the card.  The sum over k goes in blocks of 128, the blocks that one weight scale covers:
//     acc += scale * sum_{k in block} x[m][k] * code[k][n],
// the inner sum on the matrix cores with the codes widened exactly, so no dequantized weight is
// rounded.  Two workgroups share a compute unit, one computing while the other waits.
//
// What bounds it: on 8192 tokens of 8 experts with widths 7168 and 2048 the four products run at
// 830 to 960 TFLOP/s over many launches (up 0.51 ms, down 0.29, backward 0.28 and 0.54), single ones at
// up to 1100, and at 840 to 1090 on one dense 4096 x 4096 expert, where a plain bfloat16 library
// product reaches 1340 to 1400.  No one thing ends it.  The matrix cores are busy for 45 to 56 % of
// the cycles; the waves wait for 35 to 41 % of theirs until an instruction can issue (matrix
// instructions, the codes' widening, which both row halves of a tile do, and the rescaling between blocks)
// and for 20 to 29 % on data and barriers; the clock is at 1.7 to 2.0 GHz of 2.4, so power has its share: a
// wave of 128 x 64, which reads a quarter more from LDS and widens half as many codes, needs 4 to 7 % fewer
// cycles and 4 to 7 % more time.  Up reads 980 MB of HBM for 350 MB of operands.
// Small problems are bound by the chain of one tile: about 5 us and 1.5 us per scale block.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "ffn.h"
#include "ffn_rows.h"

namespace fp8z1 {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;  // tile rows
constexpr int kStep = 64;   // k per LDS stage
constexpr int kABytes = kRows * kStep * 2;

// 8 elements of a row, the first `count` of which are there: in one access, at any alignment
typedef uint32_t v4u_a2_global_t __attribute__((ext_vector_type(4), aligned(2), address_space(1)));
__device__ __forceinline__ void store_row8(uint16_t* to, const uint32_t (&x)[4], int count) {
  if (count == 8) {
    *(v4u_a2_global_t*)(to) = v4u_v_t{x[0], x[1], x[2], x[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) to[i] = static_cast<uint16_t>(x[i / 2] >> (16 * (i % 2)));
  }
}
__device__ __forceinline__ void load_row8(const uint16_t* from, uint32_t (&x)[4], int count) {
  if (count == 8) {
    const v4u_v_t v = *(const v4u_a2_global_t*)(from);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) x[i / 2] |= static_cast<uint32_t>(from[i]) << (16 * (i % 2));
  }
}

// h and u of 8 columns of a row, for kFfnDownBwd
struct Kept {
  uint32_t h[4], u[4];
};
template <int KIND>
__device__ __forceinline__ Kept load_kept(const FfnArgs& p, int64_t at, int count) {
  Kept k = {};
  if constexpr (KIND == kFfnDownBwd)
    if (count > 0) {
      load_row8(p.h + at, k.h, count);
      load_row8(p.u + at, k.u, count);
    }
  return k;
}

// 8 columns of a row, rounded to the result's type.
template <class H>
__device__ __forceinline__ void put8(const float (&f)[8], uint16_t* to, int count) {
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    o[k] = static_cast<uint32_t>(H::from_f32(f[2 * k])) | static_cast<uint32_t>(H::from_f32(f[2 * k + 1])) << 16;
  store_row8(to, o, count);
}

// y = res + act(x + bias) of 8 columns from column n of a row on, and x + bias (what the backward pass
// needs) where it is wanted; both are rounded once.  `bias` is the expert's.
// The choices are the launch's, each taken once for the 8 columns.
template <class H>
__device__ __forceinline__ void finish_linear(const FfnArgs& p, int64_t at, int32_t n, int count, const float (&x)[8]) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i];
  uint32_t r[4] = {};
  if (p.res) load_row8(p.res + at, r, count);
  if (p.bias) {
    if (count == 8) {
      const float4 b0 = ld_global_a4(p.bias + n), b1 = ld_global_a4(p.bias + n + 4);
      const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += b[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < count) y[i] += p.bias[n + i];
    }
  }
  if (p.o1) put8<H>(y, p.o1 + at, count);
  if (p.act == FP8Z1_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = act_value(FP8Z1_ACT_SILU, y[i]);
  } else if (p.act == FP8Z1_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = act_value(FP8Z1_ACT_GELU, y[i]);
  }
  if (p.res)
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += H::to_f32(static_cast<uint16_t>(r[i / 2] >> (16 * (i % 2))));
  put8<H>(y, p.o0 + at, count);
}

// The results of 8 columns of a row, of which `count` are there (for kFfnUp x: gate, v: up).
// Each is rounded once, from float32 to the activations' 16 bits, which is what the matrix instructions
// of the next product take and what a training step keeps: a between up and down, dh and du before dx
// (so y and dx lie 1.4 times as far from the 64-bit result as after a single rounding at their end).
template <class H, int KIND>
__device__ __forceinline__ void finish8(const FfnArgs& p, int64_t at, int32_t n, int count, const float (&x)[8],
                                        const float (&v)[8], const Kept& kept) {
  auto put = [&](const float (&f)[8], uint16_t* to) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = static_cast<uint32_t>(H::from_f32(f[2 * k])) | static_cast<uint32_t>(H::from_f32(f[2 * k + 1])) << 16;
    store_row8(to + at, o, count);
  };
  if (count <= 0) return;
  if (KIND == kFfnUp) {
    float a[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = act_value(p.act, x[k]) * v[k];
    put(a, p.o0);
    if (p.o1) {
      put(x, p.o1);
      put(v, p.o2);
    }
  } else if (KIND == kFfnDownBwd) {
    float dh[8], du[8], a[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float h = H::to_f32(static_cast<uint16_t>(kept.h[k / 2] >> (16 * (k % 2))));
      const float u = H::to_f32(static_cast<uint16_t>(kept.u[k / 2] >> (16 * (k % 2))));
      float value, slope;
      act_both(p.act, h, value, slope);
      dh[k] = x[k] * u * slope;
      du[k] = x[k] * value;
      a[k] = value * u;
    }
    put(dh, p.o0);
    put(du, p.o1);
    if (p.o2) put(a, p.o2);
  } else if (KIND == kLinear) {
    finish_linear<H>(p, at, n, count, x);
  } else {
    put(x, p.o0);
  }
}

// A wave's results on their way to memory: 64 rows of 64 float32 in LDS (for kFfnUp 32 gate
// and 32 up columns), so that the rows leave 16 bytes per lane and 128 bytes in a row, by a
// loop of little code: from the accumulators directly, 2 bytes at a time, the results took
// a quarter of a large problem's time, and their unrolled code, read once, most of a
// small one's.  Chunk c (16 bytes) of row r sits at c ^ (r mod 16).  What a lane writes there another
// lane of its wave reads, and the next turn's results go over it: handed_over() stands between.
constexpr int kResultBytes = 4 * 64 * 64 * 4;
__device__ __forceinline__ int result_at(int r, int c) { return r * 256 + ((c ^ (r & 15)) << 4); }

// 32 x 32 tile (i, j): lane l holds of row l % 32 the columns 8 q + 4 (l / 32) + 0..3.
__device__ __forceinline__ void lay_tile(const f32x16& x, uint8_t* to, int i, int j) {
  const int lane = threadIdx.x & 63, r = i * 32 + (lane & 31);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<f32x4*>(to + result_at(r, j * 8 + q * 2 + (lane >> 5))) =
        f32x4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
}

// LDS accesses of the wave's lanes stay on their side of this.  The hardware runs a wave's LDS
// accesses in order, so it costs no instruction: it keeps the compiler, which sees a lane's own
// addresses only, from moving a read of another lane's values over their write.
__device__ __forceinline__ void handed_over() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void read8(const uint8_t* from, int r, int c, float (&x)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(from + result_at(r, c));
  const f32x4 b = *reinterpret_cast<const f32x4*>(from + result_at(r, c + 1));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[k] = a[k];
    x[4 + k] = b[k];
  }
}

// The 64 rows laid out, from row m and column n of the results on.
template <class H, int KIND>
__device__ __forceinline__ void store_rows(const FfnArgs& p, const uint8_t* from, int32_t m, int32_t hi, int32_t n) {
  constexpr int kPer = KIND == kFfnUp ? 4 : 8;  // 8-column groups per row
  const int lane = threadIdx.x & 63, c = lane % kPer;
  auto place = [&](int turn, int& r, int& count) {
    r = turn * (64 / kPer) + lane / kPer;
    count = m + r < hi ? min(p.N - n - 8 * c, 8) : 0;
    return static_cast<int64_t>(m + r) * p.N + n + 8 * c;
  };
  int r, count;
  int64_t at = place(0, r, count);
  Kept kept = load_kept<KIND>(p, at, count);
#pragma unroll 1
  for (int turn = 0; turn < kPer; ++turn) {
    int rn, cn;
    const int64_t an = place(turn + 1, rn, cn);
    const Kept next = load_kept<KIND>(p, an, turn + 1 < kPer ? cn : 0);
    float x[8], v[8] = {};
    read8(from, r, 2 * c, x);
    if (KIND == kFfnUp) read8(from, r, 8 + 2 * c, v);
    finish8<H, KIND>(p, at, n + 8 * c, count, x, v, kept);
    r = rn;
    count = cn;
    at = an;
    kept = next;
  }
}

// Part `at` of the split tiles in the workspace: the accumulators of all threads, float4 by
// float4, so that each store of a wave is 1 KB in a row.
template <int NT>
__device__ __forceinline__ f32x4* part_at(float* part, int32_t at) {
  return reinterpret_cast<f32x4*>(part) + static_cast<int64_t>(at) * (2 * NT * 4 * kThreads);
}

// Whether the block scales that a tile multiplies by are positive, finite and within a
// factor 2^40 of each other.  Every wave looks at all of them, so all agree.
__device__ __forceinline__ bool scales_close(const float* s, int32_t count, int32_t stride, float& lo, float& hi) {
  bool ok = true;
  for (int32_t i = threadIdx.x & 63; i < count; i += 64) {
    const float x = s[static_cast<int64_t>(i) * stride];
    ok = ok && x > 0.0f && x < 3e38f;
    lo = fminf(lo, x);
    hi = fmaxf(hi, x);
  }
  return ok;
}

// Chunk c of row r of an LDS tile sits at position c ^ swizzle(r) of the row.  LDS serves 256
// bytes at a time: 16 lanes of a 16-byte read (16 rows of one chunk) or 32 lanes of a
// transposing 8-byte read (8 rows of two neighbouring chunks), which the swizzle
// spreads over all 16 places; with the lower 3 bits of the row alone half of the
// LDS cycles were conflicts.
__device__ __forceinline__ int swizzle_a(int r) { return (r >> 1) & 7; }  // rows of 128 bytes
__device__ __forceinline__ int swizzle_b(int r) { return (r >> 2) & 3; }  // rows of 64 bytes
template <int BYTES>
__device__ __forceinline__ int swizzle_t(int r) {  // transposed reads, rows of 128 or 256 bytes
  return BYTES == 256 ? (r & 7) << 1 : ((r >> 1) & 3) << 1;
}

// NT: 32-column tiles per wave (2 or 4).  DIRECT: rows of activations and codes are 4-byte aligned,
// so a stage goes from memory to LDS by direct copies (what they bring past the end of k is
// cleared in LDS); otherwise through registers, with the bytes outside a row left out.
//
// The accumulator holds the sum in units of the current block's scale: between blocks
// it is multiplied by scale_before / scale_now and the matrix cores add the next block's
// code products right into it, so no second set of registers is needed for the partial
// sums and a wave can own 64 x 128.  That product stays harmless while the tile's scales
// are within 2^40 of each other; a tile with scales further apart (or not positive and finite)
// sums each block apart and adds scale * sum, in a pass for each of its wave's tile columns.
template <class H, int KIND, int NT, bool DIRECT>
__global__ __launch_bounds__(kThreads, 2) void ffn_tile_kernel(FfnArgs p, int32_t ncols) {
  constexpr bool kTrans = KIND == kFfnDownBwd || KIND == kFfnUpBwd || KIND == kLinearBwd;  // weights run along n
  constexpr bool kUp = KIND == kFfnUp;
  constexpr int kB2 = NT * 64;                  // weight rows (or columns) of a stage
  constexpr int kCols = kUp ? kB2 / 2 : kB2;    // output columns of a tile
  constexpr int kSeg = KIND == kFfnUpBwd ? 2 : 1;  // products added up
  constexpr int kBBytes = kB2 * kStep;
  constexpr int kBC = kBBytes / 16 / kThreads;  // 16-byte chunks per thread and stage: 2 or 4
  constexpr int kBPer = kTrans ? kB2 / 16 : 4;  // chunks per row of B's stage
  typedef typename H::v8 v8;
  // two stages in LDS, each copied while the other is computed; then the waves' results
  constexpr int kStageBytes = kABytes + kBBytes;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStageBytes > kResultBytes ? 2 * kStageBytes : kResultBytes];
  uint8_t* const sa0 = lds;
  uint8_t* const sb0 = lds + kABytes;
  uint8_t* const sa1 = sa0 + kStageBytes;
  uint8_t* const sb1 = sb0 + kStageBytes;

  const int32_t kb = (p.K + kB - 1) / kB, blocks = kSeg * kb;  // scale blocks of k, each two stages
  int32_t rowtiles, e, lo, hi, m0, col;
  Run first;
  const int32_t item = static_cast<int32_t>(blockIdx.x);
  const Plan plan = plan_tiles<kRows>(p.offsets, p.T, p.E, ncols, blocks, p.part ? p.split_from : 0, rowtiles, first);
  if (item >= plan.items()) return;
  const bool split = item >= plan.whole;
  const int32_t rest = plan.tiles - plan.whole;
  const int32_t id = split ? plan.whole + (item - plan.whole) % rest : xcd_run(item, plan.whole);
  const int32_t sp = split ? (item - plan.whole) / rest : 0, parts = split ? plan.splits : 1;
  const int32_t q0 = blocks * sp / parts, q1 = blocks * (sp + 1) / parts;
  if (!find_tile<kRows>(p.offsets, p.T, p.E, ncols, rowtiles, first, id, e, lo, hi, m0, col)) return;
  const int32_t n0 = col * kCols;
  if (KIND == kLinear && p.bias) p.bias += static_cast<int64_t>(e) * p.N;
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6), wm = w >> 1, wn = w & 1;
  const int32_t N = p.N, K = p.K;
  const int32_t nb = (N + kB - 1) / kB;

  // This thread's 16-byte chunks of a stage, positions id = t + 256 j of the LDS tile.
  // Their addresses are a base that is the same for the workgroup and moves with k,
  // plus a 32-bit offset that stays; rows past the end repeat the last one.
  uint32_t aoff[4], boff[kBC];
  int32_t ac[4], bn[kBC], br[kBC];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int id = t + kThreads * j, r = id >> 3;
    ac[j] = ((id & 7) ^ swizzle_a(r)) * 16;
    aoff[j] = static_cast<uint32_t>(min(r, hi - 1 - m0)) * static_cast<uint32_t>(K) * 2 + ac[j];
  }
#pragma unroll
  for (int j = 0; j < kBC; ++j) {
    const int id = t + kThreads * j, r = id / kBPer;
    if (kTrans) {
      const int c = ((id % kBPer) ^ swizzle_t<kB2>(r)) * 16;
      br[j] = r;
      bn[j] = N - n0 - c;  // bytes of the chunk inside the row
      // (direct copies: a chunk past the row, whose columns are not stored, is another's)
      boff[j] = static_cast<uint32_t>(r) * static_cast<uint32_t>(N) + (DIRECT && bn[j] <= 0 ? 0 : c);
    } else {
      const int c = ((id & 3) ^ swizzle_b(r)) * 16;
      br[j] = 0;
      bn[j] = c;
      boff[j] = static_cast<uint32_t>(min(kUp ? r % (kB2 / 2) : r, N - 1 - n0)) * static_cast<uint32_t>(K) + c;
    }
  }
  const int64_t abase = static_cast<int64_t>(m0) * K * 2;
  const int64_t bbase = static_cast<int64_t>(e) * N * K + (kTrans ? n0 : static_cast<int64_t>(n0) * K);

  uint4 ra[4], rb[kBC];
  // k0: first k of the stage within its product `seg`
  auto fetch = [&](int seg, int32_t k0, uint8_t* sa, uint8_t* sb) {
    const uint8_t* const x = (seg ? p.x1 : p.x0) + abase + 2 * static_cast<int64_t>(k0);
    const int64_t kw = kTrans ? static_cast<int64_t>(k0) * N : k0;
    const uint8_t* const wa = (seg ? p.w1 : p.w0) + bbase + kw;
    const uint8_t* const wb = kUp ? p.w1 + bbase + kw : wa;  // upper half of the stage's rows
    if (DIRECT) {  // (the buffers end with the tensors: what lies behind is not read)
      const buffer_t xb = make_buffer(x, static_cast<int64_t>(p.T - m0) * K * 2 - 2 * static_cast<int64_t>(k0));
      const int64_t left = static_cast<int64_t>(p.E) * N * K - bbase - kw;
      const buffer_t ba = make_buffer(wa, left), bb = make_buffer(wb, left);
#pragma unroll
      for (int j = 0; j < 4; ++j) copy16_to_lds(xb, aoff[j], sa + (w * 64 + kThreads * j) * 16);
#pragma unroll
      for (int j = 0; j < kBC; ++j)
        copy16_to_lds(j < kBC / 2 ? ba : bb, boff[j], sb + (w * 64 + kThreads * j) * 16);
      return;
    }
    if (k0 + kStep <= K && (!kTrans || n0 + kB2 <= N)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) ra[j] = ld16(x + aoff[j]);
#pragma unroll
      for (int j = 0; j < kBC; ++j) rb[j] = ld16((j < kBC / 2 ? wa : wb) + boff[j]);
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) ra[j] = ld16_part(x + aoff[j], (K - k0) * 2 - ac[j], k0 * 2 + ac[j]);
#pragma unroll
    for (int j = 0; j < kBC; ++j)
      rb[j] = kTrans ? ld16_part(wa + boff[j], k0 + br[j] < K ? bn[j] : 0, N - bn[j])
                     : ld16_part((j < kBC / 2 ? wa : wb) + boff[j], K - k0 - bn[j], k0 + bn[j]);
  };
  auto put = [&](uint8_t* sa, uint8_t* sb) {
    if (DIRECT) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(sa + (t + kThreads * j) * 16) = ra[j];
#pragma unroll
    for (int j = 0; j < kBC; ++j) *reinterpret_cast<uint4*>(sb + (t + kThreads * j) * 16) = rb[j];
  };

  // Clears what a stage holds past the end of k: `v` of its 64 k are there.
  auto clear_past = [&](int32_t v, uint8_t* sa, uint8_t* sb) {
    auto keep = [](uint8_t* at, int n) {  // the first n of 16 bytes
      if (n >= 16) return;
      uint4 x = *reinterpret_cast<uint4*>(at);
      uint32_t* const o[4] = {&x.x, &x.y, &x.z, &x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int in = n - 4 * i;
        *o[i] = in >= 4 ? *o[i] : in > 0 ? *o[i] & (0xffffffffu >> (32 - 8 * in)) : 0u;
      }
      *reinterpret_cast<uint4*>(at) = x;
    };
    for (int id = t; id < kABytes / 16; id += kThreads) {
      const int r = id >> 3;
      keep(sa + id * 16, 2 * v - ((id & 7) ^ swizzle_a(r)) * 16);
    }
    for (int id = t; id < kBBytes / 16; id += kThreads) {
      const int r = id / kBPer;
      keep(sb + id * 16, kTrans ? (r < v ? 16 : 0) : v - ((id & 3) ^ swizzle_b(r)) * 16);
    }
    __syncthreads();
  };

  const f32x16 zero = {};
  const int half = lane >> 5, l32 = lane & 31, l16 = lane & 15, grp = lane >> 4;
  // d[i][j - j0] += A tile i times B tile j, over one stage: LDS reads of half a stage, the
  // copies of the next stage (`next`), and the matrix instructions among the other
  // half's reads.
  auto compute = [&](const uint8_t* sa, const uint8_t* sb, auto& d, auto j0_, auto nj_, auto next) {
    constexpr int j0 = decltype(j0_)::value, nj = decltype(nj_)::value;
    uint4 a[4][2];
    uint2 b[4][nj];
    auto read = [&](int ks0) {
#pragma unroll
      for (int ks = ks0; ks < ks0 + 2; ++ks) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = wm * 64 + i * 32 + l32;
          // k of this lane: plain order where B is read transposed; otherwise the lane's
          // 16 consecutive k of a 32-wide group, 8 per step, as B's 16-byte chunk holds them
          const int c = kTrans ? ks * 2 + half : (ks >> 1) * 4 + half * 2 + (ks & 1);
          a[ks][i] = *reinterpret_cast<const uint4*>(sa + r * 128 + ((c ^ swizzle_a(r)) << 4));
        }
#pragma unroll
        for (int jj = 0; jj < nj; ++jj) {
          const int j = j0 + jj;
          if (kTrans) {
            const int r = ks * 16 + (grp >> 1) * 8 + (l16 >> 1);
            const int c = (wn * NT + j) * 2 + (grp & 1);
            const i32x2 q = read_tr8(sb + r * kB2 + ((c ^ swizzle_t<kB2>(r)) << 4) + (l16 & 1) * 8);
            b[ks][jj] = make_uint2(q.x, q.y);
          } else if (ks % 2 == 0) {
            // gate tiles first, then the up tiles of the same columns
            const int r = kUp ? (j / (NT / 2)) * (kB2 / 2) + (wn * (NT / 2) + j % (NT / 2)) * 32 + l32
                              : (wn * NT + j) * 32 + l32;
            const int c = ks + half;
            const uint4 q = *reinterpret_cast<const uint4*>(sb + r * 64 + ((c ^ swizzle_b(r)) << 4));
            b[ks][jj] = make_uint2(q.x, q.y);
            b[ks + 1][jj] = make_uint2(q.z, q.w);
          }
        }
      }
    };
    read(0);
    next();
    read(2);
    v8 bw = widen8<H>(b[0][0].x, b[0][0].y);
#pragma unroll
    for (int s = 0; s < 4 * nj; ++s) {
      const int ks = s / nj, jj = s % nj, sn = s + 1 < 4 * nj ? s + 1 : s;
      const v8 bn = widen8<H>(b[sn / nj][sn % nj].x, b[sn / nj][sn % nj].y);
#pragma unroll
      for (int i = 0; i < 2; ++i) d[i][jj] = H::mma32(bw, as_v8<H>(a[ks][i]), d[i][jj]);
      bw = bn;
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // the scales of this wave's columns: one per block of k (two matrices: one each)
  const int32_t nblk = min((n0 + (kUp ? 0 : wn * NT * 32)) / kB, nb - 1);
  const int32_t sstride = kTrans ? nb : 1;
  const int64_t sat = kTrans ? static_cast<int64_t>(e) * kb * nb + nblk : (static_cast<int64_t>(e) * nb + nblk) * kb;
  const float* const sp0 = p.s0 + sat;
  const float* const sp1 = KIND == kFfnUpBwd || kUp ? p.s1 + sat : nullptr;
  auto scale = [&](int32_t q, int which) {
    const bool second = kSeg == 2 ? q >= kb : which == 1;
    // (through the scalar cache: the scales do not change while the kernel runs)
    typedef const __attribute__((address_space(4))) float* scalar_t;
    return ((scalar_t)(second ? sp1 : sp0))[static_cast<int64_t>(kSeg == 2 && second ? q - kb : q) * sstride];
  };

  auto stage = [&](int32_t q, int32_t second, uint8_t* sa, uint8_t* sb) {
    const bool seg = kSeg == 2 && q >= kb;
    fetch(seg ? 1 : 0, (seg ? q - kb : q) * kB + second, sa, sb);
  };
  // The first stage is on its way while the scales are looked at
  stage(q0, 0, sa0, sb0);
  bool first_pass = true;

  // One pass over this item's k; `after(q)` runs after the two stages of scale block q.
  auto sweep = [&](auto& d, auto j0_, auto nj_, auto before, auto after) {
    if (!first_pass) stage(q0, 0, sa0, sb0);
    first_pass = false;
    put(sa0, sb0);
    for (int32_t q = q0; q < q1; ++q) {
      before(q);
      if (DIRECT) wait_copies();
      __syncthreads();
      const int32_t left = K - (kSeg == 2 && q >= kb ? q - kb : q) * kB;
      if (DIRECT && left < kStep) clear_past(left, sa0, sb0);
      compute(sa0, sb0, d, j0_, nj_, [&] { stage(q, kStep, sa1, sb1); });
      put(sa1, sb1);
      if (DIRECT) wait_copies();
      __syncthreads();
      if (DIRECT && left < kB) clear_past(left - kStep, sa1, sb1);
      // (the last block's turn fetches it again rather than branch)
      compute(sa1, sb1, d, j0_, nj_, [&] { stage(min(q + 1, q1 - 1), 0, sa0, sb0); });
      put(sa0, sb0);
      after(q);
    }
    if (DIRECT) wait_copies();
    __syncthreads();  // the stages are written again by the next pass
  };

  // The accumulators as results, or as a part's sums.  Tile columns from j0 on are in d, two at a
  // time (for kFfnUp one of gate and the one of up that belongs to it, NT / 2 further on).
  uint8_t* const mine = lds + w * (kResultBytes / 4);
  auto emit = [&](const auto& d, auto nj_) {
    constexpr int nj = decltype(nj_)::value;  // tile columns in d, the first of them j0
    if (split) {
      f32x4* const to = part_at<NT>(p.part, item - plan.whole);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (m0 + wm * 64 + i * 32 >= hi) break;  // (rows past the run are not joined either)
#pragma unroll
        for (int j = 0; j < nj; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            to[((i * NT + j) * 4 + r) * kThreads + t] =
                f32x4{d[i][j][4 * r], d[i][j][4 * r + 1], d[i][j][4 * r + 2], d[i][j][4 * r + 3]};
      }
      return;
    }
#pragma unroll 1
    for (int turn = 0; turn < NT / 2; ++turn) {
      auto lay = [&](auto first_) {
        constexpr int first = decltype(first_)::value;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lay_tile(d[i][first], mine, i, 0);
          lay_tile(d[i][first + (kUp ? NT / 2 : 1)], mine, i, 1);
        }
      };
      if (turn == 0)
        lay(Int<0>{});
      else
        lay(Int<NT == 2 ? 0 : kUp ? 1 : 2>{});
      handed_over();
      store_rows<H, KIND>(p, mine, m0 + wm * 64, hi, n0 + wn * (NT / 2) * (kUp ? 32 : 64) + turn * (kUp ? 32 : 64));
      handed_over();
    }
  };

  // all waves decide alike: the barriers are shared
  float slo = 3e38f, shi = 0.0f;
  bool ok = true;
#pragma unroll
  for (int b = 0; b < (kCols + kB - 1) / kB; ++b) {
    const int64_t off = static_cast<int64_t>(min(n0 / kB + b, nb - 1) - nblk) * (kTrans ? 1 : kb);
    ok = scales_close(sp0 + off, kb, sstride, slo, shi) && ok;
    if (kUp || kSeg == 2) ok = scales_close(sp1 + off, kb, sstride, slo, shi) && ok;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    slo = fminf(slo, __shfl_xor(slo, o));
    shi = fmaxf(shi, __shfl_xor(shi, o));
  }
  ok = __all(ok) && shi * 0x1p-40f <= slo;

  if (ok) {
    f32x16 acc[2][NT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = zero;
    float was[2] = {scale(q0, 0), kUp ? scale(q0, 1) : 1.0f};
    sweep(
        acc, Int<0>{}, Int<NT>{}, [&](int32_t) {},
        [&](int32_t q) {
          if (q + 1 == q1) return;
          float ratio[2];
#pragma unroll
          for (int k = 0; k < (kUp ? 2 : 1); ++k) {
            const float now = scale(q + 1, k);
            ratio[k] = was[k] / now;
            was[k] = now;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int r = 0; r < 16; ++r) acc[i][j][r] *= ratio[kUp && j >= NT / 2 ? 1 : 0];
        });
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] *= was[kUp && j >= NT / 2 ? 1 : 0];
    emit(acc, Int<NT>{});
  } else {
    // sums by blocks, one tile column at a time, in a pass each; the results wait in `sum`
    f32x16 sum[2][NT];
    auto pass = [&](auto j_) {
      constexpr int j = decltype(j_)::value;
      f32x16 part[2][1];
#pragma unroll
      for (int i = 0; i < 2; ++i) sum[i][j] = zero;
      sweep(
          part, Int<j>{}, Int<1>{}, [&](int32_t) { part[0][0] = part[1][0] = zero; },
          [&](int32_t q) {
            const float s = scale(q, kUp && j >= NT / 2 ? 1 : 0);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int r = 0; r < 16; ++r) sum[i][j][r] = fmaf(s, part[i][0][r], sum[i][j][r]);
          });
    };
    pass(Int<0>{});
    pass(Int<1>{});
    if constexpr (NT == 4) {
      pass(Int<2>{});
      pass(Int<3>{});
    }
    emit(sum, Int<NT>{});
  }
}

// The split tiles: their parts' sums added in order, and the results as above.  A workgroup takes
// half of a 32 x 32 tile of each wave: 8 columns of 32 rows per half wave, after an exchange.
template <class H, int KIND, int NT>
__global__ __launch_bounds__(kThreads) void ffn_join_kernel(FfnArgs p, int32_t ncols) {
  constexpr bool kUp = KIND == kFfnUp;
  constexpr int kCols = (kUp ? 32 : 64) * NT, kJ = kUp ? NT / 2 : NT;
  const int32_t blocks = (KIND == kFfnUpBwd ? 2 : 1) * ((p.K + kB - 1) / kB);
  int32_t rowtiles, e, lo, hi, m0, col;
  Run first;
  const Plan plan = plan_tiles<kRows>(p.offsets, p.T, p.E, ncols, blocks, p.split_from, rowtiles, first);
  const int32_t rest = plan.tiles - plan.whole, tile = static_cast<int32_t>(blockIdx.x) / (4 * kJ);
  if (tile >= rest) return;
  const int g = blockIdx.x & 1, i = (blockIdx.x >> 1) & 1, j = static_cast<int>(blockIdx.x >> 2) % kJ;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  if (!find_tile<kRows>(p.offsets, p.T, p.E, ncols, rowtiles, first, plan.whole + tile, e, lo, hi, m0, col)) return;
  if (KIND == kLinear && p.bias) p.bias += static_cast<int64_t>(e) * p.N;
  const int32_t mw = m0 + (w >> 1) * 64 + i * 32;
  if (mw >= hi) return;  // (the parts of rows past the run were not written)
  const f32x4* const from = part_at<NT>(p.part, tile) + ((i * NT + j) * 4 + 2 * g) * kThreads + t;
  const int64_t step = part_at<NT>(p.part, rest) - part_at<NT>(p.part, 0);
  constexpr int kV = (NT / 2) * 4 * kThreads;  // from gate to up
  float x[8] = {}, v[8] = {};
#pragma unroll 4
  for (int32_t s = 0; s < plan.splits; ++s)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const f32x4 a = from[s * step + r * kThreads];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[4 * r + c] += a[c];
      if (kUp) {
        const f32x4 b = from[s * step + r * kThreads + kV];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[4 * r + c] += b[c];
      }
    }
  const int32_t m = mw + (lane & 31);
  const int32_t n = col * kCols + ((w & 1) * kJ + j) * 32 + g * 16 + (lane >> 5) * 8;
  const int count = m < hi ? min(p.N - n, 8) : 0;
  const int64_t at = static_cast<int64_t>(m) * p.N + n;
  const Kept kept = load_kept<KIND>(p, at, count);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    exchange(x[k], x[4 + k]);
    if (kUp) exchange(v[k], v[4 + k]);
  }
  finish8<H, KIND>(p, at, n, count, x, v, kept);
}

// The most row tiles that T rows in E runs can make: every run may end in a partial tile.
int64_t most_row_tiles(int64_t T, int64_t E) { return T / kRows + (T < E ? T : E); }

// Whether tiles may be split: k is long enough, and if the host knows the tiles (no offsets), there
// are some to split.
bool split_pays(const FfnArgs& p, int products, int64_t tiles) {
  const int32_t blocks = products * ((p.K + kB - 1) / kB);
  return p.offsets ? blocks >= p.split_from : tile_splits(tiles, blocks, p.split_from) > 1;
}
// bytes of a round of parts
size_t part_bytes(int nt) { return sizeof(float) * kSlots * kRows * 64 * nt; }

template <class H, int KIND, int NT>
void launch_tiles(const FfnArgs& p, bool direct, int64_t tiles, int32_t ncols, hipStream_t s) {
  // a grid with room for the most parts: the rest of a round becomes at most a round of parts
  const dim3 g(static_cast<unsigned>(tiles + (p.part ? kSlots : 0))), b(kThreads);
  if (direct)
    hipLaunchKernelGGL((ffn_tile_kernel<H, KIND, NT, true>), g, b, 0, s, p, ncols);
  else if constexpr (NT == 2)
    hipLaunchKernelGGL((ffn_tile_kernel<H, KIND, 2, false>), g, b, 0, s, p, ncols);
  if (!p.part) return;
  const int64_t rest = tiles < kSlots ? tiles : kSlots - 1;
  const dim3 gj(static_cast<unsigned>(rest * 4 * (KIND == kFfnUp ? NT / 2 : NT)));
  hipLaunchKernelGGL((ffn_join_kernel<H, KIND, NT>), gj, b, 0, s, p, ncols);
}

bool misaligned(const void* p, size_t a);

template <int KIND>
int launch(FfnArgs p, int32_t dtype, void* workspace, size_t workspace_bytes, hipStream_t s, const char* what) {
  if (p.T == 0) return FP8Z1_OK;
  if (misaligned(workspace, 16)) return refuse(FP8Z1_EINVAL, what, "misaligned workspace");
  constexpr bool kTrans = KIND == kFfnDownBwd || KIND == kFfnUpBwd || KIND == kLinearBwd;
  const bool direct = !misaligned(p.x0, 4) && !misaligned(p.x1, 4) && !misaligned(p.w0, 4) && !misaligned(p.w1, 4) &&
                      (kTrans ? p.K % 2 == 0 && p.N % 4 == 0 : p.K % 4 == 0);
  // Few rows per expert (32 on average at most): the weights' read is what counts, and a tile of 128
  // rows would be mostly empty (128 tokens on 32 experts: 425 us by tiles, 250 by rows).  Above 12
  // rows the row kernel reads them slower, at 2.2 TB/s for 32 rows where tiles with direct
  // copies reach 3.5 after some 7 us more of latency: tiles from about 10^9 bytes x rows above 12.
  // (The average is all that the host knows; the row kernel keeps to it with any load, see there.)
  // (7168 x 2048, forward, rows and tiles: 1024 tokens on 32 experts 654 and 405 us, 256 on 8 169 and
  // 134, 128 on 8 122 and 138, 32 on 1 33 and 37.)
  if constexpr (!kTrans) {
    const double weights = static_cast<double>(KIND == kFfnUp ? 2 : 1) * p.E * p.N * p.K;
    if (static_cast<int64_t>(p.T) <= 32ll * p.E && (!direct || weights * (p.T - 12.0 * p.E) <= 1e9 * p.E)) {
      const bool aligned = !misaligned(p.x0, 16) && !misaligned(p.w0, 16) && !misaligned(p.w1, 16) && p.K % 16 == 0;
      if (dtype == FP8Z1_BF16)
        launch_rows<Bf16, KIND>(p, aligned, s);
      else
        launch_rows<F16, KIND>(p, aligned, s);
      return launched(what);
    }
  }
  const int64_t rows = most_row_tiles(p.T, p.E);
  const int32_t per = KIND == kFfnUp ? 32 : 64;  // columns per NT
  // 256 columns a tile where they fill the card; what goes through registers takes too many for it
  const bool wide = direct && rows * ((p.N + 4 * per - 1) / (4 * per)) >= kSlots;
  const int32_t cols = per * (wide ? 4 : 2), ncols = (p.N + cols - 1) / cols;
  const int64_t tiles = rows * ncols;
  if (tiles > 0x7fffffff - kSlots) return refuse(FP8Z1_ESHAPE, what, "too many tiles");
  p.split_from = direct ? kDirectFrom : kRegisterFrom;
  const int64_t known = p.offsets ? tiles : static_cast<int64_t>((p.T + kRows - 1) / kRows) * ncols;
  if (split_pays(p, KIND == kFfnUpBwd ? 2 : 1, known) && workspace_bytes >= part_bytes(wide ? 4 : 2))
    p.part = static_cast<float*>(workspace);
  if (dtype == FP8Z1_BF16 && wide)
    launch_tiles<Bf16, KIND, 4>(p, direct, tiles, ncols, s);
  else if (dtype == FP8Z1_BF16)
    launch_tiles<Bf16, KIND, 2>(p, direct, tiles, ncols, s);
  else if (wide)
    launch_tiles<F16, KIND, 4>(p, direct, tiles, ncols, s);
  else
    launch_tiles<F16, KIND, 2>(p, direct, tiles, ncols, s);
  return launched(what);
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

int check_product(const fp8z1_product* f, const int32_t* offsets, const char* what) {
  if (!f) return refuse(FP8Z1_EINVAL, what, "NULL description");
  if (f->dtype != FP8Z1_BF16 && f->dtype != FP8Z1_F16)
    return refuse(FP8Z1_EINVAL, what, "dtype must be FP8Z1_BF16 or FP8Z1_F16");
  if (f->x_dtype != f->dtype && f->x_dtype != FP8Z1_E4M3)
    return refuse(FP8Z1_EINVAL, what, "x_dtype must be dtype or FP8Z1_E4M3");
  if (f->act != FP8Z1_ACT_SILU && f->act != FP8Z1_ACT_GELU && f->act != FP8Z1_ACT_NONE)
    return refuse(FP8Z1_EINVAL, what, "act must be FP8Z1_ACT_SILU, FP8Z1_ACT_GELU or FP8Z1_ACT_NONE");
  if (f->T < 0 || f->T > FP8Z1_FFN_MAX_ROWS) return refuse(FP8Z1_ESHAPE, what, "T outside 0 .. 2^30");
  if (f->E < 1 || f->E > FP8Z1_FFN_MAX_EXPERTS) return refuse(FP8Z1_ESHAPE, what, "E outside 1 .. 65535");
  if (f->N < 1 || f->N > FP8Z1_FFN_MAX_WIDTH || f->K < 1 || f->K > FP8Z1_FFN_MAX_WIDTH)
    return refuse(FP8Z1_ESHAPE, what, "N and K must be 1 .. 2^20");
  if (!offsets && f->E != 1) return refuse(FP8Z1_EINVAL, what, "offsets may be NULL for one expert only");
  if (misaligned(offsets, 4)) return refuse(FP8Z1_EINVAL, what, "misaligned offsets");
  return FP8Z1_OK;
}

int check_cfg(const fp8z1_ffn* f, const int32_t* offsets, const char* what) {
  if (!f) return refuse(FP8Z1_EINVAL, what, "NULL description");
  if (f->dtype != FP8Z1_BF16 && f->dtype != FP8Z1_F16)
    return refuse(FP8Z1_EINVAL, what, "dtype must be FP8Z1_BF16 or FP8Z1_F16");
  if (f->act != FP8Z1_ACT_SILU && f->act != FP8Z1_ACT_GELU)
    return refuse(FP8Z1_EINVAL, what, "act must be FP8Z1_ACT_SILU or FP8Z1_ACT_GELU");
  if (f->T < 0 || f->T > FP8Z1_FFN_MAX_ROWS) return refuse(FP8Z1_ESHAPE, what, "T outside 0 .. 2^30");
  if (f->E < 1 || f->E > FP8Z1_FFN_MAX_EXPERTS) return refuse(FP8Z1_ESHAPE, what, "E outside 1 .. 65535");
  if (f->D < 1 || f->D > FP8Z1_FFN_MAX_WIDTH || f->F < 1 || f->F > FP8Z1_FFN_MAX_WIDTH)
    return refuse(FP8Z1_ESHAPE, what, "D and F must be 1 .. 2^20");
  if (!offsets && f->E != 1) return refuse(FP8Z1_EINVAL, what, "offsets may be NULL for one expert only");
  if (misaligned(offsets, 4)) return refuse(FP8Z1_EINVAL, what, "misaligned offsets");
  return FP8Z1_OK;
}

int check_rows(std::initializer_list<const void*> xs, const char* what) {
  for (const void* x : xs) {
    if (!x) return refuse(FP8Z1_EINVAL, what, "NULL argument");
    if (misaligned(x, 2)) return refuse(FP8Z1_EINVAL, what, "misaligned rows");
  }
  return FP8Z1_OK;
}

int check_weights(const uint8_t* codes, const float* scales, const char* what) {
  if (!codes || !scales) return refuse(FP8Z1_EINVAL, what, "NULL weights");
  if (misaligned(scales, 4)) return refuse(FP8Z1_EINVAL, what, "misaligned scales");
  return FP8Z1_OK;
}

FfnArgs base_args(const fp8z1_ffn* f, const int32_t* offsets, bool n_is_f) {
  FfnArgs p{};
  p.offsets = offsets;
  p.T = static_cast<int32_t>(f->T);
  p.E = static_cast<int32_t>(f->E);
  p.N = static_cast<int32_t>(n_is_f ? f->F : f->D);
  p.K = static_cast<int32_t>(n_is_f ? f->D : f->F);
  p.act = f->act;
  return p;
}

const uint8_t* bytes(const void* p) { return static_cast<const uint8_t*>(p); }

}  // namespace
}  // namespace fp8z1
