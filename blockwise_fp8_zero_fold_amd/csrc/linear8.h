// Products of rows in 8 bits with blockwise-FP8 weights: y = res + act(x W^T + bias), and both projections of the
// feed-forward block with the gated activation, whose result leaves in 8 bits.
//
// Of x[m][k] = sx[m][q] cx[m][k] and w[n][k] = sw[q][n / 128] cw[n][k], q = k / 128, the codes' products are summed
// over a block q of k on the matrix cores, without rounding a dequantized operand, and
//     acc[m][n] += (sx[m][q] sw[q]) sum_{k in q} cx[m][k] cw[n][k]
// adds the block to the float32 sum.
//
// The 8-bit matrix instruction (32x32x64, twice the 16-bit one's rate) adds the products of 8 consecutive k as
// fixed-point numbers with 13 bits below the largest one's power of two and cuts off the rest: errors of 1.5e-5 to 1e-4
// of a result, far below a rounding to 16 bits (4e-3, 5e-4), so y = res + act(p) is summed that way.  The
// result of gate and up leaves with float32 scales, which are held to float32's own accuracy: there the codes
// are widened to bfloat16, which holds them exactly, and the 16-bit instruction adds in float32.  The weights are the instruction's rows, so that a lane's 16 results are of one
// row of x: one scale for all of them, and one multiply-add each per 128 products.
#pragma once

#include <hip/hip_runtime.h>

#include "ffn.h"
#include "ffn_tile.h"
#include "rows.h"
#include "rows8.h"

namespace fp8z1 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 code32(uint4 a, uint4 b) {
  return i32x8{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w),
               static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
}
// 32 x 32 += 32 x 64 codes times 64 x 32 (E4M3, the instruction's own scales 1): lane l holds 32 codes of row l % 32 of
// either, the same k of both, and gets results as the 16-bit instruction of that shape gives them.
__device__ __forceinline__ f32x16 mma8(i32x8 a, i32x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
}
__device__ __forceinline__ f32x4 mma8_16(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
}

// A wave's direct copies as copy16_to_lds makes them (64 x 16 or 64 x 4 bytes), from `soff` bytes further on: the
// buffers stay as they are while k moves.
template <int BYTES>
__device__ __forceinline__ void copy_to_lds(buffer_t b, uint32_t off, uint32_t soff, uint32_t dst) {
  static_assert(BYTES == 16 || BYTES == 4, "one dword or four");
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(dst), "v"(off), "s"(b), "s"(soff)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(dst), "v"(off), "s"(b), "s"(soff)
                 : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(
      static_cast<int>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)(p)))));
}

// All waves of the workgroup are here with their LDS accesses done, and at most LEFT of each wave's copies are on
// their way.  (A barrier of the compiler's would wait for all of them.)
template <int LEFT>
__device__ __forceinline__ void meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// ------------------------------------------------------------------------------------------------ tiles

constexpr int kCols8 = 256;               // weight rows of a tile (up: 128 of gate, 128 of up)
constexpr int kA8 = kRows * kB, kB8 = kCols8 * kB;
constexpr int kStage8 = kA8 + kB8 + kRows * 4;  // codes of x, of the weights, and x's scales
constexpr int kCopies = 13;               // of a wave for a stage
constexpr int32_t kSlots8 = 256;          // workgroups that the card runs at once: one on each compute unit

// Work items: as in ffn.h, for one workgroup per compute unit.
__host__ __device__ __forceinline__ int32_t tile_splits8(int64_t tiles, int32_t blocks) {
  const int32_t rest = static_cast<int32_t>(tiles % kSlots8);
  if (!rest || blocks < 4) return 1;
  int32_t s = kSlots8 / rest, most = blocks / (tiles < kSlots8 ? 2 : 8);
  if (tiles < kSlots8) {
    const int32_t least = static_cast<int32_t>(sqrtf(20.0f * static_cast<float>(blocks) / static_cast<float>(rest)));
    most = least < most ? least : most;
  }
  if (s > most) s = most;
  return s > 1 ? s : 1;
}
__device__ __forceinline__ Plan plan_tiles8(const FfnArgs& p, int32_t ncols, int32_t blocks, int32_t& rowtiles,
                                            Run& first) {
  Plan plan = plan_tiles<kRows>(p.offsets, p.T, p.E, ncols, blocks, 0, rowtiles, first);
  const int32_t rest = plan.tiles % kSlots8, s = p.part ? tile_splits8(plan.tiles, blocks) : 1;
  if (s > 1) {
    plan.whole = plan.tiles - rest;
    plan.splits = s;
  }
  return plan;
}
__device__ __forceinline__ float* part8_at(float* part, int32_t at) {
  return part + static_cast<int64_t>(at) * (kRows * kCols8);
}
size_t part8_bytes() { return sizeof(float) * kSlots8 * kRows * kCols8; }

// a = act(gate) * up of 8 columns from column c of the results on, with 16 neighbouring lanes on the 128
// columns of a group: h and u where they are wanted, codes and the group's scale.
typedef uint32_t v2u_a1_rw_global_t __attribute__((ext_vector_type(2), aligned(1), address_space(1)));
template <class H>
__device__ __forceinline__ void finish_up8(const FfnArgs& p, int64_t m, int32_t n, int count, const float (&x)[8],
                                           const float (&v)[8]) {
  float a[8], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = act_value(p.act, x[i]) * v[i];
    top = fmaxf(top, i < count ? fabsf(a[i]) : 0.0f);
  }
  top = fmaxf(top, permuted<0xb1>(top));
  top = fmaxf(top, permuted<0x4e>(top));
  top = fmaxf(top, permuted<0x141>(top));
  top = fmaxf(top, permuted<0x140>(top));
  if (count <= 0) return;
  const float scale = row8_scale(top, p.pow2 != 0);
  if (n % kB == 0) p.code_scales[m * ((p.N + kB - 1) / kB) + n / kB] = scale;
  const uint32_t lo = codes4(a[0], a[1], a[2], a[3], scale), hi = codes4(a[4], a[5], a[6], a[7], scale);
  uint8_t* const to = p.codes + m * p.N + n;
  if (count == 8) {
    *(v2u_a1_rw_global_t*)(to) = v2u_t{lo, hi};
  } else {
    for (int i = 0; i < count; ++i) to[i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
  }
  if (p.o1) {
    uint32_t hk[4], uk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hk[i] = static_cast<uint32_t>(H::from_f32(x[2 * i])) | static_cast<uint32_t>(H::from_f32(x[2 * i + 1])) << 16;
      uk[i] = static_cast<uint32_t>(H::from_f32(v[2 * i])) | static_cast<uint32_t>(H::from_f32(v[2 * i + 1])) << 16;
    }
    store_row8(p.o1 + m * p.N + n, hk, count);
    store_row8(p.o2 + m * p.N + n, uk, count);
  }
}

// DIRECT: rows of x and codes are 4-byte aligned, and a stage is copied to LDS directly.
//
// A workgroup of 4 waves computes 128 rows x 256 weight rows, each wave 64 x 128 as 2 x 4 matrix tiles, one wave to a
// SIMD with all its registers.  While the matrix cores work on block q out of registers, block q + 1 is read from LDS
// into others and blocks q + 2 and q + 3 are on their way to LDS.
template <class H, int KIND, bool DIRECT>
__global__ __launch_bounds__(kThreads, 1) void tile8_kernel(FfnArgs p, int32_t ncols) {
  constexpr bool kUp = KIND == kFfnUp;
  constexpr int kOut = kUp ? kCols8 / 2 : kCols8;  // output columns of a tile
  __shared__ __attribute__((aligned(16))) uint8_t lds[3 * kStage8];
  static_assert(3 * kStage8 >= kResultBytes + 2 * kRows * 4, "results use the stages' LDS");

  const int32_t kb = (p.K + kB - 1) / kB;
  int32_t rowtiles, e, lo, hi, m0, col;
  Run first;
  const int32_t item = static_cast<int32_t>(blockIdx.x);
  const Plan plan = plan_tiles8(p, ncols, kb, rowtiles, first);
  if (item >= plan.items()) return;
  const bool split = item >= plan.whole;
  const int32_t rest = plan.tiles - plan.whole;
  const int32_t id = split ? plan.whole + (item - plan.whole) % rest : xcd_run(item, plan.whole);
  const int32_t sp = split ? (item - plan.whole) / rest : 0, parts = split ? plan.splits : 1;
  const int32_t q0 = kb * sp / parts, q1 = kb * (sp + 1) / parts;
  if (!find_tile<kRows>(p.offsets, p.T, p.E, ncols, rowtiles, first, id, e, lo, hi, m0, col)) return;
  const int32_t n0 = col * kOut, N = p.N, K = p.K;
  if (KIND == kLinear && p.bias) p.bias += static_cast<int64_t>(e) * N;
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6), wm = w >> 1, wn = w & 1;
  const int half = lane >> 5, l32 = lane & 31;
  const int32_t nb = (N + kB - 1) / kB;

  // This thread's 16-byte chunks of a stage: chunk c of rows t / 8 + 32 j; rows past the end repeat the last.
  const int c16 = ((t & 7) ^ swizzle_a(t >> 3)) * 16, r0 = t >> 3;
  uint32_t aoff[4], boff[8];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    aoff[j] = static_cast<uint32_t>(min(r0 + 32 * j, hi - 1 - m0)) * static_cast<uint32_t>(K) + c16;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    boff[j] = static_cast<uint32_t>(min(r0 + 32 * (kUp ? j % 4 : j), N - 1 - n0)) * static_cast<uint32_t>(K) + c16;
  const uint32_t soff = static_cast<uint32_t>(min(t & (kRows - 1), hi - 1 - m0)) * static_cast<uint32_t>(kb) * 4;
  const int64_t abase = static_cast<int64_t>(m0) * K, bbase = (static_cast<int64_t>(e) * N + n0) * K;

  const float* const xs = p.xs + static_cast<int64_t>(m0) * kb;
  // (the buffers end with the tensors: what lies behind is not read)
  const int64_t wleft = static_cast<int64_t>(p.E) * N * K - bbase;
  const buffer_t xbuf = make_buffer(p.x0 + abase, static_cast<int64_t>(p.T - m0) * K),
                 w0buf = make_buffer(p.w0 + bbase, wleft), w1buf = make_buffer((kUp ? p.w1 : p.w0) + bbase, wleft),
                 sbuf = make_buffer(reinterpret_cast<const uint8_t*>(xs), static_cast<int64_t>(p.T - m0) * kb * 4);
  const uint32_t lds0 = lds_address(lds);
  // copy j of kCopies of the stage at LDS offset `to`
  auto copy = [&](int j, int32_t q, uint32_t to) {
    const uint32_t at = lds0 + to + w * 1024;
    if (j < 4)
      copy_to_lds<16>(xbuf, aoff[j], q * kB, at + j * (kThreads * 16));
    else if (j < 12)
      copy_to_lds<16>(j < 8 ? w0buf : w1buf, boff[j - 4], q * kB, at + kA8 + (j - 4) * (kThreads * 16));
    else  // (by two waves each: as many copies of every wave)
      copy_to_lds<4>(sbuf, soff, q * 4, lds0 + to + kA8 + kB8 + (w & 1) * 256);
  };
  // Through registers: batch b of 3, 4 of the 12 chunks, and the scales with the first.
  uint4 held[4];
  float scale_held = 0.0f;
  auto fetch = [&](int batch, int32_t q) {
    const int32_t k0 = q * kB;
    const uint8_t* const from = (batch == 0 ? p.x0 + abase : (kUp && batch == 2 ? p.w1 : p.w0) + bbase) + k0;
    const uint32_t* const off = batch == 0 ? aoff : boff + 4 * (batch - 1);
    const int n = K - k0 - c16;  // codes of the row from this chunk on
#pragma unroll
    for (int j = 0; j < 4; ++j) held[j] = k0 + kB <= K ? ld16(from + off[j]) : ld16_part(from + off[j], n, k0 + c16);
    if (batch == 0) scale_held = xs[soff / 4 + q];
  };
  auto put = [&](int batch, uint8_t* to) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(to + (t + kThreads * (4 * batch + j)) * 16) = held[j];
    if (batch == 0 && t < kRows) *reinterpret_cast<float*>(to + kA8 + kB8 + t * 4) = scale_held;
  };
  // Clears what the last stage holds past the end of k (both operands: 0 times a NaN is none).
  auto clear_past = [&](uint8_t* at) {
    const int n = K - (kb - 1) * kB - c16;
    if (n >= 16) return;
    for (int j = 0; j < 12; ++j) {
      uint4* const x = reinterpret_cast<uint4*>(at + (t + kThreads * j) * 16);
      uint4 v = *x;
      uint32_t* const o[4] = {&v.x, &v.y, &v.z, &v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int in = n - 4 * i;
        *o[i] = in >= 4 ? *o[i] : in > 0 ? *o[i] & (0xffffffffu >> (32 - 8 * in)) : 0u;
      }
      *x = v;
    }
  };

  const int swz = swizzle_a(l32);  // (that of every row read: they lie 32 apart)
  // the weights' scales of this wave's columns, one per block of k (two matrices: one each)
  const int32_t nblk = min((n0 + (kUp ? 0 : wn * 128)) / kB, nb - 1);
  const int64_t sat = (static_cast<int64_t>(e) * nb + nblk) * kb;
  typedef const __attribute__((address_space(4))) float* scalar_t;
  auto wscale = [&](int32_t q, int which) { return ((scalar_t)((which ? p.s1 : p.s0) + sat))[q]; };

  f32x16 acc[2][4];
  const f32x16 zero = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = zero;

  const bool tail = DIRECT && K % kB != 0;
  uint32_t cur = 0, next = kStage8, last = 2 * kStage8;  // LDS offsets of stages q, q + 1 and q + 2
  auto rotate = [&] {
    const uint32_t x = cur;
    cur = next;
    next = last;
    last = x;
  };
  if (DIRECT) {
#pragma unroll 1
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int j = 0; j < kCopies; ++j) copy(j, min(q0 + k, q1 - 1), k * kStage8);
    meet<2 * kCopies>();
  } else {
#pragma unroll 1
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        fetch(b, min(q0 + k, q1 - 1));
        put(b, lds + k * kStage8);
      }
    __syncthreads();
  }
  if (tail && q0 == kb - 1) {
    clear_past(lds);
    __syncthreads();
  }
  if constexpr (kUp) {
    // Gate and up: codes widened to bfloat16, which holds them, so that the sums are float32 sums (see the top).
    // A step is 32 k, chunk c of a block's 4 from both halves of the lanes, two matrix instructions for each of the
    // 8 tiles.  In its 8 slots, a tile's instructions each, the next step's chunks are read from LDS and
    // widened: a weight's when its two tiles of this step are done, x's into another set.
    typedef Bf16::v8 v8;
    v8 W[4][2], X[2][2][2];
    uint4 rw[4], rx[2];
    auto read_x = [&](uint32_t from, int c, int i) {
      rx[i] = *reinterpret_cast<const uint4*>(lds + from + (wm * 64 + i * 32 + l32) * kB + (((half * 4 + c) ^ swz) << 4));
    };
    auto read_w = [&](uint32_t from, int c, int j) {  // (two tile columns of gate, then the same of up)
      rw[j] = *reinterpret_cast<const uint4*>(lds + from + kA8 + ((j / 2) * 128 + wn * 64 + (j % 2) * 32 + l32) * kB +
                                              (((half * 4 + c) ^ swz) << 4));
    };
    auto wide_x = [&](int set, int i, int k) {
      X[set][i][k] = k ? widen8<Bf16>(rx[i].z, rx[i].w) : widen8<Bf16>(rx[i].x, rx[i].y);
    };
    auto wide_w = [&](int j, int k) { W[j][k] = k ? widen8<Bf16>(rw[j].z, rw[j].w) : widen8<Bf16>(rw[j].x, rw[j].y); };
    // acc is held in units of the current block's scale: between blocks it is multiplied by scale_before / scale_now.
    // That does no harm while all scales lie between 2^-70 and 2^20, which every wave watches; if one does not, the
    // tile is done again, block by block.
    float s[2][2], ratio[2][2];
    bool near = true;
    auto scales = [&](uint32_t from, const float (&sw)[2], float (&to)[2][2]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float sx = *reinterpret_cast<const float*>(lds + from + kA8 + kB8 + (wm * 64 + i * 32 + l32) * 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          to[i][k] = sx * sw[k];
          near = near && to[i][k] >= 0x1p-70f && to[i][k] <= 0x1p20f;
        }
      }
    };
    auto rescale = [&](int u, int r0) {
#pragma unroll
      for (int r = r0; r < r0 + 8; ++r) acc[u & 1][u >> 1][r] *= ratio[u & 1][u >> 2];
    };
    auto pin = [&] {  // (the work stays in its step: nothing of it is moved past a barrier behind it)
#pragma unroll
      for (int u = 0; u < 8; ++u) asm volatile("" : "+v"(acc[u & 1][u >> 1]));
#pragma unroll
      for (int k = 0; k < 6; ++k) asm volatile("" : "+v"(W[k >> 1][k & 1]));
#pragma unroll
      for (int k = 0; k < 4; ++k) asm volatile("" : "+v"(X[1][k >> 1][k & 1]));
    };
    // Block q; its first chunk is in X[0] and W (W[3] in rw[3]).  Leaves the next block's so.
    auto turn = [&](int32_t q) {
      const int32_t far = min(q + 3, q1 - 1), after = min(q + 1, q1 - 1);
      const float sw[2] = {wscale(after, 0), wscale(after, 1)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t from = cur;
        if (c == 3) {
          pin();
          if (DIRECT)
            meet<kCopies>();  // stage q + 1 is there, and all waves have read stage q
          else
            __syncthreads();
          if (tail && q + 2 == kb) {
            clear_past(lds + next);
            __syncthreads();
          }
          from = next;
        }
        const int set = c & 1, cn = (c + 1) & 3;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = u & 1, j = u >> 1;
          acc[i][j] = Bf16::mma32(W[j][0], X[set][i][0], acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
          if (u == 0) {
            read_x(from, cn, 0);
            read_w(from, cn, 0);
            wide_w(3, 0);
          } else if (u == 1) {
            read_x(from, cn, 1);
            read_w(from, cn, 1);
          } else if (u == 2) {
            read_w(from, cn, 2);
            wide_x(set ^ 1, 0, 0);
          } else if (u == 3) {
            wide_x(set ^ 1, 0, 1);
          } else if (u == 4) {
            wide_w(0, 1);
          } else if (u == 5) {
            read_w(from, cn, 3);
            wide_x(set ^ 1, 1, 1);
          } else if (u == 6) {
            wide_w(1, 1);
          } else {
            wide_w(2, 1);
          }
          if (c == 0 && u < 7) rescale(u + 1, 0);
          __builtin_amdgcn_sched_barrier(0);
          acc[i][j] = Bf16::mma32(W[j][1], X[set][i][1], acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
          if (u == 1) {
            wide_w(3, 1);
          } else if (u == 3) {
            wide_w(0, 0);
          } else if (u == 4) {
            wide_x(set ^ 1, 1, 0);
          } else if (u == 5) {
            wide_w(1, 0);
          } else if (u == 6) {
            wide_w(2, 0);
          }
          if (c == 0 && u < 7) rescale(u + 1, 8);
          if (c == 3) {
            if (DIRECT) {
              copy(u, far, cur);
              if (u + 8 < kCopies) copy(u + 8, far, cur);
            } else if (u < 3) {
              fetch(u, far);
              put(u, lds + cur);
            }
            if (u == 3) {
              float to[2][2];
              scales(next, sw, to);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                ratio[k >> 1][k & 1] = s[k >> 1][k & 1] * __builtin_amdgcn_rcpf(to[k >> 1][k & 1]);
                s[k >> 1][k & 1] = to[k >> 1][k & 1];
              }
            }
            if (u == 7) {
              rescale(0, 0);
              rescale(0, 8);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      rotate();
    };
    const float sw0[2] = {wscale(q0, 0), wscale(q0, 1)};
    scales(0, sw0, s);
#pragma unroll
    for (int k = 0; k < 4; ++k) ratio[k >> 1][k & 1] = 1.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      read_w(0, 0, j);
      if (j < 3) {
        wide_w(j, 0);
        wide_w(j, 1);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      read_x(0, 0, i);
      wide_x(0, i, 0);
      wide_x(0, i, 1);
    }
    for (int32_t q = q0; q < q1; ++q) turn(q);
    // (the last turn has fetched its own block as the next: its scales are the units still)
    if (DIRECT) wait_copies();
    int32_t* const far_apart = reinterpret_cast<int32_t*>(lds + kResultBytes);
    __syncthreads();
    if (t == 0) *far_apart = 0;
    __syncthreads();
    if (!near) *far_apart = 1;
    __syncthreads();
    if (!*far_apart) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[u & 1][u >> 1][r] *= s[u & 1][u >> 2];
    } else {
      // a pass for each tile column: the blocks' sums apart, times their scales
      auto pass = [&](auto j_) {
        constexpr int j = decltype(j_)::value;
        acc[0][j] = acc[1][j] = zero;
        for (int32_t q = q0; q < q1; ++q) {
          __syncthreads();
          if (DIRECT) {
#pragma unroll
            for (int k = 0; k < kCopies; ++k) copy(k, q, 0);
            wait_copies();
          } else {
#pragma unroll
            for (int b = 0; b < 3; ++b) {
              fetch(b, q);
              put(b, lds);
            }
          }
          __syncthreads();
          if (tail && q + 1 == kb) {
            clear_past(lds);
            __syncthreads();
          }
          f32x16 part[2] = {zero, zero};
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            read_w(0, c, j);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              read_x(0, c, i);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const v8 wk = k ? widen8<Bf16>(rw[j].z, rw[j].w) : widen8<Bf16>(rw[j].x, rw[j].y);
                const v8 xk = k ? widen8<Bf16>(rx[i].z, rx[i].w) : widen8<Bf16>(rx[i].x, rx[i].y);
                part[i] = Bf16::mma32(wk, xk, part[i]);
              }
            }
          }
          const float sw = wscale(q, j / 2);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float sx = *reinterpret_cast<const float*>(lds + kA8 + kB8 + (wm * 64 + i * 32 + l32) * 4);
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(sx * sw, part[i][r], acc[i][j][r]);
          }
        }
      };
      pass(Int<0>{});
      pass(Int<1>{});
      pass(Int<2>{});
      pass(Int<3>{});
    }
  } else {
    struct Block {
      uint4 x[2][4], w[4][4];
      float s[2];
    };
    // part u of 8 of a block's reads: 3 chunks, x first; and its scales
    auto read = [&](const uint8_t* from, Block& b, int u) {
#pragma unroll
      for (int k = 3 * u; k < 3 * u + 3; ++k) {
        const int c = k & 3, at = ((half * 4 + c) ^ swz) << 4;
        if (k < 8) {
          b.x[k >> 2][c] = *reinterpret_cast<const uint4*>(from + (wm * 64 + l32) * kB + at + (k >> 2) * (32 * kB));
        } else {
          const int j = (k - 8) >> 2;
          b.w[j][c] = *reinterpret_cast<const uint4*>(from + kA8 + (wn * 128 + j * 32 + l32) * kB + at);
        }
      }
      if (u == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          b.s[i] = *reinterpret_cast<const float*>(from + kA8 + kB8 + (wm * 64 + i * 32 + l32) * 4);
    };

    // Tile u of a block: column j = u / 2 of the weights, row i = u % 2 of x.  Its two products go to one of four
    // partial sums, which are added to acc two tiles later: a result may be read some 20 instructions after its
    // product is issued, and the additions of one tile run under the products of another.
    f32x16 part[4];
    part[2] = part[3] = zero;
    float s[2] = {};  // of the block before: its last two tiles are still to be added
    auto add = [&](int u, int r0) {
#pragma unroll
      for (int r = r0; r < r0 + 8; ++r)
        acc[u & 1][u >> 1][r] = fmaf(s[u & 1], part[u & 3][r], acc[u & 1][u >> 1][r]);
    };

    // Block q out of registers; block q + 1 from LDS to registers, block q + 3 from memory to LDS.
    auto turn = [&](int32_t q, const Block& now, Block& then) {
      if (DIRECT)
        meet<kCopies>();  // stage q + 1 is there, and all waves have read stage q
      else
        __syncthreads();
      if (tail && q + 2 == kb) {
        clear_past(lds + next);
        __syncthreads();
      }
      // (the last turns fetch the last block again rather than branch)
      const int32_t far = min(q + 3, q1 - 1);
      const float sw = wscale(q, 0);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = u & 1, j = u >> 1, before = (u + 6) & 7;
        f32x16 d = mma8(code32(now.w[j][0], now.w[j][1]), code32(now.x[i][0], now.x[i][1]), zero);
        __builtin_amdgcn_sched_barrier(0);
        read(lds + next, then, u);
        add(before, 0);
        __builtin_amdgcn_sched_barrier(0);
        part[u & 3] = mma8(code32(now.w[j][2], now.w[j][3]), code32(now.x[i][2], now.x[i][3]), d);
        __builtin_amdgcn_sched_barrier(0);
        if (DIRECT) {
          copy(u, far, cur);
          if (u + 8 < kCopies) copy(u + 8, far, cur);
        } else {
          if (u == 2 || u == 4 || u == 7) put(u / 3, lds + cur);
          if (u == 0 || u == 2 || u == 4) fetch(u / 2, far);
        }
        add(before, 8);
        if (u == 1)
#pragma unroll
          for (int k = 0; k < 2; ++k) s[k] = now.s[k] * sw;
        __builtin_amdgcn_sched_barrier(0);
      }
      // (the work stays in its turn: nothing of it is moved past the next turn's barrier)
#pragma unroll
      for (int u = 0; u < 8; ++u) asm volatile("" : "+v"(acc[u & 1][u >> 1]));
      asm volatile("" : "+v"(part[2]));
      asm volatile("" : "+v"(part[3]));
      rotate();
    };

    Block b0, b1;
#pragma unroll
    for (int u = 0; u < 8; ++u) read(lds, b0, u);
    int32_t q = q0;
    for (; q + 1 < q1; q += 2) {
      turn(q, b0, b1);
      turn(q + 1, b1, b0);
    }
    if (q < q1) turn(q, b0, b1);
#pragma unroll
    for (int u = 6; u < 8; ++u) {
      add(u, 0);
      add(u, 8);
    }
  }
  if (DIRECT) wait_copies();
  __syncthreads();  // the results take the stages' place

  uint8_t* const mine = lds + w * (kResultBytes / 4);
  const int32_t mw = m0 + wm * 64;
  if (split) {  // float32 sums [128][256], up: gate's 128 columns, then up's
    float* const to = part8_at(p.part, item - plan.whole) + static_cast<int64_t>(wm * 64) * kCols8;
#pragma unroll 1
    for (int half_ = 0; half_ < 2; ++half_) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lay_tile(half_ ? acc[i][2] : acc[i][0], mine, i, 0);
        lay_tile(half_ ? acc[i][3] : acc[i][1], mine, i, 1);
      }
      handed_over();
      const int32_t c0 = kUp ? half_ * 128 + wn * 64 : wn * 128 + half_ * 64;
      for (int k = 0; k < 8; ++k) {
        const int r = k * 8 + (lane >> 3), c = lane & 7;
        if (mw + r >= hi) continue;
        float x[8];
        read8(mine, r, 2 * c, x);
        f32x4* const o = reinterpret_cast<f32x4*>(to + static_cast<int64_t>(r) * kCols8 + c0 + 8 * c);
        o[0] = f32x4{x[0], x[1], x[2], x[3]};
        o[1] = f32x4{x[4], x[5], x[6], x[7]};
      }
      handed_over();
    }
    return;
  }
  if constexpr (!kUp) {
#pragma unroll 1
    for (int half_ = 0; half_ < 2; ++half_) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lay_tile(half_ ? acc[i][2] : acc[i][0], mine, i, 0);
        lay_tile(half_ ? acc[i][3] : acc[i][1], mine, i, 1);
      }
      handed_over();
      store_rows<H, kLinear>(p, mine, mw, hi, n0 + wn * 128 + half_ * 64);
      handed_over();
    }
  } else {
    if (p.o1) {  // h and u: 32 columns of each at a time
#pragma unroll 1
      for (int half_ = 0; half_ < 2; ++half_) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lay_tile(half_ ? acc[i][1] : acc[i][0], mine, i, 0);
          lay_tile(half_ ? acc[i][3] : acc[i][2], mine, i, 1);
        }
        handed_over();
        for (int k = 0; k < 4; ++k) {
          const int r = k * 16 + (lane >> 2), c = lane & 3;
          const int32_t n = n0 + wn * 64 + half_ * 32 + 8 * c;
          const int count = mw + r < hi ? min(N - n, 8) : 0;
          if (count <= 0) continue;
          const int64_t at = static_cast<int64_t>(mw + r) * N + n;
          float x[8], v[8];
          read8(mine, r, 2 * c, x);
          read8(mine, r, 8 + 2 * c, v);
          uint32_t hk[4], uk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hk[i] = static_cast<uint32_t>(H::from_f32(x[2 * i])) | static_cast<uint32_t>(H::from_f32(x[2 * i + 1])) << 16;
            uk[i] = static_cast<uint32_t>(H::from_f32(v[2 * i])) | static_cast<uint32_t>(H::from_f32(v[2 * i + 1])) << 16;
          }
          store_row8(p.o1 + at, hk, count);
          store_row8(p.o2 + at, uk, count);
        }
        handed_over();
      }
    }
    // a in place of gate; the largest magnitude of a row over this wave's 64 columns, then over both waves'
    float* const tops = reinterpret_cast<float*>(lds + kResultBytes);  // [2][128]
    float top[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int32_t n = n0 + wn * 64 + j * 32 + 8 * (r / 4) + 4 * half + r % 4;
          const float a = act_value(p.act, acc[i][j][r]) * acc[i][j + 2][r];
          acc[i][j][r] = a;
          top[i] = fmaxf(top[i], n < N ? fabsf(a) : 0.0f);
        }
      top[i] = fmaxf(top[i], __shfl_xor(top[i], 32));
      if (half == 0) tops[wn * kRows + wm * 64 + i * 32 + l32] = top[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = wm * 64 + i * 32 + l32;
      const float scale = row8_scale(fmaxf(top[i], tops[(1 - wn) * kRows + r]), p.pow2 != 0);
      if (wn == 0 && half == 0 && m0 + r < hi) p.code_scales[static_cast<int64_t>(m0 + r) * nb + n0 / kB] = scale;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<uint32_t*>(mine + (i * 32 + l32) * 64 + ((j * 32 + 8 * g + 4 * half) ^ ((l32 & 3) << 4))) =
              codes4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3], scale);
    }
    handed_over();
    for (int k = 0; k < 4; ++k) {
      const int r = k * 16 + (lane >> 2), c = (lane & 3) * 16;
      const int32_t n = n0 + wn * 64 + c, count = mw + r < hi ? min(N - n, 16) : 0;
      if (count <= 0) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(mine + r * 64 + (c ^ ((r & 3) << 4)));
      uint8_t* const to = p.codes + static_cast<int64_t>(mw + r) * N + n;
      typedef uint32_t v4u_a1_rw_t __attribute__((ext_vector_type(4), aligned(1), address_space(1)));
      if (count == 16) {
        *(v4u_a1_rw_t*)(to) = v4u_v_t{v.x, v.y, v.z, v.w};
      } else {
        const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < count) to[i] = static_cast<uint8_t>(words[i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

// The split tiles: their parts' sums added in order, and the results.  16 lanes take 128 columns of a row.
template <class H, int KIND>
__global__ __launch_bounds__(kThreads) void join8_kernel(FfnArgs p, int32_t ncols) {
  constexpr bool kUp = KIND == kFfnUp;
  constexpr int kOut = kUp ? kCols8 / 2 : kCols8, kLanes = kOut / 8, kTurns = kRows * kLanes / kThreads;
  const int32_t kb = (p.K + kB - 1) / kB;
  int32_t rowtiles, e, lo, hi, m0, col;
  Run first;
  const Plan plan = plan_tiles8(p, ncols, kb, rowtiles, first);
  const int32_t rest = plan.tiles - plan.whole, tile = static_cast<int32_t>(blockIdx.x) / kTurns;
  if (tile >= rest) return;
  if (!find_tile<kRows>(p.offsets, p.T, p.E, ncols, rowtiles, first, plan.whole + tile, e, lo, hi, m0, col)) return;
  if (KIND == kLinear && p.bias) p.bias += static_cast<int64_t>(e) * p.N;
  const int r = static_cast<int>(blockIdx.x % kTurns) * (kThreads / kLanes) + threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  const int32_t n = col * kOut + 8 * c, m = m0 + r, count = m < hi ? min(p.N - n, 8) : 0;
  float x[8] = {}, v[8] = {};
  if (m < hi) {  // (the parts of rows past the run were not written)
    const f32x4* from = reinterpret_cast<const f32x4*>(part8_at(p.part, tile) + static_cast<int64_t>(r) * kCols8 + 8 * c);
    const int64_t step = static_cast<int64_t>(rest) * (kRows * kCols8) / 4;
#pragma unroll 4
    for (int32_t s = 0; s < plan.splits; ++s)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f32x4 a = from[s * step + k];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * k + i] += a[i];
        if (kUp) {
          const f32x4 b = from[s * step + 128 / 4 + k];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * k + i] += b[i];
        }
      }
  }
  if constexpr (kUp)
    finish_up8<H>(p, m, n, count, x, v);
  else if (count > 0)
    finish_linear<H>(p, static_cast<int64_t>(m) * p.N + n, n, count, x);
}

// ------------------------------------------------------------------------------------------- few rows

// Few rows per expert: bound by the read of the weights, which go from memory into registers as
// the matrix instruction's operand.  A workgroup takes 16 weight rows and 16 TT rows of x; its WAVES waves share the
// blocks of k and their sums are added in order.  Up: gate's or up's 16 rows (blockIdx.x), the float32
// sums to p.part [T][2][N] for finish_rows8_kernel.
template <class H, int KIND, int WAVES, int TT, bool ALIGNED>
__global__ __launch_bounds__(WAVES * 64) void rows8_kernel(FfnArgs p) {
  constexpr bool kUp = KIND == kFfnUp;
  __shared__ f32x4 sums[WAVES][TT][64];
  int32_t e, lo, hi, t0;
  const int32_t group = static_cast<int32_t>(blockIdx.z * gridDim.y + blockIdx.y);
  if (!find_group<16 * TT>(p.offsets, p.T, p.E, group, e, lo, hi, t0)) return;
  const int32_t N = p.N, K = p.K, strips = (N + 15) / 16;
  const int which = kUp && static_cast<int32_t>(blockIdx.x) >= strips;
  const int32_t n0 = (static_cast<int32_t>(blockIdx.x) - (which ? strips : 0)) * 16;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int32_t kb = (K + kB - 1) / kB, nb = (N + kB - 1) / kB;
  const uint8_t* const wt = (which ? p.w1 : p.w0) + (static_cast<int64_t>(e) * N + min(n0 + r, N - 1)) * K + g * 32;
  const float* const sc = (which ? p.s1 : p.s0) + (static_cast<int64_t>(e) * nb + n0 / kB) * kb;
  const uint8_t* xr[TT];
  const float* xs[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int64_t row = min(t0 + 16 * i + r, hi - 1);
    xr[i] = p.x0 + row * K + g * 32;
    xs[i] = p.xs + row * kb;
  }
  struct Block {
    uint4 c[2], x[TT][2];
    float s[TT], sw;
  };
  auto load16 = [&](const uint8_t* from, int32_t left, int32_t before) {
    if (ALIGNED) return left > 0 ? *reinterpret_cast<const uint4*>(from) : make_uint4(0u, 0u, 0u, 0u);
    return ld16_part(from, left, before);
  };
  auto load = [&](int32_t q, Block& b) {
    const int32_t at = q * kB, left = K - at - g * 32;  // of this lane's 32 k
    b.sw = sc[q];
#pragma unroll
    for (int i = 0; i < 2; ++i) b.c[i] = load16(wt + at + 16 * i, left - 16 * i, at + g * 32 + 16 * i);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      b.s[t] = xs[t][q];
#pragma unroll
      for (int i = 0; i < 2; ++i) b.x[t][i] = load16(xr[t] + at + 16 * i, left - 16 * i, at + g * 32 + 16 * i);
    }
  };
  f32x4 acc[TT];
  const f32x4 zero = {};
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = zero;
  auto add = [&](const Block& b) {
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      f32x4 part = zero;
      if constexpr (kUp) {  // (float32 sums, as on tiles)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          part = Bf16::mma16(widen8<Bf16>(b.c[i].x, b.c[i].y), widen8<Bf16>(b.x[t][i].x, b.x[t][i].y), part);
          part = Bf16::mma16(widen8<Bf16>(b.c[i].z, b.c[i].w), widen8<Bf16>(b.x[t][i].z, b.x[t][i].w), part);
        }
      } else {
        part = mma8_16(code32(b.c[0], b.c[1]), code32(b.x[t][0], b.x[t][1]), zero);
      }
      const float s = b.s[t] * b.sw;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(s, part[i], acc[t][i]);
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
  for (int t = 0; t < TT; ++t) sums[w][t][lane] = acc[t];
  __syncthreads();
  if (w >= TT) return;
  f32x4 v = sums[0][w][lane];
  for (int k = 1; k < WAVES; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += sums[k][w][lane][i];
  const int32_t t = t0 + 16 * w + r;
  if (t >= hi) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t n = n0 + 4 * g + i;
    if (n >= N) continue;
    if (kUp) {
      p.part[(static_cast<int64_t>(t) * 2 + which) * N + n] = v[i];
    } else {
      const int64_t at = static_cast<int64_t>(t) * N + n;
      const float b = p.bias ? v[i] + p.bias[static_cast<int64_t>(e) * N + n] : v[i];
      const float y = linear_act(p.act, b), res = p.res ? H::to_f32(p.res[at]) : 0.0f;
      p.o0[at] = H::from_f32(p.res ? y + res : y);
      if (p.o1) p.o1[at] = H::from_f32(b);
    }
  }
}

// The gated activation of the sums in p.part, 8 columns per thread, rows of all experts alike.
template <class H>
__global__ __launch_bounds__(kThreads) void finish_rows8_kernel(FfnArgs p) {
  const int32_t groups = (p.N + kB - 1) / kB;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + threadIdx.x / 16;
  const int64_t m = unit / groups;
  const int32_t n = static_cast<int32_t>(unit % groups) * kB + (threadIdx.x % 16) * 8;
  // rows that no expert covers have no sums
  const int32_t lo = p.offsets ? p.offsets[0] : 0, hi = p.offsets ? p.offsets[p.E] : p.T;
  const int count = m < p.T && m >= lo && m < hi ? min(p.N - n, 8) : 0;
  float x[8] = {}, v[8] = {};
  if (count > 0) {
    load8<F32>(p.part + m * 2 * p.N, p.N, n, x);
    load8<F32>(p.part + (m * 2 + 1) * p.N, p.N, n, v);
  }
  finish_up8<H>(p, m, n, count, x, v);
}

template <class H, int KIND, int WAVES, int TT>
void launch_rows8_as(const FfnArgs& p, bool aligned, hipStream_t s) {
  const int64_t groups = static_cast<int64_t>(p.E) + p.T / (16 * TT);
  const int64_t turns = (groups + 65534) / 65535;  // (a grid's y ends at 65,535)
  const dim3 g(static_cast<unsigned>((p.N + 15) / 16 * (KIND == kFfnUp ? 2 : 1)),
               static_cast<unsigned>((groups + turns - 1) / turns), static_cast<unsigned>(turns));
  if (aligned)
    hipLaunchKernelGGL((rows8_kernel<H, KIND, WAVES, TT, true>), g, dim3(WAVES * 64), 0, s, p);
  else
    hipLaunchKernelGGL((rows8_kernel<H, KIND, WAVES, TT, false>), g, dim3(WAVES * 64), 0, s, p);
}

template <class H, int KIND>
void launch_rows8(const FfnArgs& p, bool aligned, hipStream_t s) {
  const bool deep = static_cast<int64_t>((p.N + 15) / 16) * (KIND == kFfnUp ? 2 : 1) * p.E < 1024;
  const bool two = static_cast<int64_t>(p.T) > 8ll * p.E;
  if (deep && two)
    launch_rows8_as<H, KIND, 8, 2>(p, aligned, s);
  else if (deep)
    launch_rows8_as<H, KIND, 8, 1>(p, aligned, s);
  else if (two)
    launch_rows8_as<H, KIND, 4, 2>(p, aligned, s);
  else
    launch_rows8_as<H, KIND, 4, 1>(p, aligned, s);
  if constexpr (KIND == kFfnUp) {
    const int64_t units = static_cast<int64_t>(p.T) * ((p.N + kB - 1) / kB);
    hipLaunchKernelGGL((finish_rows8_kernel<H>), dim3(static_cast<unsigned>((units + 15) / 16)), dim3(kThreads), 0, s, p);
  }
}

// up's sums of few rows
size_t rows8_bytes(int64_t T, int64_t N) { return sizeof(float) * 2 * static_cast<size_t>(T) * static_cast<size_t>(N); }
bool few_rows8(int64_t T, int64_t E) { return T <= 32 * E; }

template <class H, int KIND>
void launch_tiles8(const FfnArgs& p, bool direct, int64_t tiles, int32_t ncols, hipStream_t s) {
  constexpr int kTurns = KIND == kFfnUp ? 8 : 16;
  const dim3 g(static_cast<unsigned>(tiles + (p.part ? kSlots8 : 0))), b(kThreads);
  if (direct)
    hipLaunchKernelGGL((tile8_kernel<H, KIND, true>), g, b, 0, s, p, ncols);
  else
    hipLaunchKernelGGL((tile8_kernel<H, KIND, false>), g, b, 0, s, p, ncols);
  if (!p.part) return;
  const int64_t rest = tiles < kSlots8 ? tiles : kSlots8 - 1;
  hipLaunchKernelGGL((join8_kernel<H, KIND>), dim3(static_cast<unsigned>(rest * kTurns)), b, 0, s, p, ncols);
}

template <int KIND>
int launch8(FfnArgs p, int32_t dtype, void* workspace, size_t workspace_bytes, hipStream_t s, const char* what) {
  if (p.T == 0) return FP8Z1_OK;
  if (misaligned(workspace, 16)) return refuse(FP8Z1_EINVAL, what, "misaligned workspace");
  if (few_rows8(p.T, p.E) && (KIND != kFfnUp || workspace_bytes >= rows8_bytes(p.T, p.N))) {
    const bool aligned = !misaligned(p.x0, 16) && !misaligned(p.w0, 16) && !misaligned(p.w1, 16) && p.K % 16 == 0;
    p.part = static_cast<float*>(workspace);
    if (dtype == FP8Z1_BF16)
      launch_rows8<Bf16, KIND>(p, aligned, s);
    else
      launch_rows8<F16, KIND>(p, aligned, s);
    return launched(what);
  }
  const bool direct = !misaligned(p.x0, 4) && !misaligned(p.w0, 4) && !misaligned(p.w1, 4) && p.K % 4 == 0;
  const int32_t per = KIND == kFfnUp ? kCols8 / 2 : kCols8, ncols = (p.N + per - 1) / per;
  const int64_t tiles = most_row_tiles(p.T, p.E) * ncols;
  if (tiles > 0x7fffffff / kThreads - kSlots8) return refuse(FP8Z1_ESHAPE, what, "too many tiles");
  const int32_t kb = (p.K + kB - 1) / kB;
  const int64_t known = p.offsets ? tiles : static_cast<int64_t>((p.T + kRows - 1) / kRows) * ncols;
  if ((p.offsets ? kb >= 4 : tile_splits8(known, kb) > 1) && workspace_bytes >= part8_bytes())
    p.part = static_cast<float*>(workspace);
  if (dtype == FP8Z1_BF16)
    launch_tiles8<Bf16, KIND>(p, direct, tiles, ncols, s);
  else
    launch_tiles8<F16, KIND>(p, direct, tiles, ncols, s);
  return launched(what);
}

}  // namespace
}  // namespace fp8z1
