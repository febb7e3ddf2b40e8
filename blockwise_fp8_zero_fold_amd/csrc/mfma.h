// Matrix-core helpers of the feed-forward kernels: 16-bit element types, the
// FP8 -> 16-bit widening of weight codes, the direct global -> LDS copy and the
// transposing LDS reads of gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8z1 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// Operand layout of the two matrix instructions used (documented; both operands
// alike): lane l of 32x32x16 holds row l % 32 at k = 8 * (l / 32) + 0..7 and gets
// results (row 8 * (i / 4) + 4 * (l / 32) + i % 4, column l % 32), i = 0..15; lane l
// of 16x16x32 holds row l % 16 at k = 8 * (l / 16) + 0..7 and gets results
// (row 4 * (l / 16) + i, column l % 16), i = 0..3.  Any other assignment of k to
// lanes gives the same sums as long as both operands use it.
//
// An E4M3 code has 4 significant bits and an exponent from -9 to 8, so both
// 16-bit types hold it exactly: codes are widened without rounding and the block
// scale multiplies the float32 partial sum.
struct Bf16 {
  typedef bf16x8 v8;
  static __device__ __forceinline__ f32x16 mma32(v8 a, v8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma16(v8 a, v8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  template <bool HI>
  static __device__ __forceinline__ uint32_t widen2(int w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  }
  static __device__ __forceinline__ float to_f32(uint16_t x) {
    return __uint_as_float(static_cast<uint32_t>(x) << 16);
  }
  static __device__ __forceinline__ uint16_t from_f32(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
  }
};

struct F16 {
  typedef f16x8 v8;
  static __device__ __forceinline__ f32x16 mma32(v8 a, v8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma16(v8 a, v8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  template <bool HI>
  static __device__ __forceinline__ uint32_t widen2(int w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  }
  static __device__ __forceinline__ float to_f32(uint16_t x) {
    return static_cast<float>(__builtin_bit_cast(_Float16, x));
  }
  static __device__ __forceinline__ uint16_t from_f32(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
  }
};

// 8 codes -> 8 elements
template <class H>
__device__ __forceinline__ typename H::v8 widen8(uint32_t lo, uint32_t hi) {
  const uint4 r = make_uint4(H::template widen2<false>(lo), H::template widen2<true>(lo),
                             H::template widen2<false>(hi), H::template widen2<true>(hi));
  return __builtin_bit_cast(typename H::v8, r);
}

template <class H>
__device__ __forceinline__ typename H::v8 as_v8(uint4 x) {
  return __builtin_bit_cast(typename H::v8, x);
}

// 16 bytes at any alignment, one load (gfx950 runs in unaligned-access mode)
typedef uint32_t v4u_a1_global_t __attribute__((ext_vector_type(4), aligned(1), address_space(1)));
typedef uint32_t v4u_v_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  const v4u_v_t r = *(const v4u_a1_global_t*)(p);
  return make_uint4(r.x, r.y, r.z, r.w);
}

// The first `n` of the 16 bytes at p, zeros after them (n may be <= 0 or >= 16), for a p that
// lies `before` bytes behind the start of its row: the 16 bytes that end with the n-th are
// read and shifted down, so that only bytes of the row are touched; rows of less than
// 16 bytes are read byte by byte.
__device__ __forceinline__ uint4 ld16_part(const uint8_t* p, int n, int before) {
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if (n <= 0) return r;
  const int back = n < 16 ? 16 - n : 0;
  if (back <= before) {
    r = ld16(p - back);
    if (back) {
      uint64_t lo = r.x | static_cast<uint64_t>(r.y) << 32, hi = r.z | static_cast<uint64_t>(r.w) << 32;
      const int bits = 8 * (back & 7);
      if (back >= 8) {
        lo = hi;
        hi = 0;
      }
      if (bits) {
        lo = lo >> bits | hi << (64 - bits);
        hi >>= bits;
      }
      r = make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                     static_cast<uint32_t>(hi >> 32));
    }
    return r;
  }
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const uint32_t b = static_cast<uint32_t>(p[i]) << (8 * (i & 3));
    w[0] |= i < 4 ? b : 0u;
    w[1] |= i >= 4 && i < 8 ? b : 0u;
    w[2] |= i >= 8 && i < 12 ? b : 0u;
    w[3] |= i >= 12 ? b : 0u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A wave's direct copy of 64 x 16 bytes from global memory to 1 KB of LDS: lane l's bytes,
// at `off` bytes (4-byte aligned, its own for each lane) behind the buffer's base,
// land at dst + 16 l.  The buffer is `size` bytes long at most; base and size are the
// same for the wave, so the only vector register that an address takes is the offset.
// Written as assembly so that the compiler does not make every later LDS read wait for the
// copy (it cannot tell that a read is of another stage); it has no register output.
// The caller waits with wait_copies() before the barrier that hands the stage over.  (m0, the copy's
// LDS address, is not a register that the compiler keeps values in, and nothing else here uses it.)
typedef int buffer_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ buffer_t make_buffer(const uint8_t* base, int64_t size) {
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  if (size < 0) size = 0;  // a base past the tensor: nothing is read
  return buffer_t{__builtin_amdgcn_readfirstlane(static_cast<int>(at)),
                  __builtin_amdgcn_readfirstlane(static_cast<int>(at >> 32) & 0xffff),
                  __builtin_amdgcn_readfirstlane(static_cast<int>(size < 0x7fffffff ? size : 0x7fffffff)), 0x00027000};
}
__device__ __forceinline__ void copy16_to_lds(buffer_t b, uint32_t off, uint8_t* dst) {
  const uint32_t at = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)(dst)));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(static_cast<int>(at))), "v"(off), "s"(b)
               : "memory");
}
// 32 x 32 results with rows n and columns m: lane l holds, of column m = l % 32, rows
// 8 q + 4 (l / 32) + 0..3 as its value group q = 0..3.  exchange(x, y) of the k-th values of two
// neighbouring groups 2g and 2g + 1, k = 0..3, leaves the x then y of the lower lanes rows
// 16 g + 0..7 and of the upper lanes rows 16 g + 8..15, in order.
__device__ __forceinline__ void exchange(float& x, float& y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  x = __uint_as_float(r[0]);
  y = __uint_as_float(r[1]);
}

// until at most LEFT of the copies (and other memory operations) last issued are on their way
template <int LEFT = 0>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
}

// Transposing reads, per group of 16 lanes.  16-bit: lane 4r + c names the 8 bytes
// of row r, columns 4c..4c+3, and lane i receives column i of the four rows.
// 8-bit: lane 2r + c names the 8 bytes of row r, columns 8c..8c+7, and lane i
// receives column i of the eight rows.
__device__ __forceinline__ i32x2 read_tr16(const uint8_t* p) {
  return __builtin_bit_cast(
      i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p)));
}
__device__ __forceinline__ i32x2 read_tr8(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(p));
}

}  // namespace fp8z1
