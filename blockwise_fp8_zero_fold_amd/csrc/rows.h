// Rows of 16-bit or float32 elements, 8 to a thread: how they are loaded, widened and stored, and sums
// over a wave.
#pragma once

#include <hip/hip_runtime.h>

#include "mfma.h"

namespace fp8z1 {

struct F32 {
  static __device__ __forceinline__ float to_f32(float x) { return x; }
  static __device__ __forceinline__ float from_f32(float x) { return x; }
};
template <class H>
struct Elem {
  typedef uint16_t type;
};
template <>
struct Elem<F32> {
  typedef float type;
};

// 8 consecutive elements of a row from column c, in 16-byte accesses at any
// alignment of the elements (gfx950 runs in unaligned-access mode); those past the end
// are 0 and not stored.
typedef uint32_t v4u_a2_global_t __attribute__((ext_vector_type(4), aligned(2), address_space(1)));

// the elements as they lie in memory (so that a row can be on its way while the row before it
// is computed), and their values
template <class H>
struct Raw8 {
  v4u_v_t x[sizeof(typename Elem<H>::type) * 8 / 16];
};

template <class H>
__device__ __forceinline__ Raw8<H> fetch8(const void* row, int32_t C, int32_t c) {
  typedef typename Elem<H>::type E;
  constexpr int kVecs = sizeof(E) * 8 / 16;
  const E* p = static_cast<const E*>(row) + c;
  Raw8<H> r;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) r.x[i] = v4u_v_t{0u, 0u, 0u, 0u};
  if (c + 8 <= C) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) r.x[i] = ((const v4u_a2_global_t*)(p))[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < C) {
        if constexpr (sizeof(E) == 2)
          r.x[0][i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i % 2));
        else
          r.x[i / 4][i % 4] = __float_as_uint(p[i]);
      }
  }
  return r;
}

template <class H>
__device__ __forceinline__ void widen8f(const Raw8<H>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(typename Elem<H>::type) == 2)
      v[i] = H::to_f32(static_cast<uint16_t>(r.x[0][i / 2] >> (16 * (i % 2))));
    else
      v[i] = __uint_as_float(r.x[i / 4][i % 4]);
  }
}

template <class H>
__device__ __forceinline__ void load8(const void* row, int32_t C, int32_t c, float (&v)[8]) {
  widen8f<H>(fetch8<H>(row, C, c), v);
}

// STREAM: with the non-temporal hint (where: see launch_join)
template <class H, bool STREAM = false>
__device__ __forceinline__ void store8(void* row, int32_t C, int32_t c, const float (&v)[8]) {
  typedef typename Elem<H>::type E;
  constexpr int kVecs = sizeof(E) * 8 / 16;
  E* p = static_cast<E*>(row) + c;
  if (c + 8 <= C) {
    v4u_v_t x[kVecs];
    if (sizeof(E) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[0][i] = static_cast<uint32_t>(H::from_f32(v[2 * i])) | static_cast<uint32_t>(H::from_f32(v[2 * i + 1])) << 16;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[(i / 4) % kVecs][i % 4] = __float_as_uint(v[i]);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (STREAM)
        __builtin_nontemporal_store(x[i], (v4u_a2_global_t*)(p) + i);
      else
        ((v4u_a2_global_t*)(p))[i] = x[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < C) p[i] = H::from_f32(v[i]);
  }
}

template <class H>
__device__ __forceinline__ const void* row_of(const void* p, int64_t row, int32_t C) {
  return static_cast<const typename Elem<H>::type*>(p) + row * C;
}
template <class H>
__device__ __forceinline__ void* row_of(void* p, int64_t row, int32_t C) {
  return static_cast<typename Elem<H>::type*>(p) + row * C;
}

// Sum over the wave, the same in every lane: pairs, fours, eights and sixteens by lane
// permutations within the vector unit, the last two steps through LDS.
template <int CTRL>
__device__ __forceinline__ float permuted(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_fsum(float v) {
  v += permuted<0xb1>(v);   // lanes 1 0 3 2 of each four
  v += permuted<0x4e>(v);   // lanes 2 3 0 1 of each four
  v += permuted<0x141>(v);  // each eight mirrored
  v += permuted<0x140>(v);  // each sixteen mirrored
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

}  // namespace fp8z1
