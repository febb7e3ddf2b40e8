// The join between two blocks of a residual network, in one pass over its rows:
//   p = y rstd(y) (o + w_post)              norm after the block (or p = y)
//   z = res_scale res + block_scale gate p  gate and residual scale
//   n = z rstd(z) (o + w_pre)               norm before the next block
// with rstd(x) = 1 / sqrt(mean(x^2) + eps), and its backward pass.  Everything between
// the loads and the stores is float32; z is not rounded before it is normalized.
//
// A workgroup keeps a whole row in registers, 8 elements per thread and chunk, and walks
// over rows with the weights held in registers, so each tensor is read or written
// once and the weights once per workgroup.  The kernels are bound by HBM bandwidth: 8192 rows of
// 7168, bfloat16 with a float32 residual and a channel gate, take 120 to 126 us forward (5.6 to 5.9
// TB/s) and 200 to 208 us backward (5.1 to 5.3 TB/s, with the column sums' 7 us).  Two rows take 4.6 us.
// Other widths, forward and backward, 8192 rows: 1024 22 and 40 us, 4096 75 and 125, 5120 93 and 149, 8192 139
// and 235, 16,384 353 and 1590.  Backward, rows that are no multiple of 8 wide are loaded when they are needed
// instead of a row ahead (7001: 290 us), and above 8192, where a thread holds two chunks, 143 to 238
// registers spill (8200: 1150 us); up to 8192 2 to 11 do.  The forward pass spills none.
//
// With n in 8 bits (EIGHT) the same pass finds each group's largest magnitude and writes codes and scales, besides n in
// 16 bits or in its place: 8192 rows of 7168 as above, n kept too, 143 us (0.77 GB, 5.35 TB/s); two rows 5.4.
#include <hip/hip_runtime.h>

#include "device_util.h"
#include "ffn_refuse.h"
#include "mfma.h"
#include "norm_plan.h"
#include "rows.h"
#include "rows8.h"

namespace fp8z1 {
namespace {

struct NormArgs {
  const void *y, *res, *gate;  // backward: res is the kept z
  const float *w_post, *w_pre;
  void *z, *n;  // forward outputs
  uint8_t* codes;  // n in 8 bits, and its scales [T][groups of 128]
  float* scales;
  int32_t pow2;
  // backward
  const void *dz, *dn;
  void *dy, *dres, *dgate;
  float* part;       // [3][gridDim.x][C]: dw_post, dw_pre, dgate; or NULL with one workgroup:
  float* direct[3];  // the gradients themselves
  int32_t T, C, gate_kind, want_post, want_pre, want_gate;
  int32_t waves;  // per row (backward)
  float eps, res_scale, block_scale, offset;
};

// Sums of N values over the `waves` waves of a row, in a fixed order; every thread of the row
// gets them.  A workgroup may hold several rows, each with its own consecutive waves.
// `lds` holds 16 N floats; calls in a row use different ones, so one barrier each is
// enough (a set is written again only after the next set's barrier).
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* lds, int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_fsum(v[i]);
  if (waves == 1) return;
  const int w = threadIdx.x >> 6, w0 = w / waves * waves;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) lds[w * N + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lds[w0 * N + i];
  for (int k = 1; k < waves; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += lds[(w0 + k) * N + i];
}

__device__ __forceinline__ float rstd_of(float sum, int32_t C, float eps) {
  return 1.0f / sqrtf(sum / static_cast<float>(C) + eps);
}

// o + w, or 1 where there is no weight
__device__ __forceinline__ void load_weight(const float* w, int32_t C, int32_t c, float offset, float (&v)[8]) {
  if (w) {
    load8<F32>(w, C, c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += offset;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.0f;
  }
}

// the gate's values of a row, times block_scale
template <class H>
__device__ __forceinline__ void load_gate(const NormArgs& a, int64_t row, int32_t c, float (&g)[8]) {
  if (a.gate_kind == FP8Z1_GATE_CHANNEL) {
    load8<F32>(a.gate, a.C, c, g);
  } else if (a.gate_kind == FP8Z1_GATE_FULL) {
    load8<H>(row_of<H>(a.gate, row, a.C), a.C, c, g);
  } else {
    const float x = a.gate_kind == FP8Z1_GATE_TOKEN ? static_cast<const float*>(a.gate)[row] : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = x;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] *= a.block_scale;
}

// n in 8 bits: 16 neighbouring threads hold a group of 128 columns, whose largest magnitude they find by
// lane permutations (NaN are passed over: they are NaN as codes).
typedef uint32_t v2u_a1_global_t __attribute__((ext_vector_type(2), aligned(1), address_space(1)));
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t row, int32_t c, const float (&n)[8]) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, c + i < a.C ? fabsf(n[i]) : 0.0f);
  top = fmaxf(top, permuted<0xb1>(top));
  top = fmaxf(top, permuted<0x4e>(top));
  top = fmaxf(top, permuted<0x141>(top));
  top = fmaxf(top, permuted<0x140>(top));
  if (c >= a.C) return;
  const float scale = row8_scale(top, a.pow2 != 0);
  if (c % kB == 0) a.scales[row * ((a.C + kB - 1) / kB) + c / kB] = scale;
  const Over8 over = over8(scale);
  const uint32_t lo = codes4(n[0], n[1], n[2], n[3], over), hi = codes4(n[4], n[5], n[6], n[7], over);
  uint8_t* const to = a.codes + row * a.C + c;
  if (c + 8 <= a.C) {
    *(v2u_a1_global_t*)(to) = v2u_t{lo, hi};
  } else {
    for (int i = 0; i < 8; ++i)
      if (c + i < a.C) to[i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
  }
}

template <class H, class R, int CH, bool STREAM, bool EIGHT>
__global__ __launch_bounds__(1024) void norm_join_kernel(NormArgs a) {
  __shared__ float lds[2][16];
  constexpr bool kHold = CH == 1;  // weights kept in registers over the rows
  const int waves = blockDim.x >> 6;
  auto col = [&](int ch) { return static_cast<int32_t>(ch * blockDim.x + threadIdx.x) * 8; };
  float wpost[CH][8], wpre[CH][8], gate[CH][8];
#pragma unroll
  for (int ch = 0; ch < CH; ++ch)
    if (kHold) {
      load_weight(a.w_post, a.C, col(ch), a.offset, wpost[ch]);
      load_weight(a.w_pre, a.C, col(ch), a.offset, wpre[ch]);
      if (a.gate_kind == FP8Z1_GATE_CHANNEL) load_gate<H>(a, 0, col(ch), gate[ch]);
    }
  for (int32_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    float y[CH][8], z[CH][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      if (a.y) load8<H>(row_of<H>(a.y, row, a.C), a.C, col(ch), y[ch]);
      load8<R>(row_of<R>(a.res, row, a.C), a.C, col(ch), z[ch]);
      if (!kHold) {
        load_weight(a.w_post, a.C, col(ch), a.offset, wpost[ch]);
        load_weight(a.w_pre, a.C, col(ch), a.offset, wpre[ch]);
      }
      if (a.y && (!kHold || a.gate_kind != FP8Z1_GATE_CHANNEL)) load_gate<H>(a, row, col(ch), gate[ch]);
      if (a.y)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] = fmaf(y[ch][i], y[ch][i], sum[0]);
    }
    float r = 1.0f;
    if (a.w_post) {
      row_sums<1>(sum, lds[0], waves);
      r = rstd_of(sum[0], a.C, a.eps);
    }
    sum[0] = 0.0f;
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[ch][i] *= a.res_scale;
        if (a.y) z[ch][i] = fmaf(gate[ch][i], y[ch][i] * r * wpost[ch][i], z[ch][i]);
        sum[0] = fmaf(z[ch][i], z[ch][i], sum[0]);
      }
      if (a.z) store8<R, STREAM>(row_of<R>(a.z, row, a.C), a.C, col(ch), z[ch]);
    }
    if (a.n || EIGHT) {
      row_sums<1>(sum, lds[1], waves);
      r = rstd_of(sum[0], a.C, a.eps);
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[ch][i] = z[ch][i] * r * wpre[ch][i];
        if (!EIGHT || a.n) store8<H, STREAM>(row_of<H>(a.n, row, a.C), a.C, col(ch), z[ch]);
        if (EIGHT) store_codes(a, row, col(ch), z[ch]);
      }
    }
    if (!(a.w_post && (a.n || EIGHT))) __syncthreads();  // only one of the two LDS sets is used per row
  }
}

// Backward.  With v = dn (o + w_pre), z^ = z rstd(z):
//   d    = dz + rstd(z) (v - z^ mean(v z^))        gradient at z
//   dres = res_scale d,  dgate = block_scale d p,  dp = block_scale gate d
//   dy   = rstd(y) (dp (o + w_post) - y^ mean(dp (o + w_post) y^))
//   dw_pre = sum dn z^,  dw_post = sum dp y^,  and dgate summed over what it was broadcast to.
// Two rounds of row sums; the sums over rows are kept per thread (each owns its
// columns), written per workgroup and added in order by the kernel below, so no
// atomics decide their order.
//
// AHEAD (16-byte aligned rows of at most 8192): while a row is computed the next one is copied
// to LDS, where each thread finds its own elements, so the loads overlap the row sums;
// the registers are full with the weights and the column sums.
template <class H, class R, int CH, bool AHEAD>
__global__ __launch_bounds__(1024) void norm_join_bwd_kernel(NormArgs a) {
  __shared__ float lds[2][48];
  extern __shared__ __attribute__((aligned(16))) uint8_t ahead[];
  constexpr bool kHold = CH == 1;
  constexpr int kR = sizeof(typename Elem<R>::type) / 2, kH = sizeof(typename Elem<H>::type) / 2;  // KB of a wave's 512
  const int rt = a.waves * 64, sub = static_cast<int>(threadIdx.x) / rt, t = static_cast<int>(threadIdx.x) - sub * rt;
  const int rows = blockDim.x / rt;  // rows at a time
  auto col = [&](int ch) { return static_cast<int32_t>(ch * rt + t) * 8; };
  float wpost[CH][8], wpre[CH][8], gate[CH][8], spost[CH][8], spre[CH][8], sgate[CH][8];
#pragma unroll
  for (int ch = 0; ch < CH; ++ch) {
    if (kHold) {
      load_weight(a.w_post, a.C, col(ch), a.offset, wpost[ch]);
      load_weight(a.w_pre, a.C, col(ch), a.offset, wpre[ch]);
      if (a.gate_kind == FP8Z1_GATE_CHANNEL) load_gate<H>(a, 0, col(ch), gate[ch]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) spost[ch][i] = spre[ch][i] = sgate[ch][i] = 0.0f;
  }
  const float inv = 1.0f / static_cast<float>(a.C);

  // a wave's part of LDS: y, dn, z, dz and a full gate of its 512 columns; 16 bytes per lane and copy
  const int lane = threadIdx.x & 63;
  const int32_t c = t * 8, cin = min(c, a.C - 8);  // (lanes past the row copy its end)
  const bool full = a.gate_kind == FP8Z1_GATE_FULL;
  uint8_t* const mine =
      ahead + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * ((2 * kH + 2 * kR + (full ? kH : 0)) * 1024);
  auto copy_row = [&](int32_t row) {
    auto one = [&](const void* p, int per, int at) {  // per: 2-byte units of an element
      const int64_t bytes = static_cast<int64_t>(a.C) * 2 * per;
      const buffer_t b = make_buffer(static_cast<const uint8_t*>(p) + row * bytes, bytes);
      for (int i = 0; i < per; ++i) copy16_to_lds(b, static_cast<uint32_t>(cin * 2 * per + 16 * i), mine + (at + i) * 1024);
    };
    if (a.y) one(a.y, kH, 0);
    if (a.dn) {
      one(a.dn, kH, kH);
      one(a.res, kR, 2 * kH);
    }
    if (a.dz) one(a.dz, kR, 2 * kH + kR);
    if (full) one(a.gate, kH, 2 * kH + 2 * kR);
  };
  auto take = [&](auto tag, int at, float(&v)[8]) {
    typedef decltype(tag) T;
    Raw8<T> r;
#pragma unroll
    for (size_t i = 0; i < sizeof(r) / 16; ++i)
      r.x[i] = *reinterpret_cast<const v4u_v_t*>(mine + (at + i) * 1024 + lane * 16);
    widen8f<T>(r, v);
    if (c >= a.C)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  };
  const int32_t step = static_cast<int32_t>(gridDim.x) * rows, last = a.T - 1;
  const int32_t usub = __builtin_amdgcn_readfirstlane(sub);
  int32_t base = static_cast<int32_t>(blockIdx.x) * rows;
  if (AHEAD && base < a.T) copy_row(min(base + usub, last));

  // (all rows of a workgroup take the same number of turns: the barriers are shared; a turn
  // past the end repeats the last row and adds and writes nothing)
  for (; base < a.T; base += step) {
    const bool live = base + usub < a.T;
    const int32_t row = min(base + usub, last);
    float y[CH][8], z[CH][8], d[CH][8], dn[CH][8];
    float s1[3] = {0.0f, 0.0f, 0.0f};
    if (AHEAD) wait_copies();
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      if (AHEAD) {
        if (a.y) take(H{}, 0, y[ch]);
        if (a.dn) {
          take(H{}, kH, dn[ch]);
          take(R{}, 2 * kH, z[ch]);
        }
        if (a.dz) take(R{}, 2 * kH + kR, d[ch]);
      } else {
        if (a.y) load8<H>(row_of<H>(a.y, row, a.C), a.C, col(ch), y[ch]);
        if (a.dn) {
          load8<H>(row_of<H>(a.dn, row, a.C), a.C, col(ch), dn[ch]);
          load8<R>(row_of<R>(a.res, row, a.C), a.C, col(ch), z[ch]);
        }
        if (a.dz) load8<R>(row_of<R>(a.dz, row, a.C), a.C, col(ch), d[ch]);
      }
      if (!a.dz)
#pragma unroll
        for (int i = 0; i < 8; ++i) d[ch][i] = 0.0f;
      if (!kHold) {
        load_weight(a.w_post, a.C, col(ch), a.offset, wpost[ch]);
        load_weight(a.w_pre, a.C, col(ch), a.offset, wpre[ch]);
      }
      if (a.y && (!kHold || a.gate_kind != FP8Z1_GATE_CHANNEL)) {
        if (AHEAD && full) {
          take(H{}, 2 * kH + 2 * kR, gate[ch]);
#pragma unroll
          for (int i = 0; i < 8; ++i) gate[ch][i] *= a.block_scale;
        } else {
          load_gate<H>(a, row, col(ch), gate[ch]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (a.y) s1[0] = fmaf(y[ch][i], y[ch][i], s1[0]);
        if (a.dn) {
          s1[1] = fmaf(z[ch][i], z[ch][i], s1[1]);
          s1[2] = fmaf(dn[ch][i] * wpre[ch][i], z[ch][i], s1[2]);
        }
      }
    }
    if (AHEAD && base + step < a.T) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this row's elements have left LDS
      copy_row(min(base + step + usub, last));
    }
    row_sums<3>(s1, lds[0], a.waves);
    const float ry = a.w_post ? rstd_of(s1[0], a.C, a.eps) : 1.0f;
    const float rz = rstd_of(s1[1], a.C, a.eps);
    const float mz = s1[2] * rz * rz * inv;  // mean(v z^) rstd(z)
    float s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (a.dn) {
          d[ch][i] = fmaf(rz, fmaf(-z[ch][i], mz, dn[ch][i] * wpre[ch][i]), d[ch][i]);
          if (live) spre[ch][i] = fmaf(dn[ch][i], z[ch][i] * rz, spre[ch][i]);
        }
        if (a.y) {
          y[ch][i] *= ry;  // y^ (or y)
          const float p = y[ch][i] * wpost[ch][i];
          const float dp = gate[ch][i] * d[ch][i];
          if (live) {
            spost[ch][i] = fmaf(dp, y[ch][i], spost[ch][i]);
            sgate[ch][i] = fmaf(d[ch][i], p, sgate[ch][i]);
          }
          s2[0] = fmaf(dp, p, s2[0]);
          s2[1] = fmaf(d[ch][i], p, s2[1]);
        }
      }
      if (live && a.dres) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = a.res_scale * d[ch][i];
        store8<R>(row_of<R>(a.dres, row, a.C), a.C, col(ch), o);
      }
    }
    row_sums<2>(s2, lds[1], a.waves);
    const float my = s2[0] * inv;  // mean(dp (o + w_post) y^)
    if (live && a.y)
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        float o[8];
        if (a.gate_kind == FP8Z1_GATE_FULL && a.dgate) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = a.block_scale * d[ch][i] * (y[ch][i] * wpost[ch][i]);
          store8<H>(row_of<H>(a.dgate, row, a.C), a.C, col(ch), o);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i] = gate[ch][i] * d[ch][i];
          if (a.w_post) o[i] = ry * fmaf(-y[ch][i], my, o[i] * wpost[ch][i]);
        }
        if (a.dy) store8<H>(row_of<H>(a.dy, row, a.C), a.C, col(ch), o);
      }
    if (a.gate_kind == FP8Z1_GATE_TOKEN && a.dgate && live && t == 0)
      static_cast<float*>(a.dgate)[row] = a.block_scale * s2[1];
  }
  // the rows' column sums: added in order through LDS, then one set per workgroup
  const int64_t set = static_cast<int64_t>(gridDim.x) * a.C;
  auto finish = [&](float(&v)[CH][8], int which, float scale) {
    if constexpr (CH == 1)
      if (rows > 1) {
        float* const all = reinterpret_cast<float*>(ahead);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) all[i * blockDim.x + threadIdx.x] = v[0][i];
        __syncthreads();
        if (sub == 0)
          for (int k = 1; k < rows; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[0][i] += all[i * blockDim.x + k * rt + t];
      }
    if (sub != 0) return;
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[ch][i] *= scale;
      store8<F32>(a.part ? a.part + which * set + blockIdx.x * static_cast<int64_t>(a.C) : a.direct[which], a.C, col(ch),
                  v[ch]);
    }
  };
  if (a.want_post) finish(spost, 0, 1.0f);
  if (a.want_pre) finish(spre, 1, 1.0f);
  if (a.want_gate) finish(sgate, 2, a.block_scale);
}

// Column sums of the workgroups' partial sums (blockIdx.y: which gradient), in a fixed
// order: wave w of 16 takes rows w, w + 16, ... (16 at a time, all of a usual call's 256, so
// that their loads are on their way together), then the waves' sums are added in order.
__global__ __launch_bounds__(1024) void norm_columns_kernel(const float* __restrict__ part, int32_t groups, int32_t C,
                                                            float* o0, float* o1, float* o2) {
  __shared__ float lds[16][64];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int32_t c = static_cast<int32_t>(blockIdx.x) * 64 + lane;
  const float* p = part + static_cast<int64_t>(blockIdx.y) * groups * C;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < C)
    for (int32_t g = w; g < groups; g += 256) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = p[static_cast<int64_t>(min(g + 16 * i, groups - 1)) * C + c];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i & 3] += g + 16 * i < groups ? x[i] : 0.0f;
    }
  lds[w][lane] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (w == 0 && c < C) {
    float sum = lds[0][lane];
#pragma unroll
    for (int k = 1; k < 16; ++k) sum += lds[k][lane];
    out[c] = sum;
  }
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

constexpr int64_t kMaxC = FP8Z1_NORM_MAX_WIDTH;

int check_norm(const fp8z1_norm* f, const void* y, const float* w_post, const void* gate, const char* what) {
  if (!f) return refuse(FP8Z1_EINVAL, what, "NULL description");
  if (f->dtype != FP8Z1_BF16 && f->dtype != FP8Z1_F16 && f->dtype != FP8Z1_F32)
    return refuse(FP8Z1_EINVAL, what, "dtype must be FP8Z1_F32, FP8Z1_BF16 or FP8Z1_F16");
  if (f->res_dtype != f->dtype && f->res_dtype != FP8Z1_F32)
    return refuse(FP8Z1_EINVAL, what, "res_dtype must be dtype or FP8Z1_F32");
  if (f->gate < FP8Z1_GATE_NONE || f->gate > FP8Z1_GATE_FULL) return refuse(FP8Z1_EINVAL, what, "unknown gate kind");
  if (f->T < 0 || f->T > FP8Z1_FFN_MAX_ROWS) return refuse(FP8Z1_ESHAPE, what, "T outside 0 .. 2^30");
  if (f->C < 1 || f->C > kMaxC) return refuse(FP8Z1_ESHAPE, what, "C outside 1 .. 16384");
  if (!(f->eps >= 0.0f)) return refuse(FP8Z1_EINVAL, what, "eps must be >= 0");
  if (!y && f->T && (w_post || f->gate != FP8Z1_GATE_NONE))
    return refuse(FP8Z1_EINVAL, what, "a norm after the block or a gate needs y");
  if ((f->gate != FP8Z1_GATE_NONE) != (gate != nullptr) && f->T)
    return refuse(FP8Z1_EINVAL, what, "gate pointer and gate kind disagree");
  return FP8Z1_OK;
}

NormArgs base_args(const fp8z1_norm* f, const void* y, const void* res, const float* w_post, const void* gate,
                   const float* w_pre) {
  NormArgs a{};
  a.y = y;
  a.res = res;
  a.gate = gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.T = static_cast<int32_t>(f->T);
  a.C = static_cast<int32_t>(f->C);
  a.gate_kind = f->gate;
  a.eps = f->eps;
  a.res_scale = f->res_scale;
  a.block_scale = f->block_scale;
  a.offset = f->weight_offset;
  return a;
}

bool rows_aligned(const NormArgs& a) {
  return !misaligned(a.y, 16) && !misaligned(a.res, 16) && !misaligned(a.dz, 16) && !misaligned(a.dn, 16) &&
         (a.gate_kind != FP8Z1_GATE_FULL || !misaligned(a.gate, 16));
}

// The forward pass stores z and n with the non-temporal hint while they take no more than half of the
// L2 caches, and without it above, where it would push them out of the caches that the next calls
// read them from.  A join, an up projection of n and a join of z, with and without the hint (bfloat16,
// float32 residual): 256 x 7168 31.8 and 33.1 us, 2048 x 1024 30.1 and 31.4, 512 x 7168 47.0 and 45.6, 4096 x
// 1024 41.5 and 38.2, 2048 x 7168 110 and 105, 3000 x 5120 127 and 116.  (The join alone, which leaves
// its stores to others: 512 x 7168 11.1 and 12.7, 8192 x 7168 121 and 120, x 8192 144 and 137.)  The backward
// pass stores without (221 and 211).
constexpr int64_t kHalfOfL2 = kXcds * (4LL << 20) / 2;
template <class H, class R, bool EIGHT>
void launch_join(const NormArgs& a, dim3 g, dim3 b, hipStream_t s) {
  const int64_t n = EIGHT && !a.n ? 0 : sizeof(typename Elem<H>::type);
  const int64_t bytes = static_cast<int64_t>(a.T) * a.C * (n + EIGHT + sizeof(typename Elem<R>::type));
  const bool one = a.C <= 8192, hint = bytes <= kHalfOfL2;
  if (one && hint)
    hipLaunchKernelGGL((norm_join_kernel<H, R, 1, true, EIGHT>), g, b, 0, s, a);
  else if (one)
    hipLaunchKernelGGL((norm_join_kernel<H, R, 1, false, EIGHT>), g, b, 0, s, a);
  else if (hint)
    hipLaunchKernelGGL((norm_join_kernel<H, R, 2, true, EIGHT>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((norm_join_kernel<H, R, 2, false, EIGHT>), g, b, 0, s, a);
}

template <class H, class R, bool BWD>
void launch_typed(const NormArgs& a, dim3 g, dim3 b, hipStream_t s) {
  const bool one = a.C <= 8192;
  // LDS: the next row's elements, or the sums of several rows (32 bytes per thread, no more)
  const size_t h = sizeof(typename Elem<H>::type), r = sizeof(typename Elem<R>::type);
  const size_t bytes = (2 * h + 2 * r + (a.gate_kind == FP8Z1_GATE_FULL ? h : 0)) * 8 * b.x;
  if (BWD && one && a.C % 8 == 0 && rows_aligned(a) && bytes <= 159 * 1024)  // of 160 KB
    hipLaunchKernelGGL((norm_join_bwd_kernel<H, R, 1, true>), g, b, bytes, s, a);
  else if (BWD && one)
    hipLaunchKernelGGL((norm_join_bwd_kernel<H, R, 1, false>), g, b, 32 * b.x, s, a);
  else if (BWD)
    hipLaunchKernelGGL((norm_join_bwd_kernel<H, R, 2, false>), g, b, 0, s, a);
  else if (a.codes)
    launch_join<H, R, true>(a, g, b, s);
  else
    launch_join<H, R, false>(a, g, b, s);
}

template <bool BWD>
void launch(const fp8z1_norm* f, const NormArgs& a, int64_t groups, int64_t rows, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(groups)), b(static_cast<unsigned>(rows * norm_threads(f->C)));
  const bool wide = f->res_dtype == FP8Z1_F32;
  if (f->dtype == FP8Z1_F32)
    launch_typed<F32, F32, BWD>(a, g, b, s);
  else if (f->dtype == FP8Z1_BF16 && wide)
    launch_typed<Bf16, F32, BWD>(a, g, b, s);
  else if (f->dtype == FP8Z1_BF16)
    launch_typed<Bf16, Bf16, BWD>(a, g, b, s);
  else if (wide)
    launch_typed<F16, F32, BWD>(a, g, b, s);
  else
    launch_typed<F16, F16, BWD>(a, g, b, s);
}

size_t elem_size(int32_t dtype) { return dtype == FP8Z1_F32 ? 4 : 2; }

// Every pointer aligned to its elements
int check_alignment(const fp8z1_norm* f, std::initializer_list<const void*> act, std::initializer_list<const void*> res,
                    std::initializer_list<const void*> f32, std::initializer_list<const void*> gates,
                    const char* what) {
  bool bad = false;
  for (const void* p : act) bad |= misaligned(p, elem_size(f->dtype));
  for (const void* p : res) bad |= misaligned(p, elem_size(f->res_dtype));
  for (const void* p : f32) bad |= misaligned(p, 4);
  for (const void* p : gates) bad |= misaligned(p, f->gate == FP8Z1_GATE_FULL ? elem_size(f->dtype) : 4);
  return bad ? refuse(FP8Z1_EINVAL, what, "misaligned argument") : FP8Z1_OK;
}

}  // namespace
}  // namespace fp8z1

using namespace fp8z1;

extern "C" int fp8z1_norm_join(const fp8z1_norm* f, const void* y, const void* res, const float* w_post,
                               const void* gate, const float* w_pre, void* z, void* n, void* stream) {
  const char* what = "norm_join";
  int rc = check_norm(f, y, w_post, gate, what);
  if (rc) return rc;
  if (f->T == 0) return FP8Z1_OK;
  if (!res || (!z && !n)) return refuse(FP8Z1_EINVAL, "norm_join", "NULL argument");
  rc = check_alignment(f, {y, n}, {res, z}, {w_post, w_pre}, {gate}, what);
  if (rc) return rc;
  NormArgs a = base_args(f, y, res, w_post, gate, w_pre);
  a.z = z;
  a.n = n;
  launch<false>(f, a, norm_fwd_groups(f->T, f->C), 1, static_cast<hipStream_t>(stream));
  return launched("norm_join");
}

extern "C" int fp8z1_norm_join8(const fp8z1_norm* f, const void* y, const void* res, const float* w_post,
                                const void* gate, const float* w_pre, void* z, void* n, uint8_t* codes, float* scales,
                                int32_t scale_rule, void* stream) {
  const char* what = "norm_join8";
  int rc = check_norm(f, y, w_post, gate, what);
  if (rc) return rc;
  if (scale_rule != FP8Z1_SCALE_AMAX && scale_rule != FP8Z1_SCALE_POW2)
    return refuse(FP8Z1_EINVAL, what, "scale_rule must be FP8Z1_SCALE_AMAX or FP8Z1_SCALE_POW2");
  if (f->T == 0) return FP8Z1_OK;
  if (!res || !codes || !scales) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  rc = check_alignment(f, {y, n}, {res, z}, {w_post, w_pre, scales}, {gate}, what);
  if (rc) return rc;
  NormArgs a = base_args(f, y, res, w_post, gate, w_pre);
  a.z = z;
  a.n = n;
  a.codes = codes;
  a.scales = scales;
  a.pow2 = scale_rule == FP8Z1_SCALE_POW2;
  launch<false>(f, a, norm_fwd_groups(f->T, f->C), 1, static_cast<hipStream_t>(stream));
  return launched(what);
}

extern "C" int fp8z1_norm_join_bwd_workspace_bytes(const fp8z1_norm* f, size_t* bytes) {
  if (!bytes) return refuse(FP8Z1_EINVAL, "norm_join_bwd_workspace_bytes", "NULL argument");
  if (!f) return refuse(FP8Z1_EINVAL, "norm_join_bwd_workspace_bytes", "NULL description");
  if (f->T < 0 || f->T > FP8Z1_FFN_MAX_ROWS || f->C < 1 || f->C > kMaxC)
    return refuse(FP8Z1_ESHAPE, "norm_join_bwd_workspace_bytes", "T or C out of range");
  *bytes = sizeof(float) * 3 * static_cast<size_t>(norm_bwd_groups(f->T, f->C).count) * static_cast<size_t>(f->C);
  return FP8Z1_OK;
}

extern "C" int fp8z1_norm_join_bwd(const fp8z1_norm* f, const void* dz, const void* dn, const void* y, const void* z,
                                   const float* w_post, const void* gate, const float* w_pre, void* dy, void* dres,
                                   float* dw_post, void* dgate, float* dw_pre, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  const char* what = "norm_join_bwd";
  int rc = check_norm(f, y, w_post, gate, what);
  if (rc) return rc;
  if (f->T && !dz && !dn) return refuse(FP8Z1_EINVAL, "norm_join_bwd", "dz and dn are both NULL");
  if (f->T && dn && !z) return refuse(FP8Z1_EINVAL, "norm_join_bwd", "dn needs z");
  if (f->T && dy && !y) return refuse(FP8Z1_EINVAL, "norm_join_bwd", "dy needs y");
  if ((dw_post && !w_post) || (dw_pre && !w_pre)) return refuse(FP8Z1_EINVAL, "norm_join_bwd", "gradient of no weight");
  if (dgate && f->gate == FP8Z1_GATE_NONE) return refuse(FP8Z1_EINVAL, "norm_join_bwd", "gradient of no gate");
  rc = check_alignment(f, {y, dn, dy}, {z, dz, dres}, {w_post, w_pre, dw_post, dw_pre}, {gate, dgate}, what);
  if (rc) return rc;
  float* gate_cols = f->gate == FP8Z1_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
  const bool sums = dw_post || dw_pre || gate_cols;
  const NormGroups groups = norm_bwd_groups(f->T, f->C);
  if (sums && f->T) {
    size_t need = 0;
    rc = fp8z1_norm_join_bwd_workspace_bytes(f, &need);
    if (rc) return rc;
    if (!workspace || workspace_bytes < need) return refuse(FP8Z1_EINVAL, "norm_join_bwd", "workspace too small");
    if (misaligned(workspace, 16)) return refuse(FP8Z1_EINVAL, "norm_join_bwd", "misaligned workspace");
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (f->T) {
    NormArgs a = base_args(f, y, z, w_post, gate, w_pre);
    a.dz = dz;
    a.dn = dn;
    a.dy = dy;
    a.dres = dres;
    a.dgate = dgate;
    a.part = groups.count > 1 ? static_cast<float*>(workspace) : nullptr;
    a.direct[0] = dw_post;
    a.direct[1] = dw_pre;
    a.direct[2] = gate_cols;
    a.want_post = dw_post != nullptr;
    a.want_pre = dw_pre != nullptr;
    a.want_gate = gate_cols != nullptr;
    a.waves = norm_threads(f->C) / 64;
    launch<true>(f, a, groups.count, groups.rows, s);
    rc = launched("norm_join_bwd");
    if (rc) return rc;
  }
  if (sums && (f->T == 0 || groups.count > 1)) {
    hipLaunchKernelGGL(norm_columns_kernel, dim3(static_cast<unsigned>((f->C + 63) / 64), 3), dim3(1024), 0, s,
                       static_cast<const float*>(workspace), static_cast<int32_t>(f->T ? groups.count : 0), static_cast<int32_t>(f->C),
                       dw_post, dw_pre, gate_cols);
    rc = launched("norm_join_bwd");
  }
  return rc;
}
