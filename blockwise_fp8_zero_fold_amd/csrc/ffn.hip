// The feed-forward block over blockwise-FP8 weights, tokens sorted by expert: both
// projections with the gated activation, the down projection, and the backward pass
// with respect to the activations.
//
// One tile kernel serves all four calls.  A workgroup of 4 waves computes 128 rows
// (tokens of one expert) x 128 columns; each wave 64 x 64, as 2 x 2 matrix tiles of
// 32 x 32.  The sum over k goes in blocks of 128, the blocks that one weight scale
// covers:  acc += scale * sum_{k in block} x[m][k] * code[k][n],  the inner sum on the
// matrix cores with the codes widened exactly, so no dequantized weight is rounded.
#include <hip/hip_runtime.h>

#include "ffn.h"

namespace fp8z1 {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;           // tile rows
constexpr int kStep = 64;            // k per LDS stage
constexpr int kABytes = kRows * kStep * 2;
constexpr int kBBytes = 128 * kStep;

template <class H, int KIND>
__global__ __launch_bounds__(kThreads, 2) void ffn_tile_kernel(FfnArgs p, int32_t ncols) {
  constexpr bool kTrans = KIND == kFfnDownBwd || KIND == kFfnUpBwd;  // weights run along n
  constexpr int kCols = KIND == kFfnUp ? 64 : 128;                   // columns of a tile (per matrix)
  constexpr int kSeg = KIND == kFfnUpBwd ? 2 : 1;                    // products added up
  typedef typename H::v8 v8;
  __shared__ __attribute__((aligned(16))) uint8_t sa[2][kABytes];
  __shared__ __attribute__((aligned(16))) uint8_t sb[2][kBBytes];

  int32_t e, lo, hi, m0, col;
  if (!find_tile<kRows>(p.offsets, p.T, p.E, ncols, static_cast<int32_t>(blockIdx.x), e, lo, hi, m0, col)) return;
  const int32_t n0 = col * kCols;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, wm = w >> 1, wn = w & 1;
  const int32_t N = p.N, K = p.K;
  const int32_t nb = (N + kB - 1) / kB, kb = (K + kB - 1) / kB;

  // This thread's 16-byte chunks of a stage: chunk position id = t + 256 j of the LDS
  // tile.  Chunk c of row r sits at position c ^ swizzle(r), which spreads the rows
  // that a wave reads at once over the banks.
  int64_t aoff[4], boff[2];  // byte offsets of the chunks at k = 0
  int32_t ac[4], bn[2], br[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int id = t + kThreads * j, r = id >> 3;
    ac[j] = ((id & 7) ^ (r & 7)) * 16;
    aoff[j] = static_cast<int64_t>(min(m0 + r, hi - 1)) * K * 2 + ac[j];
  }
  const uint8_t* b0[2];
  const uint8_t* b1[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int id = t + kThreads * j;
    const int64_t ebase = static_cast<int64_t>(e) * N * K;
    if (kTrans) {
      const int r = id >> 3, c = ((id & 7) ^ (r & 7)) * 16;
      br[j] = r;
      bn[j] = N - n0 - c;  // bytes of the chunk inside the row
      boff[j] = ebase + static_cast<int64_t>(r) * N + n0 + c;
      b0[j] = p.w0;
      b1[j] = p.w1;
    } else {
      const int r = id >> 2, c = ((id & 3) ^ ((r >> 1) & 3)) * 16;
      const int32_t n = min(n0 + (KIND == kFfnUp ? (r & 63) : r), N - 1);
      br[j] = 0;
      bn[j] = c;
      boff[j] = ebase + static_cast<int64_t>(n) * K + c;
      b0[j] = KIND == kFfnUp && r >= 64 ? p.w1 : p.w0;
      b1[j] = nullptr;
    }
  }

  uint4 ra[4], rb[2];
  // k0: first k of the stage within its product `seg`
  auto load = [&](int seg, int32_t k0) {
    const uint8_t* x = seg ? p.x1 : p.x0;
#pragma unroll
    for (int j = 0; j < 4; ++j) ra[j] = ld16_part(x + aoff[j] + 2 * static_cast<int64_t>(k0), (K - k0) * 2 - ac[j]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (kTrans)
        rb[j] = ld16_part((seg ? b1[j] : b0[j]) + boff[j] + static_cast<int64_t>(k0) * N,
                          k0 + br[j] < K ? bn[j] : 0);
      else
        rb[j] = ld16_part(b0[j] + boff[j] + k0, K - k0 - bn[j]);
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(&sa[buf][(t + kThreads * j) * 16]) = ra[j];
#pragma unroll
    for (int j = 0; j < 2; ++j) *reinterpret_cast<uint4*>(&sb[buf][(t + kThreads * j) * 16]) = rb[j];
  };

  f32x16 acc[2][2], part[2][2];
  const f32x16 zero = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = part[i][j] = zero;

  const int half = lane >> 5, l32 = lane & 31, l16 = lane & 15, grp = lane >> 4;
  auto compute = [&](int buf, bool first) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      v8 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wm * 64 + i * 32 + l32;
        // k of this lane: plain order where B is read transposed; otherwise the lane's
        // 16 consecutive k of a 32-wide group, 8 per step, as B's 16-byte chunk holds them
        const int c = kTrans ? ks * 2 + half : (ks >> 1) * 4 + half * 2 + (ks & 1);
        a[i] = as_v8<H>(*reinterpret_cast<const uint4*>(&sa[buf][r * 128 + ((c ^ (r & 7)) << 4)]));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (kTrans) {
          const int r = ks * 16 + (grp >> 1) * 8 + (l16 >> 1);
          const int c = wn * 4 + j * 2 + (grp & 1);
          const i32x2 q = read_tr8(&sb[buf][r * 128 + ((c ^ (r & 7)) << 4) + (l16 & 1) * 8]);
          b[j] = widen8<H>(q.x, q.y);
        } else {
          const int r = KIND == kFfnUp ? j * 64 + wn * 32 + l32 : wn * 64 + j * 32 + l32;
          const int c = (ks >> 1) * 2 + half;
          const uint2 q =
              *reinterpret_cast<const uint2*>(&sb[buf][r * 64 + ((c ^ ((r >> 1) & 3)) << 4) + (ks & 1) * 8]);
          b[j] = widen8<H>(q.x, q.y);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) part[i][j] = H::mma32(a[i], b[j], first && ks == 0 ? zero : part[i][j]);
    }
  };

  const int32_t blocks = kSeg * kb;  // scale blocks of k, each two stages
  load(0, 0);
  store(0);
  __syncthreads();
  for (int32_t q = 0; q < blocks; ++q) {
    const int seg = q >= kb ? 1 : 0;
    const int32_t kq = q - seg * kb;
    float s[2];
    if (kTrans) {
      const float* sp = seg ? p.s1 : p.s0;
      s[0] = s[1] = sp[(static_cast<int64_t>(e) * kb + kq) * nb + min((n0 + wn * 64) / kB, nb - 1)];
    } else {
      const int64_t at = (static_cast<int64_t>(e) * nb + min((n0 + (KIND == kFfnUp ? 0 : wn * 64)) / kB, nb - 1)) * kb + kq;
      s[0] = p.s0[at];
      s[1] = KIND == kFfnUp ? p.s1[at] : s[0];
    }
    load(seg, kq * kB + kStep);
    compute(0, true);
    store(1);
    __syncthreads();
    if (q + 1 < blocks) load(q + 1 >= kb ? 1 : 0, (q + 1 >= kb ? q + 1 - kb : q + 1) * kB);
    compute(1, false);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(s[j], part[i][j][r], acc[i][j][r]);
    if (q + 1 < blocks) store(0);
    __syncthreads();
  }

  // results: lane l holds column l % 32 of each 32 x 32 tile
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int32_t m = m0 + wm * 64 + i * 32 + (r >> 2) * 8 + half * 4 + (r & 3);
      if (m >= hi) continue;
      if (KIND == kFfnUp) {
        const int32_t n = n0 + wn * 32 + l32;
        if (n >= N) continue;
        const int64_t at = static_cast<int64_t>(m) * N + n;
        const float h = acc[i][0][r], u = acc[i][1][r];
        p.o0[at] = H::from_f32(act_value(p.act, h) * u);
        if (p.o1) {
          p.o1[at] = H::from_f32(h);
          p.o2[at] = H::from_f32(u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int32_t n = n0 + wn * 64 + j * 32 + l32;
          if (n >= N) continue;
          const int64_t at = static_cast<int64_t>(m) * N + n;
          const float x = acc[i][j][r];
          if (KIND == kFfnDownBwd) {
            const float h = H::to_f32(p.h[at]), u = H::to_f32(p.u[at]);
            float f, slope;
            act_both(p.act, h, f, slope);
            p.o0[at] = H::from_f32(x * u * slope);
            p.o1[at] = H::from_f32(x * f);
            if (p.o2) p.o2[at] = H::from_f32(f * u);
          } else {
            p.o0[at] = H::from_f32(x);
          }
        }
      }
    }
}

// The most row tiles that T rows in E runs can make: every run may end in a partial tile.
int64_t most_row_tiles(int64_t T, int64_t E) { return T / kRows + (T < E ? T : E); }

template <int KIND>
int launch(const FfnArgs& p, int32_t dtype, hipStream_t s, const char* what) {
  if (p.T == 0) return FP8Z1_OK;
  const int32_t cols = KIND == kFfnUp ? 64 : 128, ncols = (p.N + cols - 1) / cols;
  const int64_t grid = most_row_tiles(p.T, p.E) * ncols;
  if (grid > 0x7fffffff) return set_error(FP8Z1_ESHAPE, std::string(what) + ": too many tiles");
  const dim3 g(static_cast<unsigned>(grid)), b(kThreads);
  if (dtype == FP8Z1_BF16)
    hipLaunchKernelGGL((ffn_tile_kernel<Bf16, KIND>), g, b, 0, s, p, ncols);
  else
    hipLaunchKernelGGL((ffn_tile_kernel<F16, KIND>), g, b, 0, s, p, ncols);
  return check_hip(hipGetLastError(), what);
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

int check_cfg(const fp8z1_ffn* f, const int32_t* offsets, const char* what) {
  const std::string w(what);
  if (!f) return set_error(FP8Z1_EINVAL, w + ": NULL description");
  if (f->dtype != FP8Z1_BF16 && f->dtype != FP8Z1_F16)
    return set_error(FP8Z1_EINVAL, w + ": dtype must be FP8Z1_BF16 or FP8Z1_F16");
  if (f->act != FP8Z1_ACT_SILU && f->act != FP8Z1_ACT_GELU)
    return set_error(FP8Z1_EINVAL, w + ": act must be FP8Z1_ACT_SILU or FP8Z1_ACT_GELU");
  if (f->T < 0 || f->T > FP8Z1_FFN_MAX_ROWS) return set_error(FP8Z1_ESHAPE, w + ": T outside 0 .. 2^30");
  if (f->E < 1 || f->E > FP8Z1_FFN_MAX_EXPERTS) return set_error(FP8Z1_ESHAPE, w + ": E outside 1 .. 65535");
  if (f->D < 1 || f->D > FP8Z1_FFN_MAX_WIDTH || f->F < 1 || f->F > FP8Z1_FFN_MAX_WIDTH)
    return set_error(FP8Z1_ESHAPE, w + ": D and F must be 1 .. 2^20");
  if (!offsets && f->E != 1) return set_error(FP8Z1_EINVAL, w + ": offsets may be NULL for one expert only");
  if (misaligned(offsets, 4)) return set_error(FP8Z1_EINVAL, w + ": misaligned offsets");
  return FP8Z1_OK;
}

int check_rows(std::initializer_list<const void*> xs, const char* what) {
  for (const void* x : xs) {
    if (!x) return set_error(FP8Z1_EINVAL, std::string(what) + ": NULL argument");
    if (misaligned(x, 2)) return set_error(FP8Z1_EINVAL, std::string(what) + ": misaligned rows");
  }
  return FP8Z1_OK;
}

int check_weights(const uint8_t* codes, const float* scales, const char* what) {
  if (!codes || !scales) return set_error(FP8Z1_EINVAL, std::string(what) + ": NULL weights");
  if (misaligned(scales, 4)) return set_error(FP8Z1_EINVAL, std::string(what) + ": misaligned scales");
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

using namespace fp8z1;

extern "C" int fp8z1_ffn_up(const fp8z1_ffn* f, const void* x, const uint8_t* gate_codes, const float* gate_scales,
                            const uint8_t* up_codes, const float* up_scales, const int32_t* offsets, void* h, void* u,
                            void* a, void* stream) {
  const char* what = "ffn_up";
  int rc = check_cfg(f, offsets, what);
  if (!rc && f->T) rc = check_rows({x, a}, what);
  if (!rc && f->T && (h || u)) rc = check_rows({h, u}, what);
  if (!rc) rc = check_weights(gate_codes, gate_scales, what);
  if (!rc) rc = check_weights(up_codes, up_scales, what);
  if (rc) return rc;
  FfnArgs p = base_args(f, offsets, true);
  p.x0 = bytes(x);
  p.w0 = gate_codes;
  p.w1 = up_codes;
  p.s0 = gate_scales;
  p.s1 = up_scales;
  p.o0 = static_cast<uint16_t*>(a);
  p.o1 = static_cast<uint16_t*>(h);
  p.o2 = static_cast<uint16_t*>(u);
  return launch<kFfnUp>(p, f->dtype, static_cast<hipStream_t>(stream), what);
}

extern "C" int fp8z1_ffn_down(const fp8z1_ffn* f, const void* a, const uint8_t* down_codes, const float* down_scales,
                              const int32_t* offsets, void* y, void* stream) {
  const char* what = "ffn_down";
  int rc = check_cfg(f, offsets, what);
  if (!rc && f->T) rc = check_rows({a, y}, what);
  if (!rc) rc = check_weights(down_codes, down_scales, what);
  if (rc) return rc;
  FfnArgs p = base_args(f, offsets, false);
  p.x0 = bytes(a);
  p.w0 = down_codes;
  p.s0 = down_scales;
  p.o0 = static_cast<uint16_t*>(y);
  return launch<kFfnDown>(p, f->dtype, static_cast<hipStream_t>(stream), what);
}

extern "C" int fp8z1_ffn_down_bwd(const fp8z1_ffn* f, const void* dy, const uint8_t* down_codes,
                                  const float* down_scales, const void* h, const void* u, const int32_t* offsets,
                                  void* dh, void* du, void* a, void* stream) {
  const char* what = "ffn_down_bwd";
  int rc = check_cfg(f, offsets, what);
  if (!rc && f->T) rc = check_rows({dy, h, u, dh, du}, what);
  if (!rc && misaligned(a, 2)) rc = set_error(FP8Z1_EINVAL, "ffn_down_bwd: misaligned rows");
  if (!rc) rc = check_weights(down_codes, down_scales, what);
  if (rc) return rc;
  FfnArgs p = base_args(f, offsets, true);
  p.x0 = bytes(dy);
  p.w0 = down_codes;
  p.s0 = down_scales;
  p.h = static_cast<const uint16_t*>(h);
  p.u = static_cast<const uint16_t*>(u);
  p.o0 = static_cast<uint16_t*>(dh);
  p.o1 = static_cast<uint16_t*>(du);
  p.o2 = static_cast<uint16_t*>(a);
  return launch<kFfnDownBwd>(p, f->dtype, static_cast<hipStream_t>(stream), what);
}

extern "C" int fp8z1_ffn_up_bwd(const fp8z1_ffn* f, const void* dh, const void* du, const uint8_t* gate_codes,
                                const float* gate_scales, const uint8_t* up_codes, const float* up_scales,
                                const int32_t* offsets, void* dx, void* stream) {
  const char* what = "ffn_up_bwd";
  int rc = check_cfg(f, offsets, what);
  if (!rc && f->T) rc = check_rows({dh, du, dx}, what);
  if (!rc) rc = check_weights(gate_codes, gate_scales, what);
  if (!rc) rc = check_weights(up_codes, up_scales, what);
  if (rc) return rc;
  FfnArgs p = base_args(f, offsets, false);
  p.x0 = bytes(dh);
  p.x1 = bytes(du);
  p.w0 = gate_codes;
  p.w1 = up_codes;
  p.s0 = gate_scales;
  p.s1 = up_scales;
  p.o0 = static_cast<uint16_t*>(dx);
  return launch<kFfnUpBwd>(p, f->dtype, static_cast<hipStream_t>(stream), what);
}
