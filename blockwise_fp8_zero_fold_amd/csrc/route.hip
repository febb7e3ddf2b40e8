// The router: each token's k best of E experts by score, and their weights; and its gradient.
//   softmax  p_e = exp(l_e) / sum exp(l)          logistic  p_e = 1 / (1 + exp(-l_e))
//   choice   the k largest of p_e + bias_e (without a bias of l_e, which has the same order), the lowest
//            index among equals
//   weight   w_j = scale p_j, or scale p_j / sum of the chosen p
// Gradient, with d_j = dw_j scale (d_j = scale (dw_j - sum_i dw_i p_i / S) / S where normalized, S the sum of
// the chosen):  softmax  dl_e = p_e (d_e - sum_j d_j p_j),  logistic  dl_e = d_e p_e (1 - p_e),  d_e = 0 for
// experts that are not chosen.  Where softmax weights are normalized the other experts' scores cancel:
// w_j = scale exp(l_j) / sum of the chosen exp(l), dl_j = w_j (dw_j - sum_i dw_i w_i / scale).
//
// A wave takes a token, its scores in registers (1 to 16 a lane, consecutive experts), and finds the k
// largest by k rounds of a maximum over the wave.  With a bias the ranks are computed and compared in
// 64 bits, since two experts' sums may differ by less than a float32 rounding; logits are ranked as they are.
//
// Many tokens: bound by the issue of vector instructions, not by the reads.  8192 tokens of 256 experts in float32, 8
// choices, take 11 us forward and 6 to 7 backward, where 8.4 MB and twice that cost 2 and 3: 562 vector instructions a
// wave (255 backward), 8 waves on each SIMD, 4 cycles each are 18,000 (8,200) of the 23,000 (12,600) cycles that the
// kernel is busy.  With a bias 906, some of them on 64 bits: 15 (logistic) to 16 us.  Few tokens: bound by the latency
// of the k rounds, which come one after another.  4 tokens of 64 experts with a bias take 4.3 us in a graph, an empty
// launch 2 to 3; eager calls take 9, the host's time.
#include <hip/hip_runtime.h>

#include "device_util.h"
#include "ffn_refuse.h"
#include "rows.h"

namespace fp8z1 {
namespace {

constexpr int kRouteWaves = 4;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* experts;  // forward out, backward in
  float* weights;
  const float* dweights;
  void* dlogits;
  int32_t T, E, k, sigmoid, normalize;
  float scale;
};

template <class H>
__device__ __forceinline__ float one_f32(const void* p, int64_t at) {
  return H::to_f32(static_cast<const typename Elem<H>::type*>(p)[at]);
}

// Largest value over the wave, the same in every lane
__device__ __forceinline__ float wave_most(float v) {
  v = fmaxf(v, permuted<0xb1>(v));
  v = fmaxf(v, permuted<0x4e>(v));
  v = fmaxf(v, permuted<0x141>(v));
  v = fmaxf(v, permuted<0x140>(v));
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
template <int CTRL>
__device__ __forceinline__ double permuted(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double wave_most(double v) {
  v = fmax(v, permuted<0xb1>(v));
  v = fmax(v, permuted<0x4e>(v));
  v = fmax(v, permuted<0x141>(v));
  v = fmax(v, permuted<0x140>(v));
  v = fmax(v, __shfl_xor(v, 16));
  return fmax(v, __shfl_xor(v, 32));
}

// What an expert that cannot be chosen ranks as: a logit of -inf or NaN, one already chosen, one past E
template <class K>
__device__ __forceinline__ K no_rank() {
  return -__builtin_huge_val();
}

// NV: scores per lane.  K: float (ranks are the logits) or double (ranks are score + bias).
template <class H, class K, int NV>
__device__ __forceinline__ void route_token(const RouteArgs& a, int32_t t) {
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(t) * a.E;
  float l[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int32_t e = lane * NV + i;
    l[i] = e < a.E ? one_f32<H>(a.logits, row + e) : -__builtin_huge_valf();
  }
  constexpr bool kBias = sizeof(K) == 8;
  // softmax over all experts, where it is needed: its weights as they are, or ranks with a bias
  float top = -__builtin_huge_valf(), total = 0.0f;
  bool nan = false;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      top = fmaxf(top, l[i]);
      nan |= l[i] != l[i];
    }
    top = wave_most(top);
    // (an infinite logit has no softmax either: inf - inf)
    nan = __any(nan) || top == __builtin_huge_valf();
    if (!a.normalize) {
#pragma unroll
      for (int i = 0; i < NV; ++i) total += l[i] > -__builtin_huge_valf() ? expf(l[i] - top) : 0.0f;
      total = wave_fsum(total);
    }
  }
  K rank[NV];
  if constexpr (kBias) {
    double p[NV], sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = l[i] > -__builtin_huge_valf();
      p[i] = !in ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l[i])))
                                   : l[i] == top ? 1.0 : exp(static_cast<double>(l[i]) - static_cast<double>(top));
      sum += p[i];
    }
    if (!a.sigmoid) {
      sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < NV; ++i) p[i] /= sum;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = l[i] > -__builtin_huge_valf();
      const double r = in ? p[i] + static_cast<double>(a.bias[min(lane * NV + i, a.E - 1)]) : no_rank<double>();
      // (a bias of NaN or -inf ranks last, but can be chosen)
      rank[i] = !in ? r : r >= -1.7e308 ? r : -1.7e308;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) rank[i] = l[i] == l[i] ? l[i] : no_rank<float>();
  }

  // round j's expert and logit go to lane j
  int32_t mine = -1;
  float chosen = -__builtin_huge_valf();
  for (int32_t j = 0; j < a.k; ++j) {
    K best = rank[0];
    int at = 0;
    float bl = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i)
      if (rank[i] > best) {
        best = rank[i];
        at = i;
        bl = l[i];
      }
    const K most = wave_most(best);
    if (!(most > no_rank<K>())) break;  // nothing left to choose
    const int who = __builtin_ctzll(__ballot(best == most));
    const int32_t e = __builtin_amdgcn_readlane(lane * NV + at, who);
    const float le = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bl), who));
    if (lane == j) {
      mine = e;
      chosen = le;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane == who && i == at) rank[i] = no_rank<K>();
  }

  float w = 0.0f;
  if (mine >= 0 || nan) {
    if (a.sigmoid)
      w = 1.0f / (1.0f + expf(-chosen));
    else if (!a.normalize)
      w = expf(chosen - top) / total;
  }
  if (a.normalize) {
    const float high = wave_most(chosen);
    // relative to the largest chosen; of the logistic function only where it is exp to within a rounding
    // (there its sum may be too small for float32)
    if (!a.sigmoid || high < -40.0f) w = mine >= 0 ? expf(chosen - high) : 0.0f;
    const float sum = wave_fsum(w);
    w = mine >= 0 ? w / sum : 0.0f;
  }
  if (lane < a.k) {
    const int64_t at = static_cast<int64_t>(t) * a.k + lane;
    a.experts[at] = mine;
    a.weights[at] = mine < 0 ? 0.0f : nan ? __builtin_nanf("") : a.scale * w;
  }
}

// Backward: the scores again, the chosen ones' gradients d_j in lane j.
template <class H, int NV>
__device__ __forceinline__ void route_bwd_token(const RouteArgs& a, int32_t t) {
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(t) * a.E;
  int32_t e = -1;
  float dw = 0.0f, chosen = -__builtin_huge_valf();
  if (lane < a.k) {
    const int64_t at = static_cast<int64_t>(t) * a.k + lane;
    e = a.experts[at];
    if (e < 0 || e >= a.E) e = -1;
    if (e >= 0) {
      dw = a.dweights[at];
      chosen = one_f32<H>(a.logits, row + e);
    }
  }
  const bool whole = !a.sigmoid && !a.normalize;  // every expert's score has a gradient
  float p[NV], d, rest = 0.0f;                    // dl_e = d_e - rest p_e
  if (whole) {
    float top = -__builtin_huge_valf(), total = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t at = lane * NV + i;
      p[i] = at < a.E ? one_f32<H>(a.logits, row + at) : -__builtin_huge_valf();
      top = fmaxf(top, p[i]);
      nan |= p[i] != p[i];
    }
    top = wave_most(top);
    nan = __any(nan);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] = p[i] > -__builtin_huge_valf() ? expf(p[i] - top) : 0.0f;
      total += p[i];
    }
    total = nan ? __builtin_nanf("") : wave_fsum(total);
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = total == 0.0f ? 0.0f : p[i] / total;  // (0: every expert is masked)
    d = e >= 0 && total != 0.0f ? a.scale * dw * (expf(chosen - top) / total) : 0.0f;
    rest = wave_fsum(d);
  } else {
    float w = 0.0f, slope = 1.0f;
    if (e >= 0 && a.sigmoid) {
      const float x = expf(-fabsf(chosen)), q = 1.0f / (1.0f + x);  // of |l|
      w = chosen >= 0.0f ? q : x * q;
      slope = chosen >= 0.0f ? x * q : q;  // 1 - p without cancellation
    }
    if (a.normalize) {
      const float high = wave_most(chosen);
      if (!a.sigmoid || high < -40.0f) w = e >= 0 ? expf(chosen - high) : 0.0f;
      const float sum = wave_fsum(w);
      w = e >= 0 ? w / sum : 0.0f;
      const float mean = wave_fsum(dw * w);
      d = e >= 0 ? a.scale * w * (dw - mean) * slope : 0.0f;
    } else {
      d = e >= 0 ? a.scale * dw * w * slope : 0.0f;
    }
  }
  float g[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) g[i] = whole ? -(rest * p[i]) : 0.0f;
  for (int32_t j = 0; j < a.k; ++j) {
    const int32_t at = __builtin_amdgcn_readlane(e, j);
    const float dj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(d), j));
    if (at < 0) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane * NV + i == at) g[i] += dj;
  }
  typedef typename Elem<H>::type E;
  E* const out = static_cast<E*>(a.dlogits) + row;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int32_t at = lane * NV + i;
    if (at < a.E) out[at] = H::from_f32(g[i]);
  }
}

template <class H, class K, int NV, bool BWD>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a) {
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWaves + (threadIdx.x >> 6); t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kRouteWaves) {
    if constexpr (BWD)
      route_bwd_token<H, NV>(a, static_cast<int32_t>(t));
    else
      route_token<H, K, NV>(a, static_cast<int32_t>(t));
  }
}

template <class H, int NV, bool BWD>
void launch_route(const RouteArgs& a, hipStream_t s) {
  const int64_t groups = (static_cast<int64_t>(a.T) + kRouteWaves - 1) / kRouteWaves;
  const dim3 g(static_cast<unsigned>(groups < (1 << 21) ? groups : 1 << 21)), b(64 * kRouteWaves);
  if (!BWD && a.bias)
    hipLaunchKernelGGL((route_kernel<H, double, NV, BWD>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((route_kernel<H, float, NV, BWD>), g, b, 0, s, a);
}

template <class H, bool BWD>
void launch_width(const RouteArgs& a, hipStream_t s) {
  if (a.E <= 64)
    launch_route<H, 1, BWD>(a, s);
  else if (a.E <= 128)
    launch_route<H, 2, BWD>(a, s);
  else if (a.E <= 256)
    launch_route<H, 4, BWD>(a, s);
  else if (a.E <= 512)
    launch_route<H, 8, BWD>(a, s);
  else
    launch_route<H, 16, BWD>(a, s);
}

template <bool BWD>
int launch(const fp8z1_router* f, const RouteArgs& a, hipStream_t s, const char* what) {
  if (f->dtype == FP8Z1_F32)
    launch_width<F32, BWD>(a, s);
  else if (f->dtype == FP8Z1_BF16)
    launch_width<Bf16, BWD>(a, s);
  else
    launch_width<F16, BWD>(a, s);
  return launched(what);
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

int check_router(const fp8z1_router* f, const char* what) {
  if (!f) return refuse(FP8Z1_EINVAL, what, "NULL description");
  if (f->dtype != FP8Z1_F32 && f->dtype != FP8Z1_BF16 && f->dtype != FP8Z1_F16)
    return refuse(FP8Z1_EINVAL, what, "dtype must be FP8Z1_BF16, FP8Z1_F16 or FP8Z1_F32");
  if (f->score != FP8Z1_SCORE_SOFTMAX && f->score != FP8Z1_SCORE_SIGMOID)
    return refuse(FP8Z1_EINVAL, what, "score must be FP8Z1_SCORE_SOFTMAX or FP8Z1_SCORE_SIGMOID");
  if (f->T < 0 || f->T > FP8Z1_FFN_MAX_ROWS) return refuse(FP8Z1_ESHAPE, what, "T outside 0 .. 2^30");
  if (f->E < 1 || f->E > FP8Z1_ROUTE_MAX_EXPERTS) return refuse(FP8Z1_ESHAPE, what, "E outside 1 .. 1024");
  if (f->k < 1 || f->k > FP8Z1_ROUTE_MAX_CHOICES || f->k > f->E)
    return refuse(FP8Z1_ESHAPE, what, "k outside 1 .. 32 or more than E");
  if (!(f->scale - f->scale == 0.0f)) return refuse(FP8Z1_EINVAL, what, "scale must be finite");
  return FP8Z1_OK;
}

RouteArgs base_args(const fp8z1_router* f, const void* logits) {
  RouteArgs a{};
  a.logits = logits;
  a.T = static_cast<int32_t>(f->T);
  a.E = f->E;
  a.k = f->k;
  a.sigmoid = f->score == FP8Z1_SCORE_SIGMOID;
  a.normalize = f->normalize != 0;
  a.scale = f->scale;
  return a;
}

size_t elem_size(int32_t dtype) { return dtype == FP8Z1_F32 ? 4 : 2; }

}  // namespace
}  // namespace fp8z1

using namespace fp8z1;

extern "C" int fp8z1_route(const fp8z1_router* f, const void* logits, const float* bias, int32_t* experts, float* weights,
                           void* stream) {
  const char* what = "route";
  const int rc = check_router(f, what);
  if (rc) return rc;
  if (misaligned(bias, 4)) return refuse(FP8Z1_EINVAL, what, "misaligned bias");
  if (f->T == 0) return FP8Z1_OK;
  if (!logits || !experts || !weights) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  if (misaligned(logits, elem_size(f->dtype)) || misaligned(experts, 4) || misaligned(weights, 4))
    return refuse(FP8Z1_EINVAL, what, "misaligned argument");
  RouteArgs a = base_args(f, logits);
  a.bias = bias;
  a.experts = experts;
  a.weights = weights;
  return launch<false>(f, a, static_cast<hipStream_t>(stream), what);
}

extern "C" int fp8z1_route_bwd(const fp8z1_router* f, const void* logits, const int32_t* experts, const float* dweights,
                               void* dlogits, void* stream) {
  const char* what = "route_bwd";
  const int rc = check_router(f, what);
  if (rc) return rc;
  if (f->T == 0) return FP8Z1_OK;
  if (!logits || !experts || !dweights || !dlogits) return refuse(FP8Z1_EINVAL, what, "NULL argument");
  if (misaligned(logits, elem_size(f->dtype)) || misaligned(dlogits, elem_size(f->dtype)) || misaligned(experts, 4) ||
      misaligned(dweights, 4))
    return refuse(FP8Z1_EINVAL, what, "misaligned argument");
  RouteArgs a = base_args(f, logits);
  a.experts = const_cast<int32_t*>(experts);
  a.dweights = dweights;
  a.dlogits = dlogits;
  return launch<true>(f, a, static_cast<hipStream_t>(stream), what);
}
