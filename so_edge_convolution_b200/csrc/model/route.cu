// route.cu -- routing to experts: scores, selection and the logits' gradient.
//
// One warp per token.  Experts are ranked by a 64-bit key in the order of
// their selection scores: 0 for an expert that may not be chosen, 1 for NaN,
// then the numbers.  Without a bias the logits themselves give the order;
// with one, c = s + bias is formed in 64 bits.
#include <math.h>

#include "model_common.cuh"

namespace so2 {

struct RouteArgs {
  int K, top_k, n_groups, top_groups, group_top, per;
  int softmax, renorm;
  float scale;
};

__device__ __forceinline__ uint64_t order_key(double c, bool dead) {
  if (dead || c == -INFINITY) return 0;
  if (c != c) return 1;
  const long long b = __double_as_longlong(c + 0.0);  // -0 to +0
  return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The largest key of the warp and the lowest index that has it.
__device__ __forceinline__ void warp_best(uint64_t &key, int &idx) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t k = __shfl_xor_sync(0xffffffffu, key, o);
    const int i = __shfl_xor_sync(0xffffffffu, idx, o);
    if (k > key || (k == key && i < idx)) key = k, idx = i;
  }
}

__device__ __forceinline__ float sigmoid_f(float x) { return 1.f / (1.f + expf(-x)); }

constexpr int ROUTE_WARPS = 4;

// Shared memory per warp: keys [K] u64, chosen [top_k] f32, group keys [n_groups] u64.
template <int NPL, typename T>  // NPL experts a lane: e = lane + 32 i
__global__ void k_route(RouteArgs a, int64_t n, const T *__restrict__ logits,
                        const float *__restrict__ bias, float *__restrict__ weights,
                        int *__restrict__ index, int *__restrict__ counts) {
  extern __shared__ uint64_t sm[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint64_t *keys = sm + (size_t)w * (a.K + a.n_groups + a.top_k), *gkeys = keys + a.K;
  double *cs = reinterpret_cast<double *>(keys);
  float *picked = reinterpret_cast<float *>(gkeys + a.n_groups);
  for (int64_t t = blockIdx.x * (int64_t)ROUTE_WARPS + w; t < n;
       t += (int64_t)gridDim.x * ROUTE_WARPS) {
    float x[NPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      x[i] = e < a.K ? to_f32(logits[t * a.K + e]) : -INFINITY;
      m = fmaxf(m, x[i]);
    }
    m = warp_max(m);
    const float m0 = m == -INFINITY ? 0.f : m;  // a row without any expert
    float z = 0.f;
    if (a.softmax) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) z += expf(x[i] - m0);
      z = warp_sum(z);
    }
    // selection keys
    const bool by_score = bias != nullptr || (a.top_groups < a.n_groups && a.group_top > 1);
    double z64 = 0.0;
    if (by_score && a.softmax) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) z64 += exp((double)x[i] - m0);
      z64 = warp_sum(z64);
    }
    uint64_t key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      const bool dead = x[i] == -INFINITY;
      double c = x[i];
      if (by_score) {
        c = a.softmax ? exp((double)x[i] - m0) / z64 : 1.0 / (1.0 + exp(-(double)x[i]));
        if (bias && e < a.K) c += bias[e];
      }
      key[i] = e < a.K ? order_key(bias ? c : (double)x[i], dead) : 0;
      if (e < a.K && a.top_groups < a.n_groups) cs[e] = dead ? -INFINITY : c;
    }
    if (a.top_groups < a.n_groups) {
      __syncwarp();
      for (int g = lane; g < a.n_groups; g += 32) {
        double b0 = -INFINITY, b1 = -INFINITY;  // NaN ranks below every number
        bool nan = false;
        for (int j = 0; j < a.per; ++j) {
          const double c = cs[g * a.per + j];
          if (c != c) { nan = true; continue; }
          if (c > b0) b1 = b0, b0 = c;
          else if (c > b1) b1 = c;
        }
        // a NaN counts where too few numbers are left
        const bool use2 = a.group_top > 1;
        double s = b0;
        if (use2 && b1 != -INFINITY) s += b1;
        const bool short_ = b0 == -INFINITY || (use2 && b1 == -INFINITY);
        gkeys[g] = nan && short_ ? 1 : order_key(s, b0 == -INFINITY);
      }
      __syncwarp();
      // group g stays if fewer than top_groups groups come before it
      uint64_t keep = 0;  // of this lane's experts
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        if (e >= a.K) continue;
        const int g = e / a.per;
        const uint64_t k = gkeys[g];
        int before = 0;
        for (int h = 0; h < a.n_groups; ++h)
          before += gkeys[h] > k || (gkeys[h] == k && h < g);
        if (before < a.top_groups) keep |= 1ull << i;
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (!((keep >> i) & 1)) key[i] = 0;
      __syncwarp();
    }
    // weights of all experts, or the top_k rounds of selection
    float total = 0.f;
    if (a.top_k == a.K) {
      float mc = -INFINITY;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (key[i]) mc = fmaxf(mc, x[i]);
      mc = warp_max(mc);
      float s[NPL];
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        s[i] = 0.f;
        if (key[i])
          s[i] = !a.softmax ? sigmoid_f(x[i])
                 : a.renorm ? expf(x[i] - mc)
                            : expf(x[i] - m0) / z;
        total += s[i];
      }
      total = warp_sum(total);
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        if (e >= a.K) continue;
        float v = s[i];
        if (a.renorm) v = total == 0.f ? 0.f : v / total;
        weights[t * a.K + e] = key[i] ? v * a.scale : 0.f;
        index[t * a.K + e] = key[i] ? e : -1;
        if (counts && key[i]) atomicAdd(&counts[e], 1);
      }
      continue;
    }
    float mc = 0.f;
    for (int j = 0; j < a.top_k; ++j) {
      uint64_t bk = 0;
      int be = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (key[i] > bk) bk = key[i], be = lane + 32 * i;
      warp_best(bk, be);
      const bool live = bk != 0;
      float xv = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (live && be == lane + 32 * i) xv = x[i], key[i] = 0;
      if (live) xv = __shfl_sync(0xffffffffu, xv, be & 31);
      if (lane == 0) {
        picked[j] = xv;
        index[t * a.top_k + j] = live ? be : -1;
        if (counts && live) atomicAdd(&counts[be], 1);
      }
      if (live) mc = j == 0 ? xv : fmaxf(mc, xv);
    }
    __syncwarp();
    for (int pass = 0; pass < 2; ++pass) {
      // pass 0: the sum of the chosen scores; pass 1: the weights
      for (int j = lane; j < a.top_k; j += 32) {
        const bool live = index[t * a.top_k + j] >= 0;
        float s = 0.f;
        if (live)
          s = !a.softmax ? sigmoid_f(picked[j])
              : a.renorm ? expf(picked[j] - mc)
                         : expf(picked[j] - m0) / z;
        if (pass == 0)
          total += s;
        else
          weights[t * a.top_k + j] =
              !live ? 0.f : (a.renorm ? (total == 0.f ? 0.f : s / total) : s) * a.scale;
      }
      if (pass == 0) total = warp_sum(total);
    }
    __syncwarp();
  }
}

// Shared memory per warp: gs [K] f32, chosen flags in its own array.
template <int NPL, typename T>
__global__ void k_route_grad(RouteArgs a, int64_t n, const T *__restrict__ logits,
                             const int *__restrict__ index, const float *__restrict__ gw,
                             float *__restrict__ grad) {
  extern __shared__ float gsm[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float *gs = gsm + (size_t)w * a.K;
  for (int64_t t = blockIdx.x * (int64_t)ROUTE_WARPS + w; t < n;
       t += (int64_t)gridDim.x * ROUTE_WARPS) {
    float x[NPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      x[i] = e < a.K ? to_f32(logits[t * a.K + e]) : -INFINITY;
      m = fmaxf(m, x[i]);
      if (e < a.K) gs[e] = 0.f;
    }
    m = warp_max(m);
    const float m0 = m == -INFINITY ? 0.f : m;
    float z = 1.f;
    if (a.softmax && !a.renorm) {
      z = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) z += expf(x[i] - m0);
      z = warp_sum(z);
    }
    // the chosen logits' largest, the sum of the chosen scores
    float mc = -INFINITY, total = 0.f, dot = 0.f;
    if (a.renorm) {
      for (int j = lane; j < a.top_k; j += 32) {
        const int e = index[t * a.top_k + j];
        if (e >= 0 && e < a.K) mc = fmaxf(mc, to_f32(logits[t * a.K + e]));
      }
      mc = warp_max(mc);
      if (mc == -INFINITY) mc = 0.f;  // no slot in use
      for (int j = lane; j < a.top_k; j += 32) {
        const int e = index[t * a.top_k + j];
        if (e >= 0 && e < a.K) {
          const float v = to_f32(logits[t * a.K + e]);
          total += a.softmax ? expf(v - mc) : sigmoid_f(v);
        }
      }
      total = warp_sum(total);
      for (int j = lane; j < a.top_k; j += 32) {
        const int e = index[t * a.top_k + j];
        if (e >= 0 && e < a.K && total != 0.f) {
          const float v = to_f32(logits[t * a.K + e]);
          dot += gw[t * a.top_k + j] * ((a.softmax ? expf(v - mc) : sigmoid_f(v)) / total);
        }
      }
      dot = warp_sum(dot);
    }
    __syncwarp();
    // gradients of the scores (an expert named twice adds up, in slot order)
    if (lane == 0)
      for (int j = 0; j < a.top_k; ++j) {
        const int e = index[t * a.top_k + j];
        if (e < 0 || e >= a.K || (a.renorm && total == 0.f)) continue;
        const float v = to_f32(logits[t * a.K + e]);
        const float g = (gw[t * a.top_k + j] - dot) * a.scale;
        float d;  // score times (for softmax) or derivative times the gradient
        if (a.softmax)
          d = a.renorm ? expf(v - mc) / total * g : g;
        else
          d = (a.renorm ? g / total : g) * sigmoid_f(v) * sigmoid_f(-v);
        gs[e] += d;
      }
    __syncwarp();
    float sdot = 0.f;
    if (a.softmax && !a.renorm) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        if (e < a.K && gs[e] != 0.f) sdot += expf(x[i] - m0) / z * gs[e];
      }
      sdot = warp_sum(sdot);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      if (e >= a.K) continue;
      float g = gs[e];
      if (a.softmax && !a.renorm) g = z == 0.f ? 0.f : expf(x[i] - m0) / z * (g - sdot);
      grad[t * a.K + e] = g;
    }
    __syncwarp();
  }
}

}  // namespace so2

using namespace so2;

namespace {

bool route_ok(const so2conv_route_desc *d) {
  if (d->n_experts < 1 || d->n_experts > 1024) return false;
  if (d->top_k < 1 || d->top_k > d->n_experts) return false;
  if (d->n_groups < 1 || d->n_groups > d->n_experts || d->n_experts % d->n_groups) return false;
  if (d->top_groups < 1 || d->top_groups > d->n_groups) return false;
  const int per = d->n_experts / d->n_groups;
  if (d->group_top < 1 || d->group_top > 2 || d->group_top > per) return false;
  if (d->top_k > d->top_groups * per) return false;
  if (d->score != SO2_SCORE_SOFTMAX && d->score != SO2_SCORE_SIGMOID) return false;
  if (d->renormalise != 0 && d->renormalise != 1) return false;
  return dtype_ok(d->dtype);
}

RouteArgs route_args(const so2conv_route_desc *d) {
  RouteArgs a;
  a.K = d->n_experts;
  a.top_k = d->top_k;
  a.n_groups = d->n_groups;
  a.top_groups = d->top_groups;
  a.group_top = d->group_top;
  a.per = d->n_experts / d->n_groups;
  a.softmax = d->score == SO2_SCORE_SOFTMAX;
  a.renorm = d->renormalise;
  a.scale = d->scale;
  return a;
}

so2_status route_checks(const so2conv_route_desc *d, int64_t n, const void *logits) {
  if (!d) return SO2_ERR_INVALID_ARG;
  if (!route_ok(d)) return SO2_ERR_UNSUPPORTED;
  if (!(d->scale - d->scale == 0.f) || d->scale == 0.f) return SO2_ERR_INVALID_ARG;
  if (n < 0 || n > (1ll << 30)) return SO2_ERR_INVALID_ARG;
  if (n > 0 && (!logits || !aligned_to(logits, dtype_size(d->dtype)))) return SO2_ERR_INVALID_ARG;
  return SO2_OK;
}

// Experts a lane, as a compile-time power of two.
#define ROUTE_DISPATCH(K, ...)                                   \
  if ((K) <= 32) { constexpr int NPL = 1; __VA_ARGS__; }         \
  else if ((K) <= 64) { constexpr int NPL = 2; __VA_ARGS__; }    \
  else if ((K) <= 128) { constexpr int NPL = 4; __VA_ARGS__; }   \
  else if ((K) <= 256) { constexpr int NPL = 8; __VA_ARGS__; }   \
  else if ((K) <= 512) { constexpr int NPL = 16; __VA_ARGS__; }  \
  else { constexpr int NPL = 32; __VA_ARGS__; }

int route_grid(int64_t n) {
  const int64_t want = ceil_div(n, ROUTE_WARPS);
  return (int)(want < MODEL_SMS * 16 ? want : MODEL_SMS * 16);
}

template <int NPL, typename T>
so2_status run_route(const RouteArgs &a, int64_t n, const void *logits, const float *bias,
                     float *weights, int32_t *index, int32_t *counts, cudaStream_t s) {
  const int smem = ROUTE_WARPS * (a.K + a.n_groups + a.top_k) * 8;
  if (smem > 48 * 1024)
    MODEL_CK(cudaFuncSetAttribute(k_route<NPL, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  k_route<NPL, T><<<route_grid(n), 32 * ROUTE_WARPS, smem, s>>>(
      a, n, static_cast<const T *>(logits), bias, weights, index, counts);
  MODEL_CKL();
  return SO2_OK;
}

template <int NPL, typename T>
so2_status run_route_grad(const RouteArgs &a, int64_t n, const void *logits, const int32_t *index,
                          const float *gw, float *grad, cudaStream_t s) {
  const int smem = ROUTE_WARPS * a.K * 4;
  k_route_grad<NPL, T><<<route_grid(n), 32 * ROUTE_WARPS, smem, s>>>(
      a, n, static_cast<const T *>(logits), index, gw, grad);
  MODEL_CKL();
  return SO2_OK;
}

}  // namespace

extern "C" {

so2_status so2conv_route_forward(const so2conv_route_desc *d, int64_t n, const void *logits,
                                 const float *bias, float *weights, int32_t *index,
                                 int32_t *counts, so2_stream_t stream) {
  so2_status r = route_checks(d, n, logits);
  if (r != SO2_OK) return r;
  if (n > 0 && (!weights || !index)) return SO2_ERR_INVALID_ARG;
  if (!aligned_to(weights, 4) || !aligned_to(index, 4) || !aligned_to(bias, 4) ||
      !aligned_to(counts, 4))
    return SO2_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (counts) MODEL_CK(cudaMemsetAsync(counts, 0, sizeof(int32_t) * d->n_experts, s));
  if (n == 0) return SO2_OK;
  const RouteArgs a = route_args(d);
  if (d->dtype == SO2_F32)
    ROUTE_DISPATCH(a.K, return run_route<NPL, float>(a, n, logits, bias, weights, index, counts, s))
  ROUTE_DISPATCH(a.K, return run_route<NPL, __nv_bfloat16>(a, n, logits, bias, weights, index, counts, s))
}

so2_status so2conv_route_backward(const so2conv_route_desc *d, int64_t n, const void *logits,
                                  const int32_t *index, const float *gw, float *grad,
                                  so2_stream_t stream) {
  so2_status r = route_checks(d, n, logits);
  if (r != SO2_OK) return r;
  if (n > 0 && (!index || !gw || !grad)) return SO2_ERR_INVALID_ARG;
  if (!aligned_to(index, 4) || !aligned_to(gw, 4) || !aligned_to(grad, 4)) return SO2_ERR_INVALID_ARG;
  if (n == 0) return SO2_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RouteArgs a = route_args(d);
  if (d->dtype == SO2_F32)
    ROUTE_DISPATCH(a.K, return run_route_grad<NPL, float>(a, n, logits, index, gw, grad, s))
  ROUTE_DISPATCH(a.K, return run_route_grad<NPL, __nv_bfloat16>(a, n, logits, index, gw, grad, s))
}

}  // extern "C"
