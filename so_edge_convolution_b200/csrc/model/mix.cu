// mix.cu -- mixing of experts' weights, and its gradients.
//
// The slots (t, j) that name an expert form its list, in slot order; a small
// kernel builds the lists once per backward call.  With every expert in order
// (no index) slot (t, e) names expert e, and no lists are needed.
#include "model_common.cuh"

namespace so2 {

// ---- forward -----------------------------------------------------------------
template <int V, typename TE, typename TO>
__global__ void k_mix(int64_t n_systems, int K, int top_k, int64_t n, const TE *__restrict__ experts,
                      const float *__restrict__ weights, const int *__restrict__ index,
                      TO *__restrict__ out, DevStatus *st) {
  const int64_t c = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) * V;
  if (c >= n) return;
  for (int64_t t = blockIdx.y; t < n_systems; t += gridDim.y) {
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int j = 0; j < top_k; ++j) {
      const int64_t p = t * top_k + j;
      const int e = index ? index[p] : j;
      if (e < 0 || e >= K) {
        if (e != -1 && c == 0) raise_error(st, SO2_ERR_INDEX, (int)p);
        continue;
      }
      const float w = weights[p];
      float x[V];
      load_vec<V>(experts + e * n + c, x);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(w, x[v], acc[v]);
    }
    store_vec<V>(out + t * n + c, acc);
  }
}

// ---- backward ------------------------------------------------------------------
// Lists of the slots by expert: offsets [K+1], slots in slot order.
__global__ void k_mix_lists(int n_slots, int K, const int *__restrict__ index,
                            int *__restrict__ offsets, int *__restrict__ list, DevStatus *st) {
  for (int p = threadIdx.x; p < n_slots; p += blockDim.x) {
    const int e = index[p];
    if (e < -1 || e >= K) raise_error(st, SO2_ERR_INDEX, p);
  }
  for (int e = threadIdx.x; e < K; e += blockDim.x) {
    int c = 0;
    for (int p = 0; p < n_slots; ++p) c += index[p] == e;
    offsets[e + 1] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    offsets[0] = 0;
    for (int e = 0; e < K; ++e) offsets[e + 1] += offsets[e];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < K; e += blockDim.x) {
    int at = offsets[e];
    for (int p = 0; p < n_slots; ++p)
      if (index[p] == e) list[at++] = p;
  }
}

template <int V>
__global__ void k_mix_grad_experts(int64_t n_systems, int K, int top_k, int64_t n,
                                   const float *__restrict__ weights,
                                   const int *__restrict__ offsets, const int *__restrict__ list,
                                   const float *__restrict__ grad, float *__restrict__ ge) {
  const int64_t c = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) * V;
  if (c >= n) return;
  for (int e = blockIdx.y; e < K; e += gridDim.y) {
    const int a = offsets ? offsets[e] : 0, b = offsets ? offsets[e + 1] : (int)n_systems;
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int q = a; q < b; ++q) {
      const int p = offsets ? list[q] : q * top_k + e;
      const float w = weights[p];
      float g[V];
      load_vec<V>(grad + (int64_t)(p / top_k) * n + c, g);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(w, g[v], acc[v]);
    }
    store_vec<V>(ge + e * n + c, acc);
  }
}

constexpr int DOT_SPLITS = 16;

template <int V, typename TE>
__global__ void k_mix_dots(int64_t n_slots, int K, int top_k, int64_t n,
                           const TE *__restrict__ experts, const int *__restrict__ index,
                           const float *__restrict__ grad, float *__restrict__ part) {
  __shared__ float ws[8];
  for (int64_t p = blockIdx.y; p < n_slots; p += gridDim.y) {
    const int e = index ? index[p] : (int)(p % top_k);
    float s = 0.f;
    if (e >= 0 && e < K) {
      const TE *x = experts + e * n;
      const float *g = grad + (p / top_k) * n;
      for (int64_t c = (blockIdx.x * 256ll + threadIdx.x) * V; c < n; c += DOT_SPLITS * 256ll * V) {
        float a[V], b[V];
        load_vec<V>(x + c, a);
        load_vec<V>(g + c, b);
#pragma unroll
        for (int v = 0; v < V; ++v) s = fmaf(a[v], b[v], s);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = 0.f;
      for (int i = 0; i < 8; ++i) s += ws[i];
      part[blockIdx.x * n_slots + p] = s;
    }
    __syncthreads();
  }
}

__global__ void k_mix_dots_join(int64_t n_slots, int splits, const float *__restrict__ part,
                                float *__restrict__ gw) {
  const int64_t p = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (p >= n_slots) return;
  float s = 0.f;
  for (int i = 0; i < splits; ++i) s += part[i * n_slots + p];
  gw[p] = s;
}

}  // namespace so2

using namespace so2;

namespace {

struct MixPlan {
  size_t status, offsets, list, part, total;
};

bool mix_ok(const so2conv_mix_desc *d) {
  return d->n_experts >= 1 && d->n_experts <= 4096 && d->top_k >= 1 && d->top_k <= d->n_experts &&
         d->n_weights >= 1 && d->n_weights <= (1ll << 32) && dtype_ok(d->expert_dtype) &&
         dtype_ok(d->out_dtype);
}

bool mix_size_ok(const so2conv_mix_desc *d, int64_t n_systems) {
  return n_systems >= 0 && n_systems <= 65535 && n_systems * d->top_k <= (1 << 22);
}

MixPlan mix_plan(const so2conv_mix_desc *d, int64_t n_systems, int which) {
  MixPlan p{};
  size_t c = 0;
  p.status = ws_take(c, sizeof(DevStatus));
  if (which == SO2_WS_BACKWARD) {
    const size_t slots = (size_t)(n_systems * d->top_k);
    p.offsets = ws_take(c, sizeof(int) * (d->n_experts + 1));
    p.list = ws_take(c, sizeof(int) * slots);
    p.part = ws_take(c, sizeof(float) * slots * DOT_SPLITS);
  }
  p.total = (c + 255) & ~static_cast<size_t>(255);
  return p;
}

so2_status mix_checks(const so2conv_mix_desc *d, int64_t n_systems, const void *experts,
                      const float *weights, const int32_t *index, void *ws, size_t ws_bytes,
                      int which, MixPlan &p) {
  if (!d) return SO2_ERR_INVALID_ARG;
  if (!mix_ok(d)) return SO2_ERR_UNSUPPORTED;
  if (!mix_size_ok(d, n_systems)) return SO2_ERR_INVALID_ARG;
  if (!index && d->top_k != d->n_experts) return SO2_ERR_INVALID_ARG;
  if (n_systems > 0 && (!experts || !weights)) return SO2_ERR_INVALID_ARG;
  if (!aligned_to(experts, dtype_size(d->expert_dtype)) || !aligned_to(weights, 4) ||
      !aligned_to(index, 4))
    return SO2_ERR_INVALID_ARG;
  if (!ws || !aligned_to(ws, 256)) return SO2_ERR_WORKSPACE;
  p = mix_plan(d, n_systems, which);
  if (ws_bytes < p.total) return SO2_ERR_WORKSPACE;
  return SO2_OK;
}

template <int V, typename TE, typename TO>
void launch_mix(const so2conv_mix_desc *d, int64_t n_systems, const void *experts,
                const float *weights, const int32_t *index, void *out, DevStatus *st,
                cudaStream_t s) {
  const dim3 grid((unsigned)ceil_div(d->n_weights, 256 * V), (unsigned)(n_systems < 4 ? n_systems : 4));
  k_mix<V, TE, TO><<<grid, 256, 0, s>>>(n_systems, d->n_experts, d->top_k, d->n_weights,
                                        static_cast<const TE *>(experts), weights, index,
                                        static_cast<TO *>(out), st);
}

template <typename TE, typename TO>
void launch_mix(bool vec, const so2conv_mix_desc *d, int64_t n_systems, const void *experts,
                const float *weights, const int32_t *index, void *out, DevStatus *st,
                cudaStream_t s) {
  if (vec)
    launch_mix<4, TE, TO>(d, n_systems, experts, weights, index, out, st, s);
  else
    launch_mix<1, TE, TO>(d, n_systems, experts, weights, index, out, st, s);
}

}  // namespace

extern "C" {

size_t so2conv_mix_workspace_size(const so2conv_mix_desc *desc, int64_t n_systems, int which) {
  if (!desc || !mix_ok(desc) || !mix_size_ok(desc, n_systems) ||
      (which != SO2_WS_FORWARD && which != SO2_WS_BACKWARD))
    return 0;
  return mix_plan(desc, n_systems, which).total;
}

so2_status so2conv_mix_experts_forward(const so2conv_mix_desc *d, int64_t n_systems,
                                       const void *experts, const float *weights,
                                       const int32_t *index, void *out, void *ws, size_t ws_bytes,
                                       so2_stream_t stream) {
  MixPlan p;
  so2_status r = mix_checks(d, n_systems, experts, weights, index, ws, ws_bytes, SO2_WS_FORWARD, p);
  if (r != SO2_OK) return r;
  const size_t es = dtype_size(d->expert_dtype), os = dtype_size(d->out_dtype);
  if (n_systems > 0 && (!out || !aligned_to(out, os))) return SO2_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DevStatus *st = ws_at<DevStatus>(ws, p.status);
  MODEL_CK(cudaMemsetAsync(st, 0, sizeof(DevStatus), s));
  if (n_systems == 0) return SO2_OK;
  typedef __nv_bfloat16 bf;
  const bool vec = d->n_weights % 4 == 0 && aligned_to(experts, 4 * es) && aligned_to(out, 4 * os);
  if (d->expert_dtype == SO2_F32 && d->out_dtype == SO2_F32)
    launch_mix<float, float>(vec, d, n_systems, experts, weights, index, out, st, s);
  else if (d->expert_dtype == SO2_F32)
    launch_mix<float, bf>(vec, d, n_systems, experts, weights, index, out, st, s);
  else if (d->out_dtype == SO2_F32)
    launch_mix<bf, float>(vec, d, n_systems, experts, weights, index, out, st, s);
  else
    launch_mix<bf, bf>(vec, d, n_systems, experts, weights, index, out, st, s);
  MODEL_CKL();
  return SO2_OK;
}

so2_status so2conv_mix_experts_backward(const so2conv_mix_desc *d, int64_t n_systems,
                                        const void *experts, const float *weights,
                                        const int32_t *index, const float *grad_out,
                                        float *grad_experts, float *grad_weights, void *ws,
                                        size_t ws_bytes, so2_stream_t stream) {
  MixPlan p;
  so2_status r = mix_checks(d, n_systems, experts, weights, index, ws, ws_bytes, SO2_WS_BACKWARD, p);
  if (r != SO2_OK) return r;
  if ((n_systems > 0 && !grad_out) || !aligned_to(grad_out, 4) || !aligned_to(grad_experts, 4) ||
      !aligned_to(grad_weights, 4))
    return SO2_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DevStatus *st = ws_at<DevStatus>(ws, p.status);
  MODEL_CK(cudaMemsetAsync(st, 0, sizeof(DevStatus), s));
  if (n_systems == 0) {
    if (grad_experts)
      MODEL_CK(cudaMemsetAsync(grad_experts, 0, sizeof(float) * d->n_experts * d->n_weights, s));
    return SO2_OK;
  }
  const int K = d->n_experts, k = d->top_k;
  const int64_t n = d->n_weights, slots = n_systems * k;
  int *offsets = nullptr, *list = nullptr;
  if (index) {
    offsets = ws_at<int>(ws, p.offsets);
    list = ws_at<int>(ws, p.list);
    k_mix_lists<<<1, 1024, 0, s>>>((int)slots, K, index, offsets, list, st);
    MODEL_CKL();
  }
  const size_t es = dtype_size(d->expert_dtype);
  const bool vec = n % 4 == 0 && aligned_to(experts, 4 * es) && aligned_to(grad_out, 16) &&
                   aligned_to(grad_experts, 16);
  if (grad_experts) {
    const dim3 grid((unsigned)ceil_div(n, vec ? 1024 : 256), (unsigned)(K < 4 ? K : 4));
    if (vec)
      k_mix_grad_experts<4><<<grid, 256, 0, s>>>(n_systems, K, k, n, weights, offsets, list,
                                                 grad_out, grad_experts);
    else
      k_mix_grad_experts<1><<<grid, 256, 0, s>>>(n_systems, K, k, n, weights, offsets, list,
                                                 grad_out, grad_experts);
    MODEL_CKL();
  }
  if (grad_weights) {
    float *part = ws_at<float>(ws, p.part);
    const dim3 grid(DOT_SPLITS, (unsigned)(slots < 4096 ? slots : 4096));
    typedef __nv_bfloat16 bf;
    if (d->expert_dtype == SO2_F32) {
      const float *x = static_cast<const float *>(experts);
      if (vec)
        k_mix_dots<4, float><<<grid, 256, 0, s>>>(slots, K, k, n, x, index, grad_out, part);
      else
        k_mix_dots<1, float><<<grid, 256, 0, s>>>(slots, K, k, n, x, index, grad_out, part);
    } else {
      const bf *x = static_cast<const bf *>(experts);
      if (vec)
        k_mix_dots<4, bf><<<grid, 256, 0, s>>>(slots, K, k, n, x, index, grad_out, part);
      else
        k_mix_dots<1, bf><<<grid, 256, 0, s>>>(slots, K, k, n, x, index, grad_out, part);
    }
    MODEL_CKL();
    k_mix_dots_join<<<(unsigned)ceil_div(slots, 256), 256, 0, s>>>(slots, DOT_SPLITS, part,
                                                                   grad_weights);
    MODEL_CKL();
  }
  return SO2_OK;
}

}  // extern "C"
