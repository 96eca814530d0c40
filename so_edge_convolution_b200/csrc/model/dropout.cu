// dropout.cu -- dropout whose mask comes from a counter-based generator.
#include <math.h>

#include "model_common.cuh"

namespace so2 {

long long g_model_launches = 0;

// Philox-4x32-10 (Salmon, Moraes, Dror and Shaw 2011): ten rounds of two
// 32 x 32 -> 64 bit products on a 128-bit counter.
__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t x0 = (uint32_t)block, x1 = (uint32_t)(block >> 32);
  uint32_t x2 = (uint32_t)offset, x3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)x0 * 0xD2511F53u, p1 = (uint64_t)x2 * 0xCD9E8D57u;
    const uint32_t n0 = (uint32_t)(p1 >> 32) ^ x1 ^ k0, n2 = (uint32_t)(p0 >> 32) ^ x3 ^ k1;
    x1 = (uint32_t)p1, x3 = (uint32_t)p0, x0 = n0, x2 = n2;
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
  return make_uint4(x0, x1, x2, x3);
}

__device__ __forceinline__ uint32_t word_of(uint4 w, int i) {
  return i < 2 ? (i == 0 ? w.x : w.y) : (i == 2 ? w.z : w.w);
}

// The kernels move x, the residual and out once each; the generator's twenty
// wide products a draw of four words stay below that as long as no word is
// drawn twice, so each kernel is laid out by its unit.
//
// thr = p 2^32 (2^32 drops everything); scale = 1 / (1 - p).
struct DropArgs {
  const uint64_t *rng;
  uint64_t thr;
  float scale;
};

// V values at p: kept ones scaled, the residual added, rounded once.
template <int V, typename T>
__device__ __forceinline__ void drop_store(const float (&x)[V], const float (&r)[V], bool has_res,
                                           const bool (&keep)[V], float scale, T *out) {
  float y[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    y[v] = keep[v] ? x[v] * scale : 0.f;
    if (has_res) y[v] += r[v];
  }
  store_vec<V>(out, y);
}

// One word an element: a thread takes the V / 4 draws of V consecutive
// elements; VEC where all pointers lie on a boundary of V elements.
template <int V, bool VEC, typename T>
__global__ void __launch_bounds__(256)
    k_drop_elements(int64_t total, const T *x, const T *res, DropArgs a, T *out) {
  const uint64_t seed = a.rng[0], offset = a.rng[1];
  const int64_t i0 = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) * V;
  if (i0 >= total) return;
  if (VEC && i0 + V <= total) {
    float xv[V], rv[V];
    load_vec<V>(x + i0, xv);
    if (res) load_vec<V>(res + i0, rv);
    bool keep[V];
#pragma unroll
    for (int g = 0; g < V / 4; ++g) {
      const uint4 w = philox((uint64_t)(i0 >> 2) + g, offset, seed);
      keep[4 * g] = w.x >= a.thr, keep[4 * g + 1] = w.y >= a.thr;
      keep[4 * g + 2] = w.z >= a.thr, keep[4 * g + 3] = w.w >= a.thr;
    }
    drop_store<V>(xv, rv, res != nullptr, keep, a.scale, out + i0);
    return;
  }
  for (int g = 0; g < V / 4; ++g) {
    const uint4 w = philox((uint64_t)(i0 >> 2) + g, offset, seed);
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + 4 * g + j;
      if (i >= total) return;
      const float xv[1] = {to_f32(x[i])}, rv[1] = {res ? to_f32(res[i]) : 0.f};
      const bool keep[1] = {word_of(w, j) >= a.thr};
      drop_store<1>(xv, rv, res != nullptr, keep, a.scale, out + i);
    }
  }
}

// One word a (node, channel): a thread draws for V channels of a node and
// takes them through its share of the components.  V is 1, or a multiple of 4
// that divides the channels.
template <int V, typename T>
__global__ void __launch_bounds__(256)
    k_drop_channels(int64_t n, int n_comp, int channels, int share, const T *x, const T *res,
                    DropArgs a, T *out) {
  const uint64_t seed = a.rng[0], offset = a.rng[1];
  const int groups = channels / V;
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (id >= n * groups) return;
  const int64_t i = id / groups;
  const int c = (int)(id - i * groups) * V;
  const uint64_t m = (uint64_t)(i * channels + c);
  bool keep[V];
  if constexpr (V == 1) {
    keep[0] = word_of(philox(m >> 2, offset, seed), (int)(m & 3)) >= a.thr;
  } else {
#pragma unroll
    for (int g = 0; g < V / 4; ++g) {
      const uint4 w = philox((m >> 2) + g, offset, seed);
      keep[4 * g] = w.x >= a.thr, keep[4 * g + 1] = w.y >= a.thr;
      keep[4 * g + 2] = w.z >= a.thr, keep[4 * g + 3] = w.w >= a.thr;
    }
  }
  const int s0 = blockIdx.y * share, s1 = s0 + share < n_comp ? s0 + share : n_comp;
  const int64_t at = i * n_comp * channels + c;
#pragma unroll 4
  for (int s = s0; s < s1; ++s) {
    const int64_t p = at + (int64_t)s * channels;
    float xv[V], rv[V];
    load_vec<V>(x + p, xv);
    if (res) load_vec<V>(res + p, rv);
    drop_store<V>(xv, rv, res != nullptr, keep, a.scale, out + p);
  }
}

// One word a row: a warp takes a share of a row; a dropped row is not read.
template <int V, typename T>
__global__ void __launch_bounds__(256)
    k_drop_rows(int64_t n, int64_t row, int64_t share, const T *x, const T *res,
                const int64_t *__restrict__ rows, DropArgs a, T *out) {
  const uint64_t seed = a.rng[0], offset = a.rng[1];
  const int64_t i = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (i >= n) return;
  const uint64_t m = rows ? (uint64_t)rows[i] : (uint64_t)i;
  const bool keep1 = word_of(philox(m >> 2, offset, seed), (int)(m & 3)) >= a.thr;
  const int64_t c0 = blockIdx.y * share, c1 = c0 + share < row ? c0 + share : row;
  bool keep[V];
#pragma unroll
  for (int v = 0; v < V; ++v) keep[v] = keep1;
#pragma unroll 4
  for (int64_t c = c0 + (threadIdx.x & 31) * V; c < c1; c += 32 * V) {
    const int64_t p = i * row + c;
    float xv[V], rv[V];
    if (keep1) load_vec<V>(x + p, xv);
    if (res) load_vec<V>(res + p, rv);
    drop_store<V>(xv, rv, res != nullptr, keep, a.scale, out + p);
  }
}

template <typename T>
void launch_dropout(const so2conv_dropout_desc *d, int64_t n, const T *x, const T *res,
                    const int64_t *rows, DropArgs a, T *out, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);  // 16-byte vectors
  const bool vec = aligned_to(x, 16) && aligned_to(res, 16) && aligned_to(out, 16);
  const int64_t row = (int64_t)d->n_comp * d->channels;
  if (d->unit == SO2_DROP_ELEMENT) {
    const int64_t total = n * row;
    const unsigned grid = (unsigned)ceil_div(total, 256 * V);
    if (vec)
      k_drop_elements<V, true, T><<<grid, 256, 0, s>>>(total, x, res, a, out);
    else
      k_drop_elements<V, false, T><<<grid, 256, 0, s>>>(total, x, res, a, out);
  } else if (d->unit == SO2_DROP_CHANNEL) {
    const bool wide = vec && d->channels % V == 0;
    const int64_t threads = n * (d->channels / (wide ? V : 1));
    // split the components where nodes and channels alone leave SMs idle, but
    // keep four of them to a draw
    int64_t parts = ceil_div(MODEL_SMS * 2048, threads);
    if (parts > d->n_comp / 4) parts = d->n_comp / 4;
    if (parts < 1) parts = 1;
    const int share = (int)ceil_div(d->n_comp, parts);
    const dim3 grid((unsigned)ceil_div(threads, 256), (unsigned)ceil_div(d->n_comp, share));
    if (wide)
      k_drop_channels<V, T><<<grid, 256, 0, s>>>(n, d->n_comp, d->channels, share, x, res, a, out);
    else
      k_drop_channels<1, T><<<grid, 256, 0, s>>>(n, d->n_comp, d->channels, share, x, res, a, out);
  } else {
    const bool wide = vec && row % V == 0;
    // likewise: a warp a row, or shares of at least four vectors a lane
    const int64_t least = 4 * 32 * (wide ? V : 1);
    int64_t parts = ceil_div(MODEL_SMS * 64, n);
    if (parts > row / least) parts = row / least;
    if (parts < 1) parts = 1;
    if (parts > 65535) parts = 65535;
    const int64_t share = ceil_div(ceil_div(row, parts), V) * V;
    const dim3 grid((unsigned)ceil_div(n, 8), (unsigned)ceil_div(row, share));
    if (wide)
      k_drop_rows<V, T><<<grid, 256, 0, s>>>(n, row, share, x, res, rows, a, out);
    else
      k_drop_rows<1, T><<<grid, 256, 0, s>>>(n, row, share, x, res, rows, a, out);
  }
}

}  // namespace so2

using namespace so2;

extern "C" so2_status so2conv_dropout(const so2conv_dropout_desc *d, int64_t n, const void *x,
                                      const void *residual, const int64_t *rows,
                                      const uint64_t *rng, void *out, so2_stream_t stream) {
  if (!d) return SO2_ERR_INVALID_ARG;
  if (d->channels < 1 || d->channels > 65536 || d->n_comp < 1 || d->n_comp > 1024 ||
      !dtype_ok(d->dtype) || d->unit < SO2_DROP_ELEMENT || d->unit > SO2_DROP_ROW)
    return SO2_ERR_UNSUPPORTED;
  if (!(d->p >= 0.f && d->p <= 1.f)) return SO2_ERR_INVALID_ARG;
  if (n < 0 || n > (1ll << 30) || !rng) return SO2_ERR_INVALID_ARG;
  if (rows && d->unit != SO2_DROP_ROW) return SO2_ERR_INVALID_ARG;
  if (!aligned_to(rng, 8) || !aligned_to(rows, 8)) return SO2_ERR_INVALID_ARG;
  if (n > (1ll << 38) / ((int64_t)d->n_comp * d->channels)) return SO2_ERR_INVALID_ARG;
  if (n == 0) return SO2_OK;
  const size_t es = dtype_size(d->dtype);
  if (!x || !out || !aligned_to(x, es) || !aligned_to(out, es) || !aligned_to(residual, es))
    return SO2_ERR_INVALID_ARG;
  const double p = d->p;
  const uint64_t thr = (uint64_t)llrint(p * 4294967296.0);
  const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const DropArgs a{rng, thr, scale};
  typedef __nv_bfloat16 bf;
  if (d->dtype == SO2_F32)
    launch_dropout<float>(d, n, static_cast<const float *>(x), static_cast<const float *>(residual),
                          rows, a, static_cast<float *>(out), s);
  else
    launch_dropout<bf>(d, n, static_cast<const bf *>(x), static_cast<const bf *>(residual), rows, a,
                       static_cast<bf *>(out), s);
  MODEL_CKL();
  return SO2_OK;
}
