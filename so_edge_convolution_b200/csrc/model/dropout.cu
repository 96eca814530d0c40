// dropout.cu -- dropout whose mask comes from a counter-based generator.
#include <math.h>

#include "model_common.cuh"

namespace so2 {

long long g_model_launches = 0;

// Philox-4x32-10 (Salmon, Moraes, Dror and Shaw 2011): ten rounds of two
// 32 x 32 -> 64 bit products on a 128-bit counter.
struct PhiloxKey {
  uint64_t seed, offset;
  __device__ __forceinline__ PhiloxKey(const uint64_t *rng) : seed(rng[0]), offset(rng[1]) {}
};

__device__ __forceinline__ uint4 philox(uint64_t block, const PhiloxKey &key) {
  uint32_t x0 = (uint32_t)block, x1 = (uint32_t)(block >> 32);
  uint32_t x2 = (uint32_t)key.offset, x3 = (uint32_t)(key.offset >> 32);
  uint32_t k0 = (uint32_t)key.seed, k1 = (uint32_t)(key.seed >> 32);
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

// The kernels move x, the residual and out once each and are laid out by their
// unit, so that a thread draws for all that it moves.  (Some words are drawn
// more than once: by each share of a node's components or of a row, by all
// lanes of a row's warp, and, where vectors do not fit, for one unit of four.)
struct DropArgs {
  const uint64_t *rng;
  uint32_t thr;  // p 2^32; p = 1 does not get here as elements or channels
  bool none;     // p = 1: no row is kept
  float scale;   // 1 / (1 - p)
  __device__ __forceinline__ bool keep(uint32_t w) const { return w >= thr; }
};

// V values as they lie in memory: 16 bytes, or one value.
template <int V, typename T>
struct Raw {
  uint4 v;
  __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float (&r)[V]) const {
    load_vec<V>(reinterpret_cast<const T *>(&v), r);
  }
};
template <typename T>
struct Raw<1, T> {
  T v;
  __device__ __forceinline__ void load(const T *p) { v = *p; }
  __device__ __forceinline__ void get(float (&r)[1]) const { r[0] = to_f32(v); }
};

// Kept values scaled, the residual added, rounded once.
template <int V, bool RES, typename T>
__device__ __forceinline__ void drop_store(const Raw<V, T> &x, const Raw<V, T> &res,
                                           const bool (&keep)[V], float scale, T *out) {
  float y[V], r[V];
  x.get(y);
  if (RES) res.get(r);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    y[v] = keep[v] ? y[v] * scale : 0.f;
    if (RES) y[v] += r[v];
  }
  store_vec<V>(out, y);
}

// Which of V units from m on stay; m is a multiple of 4 (or V is 1).
template <int V>
__device__ __forceinline__ void drop_mask(uint64_t m, const PhiloxKey &key, const DropArgs &a,
                                          bool (&keep)[V]) {
  if constexpr (V == 1) {
    keep[0] = a.keep(word_of(philox(m >> 2, key), (int)(m & 3)));
  } else {
#pragma unroll
    for (int g = 0; g < V / 4; ++g) {
      const uint4 w = philox((m >> 2) + g, key);
      keep[4 * g] = a.keep(w.x), keep[4 * g + 1] = a.keep(w.y);
      keep[4 * g + 2] = a.keep(w.z), keep[4 * g + 3] = a.keep(w.w);
    }
  }
}

// One word an element: a thread takes the V / 4 draws of V consecutive
// elements, ITEMS times over, with all loads issued first.  The generator's
// integer products bound this kernel as much as memory does: 64 M bf16
// elements take 41 us with one round in place of ten (the copy rate), 55 with
// seven and 66 with all ten.  Several draws a thread hide each other's
// latency (72 us with one item, 68 with four, 66 with five blocks an SM on top).
// VEC where all pointers lie on a boundary of V elements.
constexpr int DROP_ITEMS = 4;

template <int V, bool VEC, bool RES, typename T>
__global__ void __launch_bounds__(256, 5)
    k_drop_elements(int64_t total, const T *x, const T *res, DropArgs a, T *out) {
  const int64_t first = (int64_t)blockIdx.x * (256 * V * DROP_ITEMS) + threadIdx.x * V;
  if (first >= total) return;
  if (VEC && first + (DROP_ITEMS - 1) * 256 * V + V <= total) {
    Raw<V, T> xv[DROP_ITEMS], rv[DROP_ITEMS];
#pragma unroll
    for (int k = 0; k < DROP_ITEMS; ++k) {
      xv[k].load(x + first + k * 256 * V);
      if (RES) rv[k].load(res + first + k * 256 * V);
    }
    const PhiloxKey key(a.rng);
    bool keep[DROP_ITEMS][V];
#pragma unroll
    for (int k = 0; k < DROP_ITEMS; ++k)
      drop_mask<V>((uint64_t)(first + k * 256 * V), key, a, keep[k]);
#pragma unroll
    for (int k = 0; k < DROP_ITEMS; ++k)
      drop_store<V, RES>(xv[k], rv[k], keep[k], a.scale, out + first + k * 256 * V);
    return;
  }
  const PhiloxKey key(a.rng);
  for (int k = 0; k < DROP_ITEMS; ++k) {
    const int64_t i0 = first + k * 256 * V;
    if (i0 >= total) return;
    bool keep[V];
    drop_mask<V>((uint64_t)i0, key, a, keep);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (i0 + v >= total) continue;
      Raw<1, T> xv, rv;
      xv.load(x + i0 + v);
      if (RES) rv.load(res + i0 + v);
      const bool kv[1] = {keep[v]};
      drop_store<1, RES>(xv, rv, kv, a.scale, out + i0 + v);
    }
  }
}

// One word a (node, channel): a thread draws for V channels of a node and
// takes them through its share of the components.  V is 1, or a multiple of 4
// that divides the channels.
template <int V, bool RES, typename T>
__global__ void __launch_bounds__(256)
    k_drop_channels(int64_t n, int n_comp, int channels, int share, const T *x, const T *res,
                    DropArgs a, T *out) {
  const int groups = channels / V;
  const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (id >= n * groups) return;
  const int64_t i = id / groups;
  const int c = (int)(id - i * groups) * V;
  bool keep[V];
  drop_mask<V>((uint64_t)(i * channels + c), PhiloxKey(a.rng), a, keep);
  const int s0 = blockIdx.y * share, s1 = s0 + share < n_comp ? s0 + share : n_comp;
  const int64_t at = i * n_comp * channels + c;
  // four components' loads before their stores (out may be x or the residual,
  // so the compiler keeps that order)
  constexpr int B = 4;
  for (int s = s0; s < s1; s += B) {
    Raw<V, T> xv[B], rv[B];
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (s + b < s1) {
        xv[b].load(x + at + (int64_t)(s + b) * channels);
        if (RES) rv[b].load(res + at + (int64_t)(s + b) * channels);
      }
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (s + b < s1)
        drop_store<V, RES>(xv[b], rv[b], keep, a.scale, out + at + (int64_t)(s + b) * channels);
  }
}

// One word a row: a warp takes a share of a row; a dropped row is not read.
template <int V, bool RES, typename T>
__global__ void __launch_bounds__(256)
    k_drop_rows(int64_t n, int64_t row, int64_t share, const T *x, const T *res,
                const int64_t *__restrict__ rows, DropArgs a, T *out) {
  const int64_t i = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (i >= n) return;
  const uint64_t m = rows ? (uint64_t)rows[i] : (uint64_t)i;
  const bool keep1 =
      !a.none && a.keep(word_of(philox(m >> 2, PhiloxKey(a.rng)), (int)(m & 3)));
  const int64_t c0 = blockIdx.y * share, c1 = c0 + share < row ? c0 + share : row;
  bool keep[V];
#pragma unroll
  for (int v = 0; v < V; ++v) keep[v] = keep1;
  constexpr int B = 4;
  for (int64_t c = c0 + (threadIdx.x & 31) * V; c < c1; c += B * 32 * V) {
    const int64_t p = i * row + c;
    Raw<V, T> xv[B] = {}, rv[B];
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (c + b * 32 * V < c1) {
        if (keep1) xv[b].load(x + p + b * 32 * V);
        if (RES) rv[b].load(res + p + b * 32 * V);
      }
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (c + b * 32 * V < c1)
        drop_store<V, RES>(xv[b], rv[b], keep, a.scale, out + p + b * 32 * V);
  }
}

template <bool RES, typename T>
void launch_dropout(const so2conv_dropout_desc *d, int64_t n, const T *x, const T *res,
                    const int64_t *rows, DropArgs a, T *out, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);  // 16-byte vectors
  const bool vec = aligned_to(x, 16) && aligned_to(res, 16) && aligned_to(out, 16);
  const int64_t row = (int64_t)d->n_comp * d->channels;
  if (d->unit == SO2_DROP_ELEMENT && !a.none) {
    const int64_t total = n * row;
    const unsigned grid = (unsigned)ceil_div(total, 256 * V * DROP_ITEMS);
    if (vec)
      k_drop_elements<V, true, RES, T><<<grid, 256, 0, s>>>(total, x, res, a, out);
    else
      k_drop_elements<V, false, RES, T><<<grid, 256, 0, s>>>(total, x, res, a, out);
  } else if (d->unit == SO2_DROP_CHANNEL && !a.none) {
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
      k_drop_channels<V, RES, T><<<grid, 256, 0, s>>>(n, d->n_comp, d->channels, share, x, res, a, out);
    else
      k_drop_channels<1, RES, T><<<grid, 256, 0, s>>>(n, d->n_comp, d->channels, share, x, res, a, out);
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
      k_drop_rows<V, RES, T><<<grid, 256, 0, s>>>(n, row, share, x, res, rows, a, out);
    else
      k_drop_rows<1, RES, T><<<grid, 256, 0, s>>>(n, row, share, x, res, rows, a, out);
  }
}

template <typename T>
void launch_dropout(const so2conv_dropout_desc *d, int64_t n, const void *x, const void *res,
                    const int64_t *rows, DropArgs a, void *out, cudaStream_t s) {
  const T *xt = static_cast<const T *>(x), *rt = static_cast<const T *>(res);
  if (res)
    launch_dropout<true, T>(d, n, xt, rt, rows, a, static_cast<T *>(out), s);
  else
    launch_dropout<false, T>(d, n, xt, rt, rows, a, static_cast<T *>(out), s);
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
  const DropArgs a{rng, (uint32_t)thr, thr > 0xffffffffull, scale};
  if (d->dtype == SO2_F32)
    launch_dropout<float>(d, n, x, residual, rows, a, out, s);
  else
    launch_dropout<__nv_bfloat16>(d, n, x, residual, rows, a, out, s);
  MODEL_CKL();
  return SO2_OK;
}
