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

// thr = p 2^32 (2^32 drops everything); scale = 1 / (1 - p).
template <typename T>
__global__ void k_dropout(int64_t total, int n_comp, int channels, int unit,
                          const T *x, const T *res, const int64_t *__restrict__ rows,
                          const uint64_t *__restrict__ rng, uint64_t thr, float scale, T *out) {
  const uint64_t seed = rng[0], offset = rng[1];
  const int64_t row = (int64_t)n_comp * channels;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    uint64_t m = i;
    if (unit == SO2_DROP_CHANNEL)
      m = (i / row) * channels + i % channels;
    else if (unit == SO2_DROP_ROW)
      m = rows ? (uint64_t)rows[i / row] : (uint64_t)(i / row);
    const uint32_t u = word_of(philox(m >> 2, offset, seed), (int)(m & 3));
    float v = u >= thr ? to_f32(x[i]) * scale : 0.f;
    if (res) v += to_f32(res[i]);
    out[i] = from_f32<T>(v);
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
  if (n == 0) return SO2_OK;
  const size_t es = dtype_size(d->dtype);
  if (!x || !out || !aligned_to(x, es) || !aligned_to(out, es) || !aligned_to(residual, es))
    return SO2_ERR_INVALID_ARG;
  const double p = d->p;
  const uint64_t thr = (uint64_t)llrint(p * 4294967296.0);
  const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
  const int64_t total = n * d->n_comp * d->channels;
  const int grid = (int)(ceil_div(total, 256) < MODEL_SMS * 16 ? ceil_div(total, 256) : MODEL_SMS * 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->dtype == SO2_F32)
    k_dropout<float><<<grid, 256, 0, s>>>(total, d->n_comp, d->channels, d->unit,
                                          static_cast<const float *>(x),
                                          static_cast<const float *>(residual), rows, rng, thr,
                                          scale, static_cast<float *>(out));
  else
    k_dropout<__nv_bfloat16><<<grid, 256, 0, s>>>(
        total, d->n_comp, d->channels, d->unit, static_cast<const __nv_bfloat16 *>(x),
        static_cast<const __nv_bfloat16 *>(residual), rows, rng, thr, scale,
        static_cast<__nv_bfloat16 *>(out));
  MODEL_CKL();
  return SO2_OK;
}
