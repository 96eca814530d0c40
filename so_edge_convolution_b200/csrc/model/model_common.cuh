// model_common.cuh -- shared pieces of the model operators (so2model.h).
#pragma once

#include "../common.cuh"
#include "../../../include/so2model.h"

namespace so2 {

// Kernels launched by the model operators; so2conv_launch_count adds it.
extern long long g_model_launches;

#define MODEL_CK(call)                              \
  do {                                              \
    if ((call) != cudaSuccess) return SO2_ERR_CUDA; \
  } while (0)

#define MODEL_CKL()                                                \
  do {                                                             \
    ++g_model_launches;                                            \
    if (cudaPeekAtLastError() != cudaSuccess) return SO2_ERR_CUDA; \
  } while (0)

constexpr int MODEL_SMS = 148;  // B200

// Shared memory for a launch of `bytes`.  The limit belongs to the kernel and not
// to the launch, so it is always set to the most that any call takes: calls of
// several host threads then never lower it under one another.
template <typename K>
bool allow_smem(K kernel, int bytes, int most) {
  return bytes <= 48 * 1024 ||
         cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess;
}

inline bool dtype_ok(int32_t d) { return d == SO2_F32 || d == SO2_BF16; }
inline size_t dtype_size(int32_t d) { return d == SO2_BF16 ? 2 : 4; }
inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline size_t ws_take(size_t &cur, size_t bytes) {
  cur = (cur + 255) & ~static_cast<size_t>(255);
  const size_t at = cur;
  cur += bytes;
  return at;
}

template <typename T>
T *ws_at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<char *>(ws) + off);
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// V consecutive values as f32; V = 4 and 8 need the alignment of V values.
template <int V, typename T>
__device__ __forceinline__ void load_vec(const T *__restrict__ p, float (&r)[V]) {
  if constexpr (V == 1) {
    r[0] = to_f32(*p);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(p + i);
      r[i] = v.x, r[i + 1] = v.y, r[i + 2] = v.z, r[i + 3] = v.w;
    }
  } else if constexpr (V == 4) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    r[0] = __uint_as_float(v.x << 16), r[1] = __uint_as_float(v.x & 0xffff0000u);
    r[2] = __uint_as_float(v.y << 16), r[3] = __uint_as_float(v.y & 0xffff0000u);
  } else {
    static_assert(V == 8, "");
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[2 * i] = __uint_as_float(w[i] << 16), r[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <int V, typename T>
__device__ __forceinline__ void store_vec(T *p, const float (&r)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(r[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(p + i) = make_float4(r[i], r[i + 1], r[i + 2], r[i + 3]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]));
  } else {
    static_assert(V == 8, "");
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]),
                                               pack_bf16x2(r[4], r[5]), pack_bf16x2(r[6], r[7]));
  }
}

}  // namespace so2
