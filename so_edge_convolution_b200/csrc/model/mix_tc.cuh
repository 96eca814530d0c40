// mix_tc.cuh -- rows of a skinny product on the tensor cores, at f32 accuracy.
//
// C[r, :] = sum_s M[r, s] B[s, :] as in k_mix_rows, for row counts whose FMAs
// take longer than the bytes: 64 systems over 32 experts need 70 us of packed
// FMAs at peak (144 measured) for 1,228,800 columns, and 72 us of memory.
//
// Every f32 is the sum of three bf16 (8 + 8 + 8 bits), and six of the nine
// products of such sums keep 2^-24: hi lo, lo hi, mid mid, mid hi, hi mid,
// hi hi, added smallest first in f32 accumulators.  A bf16 operand is its own
// first part and needs three.  128 columns of B are the MMA's M, up to 64 rows
// of C its N, s its K, so both operands are MN-major and B's rows go to shared
// memory as they lie in memory: a thread splits four columns of a row into
// three 8-byte stores, with the 128-byte swizzle the MMA reads.  The next
// step's loads are in flight during the MMAs and during the previous tile's
// way from tensor memory to C; two blocks an SM overlap the rest.
//
// Infinities, NaN and values that round to infinity in bf16 do not survive
// the split (infinity times a zero part is NaN), so a tile or a matrix M that
// holds one is computed with FMAs.
#pragma once

#include "model_common.cuh"

namespace so2 {

constexpr int MIXTC_THREADS = 256, MIXTC_COLS = 128, MIXTC_MAX_S = 256, MIXTC_ROWS = 64;

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Two f32 as three pairs of bf16 whose sums have 24 bits of them.  `odd` stays
// 0 as long as every value is finite and its first part too (the remainder is
// infinite or NaN otherwise, and 0 times that is NaN).  Conversions in pairs:
// one instruction, where a single one goes through a slower unit.
__device__ __forceinline__ void split3(float a, float b, uint32_t &h, uint32_t &m, uint32_t &l, float &odd) {
  h = pack_bf16x2(a, b);
  const float ra = a - __uint_as_float(h << 16), rb = b - __uint_as_float(h & 0xffff0000u);
  odd = fmaf(ra, 0.f, fmaf(rb, 0.f, odd));
  m = pack_bf16x2(ra, rb);
  l = pack_bf16x2(ra - __uint_as_float(m << 16), rb - __uint_as_float(m & 0xffff0000u));
}

// Four columns of a row as they lie in memory.
template <typename TB> struct Quad;
template <> struct Quad<float> { float4 v; };
template <> struct Quad<__nv_bfloat16> { uint2 v; };

// Rows of s a K block holds: 32 for small sums, else 64.
__host__ __device__ constexpr int mixtc_plane(int KB) { return KB * 256; }  // 128 columns x KB rows, bytes
template <typename TB> constexpr int mixtc_parts() { return sizeof(TB) == 2 ? 1 : 3; }
template <typename TB>
inline int mixtc_smem(int KB, int blocks) {
  return 1024 + mixtc_parts<TB>() * mixtc_plane(KB) + 3 * blocks * KB * 128 + 64;
}

// Rows r0 .. r0 + min(R - r0, N) of C; N is 32 or 64, `blocks` the K blocks of S.
template <int N, int KB, typename TB, typename TC>
__global__ void __launch_bounds__(MIXTC_THREADS, 2)
    k_mix_tc(int r0, int R, int S, int blocks, int64_t n, const float *__restrict__ M, int64_t mr,
             int64_t ms, const TB *__restrict__ Bm, TC *__restrict__ C, DevStatus *st) {
  extern __shared__ uint8_t raw[];
  constexpr int PARTS = mixtc_parts<TB>(), PLANE = mixtc_plane(KB), PER = KB / 8;
  uint8_t *a_smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *m_smem = a_smem + PARTS * PLANE;       // [3][blocks][KB rows of 64 r]
  const int m_plane = blocks * KB * 128;
  uint64_t *bar = reinterpret_cast<uint64_t *>(m_smem + 3 * m_plane);
  uint32_t *slot = reinterpret_cast<uint32_t *>(bar + 1);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rows = R - r0 < N ? R - r0 : N;

  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  if (w == 0) {
    tmem_alloc(slot, 2 * N);
    tmem_relinquish();
  }
  // M's three parts, MN-major: row s holds 64 r, its 16-byte pieces swizzled by s
  float bad = 0.f;
  for (int i = tid; i < blocks * KB * 32; i += MIXTC_THREADS) {
    const int s = i >> 5, r = (i & 31) * 2;
    const float v0 = s < S && r < rows ? M[(r0 + r) * mr + s * ms] : 0.f;
    const float v1 = s < S && r + 1 < rows ? M[(r0 + r + 1) * mr + s * ms] : 0.f;
    uint32_t p[3];
    split3(v0, v1, p[0], p[1], p[2], bad);
    const int at = s * 128 + ((((r >> 3) ^ s) & 7) << 4) + (r & 7) * 2;
#pragma unroll
    for (int k = 0; k < 3; ++k) *reinterpret_cast<uint32_t *>(m_smem + k * m_plane + at) = p[k];
  }
  const bool bad_m = __syncthreads_or(bad != bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;

  const int64_t tiles = (n + MIXTC_COLS - 1) / MIXTC_COLS;
  const int64_t mine = blockIdx.x < tiles ? (tiles - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  const int64_t steps = mine * blocks;
  // A warp's rows of a block: s = w + 8 i, four columns a lane
  Quad<TB> x[PER];
  int64_t next_tile = blockIdx.x;  // of the next load
  int next_kb = 0;
  auto load = [&]() {
    const int64_t c = next_tile * MIXTC_COLS + lane * 4;
    const int s0 = next_kb * KB + w;
    const TB *from = Bm + s0 * n + c;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      x[i] = Quad<TB>{};
      if (s0 + 8 * i < S && c < n)
        x[i].v = *reinterpret_cast<const decltype(x[i].v) *>(from + 8 * i * n);
    }
    if (++next_kb == blocks) next_kb = 0, next_tile += gridDim.x;
  };
  const int put = (lane >> 4) * (KB * 128) + w * 128 + ((((lane & 15) >> 1) ^ w) << 4) + (lane & 1) * 8;
  // The tile `t` from tensor memory to C (warps w and w + 4 share its 32
  // columns w & 3 and take half of the rows each), or with FMAs.
  auto finish = [&](int64_t t, bool with_fma) {
    const int64_t c = (blockIdx.x + t * gridDim.x) * MIXTC_COLS + (w & 3) * 32 + lane;
    const int ra = (w >> 2) * (N / 2);
    if (with_fma) {
      if (c >= n) return;
      for (int r = ra; r < ra + N / 2 && r < rows; ++r) {
        float acc = 0.f;
        for (int s = 0; s < S; ++s) acc = fmaf(M[(r0 + r) * mr + s * ms], to_f32(Bm[s * n + c]), acc);
        C[(int64_t)(r0 + r) * n + c] = from_f32<TC>(acc);
      }
      return;
    }
    uint32_t v[N / 2];
    const uint32_t from = tmem + ((uint32_t)(w & 3) << 21) + (uint32_t)(t & 1) * N + ra;
    if constexpr (N == 64) tmem_ld32(from, v);
    else tmem_ld16(from, v);
    if (c >= n) return;
    TC *to = C + (int64_t)(r0 + ra) * n + c;
#pragma unroll
    for (int r = 0; r < N / 2; ++r)
      if (ra + r < rows) to[r * n] = from_f32<TC>(__uint_as_float(v[r]));
  };

  bool ok = true, bad_tile = false, bad_last = false;
  if (steps > 0) load();
  int kb = 0;
  int64_t t = 0;  // of the block's tiles
  for (int64_t step = 0; step < steps; ++step) {
    // the previous step's MMAs have read the operand and written their tile
    if (step > 0) ok = mbar_wait(bar, (uint32_t)(step - 1) & 1, st);
    if (kb == 0) bad_last = bad_tile, bad_tile = bad_m;
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      uint8_t *to = a_smem + put + i * 1024;
      if constexpr (PARTS == 1) {
        const uint2 v = x[i].v;
        odd = fmaf(__uint_as_float(v.x << 16), 0.f, fmaf(__uint_as_float(v.x & 0xffff0000u), 0.f, odd));
        odd = fmaf(__uint_as_float(v.y << 16), 0.f, fmaf(__uint_as_float(v.y & 0xffff0000u), 0.f, odd));
        *reinterpret_cast<uint2 *>(to) = v;
      } else {
        uint2 h, m, l;
        split3(x[i].v.x, x[i].v.y, h.x, m.x, l.x, odd);
        split3(x[i].v.z, x[i].v.w, h.y, m.y, l.y, odd);
        *reinterpret_cast<uint2 *>(to) = h;
        *reinterpret_cast<uint2 *>(to + PLANE) = m;
        *reinterpret_cast<uint2 *>(to + 2 * PLANE) = l;
      }
    }
    fence_async_shared();  // the operand's stores, before the MMAs read them
    tc_fence_before();     // the tensor memory reads of the tile before the last
    if (__syncthreads_or(odd != odd || !ok)) {
      if (__syncthreads_or(!ok)) {
        ok = false;
        break;
      }
      bad_tile = true;
    }
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idesc = idesc_bf16_f32(128, N, true);
      const uint32_t d = tmem + (uint32_t)(t & 1) * N;
      const uint32_t a0 = smem_u32(a_smem), b0 = smem_u32(m_smem) + kb * KB * 128;
      constexpr int ORDER[6][2] = {{0, 2}, {2, 0}, {1, 1}, {1, 0}, {0, 1}, {0, 0}};  // parts of B, of M
      uint32_t more = kb > 0;
#pragma unroll
      for (int q = 0; q < 6; ++q) {
        if (ORDER[q][0] >= PARTS) continue;
        const uint64_t da = sdesc_mn_sw128(a0 + ORDER[q][0] * PLANE, KB * 128);
        const uint64_t db = sdesc_mn_sw128(b0 + ORDER[q][1] * m_plane, KB * 128);
#pragma unroll
        for (int kk = 0; kk < KB / 16; ++kk) {
          umma_bf16(d, da + kk * 128, db + kk * 128, idesc, more);
          more = 1;
        }
      }
      umma_commit(bar);
    }
    __syncwarp();
    if (step + 1 < steps) load();
    if (kb == 0 && t > 0) {
      tc_fence_after();
      finish(t - 1, bad_last);
    }
    if (++kb == blocks) kb = 0, ++t;
  }
  if (steps > 0 && ok) ok = mbar_wait(bar, (uint32_t)(steps - 1) & 1, st);
  if (__syncthreads_or(!ok)) {
    // a wait gave up (recorded in the status word): give the MMAs in flight a
    // while longer before their tensor memory is freed
    const uint64_t since = globaltimer_ns();
    while (globaltimer_ns() - since < 200000000ull) {
    }
  } else if (steps > 0) {
    tc_fence_after();
    finish(mine - 1, bad_tile);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 0) tmem_dealloc(tmem, 2 * N);
}

}  // namespace so2
