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
// three 8-byte stores, with the 128-byte swizzle the MMA reads.  While a tile's
// MMAs run, the previous tile goes from tensor memory to C; two blocks an SM
// overlap the rest.
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

// A step: 32 rows of B by 128 columns.  Its bytes arrive through a ring of
// asynchronous copies, MIXTC_RING steps deep, of which a thread reads only what
// it copied itself (four columns of four rows): with the next step's loads in
// registers instead, 157 MB arrived at 3 TB/s.
constexpr int MIXTC_KB = 32, MIXTC_RING = 2, MIXTC_PER = MIXTC_KB / 8;
constexpr int MIXTC_PLANE = MIXTC_KB * 256;  // one part of a step as bf16, bytes
template <typename TB> constexpr int mixtc_parts() { return sizeof(TB) == 2 ? 1 : 3; }
template <typename TB> constexpr int mixtc_raw() { return MIXTC_KB * MIXTC_COLS * (int)sizeof(TB); }
template <typename TB>
inline int mixtc_smem(int blocks) {
  return 1024 + 2 * mixtc_parts<TB>() * MIXTC_PLANE + 3 * blocks * MIXTC_KB * 128 +
         MIXTC_RING * mixtc_raw<TB>() + 64;
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES)
                 : "memory");
}
// The same, or zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async_or_zero(void *dst, const void *src, bool on) {
  const int have = on ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(have)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src),
                 "n"(BYTES), "r"(have)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows r0 .. r0 + min(R - r0, N) of C; N is 32 or 64, `blocks` the steps of a tile.
template <int N, typename TB, typename TC>
__global__ void __launch_bounds__(MIXTC_THREADS, 2)
    k_mix_tc(int r0, int R, int S, int blocks, int64_t n, const float *__restrict__ M, int64_t mr,
             int64_t ms, const TB *__restrict__ Bm, TC *__restrict__ C, DevStatus *st) {
  extern __shared__ uint8_t raw[];
  constexpr int PARTS = mixtc_parts<TB>(), KB = MIXTC_KB, PLANE = MIXTC_PLANE, PER = MIXTC_PER;
  constexpr int QUAD = 4 * (int)sizeof(TB);
  uint8_t *a_smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *m_smem = a_smem + 2 * PARTS * PLANE;   // [3][blocks][KB rows of 64 r]
  const int m_plane = blocks * KB * 128;
  uint8_t *ring = m_smem + 3 * m_plane;           // [MIXTC_RING][PER][threads] four columns
  uint64_t *bar = reinterpret_cast<uint64_t *>(ring + MIXTC_RING * mixtc_raw<TB>());  // [2]
  uint32_t *slot = reinterpret_cast<uint32_t *>(bar + 2);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rows = R - r0 < N ? R - r0 : N;

  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 1, 1);
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
  int64_t next_tile = blockIdx.x;  // of the next copy
  int next_kb = 0;
  uint8_t *const own = ring + tid * QUAD;
  auto copy = [&](int64_t step) {
    if (next_tile < tiles) {
      const int64_t c = next_tile * MIXTC_COLS + lane * 4;
      const int s0 = next_kb * KB + w;
      const TB *from = Bm + s0 * n + c;
      uint8_t *to = own + (int)(step % MIXTC_RING) * mixtc_raw<TB>();
      if (c < n && s0 + 8 * (PER - 1) < S) {
#pragma unroll
        for (int i = 0; i < PER; ++i, from += 8 * n) copy_async<QUAD>(to + i * MIXTC_THREADS * QUAD, from);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i, from += 8 * n) {
          const bool on = s0 + 8 * i < S && c < n;
          copy_async_or_zero<QUAD>(to + i * MIXTC_THREADS * QUAD, on ? from : Bm, on);
        }
      }
    }
    copy_commit();
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
    TC *to = C + (int64_t)(r0 + ra) * n + c;
    const int left = c < n ? rows - ra : 0;
#pragma unroll
    for (int q = 0; q < N / 2; q += 16) {
      uint32_t v[16];
      tmem_ld16(tmem + ((uint32_t)(w & 3) << 21) + (uint32_t)(t & 1) * N + ra + q, v);
      if (left >= q + 16) {
#pragma unroll
        for (int r = 0; r < 16; ++r, to += n) *to = from_f32<TC>(__uint_as_float(v[r]));
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r, to += n)
          if (q + r < left) *to = from_f32<TC>(__uint_as_float(v[r]));
      }
    }
  };

  auto done = [&](int64_t step) { return mbar_wait(bar + (step & 1), (uint32_t)(step >> 1) & 1, st); };
  bool ok = true, bad_tile = false, bad_last = false;
#pragma unroll
  for (int i = 0; i < MIXTC_RING - 1; ++i) copy(i);
  int kb = 0;
  int64_t t = 0;  // of the block's tiles
  for (int64_t step = 0; step < steps; ++step) {
    // the MMAs of the step before the last have read their operand's buffer
    if (step > 1) ok = ok && done(step - 2);
    if (kb == 0) bad_last = bad_tile, bad_tile = bad_m;
    copy(step + MIXTC_RING - 1);  // into the slot that the last step has read
    copy_wait<MIXTC_RING - 1>();
    const uint8_t *mine_raw = own + (int)(step % MIXTC_RING) * mixtc_raw<TB>();
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      uint8_t *to = a_smem + (int)(step & 1) * (PARTS * PLANE) + put + i * 1024;
      if constexpr (PARTS == 1) {
        const uint2 v = *reinterpret_cast<const uint2 *>(mine_raw + i * MIXTC_THREADS * QUAD);
        odd = fmaf(__uint_as_float(v.x << 16), 0.f, fmaf(__uint_as_float(v.x & 0xffff0000u), 0.f, odd));
        odd = fmaf(__uint_as_float(v.y << 16), 0.f, fmaf(__uint_as_float(v.y & 0xffff0000u), 0.f, odd));
        *reinterpret_cast<uint2 *>(to) = v;
      } else {
        const float4 v = *reinterpret_cast<const float4 *>(mine_raw + i * MIXTC_THREADS * QUAD);
        uint2 h, m, l;
        split3(v.x, v.y, h.x, m.x, l.x, odd);
        split3(v.z, v.w, h.y, m.y, l.y, odd);
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
      const uint32_t a0 = smem_u32(a_smem) + (uint32_t)(step & 1) * (PARTS * PLANE), b0 = smem_u32(m_smem) + kb * KB * 128;
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
      umma_commit(bar + (step & 1));
    }
    __syncwarp();
    if (kb == 0 && t > 0) {  // (a wait that gave up shows at the next step's barrier)
      ok = __all_sync(0xffffffffu, done(step - 1));
      tc_fence_after();
      if (ok) finish(t - 1, bad_last);
    }
    if (++kb == blocks) kb = 0, ++t;
  }
  copy_wait<0>();
  if (steps > 0 && ok) ok = done(steps - 1);
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
