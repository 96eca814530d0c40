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
// it copied itself (four columns of four rows).  With the next step's loads in
// registers instead it took as long (104 and 105 us at 64 rows x 1,228,800
// columns); whole steps without a check of each row's bounds brought 85.
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
#pragma unroll 4  // (the loads of M are what a small product waits for)
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

// ---- both gradients from one split of grad_out -------------------------------------
// For up to 64 systems and 32 experts.  Of each tile of 128 columns the three
// parts of G (grad_out) and of the experts W are formed once and serve two
// products: the experts' gradient, D[column, e] = sum_t G[t, column] a[t, e],
// which reads G's rows MN-major, and the routing weights', D2[t, e] = sum over
// the columns of G[t, .] W[e, .], which reads the same bytes K-major (a
// 128-byte row of 64 columns is a row of either).  The parts of a and of W lie
// side by side as up to 96 columns of one operand, so each part of G is read
// once per product: hi [hi mid lo], mid [hi mid], lo [hi], three accumulator
// ranges that the epilogue adds.  D2 is taken out of tensor memory after each
// tile and added up in registers, a tile's 128 columns at a time.  Shared
// memory bounds it (copies in, parts out, operand reads).
// (The MMAs of D2 are 128 rows high; rows 64.. read what follows G's part in
// shared memory and are not looked at.)
// Sixteen warps copy, split and finish; a seventeenth only issues the MMAs (36 a
// tile: with one of the sixteen doing that, the others waited for it at the
// tile's barrier).
constexpr int MIXBK_WORKERS = 512, MIXBK_THREADS = MIXBK_WORKERS + 32, MIXBK_T = 64, MIXBK_E = 32;
constexpr int MIXBK_G = 3 * MIXBK_T * 256;  // G's parts, bytes
template <typename TE> constexpr int mixbk_w() { return mixtc_parts<TE>() * MIXBK_E * 256; }
template <typename TE> constexpr int mixbk_raw() { return (MIXBK_T * 4 + MIXBK_E * (int)sizeof(TE)) * MIXTC_COLS; }
template <typename TE> constexpr int mixbk_smem() {
  return 1024 + 2 * (MIXBK_G + mixbk_w<TE>()) + 2 * MIXBK_T * 128 + mixbk_raw<TE>() +
         MIXBK_T * MIXBK_E * 4 + 64;
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Eight columns of an accumulator of RANGES ranges of 32, added up.
template <int RANGES>
__device__ __forceinline__ void tmem_sum8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  tmem_ld8(taddr, r);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[j]);
#pragma unroll
  for (int q = 1; q < RANGES; ++q) {
    tmem_ld8(taddr + 32 * q, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(r[j]);
  }
}

// ge [K][n] and part[block][t][e]; NULL leaves one out (the other is the same).
template <typename TE>
__global__ void __launch_bounds__(MIXBK_THREADS, 1)
    k_mix_tc_back(int T, int K, int64_t n, const float *__restrict__ weights,
                  const TE *__restrict__ experts, const float *__restrict__ grad,
                  float *__restrict__ ge, float *__restrict__ part, DevStatus *st) {
  extern __shared__ uint8_t raw[];
  constexpr int WPARTS = mixtc_parts<TE>(), BUF = MIXBK_G + mixbk_w<TE>();
  constexpr int GPART = MIXBK_T * 256, WCHUNK = WPARTS * MIXBK_E * 128, QW = 4 * (int)sizeof(TE);
  uint8_t *planes = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t *m_smem = planes + 2 * BUF;              // [2 chunks][64 t][hi mid | lo]
  uint8_t *ring = m_smem + 2 * MIXBK_T * 128;      // a thread's own: four quads of G, two of W
  float *extra = reinterpret_cast<float *>(ring + mixbk_raw<TE>());  // [64][32] of tiles done with FMAs
  uint64_t *bar = reinterpret_cast<uint64_t *>(extra + MIXBK_T * MIXBK_E);  // [2]
  uint32_t *slot = reinterpret_cast<uint32_t *>(bar + 2);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;

  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 1, 1);
    fence_mbar_init();
  }
  if (w == 0) {
    tmem_alloc(slot, 512);
    tmem_relinquish();
  }
  for (int i = tid; i < MIXBK_T * MIXBK_E; i += MIXBK_THREADS) extra[i] = 0.f;
  float bad = 0.f;
  for (int i = tid; i < MIXBK_T * MIXBK_E / 2; i += MIXBK_THREADS) {
    const int t = i / (MIXBK_E / 2), e = i % (MIXBK_E / 2) * 2;
    const float v0 = t < T && e < K ? weights[t * K + e] : 0.f;
    const float v1 = t < T && e + 1 < K ? weights[t * K + e + 1] : 0.f;
    uint32_t p[3];
    split3(v0, v1, p[0], p[1], p[2], bad);
    auto put = [&](int chunk, int r, uint32_t v) {  // columns r, r + 1 of a chunk's row t
      *reinterpret_cast<uint32_t *>(m_smem + chunk * (MIXBK_T * 128) + t * 128 +
                                    ((((r >> 3) ^ t) & 7) << 4) + (r & 7) * 2) = v;
    };
    put(0, e, p[0]);
    put(0, 32 + e, p[1]);
    put(1, e, p[2]);
    put(1, 32 + e, 0);
  }
  const bool bad_m = __syncthreads_or(bad != bad);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;

  const int64_t tiles = (n + MIXTC_COLS - 1) / MIXTC_COLS;
  const int64_t mine = blockIdx.x < tiles ? (tiles - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  uint8_t *const own_g = ring + tid * 16, *const own_w = ring + 4 * MIXBK_WORKERS * 16 + tid * QW;
  auto copy = [&](int64_t i) {  // the block's i-th tile: rows w, w + 16, ..., four columns a lane
    if (i < mine) {
      const int64_t c = (blockIdx.x + i * gridDim.x) * MIXTC_COLS + lane * 4;
      const float *g = grad + w * n + c;
      const TE *x = experts + w * n + c;
#pragma unroll
      for (int k = 0; k < 4; ++k, g += 16 * n) {
        const bool on = w + 16 * k < T && c < n;
        copy_async_or_zero<16>(own_g + k * MIXBK_WORKERS * 16, on ? g : grad, on);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k, x += 16 * n) {
        const bool on = w + 16 * k < K && c < n;
        copy_async_or_zero<QW>(own_w + k * MIXBK_WORKERS * QW, on ? x : experts, on);
      }
    }
    copy_commit();
  };
  const int swz = ((((lane & 15) >> 1) ^ (w & 7)) << 4) + (lane & 1) * 8;
  const int put_g = (lane >> 4) * (MIXBK_T * 128) + w * 128 + swz;
  const int put_w = MIXBK_G + (lane >> 4) * WCHUNK + w * 128 + swz;
  const bool worker = w < 16;
  const int q = w & 3, e0 = (w >> 2) * 8;  // of the epilogues: tensor memory lanes 32 q.., eight experts
  float dot[8] = {};
  auto done = [&](int64_t i) { return mbar_wait(bar + (i & 1), (uint32_t)(i >> 1) & 1, st); };
  auto finish = [&](int64_t i, bool odd) {
    const int64_t c0 = (blockIdx.x + i * gridDim.x) * MIXTC_COLS, c = c0 + q * 32 + lane;
    const uint32_t from = tmem + ((uint32_t)q << 21) + (uint32_t)(i & 1) * 96 + e0;
    float v[8];
    if (!ge) {
    } else if (odd || bad_m) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
      if (c < n)
        for (int t = 0; t < T; ++t) {
          const float g = grad[t * n + c];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e0 + j < K) v[j] = fmaf(weights[t * K + e0 + j], g, v[j]);
        }
    } else {
      tmem_sum8<3>(from, v);
    }
    if (ge && c < n) {
      float *to = ge + e0 * n + c;
#pragma unroll
      for (int j = 0; j < 8; ++j, to += n)
        if (e0 + j < K) *to = v[j];
    }
    if (!part) return;
    if (odd) {  // four (t, e) a thread, its own
      const int64_t c1 = c0 + MIXTC_COLS < n ? c0 + MIXTC_COLS : n;
      for (int k = tid * 4; k < tid * 4 + 4; ++k) {
        const int t = k / MIXBK_E, e = k % MIXBK_E;
        if (t >= T || e >= K) continue;
        float s = 0.f;
        for (int64_t x = c0; x < c1; ++x) s = fmaf(grad[t * n + x], to_f32(experts[e * n + x]), s);
        extra[k] += s;
      }
    } else if (q < 2) {
      tmem_sum8<WPARTS>(from + 192, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot[j] += v[j];
    }
  };

  bool ok = true, odd_now = false, odd_last = false;
  if (worker) copy(0);
  for (int64_t i = 0; i < mine; ++i) {
    uint8_t *buf = planes + (int)(i & 1) * BUF;
    float odd = 0.f;
    if (worker) {
      copy_wait<0>();
      if (i > 1) ok = ok && done(i - 2);  // the MMAs that read this buffer
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = *reinterpret_cast<const float4 *>(own_g + k * MIXBK_WORKERS * 16);
        uint2 h, m, l;
        split3(v.x, v.y, h.x, m.x, l.x, odd);
        split3(v.z, v.w, h.y, m.y, l.y, odd);
        uint8_t *to = buf + put_g + k * 16 * 128;
        *reinterpret_cast<uint2 *>(to) = h;
        *reinterpret_cast<uint2 *>(to + GPART) = m;
        *reinterpret_cast<uint2 *>(to + 2 * GPART) = l;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint8_t *to = buf + put_w + k * 16 * 128;
        if constexpr (WPARTS == 1) {
          const uint2 v = *reinterpret_cast<const uint2 *>(own_w + k * MIXBK_WORKERS * QW);
          odd = fmaf(__uint_as_float(v.x << 16), 0.f, fmaf(__uint_as_float(v.x & 0xffff0000u), 0.f, odd));
          odd = fmaf(__uint_as_float(v.y << 16), 0.f, fmaf(__uint_as_float(v.y & 0xffff0000u), 0.f, odd));
          *reinterpret_cast<uint2 *>(to) = v;
        } else {
          const float4 v = *reinterpret_cast<const float4 *>(own_w + k * MIXBK_WORKERS * QW);
          uint2 h, m, l;
          split3(v.x, v.y, h.x, m.x, l.x, odd);
          split3(v.z, v.w, h.y, m.y, l.y, odd);
          *reinterpret_cast<uint2 *>(to) = h;
          *reinterpret_cast<uint2 *>(to + MIXBK_E * 128) = m;
          *reinterpret_cast<uint2 *>(to + 2 * MIXBK_E * 128) = l;
        }
      }
      copy(i + 1);  // (what this thread read is in registers by now)
      fence_async_shared();
      tc_fence_before();
    }
    odd_last = odd_now;
    odd_now = false;
    if (__syncthreads_or(odd != odd || !ok)) {
      if (__syncthreads_or(!ok)) {
        ok = false;
        break;
      }
      odd_now = true;
    }
    if (tid == MIXBK_WORKERS) {
      tc_fence_after();
      const uint32_t g0 = smem_u32(buf), w0 = g0 + MIXBK_G, m0 = smem_u32(m_smem);
      const uint32_t d = tmem + (uint32_t)(i & 1) * 96, d2 = d + 192;
      // Parts of the other operand that a part of G meets, as columns.  The
      // first high product clears all ranges; the small products follow it and
      // the other high ones come last, so that few roundings are of full size.
      constexpr int NG[3] = {96, 64, 32};
      constexpr int NW[3] = {32 * WPARTS, WPARTS == 1 ? 32 : 64, 32};
      if (ge) {
        const uint64_t b = sdesc_mn_sw128(m0, MIXBK_T * 128);
        auto mma = [&](int pg, int kk, bool more) {
          const uint64_t a = sdesc_mn_sw128(g0 + pg * GPART, MIXBK_T * 128);
          umma_bf16(d, a + kk * 128, b + kk * 128, idesc_bf16_f32(128, NG[pg], true), more);
        };
        mma(0, 0, false);
#pragma unroll
        for (int pg = 2; pg > 0; --pg)
#pragma unroll
          for (int kk = 0; kk < MIXBK_T / 16; ++kk) mma(pg, kk, true);
#pragma unroll
        for (int kk = 1; kk < MIXBK_T / 16; ++kk) mma(0, kk, true);
      }
      if (part) {
        auto mma = [&](int pg, int k8, bool more) {  // 16 of the tile's columns
          const uint64_t a = sdesc_k_sw128(g0 + pg * GPART + (k8 >> 2) * (MIXBK_T * 128));
          const uint64_t b = sdesc_k_sw128(w0 + (k8 >> 2) * WCHUNK);
          umma_bf16(d2, a + (k8 & 3) * 2, b + (k8 & 3) * 2, idesc_bf16_f32(128, NW[pg]), more);
        };
        mma(0, 0, false);
#pragma unroll
        for (int pg = 2; pg > 0; --pg)
#pragma unroll
          for (int k8 = 0; k8 < 8; ++k8) mma(pg, k8, true);
#pragma unroll
        for (int k8 = 1; k8 < 8; ++k8) mma(0, k8, true);
      }
      umma_commit(bar + (i & 1));
    }
    __syncwarp();
    if (worker && i > 0) {  // (a wait that gave up shows at the next tile's barrier)
      ok = __all_sync(0xffffffffu, done(i - 1));
      tc_fence_after();
      if (ok) finish(i - 1, odd_last);
    }
  }
  copy_wait<0>();
  if (mine > 0 && ok) ok = done(mine - 1);  // (every warp: the tensor memory is freed below)
  if (__syncthreads_or(!ok)) {
    // a wait gave up (recorded in the status word): give the MMAs in flight a
    // while longer before their tensor memory is freed
    const uint64_t since = globaltimer_ns();
    while (globaltimer_ns() - since < 200000000ull) {
    }
  } else if (mine > 0 && worker) {
    tc_fence_after();
    finish(mine - 1, odd_now);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 0) tmem_dealloc(tmem, 512);
  const int t = q * 32 + lane;
  if (part && worker && q < 2 && t < T)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e0 + j < K)
        part[((int64_t)blockIdx.x * T + t) * K + e0 + j] = dot[j] + extra[t * MIXBK_E + e0 + j];
}

}  // namespace so2
