// mix.cu -- mixing of experts' weights, and its gradients.
//
// The slots (t, j) that name an expert form its list, in slot order; a small
// kernel builds the lists once per backward call.  With every expert in order
// (no index) slot (t, e) names expert e, and no lists are needed.
#include "mix_tc.cuh"

namespace so2 {

// ---- every expert in order: rows of a skinny product -------------------------------
// C[r, :] = sum_s M[r, s] B[s, :], with M[r * mr + s * ms] in f32: the forward
// (r = t, s = e, B = experts) and the experts' gradient (r = e, s = t, B =
// grad_out).  A thread owns V columns and TT rows of C in registers and reads
// each row of B once for them, through a ring of asynchronous copies that
// only it reads (no block barrier in the loop).  Two rows of C share one
// packed FMA; the weights lie in shared memory, pairs of rows side by side.
constexpr int ROWS_THREADS = 128;
constexpr int ROWS_SC = 32;     // rows of B whose weights are staged together
constexpr int ROWS_DEPTH = 8;   // copies in flight
// From this many FMAs a column and step of 32 rows of B on, the tensor cores
// take the product (mix_tc.cuh): a step of theirs costs much the same whatever
// it holds.  Forward, FMA / tensor us: 1,228,800 f32 columns, R x S = 24 x 24
// 50 / 66, 32 x 16 53 / 64, 32 x 32 82 / 64, 64 x 16 97 / 79, 64 x 64 283 / 125;
// 300,000 columns, 8 x 100 23 / 84, 32 x 32 21 / 22, 64 x 32 40 / 29, 30 x 120
// 60 / 84, 64 x 128 130 / 88.  With few columns the tensor cores would win
// earlier, which the rule leaves (30 x 120: 4,864 columns 22 / 12, 20,000 22 / 17,
// 80,000 30 / 31).
constexpr int MIX_TC_FROM = 960;
// And from this many products of all (t, e) on, those go in tiles (mix_plan).
constexpr int MIX_TILES_FROM = 256;

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void fma2(uint64_t &d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
template <int TT, int V, typename TB, typename TC>
__global__ void __launch_bounds__(ROWS_THREADS)
    k_mix_rows(int R, int S, int64_t n, const float *__restrict__ M, int64_t mr, int64_t ms,
               const TB *__restrict__ Bm, TC *__restrict__ C, DevStatus *st) {
  constexpr int PAIRS = (TT + 1) / 2;
  constexpr bool RING = V > 1;
  constexpr int BYTES = V * (int)sizeof(TB);
  __shared__ __align__(16) float wts[ROWS_SC][2 * PAIRS];
  __shared__ __align__(16) unsigned char ring[RING ? ROWS_DEPTH : 1][ROWS_THREADS][RING ? BYTES : 4];
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && tid == 0) *st = DevStatus{0, 0};  // nothing here can go wrong
  const int64_t c = (blockIdx.x * (int64_t)ROWS_THREADS + tid) * V;
  const bool on = c < n;
  const TB *col = Bm + c;
  for (int r0 = 0; r0 < R; r0 += TT) {
    uint64_t acc[PAIRS][V];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[p][v] = 0;
    if constexpr (RING) {
#pragma unroll
      for (int d = 0; d < ROWS_DEPTH - 1; ++d) {
        if (on && d < S) copy_async<BYTES>(ring[d][tid], col + d * n);
        copy_commit();
      }
    }
    for (int s0 = 0; s0 < S; s0 += ROWS_SC) {
      __syncthreads();
      for (int i = tid; i < ROWS_SC * 2 * PAIRS; i += ROWS_THREADS) {
        const int s = s0 + i / (2 * PAIRS), r = r0 + i % (2 * PAIRS);
        wts[i / (2 * PAIRS)][i % (2 * PAIRS)] =
            (s < S && r < R && i % (2 * PAIRS) < TT) ? M[r * mr + s * ms] : 0.f;
      }
      __syncthreads();
      const int end = S - s0 < ROWS_SC ? S - s0 : ROWS_SC;
#pragma unroll 4
      for (int i = 0; i < end; ++i) {
        const int s = s0 + i;
        float x[V];
        if constexpr (RING) {
          const int nx = s + ROWS_DEPTH - 1;
          if (on && nx < S) copy_async<BYTES>(ring[nx % ROWS_DEPTH][tid], col + nx * n);
          copy_commit();
          copy_wait<ROWS_DEPTH - 1>();
          load_vec<V>(reinterpret_cast<const TB *>(ring[s % ROWS_DEPTH][tid]), x);
        } else {
          x[0] = on ? to_f32(col[s * n]) : 0.f;
        }
        uint64_t xx[V];
#pragma unroll
        for (int v = 0; v < V; ++v) xx[v] = pack2(x[v], x[v]);
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
          const uint64_t w = *reinterpret_cast<const uint64_t *>(&wts[i][2 * p]);
#pragma unroll
          for (int v = 0; v < V; ++v) fma2(acc[p][v], w, xx[v]);
        }
      }
    }
    if (on) {
#pragma unroll
      for (int q = 0; q < TT; ++q) {
        if (r0 + q < R) {
          float o[V];
#pragma unroll
          for (int v = 0; v < V; ++v)
            o[v] = __uint_as_float((uint32_t)(acc[q >> 1][v] >> (32 * (q & 1))));
          store_vec<V>(C + (int64_t)(r0 + q) * n + c, o);
        }
      }
    }
    if constexpr (RING) copy_wait<0>();
  }
}

// ---- forward, by index -------------------------------------------------------------
// A thread owns V columns and takes the systems of its blockIdx.y one after
// the other, four slots' rows in flight; the slots' experts and weights lie in
// shared memory, unused ones as expert -1.
constexpr int SLOT_STAGE = 4096;  // slots staged together: all of a system's at least

template <int V, typename TE, typename TO>
__global__ void __launch_bounds__(256)
    k_mix(int n_systems, int K, int top_k, int64_t n, const TE *__restrict__ experts,
          const float *__restrict__ weights, const int *__restrict__ index, TO *__restrict__ out,
          DevStatus *st) {
  __shared__ int se[SLOT_STAGE];
  __shared__ float sw[SLOT_STAGE];
  const int64_t c = (blockIdx.x * 256ll + threadIdx.x) * V;
  const int per = (n_systems + gridDim.y - 1) / gridDim.y;
  const int ta = blockIdx.y * per, tb = ta + per < n_systems ? ta + per : n_systems;
  const int together = SLOT_STAGE / top_k;
  const TE *col = experts + c;
  for (int t0 = ta; t0 < tb; t0 += together) {
    const int t1 = t0 + together < tb ? t0 + together : tb;
    __syncthreads();
    for (int i = threadIdx.x; i < (t1 - t0) * top_k; i += 256) {
      const int64_t p = (int64_t)t0 * top_k + i;
      int e = index[p];
      if (e < 0 || e >= K) {
        if (e != -1 && blockIdx.x == 0) raise_error(st, SO2_ERR_INDEX, (int)p);
        e = -1;
      }
      se[i] = e;
      sw[i] = e >= 0 ? weights[p] : 0.f;
    }
    __syncthreads();
    if (c >= n) continue;
    for (int t = t0; t < t1; ++t) {
      float acc[V];
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = 0.f;
      const int i0 = (t - t0) * top_k;
      for (int j = 0; j < top_k; j += 4) {
        float x[4][V];
        int e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          e[u] = j + u < top_k ? se[i0 + j + u] : -1;
          if (e[u] >= 0) load_vec<V>(col + e[u] * n, x[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (e[u] >= 0) {
            const float w = sw[i0 + j + u];
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(w, x[u][v], acc[v]);
          }
      }
      store_vec<V>(out + t * n + c, acc);
    }
  }
}

// ---- backward ------------------------------------------------------------------
// Lists of the slots by expert: offsets [K+1], slots in slot order.  One warp
// per expert: the slots of lower experts give its offset, its own follow.
__global__ void k_mix_lists(int n_slots, int K, const int *__restrict__ index,
                            int *__restrict__ offsets, int *__restrict__ list, DevStatus *st) {
  const int lane = threadIdx.x & 31;
  const int e = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (e >= K) return;
  if (e == 0 && lane == 0) *st = DevStatus{0, 0};  // this warp alone touches it
  __syncwarp();
  int lower = 0, mine = 0;
  for (int p0 = 0; p0 < n_slots; p0 += 32) {
    const int p = p0 + lane, v = p < n_slots ? index[p] : -1;
    lower += __popc(__ballot_sync(0xffffffffu, v >= 0 && v < e));
    mine += __popc(__ballot_sync(0xffffffffu, v == e));
    if (e == 0 && (v < -1 || v >= K)) raise_error(st, SO2_ERR_INDEX, p);
  }
  if (lane == 0) {
    offsets[e] = lower;
    if (e == K - 1) offsets[K] = lower + mine;
  }
  if (mine == 0) return;
  int at = lower;
  for (int p0 = 0; p0 < n_slots; p0 += 32) {
    const int p = p0 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, p < n_slots && index[p] == e);
    if ((m >> lane) & 1) list[at + __popc(m & ((1u << lane) - 1))] = p;
    at += __popc(m);
  }
}

// A thread owns V columns and the experts of its blockIdx.y; the expert's
// slots four at a time.  Lists of up to SLOT_STAGE slots are read from shared
// memory, longer ones from where they are.
template <int V>
__global__ void __launch_bounds__(256)
    k_mix_grad_experts(int n_slots, int K, int top_k, int64_t n, const float *__restrict__ weights,
                       const int *__restrict__ offsets, const int *__restrict__ list,
                       const float *__restrict__ grad, float *__restrict__ ge) {
  __shared__ int st[SLOT_STAGE];
  __shared__ float sw[SLOT_STAGE];
  const int per = (K + gridDim.y - 1) / gridDim.y;
  const int ea = blockIdx.y * per, eb = ea + per < K ? ea + per : K;
  const int first = ea < eb ? offsets[ea] : 0, end = ea < eb ? offsets[eb] : 0;
  const bool staged = end - first <= SLOT_STAGE;
  if (staged)
    for (int i = first + threadIdx.x; i < end; i += 256) {
      const int p = list[i];
      st[i - first] = p / top_k;
      sw[i - first] = weights[p];
    }
  __syncthreads();
  const int64_t c = (blockIdx.x * 256ll + threadIdx.x) * V;
  if (c >= n) return;
  for (int e = ea; e < eb; ++e) {
    const int a = offsets[e], b = offsets[e + 1];
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int q = a; q < b; q += 4) {
      float g[4][V], w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (q + u >= b) break;
        const int t = staged ? st[q + u - first] : list[q + u] / top_k;
        w[u] = staged ? sw[q + u - first] : weights[list[q + u]];
        load_vec<V>(grad + t * n + c, g[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (q + u >= b) break;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(w[u], g[u][v], acc[v]);
      }
    }
    store_vec<V>(ge + e * n + c, acc);
  }
}

// ---- the routing weights' gradient: products over all columns --------------------------
// Every (t, e) of a tile of 64 systems and 32 experts, over the block's share
// of the columns.  Tiles of both operands go through shared memory in four
// stages of asynchronous copies; a thread holds 8 x 4 products, two columns to
// a packed FMA (their halves are added at the end), and reads 12 vectors of
// four columns for 64 of them.  Four groups of 64 threads take every fourth
// vector.  Row pitches are 4 words off a multiple of 32, so the eight rows of
// a warp's read lie in different banks.
constexpr int DOT_T = 64, DOT_E = 32, DOT_COLS = 64, DOT_STAGES = 4;
constexpr int DOT_PITCH_G = DOT_COLS + 4;  // f32 elements
template <typename TE> constexpr int dot_pitch_e() { return DOT_COLS + 16 / (int)sizeof(TE); }
template <typename TE> constexpr int dot_stage_bytes() {
  return DOT_T * DOT_PITCH_G * 4 + DOT_E * dot_pitch_e<TE>() * (int)sizeof(TE);
}

// A thread's vectors of a stage: one column group of ROWS / 16 rows, 16 apart.
// Rows and columns outside the matrix are zero.  (VEC: vectors of four and
// asynchronous copies; otherwise single values, 64 of them side by side.)
template <int ROWS, int PITCH, bool VEC, typename T>
struct DotLoader {
  static constexpr int V = VEC ? 4 : 1, PER_ROW = DOT_COLS / V, APART = 256 / PER_ROW,
                       COUNT = ROWS / APART;
  const T *from;  // the thread's first vector of the next stage
  int64_t c, n;   // its column
  int rows;       // of its rows inside the matrix
  int put;
  __device__ __forceinline__ DotLoader(const T *src, int row0, int limit, int64_t c0, int64_t n_) : n(n_) {
    const int r = threadIdx.x / PER_ROW;
    c = c0 + threadIdx.x % PER_ROW * V;
    from = src + (int64_t)(row0 + r) * n + c;
    rows = (limit - row0 - r + APART - 1) / APART;  // may be 0 or less
    put = r * PITCH + threadIdx.x % PER_ROW * V;
  }
  __device__ __forceinline__ void load(T *dst, const T *base) {
    const T *p = from;
    if (VEC && rows >= COUNT && c < n) {
#pragma unroll
      for (int k = 0; k < COUNT; ++k, p += APART * n)
        copy_async<V * (int)sizeof(T)>(dst + put + k * APART * PITCH, p);
    } else {
#pragma unroll
      for (int k = 0; k < COUNT; ++k, p += APART * n) {
        const bool on = k < rows && c < n;
        if constexpr (VEC)
          copy_async_or_zero<V * (int)sizeof(T)>(dst + put + k * APART * PITCH, on ? p : base, on);
        else
          dst[put + k * APART * PITCH] = on ? *p : from_f32<T>(0.f);
      }
    }
    from += DOT_COLS;
    c += DOT_COLS;
  }
};

// Four columns of an operand row as two packed pairs.
__device__ __forceinline__ void dot_read(const float *p, uint64_t (&v)[2]) {
  const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(p);
  v[0] = q.x, v[1] = q.y;
}
__device__ __forceinline__ void dot_read(const __nv_bfloat16 *p, uint64_t (&v)[2]) {
  float f[4];
  load_vec<4>(p, f);
  v[0] = pack2(f[0], f[1]), v[1] = pack2(f[2], f[3]);
}

// part[split][t][e], with blockIdx.x the split, blockIdx.y the tile.
template <bool VEC, typename TE>
__global__ void __launch_bounds__(256, 2)
    k_mix_dot_tiles(int T, int K, int64_t n, const TE *__restrict__ experts,
                    const float *__restrict__ grad, float *__restrict__ part) {
  extern __shared__ __align__(16) unsigned char sm[];
  constexpr int PE = dot_pitch_e<TE>(), STAGE = dot_stage_bytes<TE>();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int tg = lane & 7, eg = (lane >> 3) + 4 * (w & 1), cg = w >> 1;
  const int etiles = (K + DOT_E - 1) / DOT_E;
  const int t0 = (blockIdx.y / etiles) * DOT_T, e0 = (blockIdx.y % etiles) * DOT_E;
  const int64_t tiles = (n + DOT_COLS - 1) / DOT_COLS;
  const int64_t first = tiles * blockIdx.x / gridDim.x, last = tiles * (blockIdx.x + 1) / gridDim.x;
  auto g_of = [&](int64_t i) { return reinterpret_cast<float *>(sm + (int)((i - first) % DOT_STAGES) * STAGE); };
  auto e_of = [&](int64_t i) {
    return reinterpret_cast<TE *>(sm + (int)((i - first) % DOT_STAGES) * STAGE + DOT_T * DOT_PITCH_G * 4);
  };
  DotLoader<DOT_T, DOT_PITCH_G, VEC, float> lg(grad, t0, T, first * DOT_COLS, n);
  DotLoader<DOT_E, PE, VEC, TE> le(experts, e0, K, first * DOT_COLS, n);
  auto load = [&](int64_t i) {
    if (i < last) {
      lg.load(g_of(i), grad);
      le.load(e_of(i), experts);
    }
    copy_commit();
  };
  uint64_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;
#pragma unroll
  for (int i = 0; i < DOT_STAGES - 1; ++i) load(first + i);
  for (int64_t i = first; i < last; ++i) {
    copy_wait<DOT_STAGES - 2>();
    __syncthreads();  // stage i is there, and everyone is done with stage i - 1
    load(i + DOT_STAGES - 1);
    const float *g = g_of(i);
    const TE *x = e_of(i);
#pragma unroll
    for (int q = cg; q < DOT_COLS / 4; q += 4) {
      uint64_t gv[8][2], xv[4][2];
#pragma unroll
      for (int a = 0; a < 8; ++a) dot_read(g + (tg + 8 * a) * DOT_PITCH_G + 4 * q, gv[a]);
#pragma unroll
      for (int b = 0; b < 4; ++b) dot_read(x + (eg + 8 * b) * PE + 4 * q, xv[b]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) fma2(acc[a][b], gv[a][h], xv[b][h]);
    }
  }
  copy_wait<0>();
  __syncthreads();
  // the four column groups' sums, in order
  float *red = reinterpret_cast<float *>(sm);  // [4][DOT_T][DOT_E]
#pragma unroll
  for (int a = 0; a < 8; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      red[(cg * DOT_T + tg + 8 * a) * DOT_E + eg + 8 * b] =
          __uint_as_float((uint32_t)acc[a][b]) + __uint_as_float((uint32_t)(acc[a][b] >> 32));
  __syncthreads();
  for (int i = tid; i < DOT_T * DOT_E; i += 256) {
    const int t = t0 + i / DOT_E, e = e0 + i % DOT_E;
    if (t < T && e < K)
      part[(int64_t)blockIdx.x * T * K + (int64_t)t * K + e] =
          (red[i] + red[DOT_T * DOT_E + i]) + (red[2 * DOT_T * DOT_E + i] + red[3 * DOT_T * DOT_E + i]);
  }
}

// Four slots of one system a warp over the block's share of the columns, which
// read the system's gradient once: part[split][slot].
template <int V, typename TE>
__global__ void __launch_bounds__(256)
    k_mix_dot_slots(int n_systems, int K, int top_k, int64_t n, const TE *__restrict__ experts,
                    const int *__restrict__ index, const float *__restrict__ grad,
                    float *__restrict__ part) {
  const int lane = threadIdx.x & 31;
  const int64_t len = ((n + gridDim.x - 1) / gridDim.x + V - 1) / V * V;
  const int64_t c0 = blockIdx.x * len, c1 = c0 + len < n ? c0 + len : n;
  const int quads = (top_k + 3) / 4;
  const int64_t jobs = (int64_t)n_systems * quads, n_slots = (int64_t)n_systems * top_k;
  for (int64_t job = blockIdx.y * 8 + (threadIdx.x >> 5); job < jobs; job += gridDim.y * 8) {
    const int64_t t = job / quads;
    const int j0 = (int)(job - t * quads) * 4;
    const float *g = grad + t * n;
    const TE *x[4];
    float s[4][V];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = j0 + u >= top_k ? -1 : index ? index[t * top_k + j0 + u] : j0 + u;
      x[u] = e >= 0 && e < K ? experts + e * n : nullptr;
#pragma unroll
      for (int v = 0; v < V; ++v) s[u][v] = 0.f;
    }
#pragma unroll 2
    for (int64_t c = c0 + lane * V; c < c1; c += 32 * V) {
      float b[V], a[4][V];
      load_vec<V>(g + c, b);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (x[u]) load_vec<V>(x[u] + c, a[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (x[u])
#pragma unroll
          for (int v = 0; v < V; ++v) s[u][v] = fmaf(a[u][v], b[v], s[u][v]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float sum = s[u][0];
#pragma unroll
      for (int v = 1; v < V; ++v) sum += s[u][v];
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0 && j0 + u < top_k) part[blockIdx.x * n_slots + t * top_k + j0 + u] = sum;
    }
  }
}

// Both gradients by index, for the systems whose gradients fit a block's shared
// memory: a block stages `cols` columns of all of them with asynchronous
// copies, forms the experts' gradient there from groups of cols / 4 threads
// (four columns a thread, an expert a group) and the slots' products from its
// warps.  grad_out is read once and nothing else passes through L2 twice but
// the experts' rows that several systems name.  part[block][slot].
constexpr int BACK_SLOTS = 2048, BACK_EXPERTS = 1024, BACK_BYTES = 96 * 1024;

template <int COLS, typename TE>
__global__ void __launch_bounds__(256)
    k_mix_back_slots(int T, int K, int top_k, int64_t n, const TE *__restrict__ experts,
                     const float *__restrict__ weights, const int *__restrict__ index,
                     const int *__restrict__ offsets, const int *__restrict__ list,
                     const float *__restrict__ grad, float *__restrict__ ge,
                     float *__restrict__ part) {
  extern __shared__ __align__(16) unsigned char sm[];
  const int slots = T * top_k, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  float *stage = reinterpret_cast<float *>(sm);  // [2][T][COLS]
  int2 *by_expert = reinterpret_cast<int2 *>(stage + 2 * T * COLS);  // the lists: system's place, weight
  int2 *by_slot = by_expert + slots;                                 // the slots: place, expert or -1
  int *off = reinterpret_cast<int *>(by_slot + slots);               // [K + 1]
  float *total = reinterpret_cast<float *>(off + K + 1);             // the slots' products so far
  const int64_t tiles = (n + COLS - 1) / COLS;
  auto load = [&](int64_t tile) {
    if (tile < tiles) {
      constexpr int VECS = COLS / 4, STEP = 256 / VECS;
      const int c = (tid % VECS) * 4;
      const int64_t at = tile * COLS + c;
      float *g = stage + (tile / gridDim.x & 1) * T * COLS;
      for (int t = tid / VECS; t < T; t += STEP)
        copy_async_or_zero<16>(g + t * COLS + c, grad + t * n + (at < n ? at : 0), at < n);
    }
    copy_commit();
  };
  load(blockIdx.x);
  const int named = offsets[K];
  for (int i = tid; i < slots; i += 256) {
    if (i < named) {
      const int p = list[i];
      by_expert[i] = make_int2(p / top_k * COLS, __float_as_int(weights[p]));
    }
    const int e = index[i];
    by_slot[i] = make_int2(i / top_k * COLS, e >= 0 && e < K ? e : -1);
  }
  for (int i = tid; i <= K; i += 256) off[i] = offsets[i];
  for (int i = tid; i < slots; i += 256) total[i] = 0.f;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    load(tile + gridDim.x);  // into the buffer that the last step is done with
    copy_wait<1>();
    __syncthreads();
    const float *g = stage + (tile / gridDim.x & 1) * T * COLS;
    const int64_t c0 = tile * COLS;
    const int have = n - c0 < COLS ? (int)(n - c0) : COLS;  // a multiple of four
    if (ge) {
      constexpr int GROUP = COLS / 4;
      const int c = (tid % GROUP) * 4;
      float *to = ge + c0 + c;
      for (int e = tid / GROUP; e < K; e += 256 / GROUP) {
        float acc[4] = {};
        const int b = off[e + 1];
        for (int q = off[e]; q < b; ++q) {
          const int2 slot = by_expert[q];
          float x[4];
          load_vec<4>(g + slot.x + c, x);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[v] = fmaf(__int_as_float(slot.y), x[v], acc[v]);
        }
        if (c < have) store_vec<4>(to + e * n, acc);
      }
    }
    if (part) {
      // S slots a warp and step, all their vectors in flight
      constexpr int H = COLS / 128, S = H >= 4 ? 2 : 4;
      for (int p = w; p < slots; p += 8 * S) {
        int2 slot[S];
        float x[S][H][4], sum[S];
#pragma unroll
        for (int u = 0; u < S; ++u) {
          slot[u] = p + 8 * u < slots ? by_slot[p + 8 * u] : make_int2(0, -1);
          sum[u] = 0.f;
          const TE *from = experts + slot[u].y * n + c0 + lane * 4;
#pragma unroll
          for (int h = 0; h < H; ++h)
            if (slot[u].y >= 0 && h * 128 + lane * 4 < have) load_vec<4>(from + h * 128, x[u][h]);
        }
#pragma unroll
        for (int u = 0; u < S; ++u)
#pragma unroll
          for (int h = 0; h < H; ++h)
            if (slot[u].y >= 0 && h * 128 + lane * 4 < have) {
              float y[4];
              load_vec<4>(g + slot[u].x + h * 128 + lane * 4, y);
#pragma unroll
              for (int v = 0; v < 4; ++v) sum[u] = fmaf(x[u][h][v], y[v], sum[u]);
            }
#pragma unroll
        for (int u = 0; u < S; ++u) {
#pragma unroll
          for (int o = 16; o; o >>= 1) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
          if (lane == 0 && p + 8 * u < slots) total[p + 8 * u] += sum[u];  // this warp's alone
        }
      }
    }
    __syncthreads();  // everyone is done with this buffer
  }
  copy_wait<0>();
  if (part)
    for (int i = tid; i < slots; i += 256) part[blockIdx.x * (int64_t)slots + i] = total[i];
}

// gw[slot] from the splits: of all (t, e) (all) or of the slots.  A lane a
// slot, so that the partial sums are read side by side; a warp takes every
// 32nd split, and the warps' sums are added in a tree.
__global__ void __launch_bounds__(1024)
    k_mix_dots_join(int64_t n_slots, int K, int top_k, const int *__restrict__ index, bool all,
                    int64_t stride, int splits, const float *__restrict__ part,
                    float *__restrict__ gw) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t p = blockIdx.x * 32ll + lane;
  float s = 0.f;
  if (p < n_slots) {
    const int e = index ? index[p] : (int)(p % top_k);
    if (e >= 0 && e < K) {
      const int64_t at = all ? (p / top_k) * K + e : p;
#pragma unroll 8
      for (int i = w; i < splits; i += 32) s += part[i * stride + at];
    }
  }
  sums[w][lane] = s;
  __syncthreads();
  s = sums[lane][w];  // of slot w, from warp `lane`
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32ll + w < n_slots) gw[blockIdx.x * 32ll + w] = s;
}

}  // namespace so2

using namespace so2;

namespace {

struct MixPlan {
  size_t status, offsets, list, part, total;
  bool tiles;  // the products of all (t, e), or of the slots alone
  int cols;    // both gradients by index together: a tile's columns, or 0
  int smem;    // and the block's shared memory
  int splits;
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
    // The products of all (t, e) in tiles of a fixed size, or of the slots one by
    // one.  Both gradients of 307,200 bf16 weights, tiles / slots in us: 33
    // systems, 4 of 64 experts 121 / 66, 8 of 64 128 / 95, 16 of 64 155 / 137.
    // Of 1,228,800 f32 weights, every expert: 4 x 8 165 / 45, 8 x 16 174 / 103,
    // 16 x 16 179 / 157, 8 x 32 192 / 254.
    p.tiles = d->top_k * 2 >= d->n_experts && n_systems * d->n_experts >= MIX_TILES_FROM;
    const int64_t per = p.tiles ? n_systems * d->n_experts : n_systems * d->top_k;  // products
    int64_t want;
    // Up to eight slots a system, and all systems' gradients of at least 128
    // columns in a block's shared memory (two blocks an SM): one kernel for both
    // gradients.  Same case, together / apart in us: 2 of 64 51 / 59, 4 of 64
    // 63 / 66, 8 of 64 86 / 95, but 16 of 64 174 / 137.
    p.cols = 0;
    if (!p.tiles && n_systems > 0 && d->top_k <= 8 && d->top_k < d->n_experts && slots <= BACK_SLOTS && d->n_experts <= BACK_EXPERTS &&
        d->n_weights % 4 == 0) {
      p.cols = 512;
      while (p.cols >= 128 && n_systems * p.cols * 8 > BACK_BYTES) p.cols /= 2;
      if (p.cols < 128) p.cols = 0;
    }
    if (p.tiles) {  // two resident blocks an SM
      const int64_t t = ceil_div(n_systems, DOT_T) * ceil_div(d->n_experts, DOT_E);
      want = ceil_div(2 * MODEL_SMS, t > 0 ? t : 1);
      if (want > ceil_div(d->n_weights, DOT_COLS)) want = ceil_div(d->n_weights, DOT_COLS);
    } else {
      want = ceil_div(d->n_weights, 2048);
    }
    // at most 16 M partial sums
    const int64_t most = per > 0 ? (16ll << 20) / per : 1;
    p.splits = (int)(want < most ? want : (most > 0 ? most : 1));
    if (p.cols) {
      // as many blocks as stay resident, which take equal shares of the tiles
      p.smem = (int)(n_systems * p.cols * 8 + slots * 20 + (d->n_experts + 1) * 4);
      int fit = 224 * 1024 / (p.smem + 1024);
      if (fit > 4) fit = 4;
      const int64_t tiles = ceil_div(d->n_weights, p.cols);
      p.splits = (int)ceil_div(tiles, ceil_div(tiles, MODEL_SMS * fit));
    }
    p.part = ws_take(c, sizeof(float) * (size_t)(per * p.splits));
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

// Rows of C a thread holds: all of them up to 32, else the fewest passes over B
// with evenly filled ones.
template <int V, typename TB, typename TC>
so2_status launch_rows_fma(int R, int S, int64_t n, const float *M, int64_t mr, int64_t ms,
                           const TB *B, TC *C, DevStatus *st, cudaStream_t s) {
  const unsigned grid = (unsigned)ceil_div(n, ROWS_THREADS * V);
  const int passes = (R + 31) / 32, tt = (R + passes - 1) / passes;
#define MIX_ROWS(TT) \
  k_mix_rows<TT, V, TB, TC><<<grid, ROWS_THREADS, 0, s>>>(R, S, n, M, mr, ms, B, C, st)
  if (tt <= 1) MIX_ROWS(1);
  else if (tt <= 2) MIX_ROWS(2);
  else if (tt <= 4) MIX_ROWS(4);
  else if (tt <= 8) MIX_ROWS(8);
  else if (tt <= 16) MIX_ROWS(16);
  else if (tt <= 24) MIX_ROWS(24);
  else MIX_ROWS(32);
#undef MIX_ROWS
  MODEL_CKL();
  return SO2_OK;
}

template <int N, typename TB, typename TC>
so2_status launch_rows_tc(int r0, int R, int S, int64_t n, const float *M, int64_t mr, int64_t ms,
                          const TB *B, TC *C, DevStatus *st, cudaStream_t s) {
  const int blocks = (S + MIXTC_KB - 1) / MIXTC_KB, smem = mixtc_smem<TB>(blocks);
  if (!allow_smem(k_mix_tc<N, TB, TC>, smem, mixtc_smem<TB>(MIXTC_MAX_S / MIXTC_KB))) return SO2_ERR_CUDA;
  const int64_t tiles = ceil_div(n, MIXTC_COLS);
  const int64_t most = MODEL_SMS * (smem <= 112 * 1024 ? 2 : 1);
  k_mix_tc<N, TB, TC><<<(unsigned)(tiles < most ? tiles : most), MIXTC_THREADS, smem, s>>>(
      r0, R, S, blocks, n, M, mr, ms, B, C, st);
  MODEL_CKL();
  return SO2_OK;
}

template <int V, typename TB, typename TC>
so2_status launch_rows(int R, int S, int64_t n, const float *M, int64_t mr, int64_t ms, const TB *B,
                       TC *C, DevStatus *st, cudaStream_t s) {
  if constexpr (V == 4) {
    const int64_t steps = ceil_div(S, MIXTC_KB);
    if (S <= MIXTC_MAX_S && R * (int64_t)S >= MIX_TC_FROM * steps) {
      MODEL_CK(cudaMemsetAsync(st, 0, sizeof(DevStatus), s));
      for (int r0 = 0; r0 < R; r0 += MIXTC_ROWS) {
        const so2_status e = R - r0 <= 32 ? launch_rows_tc<32>(r0, R, S, n, M, mr, ms, B, C, st, s)
                                          : launch_rows_tc<64>(r0, R, S, n, M, mr, ms, B, C, st, s);
        if (e != SO2_OK) return e;
      }
      return SO2_OK;
    }
  }
  return launch_rows_fma<V>(R, S, n, M, mr, ms, B, C, st, s);
}

template <int V, typename TE, typename TO>
so2_status launch_mix(const so2conv_mix_desc *d, int64_t n_systems, const void *experts,
                const float *weights, const int32_t *index, void *out, DevStatus *st,
                cudaStream_t s) {
  if constexpr (V <= 4) {
    if (!index)
      return launch_rows<V>((int)n_systems, d->n_experts, d->n_weights, weights, d->top_k, 1,
                            static_cast<const TE *>(experts), static_cast<TO *>(out), st, s);
  }
  MODEL_CK(cudaMemsetAsync(st, 0, sizeof(DevStatus), s));
  const int64_t cols = ceil_div(d->n_weights, 256 * V);
  int64_t rows = ceil_div(MODEL_SMS * 16, cols);
  if (rows > n_systems) rows = n_systems;
  k_mix<V, TE, TO><<<dim3((unsigned)cols, (unsigned)rows), 256, 0, s>>>(
      (int)n_systems, d->n_experts, d->top_k, d->n_weights, static_cast<const TE *>(experts),
      weights, index, static_cast<TO *>(out), st);
  MODEL_CKL();
  return SO2_OK;
}

template <typename TE, typename TO>
so2_status launch_mix(bool vec, const so2conv_mix_desc *d, int64_t n_systems, const void *experts,
                const float *weights, const int32_t *index, void *out, DevStatus *st,
                cudaStream_t s) {
  // by index, eight columns a thread where both sides allow it: half the
  // instructions a column of four
  if (vec && index && d->n_weights % 8 == 0 && aligned_to(experts, 16) && aligned_to(out, 16))
    return launch_mix<8, TE, TO>(d, n_systems, experts, weights, index, out, st, s);
  if (vec) return launch_mix<4, TE, TO>(d, n_systems, experts, weights, index, out, st, s);
  return launch_mix<1, TE, TO>(d, n_systems, experts, weights, index, out, st, s);
}

template <int COLS, typename TE>
so2_status mix_back_slots(const so2conv_mix_desc *d, int64_t T, const MixPlan &p, const TE *experts,
                          const float *weights, const int32_t *index, const int *offsets,
                          const int *list, const float *grad, float *ge, float *part,
                          cudaStream_t s) {
  constexpr int most = BACK_BYTES + BACK_SLOTS * 20 + (BACK_EXPERTS + 1) * 4;
  if (!allow_smem(k_mix_back_slots<COLS, TE>, p.smem, most)) return SO2_ERR_CUDA;
  k_mix_back_slots<COLS, TE><<<p.splits, 256, p.smem, s>>>(
      (int)T, d->n_experts, d->top_k, d->n_weights, experts, weights, index, offsets, list, grad, ge,
      part);
  MODEL_CKL();
  return SO2_OK;
}

template <typename TE>
so2_status mix_back_slots(const so2conv_mix_desc *d, int64_t T, const MixPlan &p,
                          const void *experts, const float *weights, const int32_t *index,
                          const int *offsets, const int *list, const float *grad, float *ge,
                          float *part, cudaStream_t s) {
  const TE *x = static_cast<const TE *>(experts);
  if (p.cols == 512)
    return mix_back_slots<512, TE>(d, T, p, x, weights, index, offsets, list, grad, ge, part, s);
  if (p.cols == 256)
    return mix_back_slots<256, TE>(d, T, p, x, weights, index, offsets, list, grad, ge, part, s);
  return mix_back_slots<128, TE>(d, T, p, x, weights, index, offsets, list, grad, ge, part, s);
}

template <typename TE>
so2_status mix_tc_back(const so2conv_mix_desc *d, int T, int blocks, const void *experts,
                       const float *weights, const float *grad, float *ge, float *part,
                       DevStatus *st, cudaStream_t s) {
  constexpr int smem = mixbk_smem<TE>();
  if (!allow_smem(k_mix_tc_back<TE>, smem, smem)) return SO2_ERR_CUDA;
  k_mix_tc_back<TE><<<blocks, MIXBK_THREADS, smem, s>>>(T, d->n_experts, d->n_weights, weights,
                                                        static_cast<const TE *>(experts), grad, ge,
                                                        part, st);
  MODEL_CKL();
  return SO2_OK;
}

template <bool VEC, typename TE>
so2_status mix_dots(const so2conv_mix_desc *d, int64_t n_systems, const MixPlan &p,
                    const void *experts, const int32_t *index, const float *grad, float *part,
                    cudaStream_t s) {
  const TE *x = static_cast<const TE *>(experts);
  if (p.tiles) {
    constexpr int red = 4 * DOT_T * DOT_E * 4;
    constexpr int smem = DOT_STAGES * dot_stage_bytes<TE>() > red ? DOT_STAGES * dot_stage_bytes<TE>() : red;
    if (!allow_smem(k_mix_dot_tiles<VEC, TE>, smem, smem)) return SO2_ERR_CUDA;
    const int64_t tiles = ceil_div(n_systems, DOT_T) * ceil_div(d->n_experts, DOT_E);
    k_mix_dot_tiles<VEC, TE><<<dim3(p.splits, (unsigned)tiles), 256, smem, s>>>(
        (int)n_systems, d->n_experts, d->n_weights, x, grad, part);
  } else {
    const int64_t rows = ceil_div(n_systems * ceil_div(d->top_k, 4), 8);
    k_mix_dot_slots<VEC ? 4 : 1, TE><<<dim3(p.splits, (unsigned)(rows < 65535 ? rows : 65535)), 256, 0, s>>>(
        (int)n_systems, d->n_experts, d->top_k, d->n_weights, x, index, grad, part);
  }
  MODEL_CKL();
  return SO2_OK;
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
  if (n_systems == 0) {
    MODEL_CK(cudaMemsetAsync(st, 0, sizeof(DevStatus), s));
    return SO2_OK;
  }
  typedef __nv_bfloat16 bf;
  const bool vec = d->n_weights % 4 == 0 && aligned_to(experts, 4 * es) && aligned_to(out, 4 * os);
  if (d->expert_dtype == SO2_F32 && d->out_dtype == SO2_F32)
    return launch_mix<float, float>(vec, d, n_systems, experts, weights, index, out, st, s);
  if (d->expert_dtype == SO2_F32)
    return launch_mix<float, bf>(vec, d, n_systems, experts, weights, index, out, st, s);
  if (d->out_dtype == SO2_F32)
    return launch_mix<bf, float>(vec, d, n_systems, experts, weights, index, out, st, s);
  return launch_mix<bf, bf>(vec, d, n_systems, experts, weights, index, out, st, s);
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
  if (!index || n_systems == 0) MODEL_CK(cudaMemsetAsync(st, 0, sizeof(DevStatus), s));
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
    k_mix_lists<<<(unsigned)ceil_div(K, 8), 256, 0, s>>>((int)slots, K, index, offsets, list, st);
    MODEL_CKL();
  }
  const size_t es = dtype_size(d->expert_dtype);
  const bool vec = n % 4 == 0 && aligned_to(experts, 4 * es) && aligned_to(grad_out, 16) &&
                   aligned_to(grad_experts, 16);
  if (index && vec && p.cols) {
    float *part = grad_weights ? ws_at<float>(ws, p.part) : nullptr;
    r = d->expert_dtype == SO2_F32
            ? mix_back_slots<float>(d, n_systems, p, experts, weights, index, offsets, list, grad_out,
                                    grad_experts, part, s)
            : mix_back_slots<__nv_bfloat16>(d, n_systems, p, experts, weights, index, offsets, list,
                                            grad_out, grad_experts, part, s);
    if (r != SO2_OK) return r;
    if (grad_weights) {
      k_mix_dots_join<<<(unsigned)ceil_div(slots, 32), 1024, 0, s>>>(
          slots, K, k, index, false, slots, p.splits, part, grad_weights);
      MODEL_CKL();
    }
    return SO2_OK;
  }
  if (!grad_experts && !grad_weights) return SO2_OK;
  // (the last case above: 174 us; it costs the same up to 64 x 32, where tiles
  // and the other kernels take 260)
  if (!index && vec && n_systems <= MIXBK_T && K <= MIXBK_E && n_systems * K >= MIX_TILES_FROM) {
    float *part = grad_weights ? ws_at<float>(ws, p.part) : nullptr;
    const int64_t tiles = ceil_div(n, MIXTC_COLS);
    const int blocks = (int)(tiles < MODEL_SMS ? tiles : MODEL_SMS);  // never over the plan's splits
    r = d->expert_dtype == SO2_F32
            ? mix_tc_back<float>(d, (int)n_systems, blocks, experts, weights, grad_out, grad_experts,
                                 part, st, s)
            : mix_tc_back<__nv_bfloat16>(d, (int)n_systems, blocks, experts, weights, grad_out,
                                         grad_experts, part, st, s);
    if (r != SO2_OK) return r;
    if (grad_weights) {
      k_mix_dots_join<<<(unsigned)ceil_div(slots, 32), 1024, 0, s>>>(
          slots, K, k, nullptr, true, n_systems * K, blocks, part, grad_weights);
      MODEL_CKL();
    }
    return SO2_OK;
  }
  if (grad_experts) {
    const int64_t cols = ceil_div(n, vec ? 1024 : 256);
    int64_t rows = ceil_div(MODEL_SMS * 8, cols);
    if (rows > K) rows = K;
    const dim3 grid((unsigned)cols, (unsigned)rows);
    if (!index) {
      r = vec ? launch_rows<4>(K, (int)n_systems, n, weights, 1, k, grad_out, grad_experts, st, s)
              : launch_rows<1>(K, (int)n_systems, n, weights, 1, k, grad_out, grad_experts, st, s);
      if (r != SO2_OK) return r;
    } else if (vec)
      k_mix_grad_experts<4><<<grid, 256, 0, s>>>((int)slots, K, k, n, weights, offsets, list,
                                                 grad_out, grad_experts);
    else
      k_mix_grad_experts<1><<<grid, 256, 0, s>>>((int)slots, K, k, n, weights, offsets, list,
                                                 grad_out, grad_experts);
    MODEL_CKL();
  }
  if (grad_weights) {
    float *part = ws_at<float>(ws, p.part);
    typedef __nv_bfloat16 bf;
    so2_status r2;
    if (d->expert_dtype == SO2_F32)
      r2 = vec ? mix_dots<true, float>(d, n_systems, p, experts, index, grad_out, part, s)
               : mix_dots<false, float>(d, n_systems, p, experts, index, grad_out, part, s);
    else
      r2 = vec ? mix_dots<true, bf>(d, n_systems, p, experts, index, grad_out, part, s)
               : mix_dots<false, bf>(d, n_systems, p, experts, index, grad_out, part, s);
    if (r2 != SO2_OK) return r2;
    k_mix_dots_join<<<(unsigned)ceil_div(slots, 32), 1024, 0, s>>>(
        slots, K, k, index, p.tiles, p.tiles ? n_systems * K : slots, p.splits, part, grad_weights);
    MODEL_CKL();
  }
  return SO2_OK;
}

}  // extern "C"
