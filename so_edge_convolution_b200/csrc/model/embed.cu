// embed.cu -- element embedding: lookup into the l = 0 rows, and the table's
// gradient by sorted tokens.
//
// Backward.  The tokens are sorted by id (stable, least significant digit
// first, 8 bits a pass), so that each id's rows are one run of the sorted
// list.  The list is cut into equal ranges, one group of lanes each; a group
// adds its rows in registers and writes every run that lies inside its range
// straight to the table's gradient.  A run that crosses ranges leaves one
// partial sum in each, which a second kernel adds in range order.  Few tokens
// and a small table need no sort: a block per id scans the tokens.  No atomics
// on floats: the order of the additions depends on the sizes and the ids alone.
#include "model_common.cuh"

namespace so2 {

// ---- forward -----------------------------------------------------------------
// A group of 2^shift lanes a node, V values a lane and step (V divides the
// channels, so a vector is an element's row or zeros, not both).  The stores
// bound it.  A grid of one block clears the status word itself.
template <int V, typename TT, typename TO>
__global__ void k_embed(int64_t n, const int64_t *__restrict__ ids, const TT *__restrict__ table,
                        int64_t n_rows, int channels, int64_t row, float scale, int64_t pad_id,
                        TO *__restrict__ out, int64_t ld_out, int shift, DevStatus *st) {
  if (gridDim.x == 1) {
    if (threadIdx.x == 0) *st = DevStatus{0, 0};
    __syncthreads();
  }
  const int64_t id0 = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int lane = (int)(id0 & ((1 << shift) - 1));
  for (int64_t i = id0 >> shift; i < n; i += ((int64_t)gridDim.x * blockDim.x) >> shift) {
    const int64_t id = ids[i];
    const bool on = id != pad_id && id >= 0 && id < n_rows;
    if (!on && id != pad_id && lane == 0) raise_error(st, SO2_ERR_INDEX, (int)(i & 0x7fffffff));
    TO *o = out + i * ld_out;
    for (int64_t c = (int64_t)lane * V; c < row; c += (int64_t)V << shift) {
      float v[V];
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = 0.f;
      if (on && c < channels) {
        load_vec<V>(table + id * channels + c, v);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] *= scale;
      }
      store_vec<V>(o + c, v);
    }
  }
}

// ---- backward: sort ------------------------------------------------------------
constexpr int SORT_THREADS = 256, SORT_WARPS = 8;
constexpr int SORT_ROUNDS = 4;                           // 32 keys of a warp each
constexpr int SORT_TILE = SORT_THREADS * SORT_ROUNDS;    // keys of a block
constexpr int SORT_BINS = 256;

// The sort key of token i: its id, or n_rows for a token without a gradient.
__device__ __forceinline__ uint32_t embed_key(const int64_t *ids, int64_t i, int64_t n_rows,
                                              int64_t pad_id, DevStatus *st) {
  const int64_t id = ids[i];
  if (id >= 0 && id < n_rows && id != pad_id) return (uint32_t)id;
  if (st && id != pad_id) raise_error(st, SO2_ERR_INDEX, (int)(i & 0x7fffffff));
  return (uint32_t)n_rows;
}

// With up to 64 tiles a scatter block adds up the tiles before its own itself,
// from hist[block][bin]; with more, k_sort_scan does, in hist[bin][block].
__host__ __device__ inline bool sort_direct(int nb) { return nb <= 64; }

// hist: keys of the block's tile by digit.  FIRST reads the ids,
// clears the status word (the scatter records bad ids) and has its blocks
// from nb on zero the table's gradient.
template <bool FIRST>
__global__ void k_sort_hist(int64_t n, const int64_t *__restrict__ ids, int64_t n_rows,
                            int64_t pad_id, const uint32_t *__restrict__ keys, int shift,
                            uint32_t mask, int nb, int *__restrict__ hist,
                            float *__restrict__ table, int64_t table_size, DevStatus *st) {
  if (FIRST && blockIdx.x >= nb) {
    const int64_t t = (blockIdx.x - nb) * (int64_t)SORT_THREADS + threadIdx.x;
    const int64_t step = (int64_t)(gridDim.x - nb) * SORT_THREADS;
    if ((reinterpret_cast<uintptr_t>(table) & 15) == 0) {
      for (int64_t i = t; i < table_size / 4; i += step)
        reinterpret_cast<float4 *>(table)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int64_t i = (table_size & ~3ll) + t; i < table_size; i += step) table[i] = 0.f;
    } else {
      for (int64_t i = t; i < table_size; i += step) table[i] = 0.f;
    }
    return;
  }
  __shared__ int h[SORT_BINS];
  if (FIRST && blockIdx.x == 0 && threadIdx.x == 0) *st = DevStatus{0, 0};
  h[threadIdx.x] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * SORT_TILE;
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const int64_t i = t0 + r * SORT_THREADS + threadIdx.x;
    uint32_t d = SORT_BINS;
    if (i < n) {
      const uint32_t k = FIRST ? embed_key(ids, i, n_rows, pad_id, nullptr) : keys[i];
      d = (k >> shift) & mask;
    }
    // one addition for the lanes of a warp that share a digit
    const unsigned same = __match_any_sync(0xffffffffu, d);
    if (d < SORT_BINS && (threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&h[d], __popc(same));
  }
  __syncthreads();
  const int64_t at = sort_direct(nb) ? (int64_t)blockIdx.x * SORT_BINS + threadIdx.x
                                     : (int64_t)threadIdx.x * nb + blockIdx.x;
  hist[at] = h[threadIdx.x];
}

// Block-wide exclusive scan of one int per thread (256 threads); *total.
__device__ __forceinline__ int block_scan256(int v, int *total) {
  __shared__ int warp_sum[SORT_WARPS];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warp_sum[w] = s;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < SORT_WARPS; ++i) {
    if (i < w) base += warp_sum[i];
    all += warp_sum[i];
  }
  __syncthreads();
  *total = all;
  return base + s - v;
}

// One block per bin: its row of hist to exclusive sums over the blocks.
__global__ void k_sort_scan(int nb, int *__restrict__ hist, int *__restrict__ totals) {
  int *row = hist + (int64_t)blockIdx.x * nb;
  int carry = 0;
  for (int b0 = 0; b0 < nb; b0 += SORT_THREADS) {
    const int b = b0 + threadIdx.x;
    const int v = b < nb ? row[b] : 0;
    int all;
    const int e = block_scan256(v, &all);
    if (b < nb) row[b] = carry + e;
    carry += all;
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// Stable scatter of the tile: a warp's 128 keys are consecutive, so the order
// inside the tile is (warp, round, lane).  A key's rank among its warp's equal
// digits comes from matching the lanes; the warps' counts and the blocks'
// sums then place it.
template <bool FIRST>
__global__ void __launch_bounds__(SORT_THREADS)
    k_sort_scatter(int64_t n, const int64_t *__restrict__ ids, int64_t n_rows, int64_t pad_id,
                   const uint32_t *__restrict__ keys_in, const int *__restrict__ perm_in, int shift,
                   uint32_t mask, const int *__restrict__ hist, const int *__restrict__ totals,
                   uint32_t *__restrict__ keys_out, int *__restrict__ perm_out, DevStatus *st) {
  __shared__ int cnt[SORT_WARPS][SORT_BINS + 1];  // the last one takes lanes beyond the list
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * SORT_TILE + w * (32 * SORT_ROUNDS);
  uint32_t k[SORT_ROUNDS], d[SORT_ROUNDS];
  int p[SORT_ROUNDS], rank[SORT_ROUNDS];
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const int64_t i = t0 + r * 32 + lane;
    k[r] = 0;
    p[r] = (int)i;
    if (i < n) {
      k[r] = FIRST ? embed_key(ids, i, n_rows, pad_id, st) : keys_in[i];
      if (!FIRST) p[r] = perm_in[i];
    }
    d[r] = i < n ? (k[r] >> shift) & mask : SORT_BINS;
  }
  int before, total;
  if (sort_direct(gridDim.x)) {
    before = total = 0;
#pragma unroll 8
    for (int b = 0; b < (int)gridDim.x; ++b) {
      const int v = hist[b * SORT_BINS + tid];
      total += v;
      if (b < (int)blockIdx.x) before += v;
    }
  } else {
    before = hist[(int64_t)tid * gridDim.x + blockIdx.x];
    total = totals[tid];
  }
#pragma unroll
  for (int i = 0; i < SORT_WARPS; ++i) cnt[i][tid] = 0;
  if (tid < SORT_WARPS) cnt[tid][SORT_BINS] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const unsigned same = __match_any_sync(0xffffffffu, d[r]);
    const int ahead = __popc(same & ((1u << lane) - 1));
    rank[r] = cnt[w][d[r]] + ahead;
    __syncwarp();
    if (ahead == 0) cnt[w][d[r]] += __popc(same);
    __syncwarp();
  }
  int unused;
  const int first = block_scan256(total, &unused);  // synchronises the block
  {
    int s = first + before;
#pragma unroll
    for (int i = 0; i < SORT_WARPS; ++i) {
      const int c = cnt[i][tid];
      cnt[i][tid] = s;
      s += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r)
    if (t0 + r * 32 + lane < n) {
      const int at = cnt[w][d[r]] + rank[r];
      keys_out[at] = k[r];
      perm_out[at] = p[r];
    }
}

// ---- backward: sums of the runs --------------------------------------------------
// One group of 2^shift lanes per range of `len` sorted tokens and slice of
// V << shift channels.  head[r]: the range's share of a run that began before
// it; tail[r]: of a run that begins in it and goes on after it.  Eight rows
// are in flight a group; the next eight keys and places are read ahead.
constexpr int RUN_ROWS = 8;  // divides len

template <int V, typename TG>
__global__ void __launch_bounds__(256)
    k_embed_runs(int64_t n, int64_t n_ranges, int len, const uint32_t *__restrict__ keys,
                 const int *__restrict__ perm, uint32_t n_rows, const TG *__restrict__ grad,
                 int64_t ld, int channels, float scale, int shift, float *__restrict__ table,
                 float *__restrict__ head, float *__restrict__ tail) {
  const int64_t id = blockIdx.x * 256ll + threadIdx.x;
  const int64_t r = id >> shift;
  const int c = ((blockIdx.y << shift) + (int)(id & ((1 << shift) - 1))) * V;
  if (r >= n_ranges || c >= channels) return;
  const int64_t a = r * len, b = a + len < n ? a + len : n;
  uint32_t cur = keys[a];
  if (cur >= n_rows) return;
  bool from_before = a > 0 && keys[a - 1] == cur;
  float acc[V];
  auto flush = [&](bool goes_on) {
    if (from_before || goes_on) {
      store_vec<V>((from_before ? head : tail) + r * channels + c, acc);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= scale;
      store_vec<V>(table + (int64_t)cur * channels + c, acc);
    }
  };
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  uint32_t k[RUN_ROWS], kn[RUN_ROWS];
  int p[RUN_ROWS], pn[RUN_ROWS];
  auto read = [&](int64_t j, uint32_t(&kk)[RUN_ROWS], int(&pp)[RUN_ROWS]) {
#pragma unroll
    for (int u = 0; u < RUN_ROWS; ++u) {
      kk[u] = j + u < b ? keys[j + u] : 0xffffffffu;
      pp[u] = j + u < b ? perm[j + u] : 0;
    }
  };
  read(a, kn, pn);
  for (int64_t j = a; j < b; j += RUN_ROWS) {
#pragma unroll
    for (int u = 0; u < RUN_ROWS; ++u) k[u] = kn[u], p[u] = pn[u];
    float g[RUN_ROWS][V];
#pragma unroll
    for (int u = 0; u < RUN_ROWS; ++u)
      if (k[u] < n_rows) load_vec<V>(grad + (int64_t)p[u] * ld + c, g[u]);
    if (j + RUN_ROWS < b) read(j + RUN_ROWS, kn, pn);
    if (k[0] == cur && k[RUN_ROWS - 1] == cur) {  // eight of one run: their sum first
#pragma unroll
      for (int v = 0; v < V; ++v)
        acc[v] += ((g[0][v] + g[1][v]) + (g[2][v] + g[3][v])) +
                  ((g[4][v] + g[5][v]) + (g[6][v] + g[7][v]));
      continue;
    }
#pragma unroll
    for (int u = 0; u < RUN_ROWS; ++u) {
      if (k[u] != cur) {
        if (j + u >= b) break;  // the list's end inside the last eight
        flush(false);
        from_before = false;
        cur = k[u];
        if (cur >= n_rows) return;  // tokens without a gradient end the list
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += g[u][v];
    }
  }
  flush(b < n && keys[b] == cur);
}

// Runs that begin in one of the block's 32 ranges and go on after it: their
// partial sums in range order.  A short run is one warp's, all warps taking
// runs of their own; a long one is the whole block's, warp w adding every
// sixteenth range from the w-th on.
constexpr int JOIN_RANGES = 32, JOIN_WARPS = 16, JOIN_ALONE = 32;

// (Thousands of partial sums of a frequent element's rows: added in 64 bits,
// so that the error stays that of the ranges' own sums.)
template <int V>
__device__ __forceinline__ void join_add(double (&acc)[V], const float *from) {
  float g[V];
  load_vec<V>(from, g);
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] += g[v];
}
template <int V>
__device__ __forceinline__ void join_store(const double (&acc)[V], float scale, float *to) {
  float r[V];
#pragma unroll
  for (int v = 0; v < V; ++v) r[v] = (float)(acc[v] * scale);
  store_vec<V>(to, r);
}

template <int V>
__global__ void __launch_bounds__(32 * JOIN_WARPS)
    k_embed_join(int64_t n, int64_t n_ranges, int len, const uint32_t *__restrict__ keys,
                 uint32_t n_rows, int channels, float scale, float *__restrict__ table,
                 const float *__restrict__ head, const float *__restrict__ tail) {
  __shared__ double part[JOIN_WARPS][32 * V];
  __shared__ int64_t last[JOIN_RANGES];  // of long runs: the last range that starts in it
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = (blockIdx.y * 32 + lane) * V;
  const int64_t r0 = blockIdx.x * (int64_t)JOIN_RANGES;
  unsigned todo;
  {  // every warp looks for itself
    const int64_t a = (r0 + lane) * len, b = a + len;
    bool begins = false;
    if (b < n) {
      const uint32_t key = keys[b - 1];
      begins = key < n_rows && keys[b] == key && (a == 0 || keys[a - 1] != key);
    }
    todo = __ballot_sync(0xffffffffu, begins);
  }
  if (w == 0) last[lane] = -1;
  __syncthreads();
  int nth = 0;
  for (unsigned m = todo; m; m &= m - 1, ++nth) {
    if (nth % JOIN_WARPS != w) continue;
    const int64_t r = r0 + __ffs(m) - 1;
    const uint32_t key = keys[r * len + len - 1];
    int64_t lo = r + 1, hi = n_ranges - 1;
    while (lo < hi) {  // 32 probes a step
      const int64_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
      const bool in = at <= hi && keys[at * len] == key;
      const int hits = __popc(__ballot_sync(0xffffffffu, in));
      const int64_t end = lo + (hits + 1) * step - 1;
      lo += hits * step;
      hi = end < hi ? end : hi;
    }
    if (lo - r > JOIN_ALONE) {
      if (lane == 0) last[r - r0] = lo;
    } else if (c < channels) {
      double acc[V] = {};
      join_add<V>(acc, tail + r * channels + c);
#pragma unroll 4
      for (int64_t q = r + 1; q <= lo; ++q) join_add<V>(acc, head + q * channels + c);
      join_store<V>(acc, scale, table + (int64_t)key * channels + c);
    }
  }
  __syncthreads();
  for (unsigned m = todo; m; m &= m - 1) {
    const int64_t r = r0 + __ffs(m) - 1, lo = last[r - r0];
    if (lo < 0) continue;
    double acc[V] = {};
    if (c < channels) {
      if (w == 0) join_add<V>(acc, tail + r * channels + c);
#pragma unroll 8
      for (int64_t q = r + 1 + w; q <= lo; q += JOIN_WARPS) join_add<V>(acc, head + q * channels + c);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) part[w][lane * V + v] = acc[v];
    __syncthreads();
    if (w == 0 && c < channels) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        acc[v] = 0.0;
#pragma unroll
        for (int i = 0; i < JOIN_WARPS; ++i) acc[v] += part[i][lane * V + v];
      }
      join_store<V>(acc, scale, table + (int64_t)keys[r * len + len - 1] * channels + c);
    }
    __syncthreads();
  }
}

// ---- backward: few tokens ------------------------------------------------------------
// One block a table row and slice of 32 V channels: each of eight warps scans
// an eighth of the ids and adds the rows that match, then the eight sums.
template <int V, typename TG>
__global__ void __launch_bounds__(256)
    k_embed_scan(int n, const int64_t *__restrict__ ids, int64_t n_rows, int64_t pad_id,
                 const TG *__restrict__ grad, int64_t ld, int channels, float scale,
                 float *__restrict__ table, DevStatus *st) {
  __shared__ float part[8][32 * V];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const int c = (blockIdx.y * 32 + lane) * V;
  const bool reports = row == 0 && blockIdx.y == 0;  // this block alone touches the status
  if (reports) {
    if (threadIdx.x == 0) *st = DevStatus{0, 0};
    __syncthreads();
  }
  const int per = ((n + 255) / 256) * 32, i0 = w * per, i1 = i0 + per < n ? i0 + per : n;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int i = i0; i < i1; i += 32) {
    const int64_t id = i + lane < i1 ? ids[i + lane] : pad_id;
    const bool bad = id != pad_id && (id < 0 || id >= n_rows);
    if (reports && bad) raise_error(st, SO2_ERR_INDEX, i + lane);
    unsigned m = __ballot_sync(0xffffffffu, i + lane < i1 && id == row && id != pad_id);
    if (c >= channels) continue;
    while (m) {  // four rows in flight
      float g[4][V];
      int j[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        j[u] = m ? i + __ffs(m) - 1 : -1;
        m &= m - 1;
        if (j[u] >= 0) load_vec<V>(grad + (int64_t)j[u] * ld + c, g[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j[u] >= 0)
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] += g[u][v];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) part[w][lane * V + v] = acc[v];
  __syncthreads();
  if (w == 0 && c < channels) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += part[i][lane * V + v];
      acc[v] = s * scale;
    }
    store_vec<V>(table + row * channels + c, acc);
  }
}

}  // namespace so2

using namespace so2;

namespace {

struct EmbedPlan {
  size_t status, keys[2], perm[2], hist, totals, head, tail, total;
  int nb, passes, bits, len;
  int64_t n_ranges;
};

bool embed_ok(const so2conv_embed_desc *d) {
  return d->n_rows >= 1 && d->n_rows < 0x7fffffff && d->channels >= 1 && d->channels <= 65536 &&
         d->n_comp >= 1 && d->n_comp <= 1024 && dtype_ok(d->table_dtype) && dtype_ok(d->out_dtype);
}

// Tokens few enough that every table row looks at all of them: the scans are
// n_rows * n / 32 steps of a warp, and a row's own tokens one eighth of n deep
// at worst.  Scan / sort in us at 128 channels: 100 rows, 128 tokens 2.3 / 12.3,
// 2,048 11.5 / 17.9, 4,096 18.1 / 19.3, 8,192 37.4 / 18.4; 2,000 rows, 2,048
// tokens 9.3 / 26.  Of large tables only the scan was timed, with cold caches
// and the call: 60,000 x 512, 69 tokens 203 us, where zeroing alone is 26, so
// the sort is likely the better one there.
bool embed_scans(const so2conv_embed_desc *d, int64_t n) {
  return n <= 4096 && d->n_rows * n <= (1 << 22);
}

// Lanes that take a row of `vectors` vectors, as a power of two.
int lane_shift(int64_t vectors) {
  int s = 0;
  while (s < 5 && (1 << s) < vectors) ++s;
  return s;
}

EmbedPlan embed_plan(const so2conv_embed_desc *d, int64_t n, int which) {
  EmbedPlan p{};
  size_t c = 0;
  p.status = ws_take(c, sizeof(DevStatus));
  if (which == SO2_WS_BACKWARD && n > 0 && !embed_scans(d, n)) {
    int bits = 1;  // of the keys 0..n_rows
    while ((d->n_rows >> bits) != 0) ++bits;
    p.passes = (bits + 7) / 8;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.nb = (int)ceil_div(n, SORT_TILE);
    // about 16 warps of ranges for each SM, which keep eight rows each in
    // flight; with 32 the runs took as long and their join 10 us more of 130
    // (a million tokens of 100 elements, 128 channels)
    p.len = (int)(ceil_div(ceil_div(n, MODEL_SMS * 16), RUN_ROWS) * RUN_ROWS);
    if (p.len < 2 * RUN_ROWS) p.len = 2 * RUN_ROWS;
    p.n_ranges = ceil_div(n, p.len);
    for (int i = 0; i < 2; ++i) {
      p.keys[i] = ws_take(c, sizeof(uint32_t) * n);
      p.perm[i] = ws_take(c, sizeof(int) * n);
    }
    p.hist = ws_take(c, sizeof(int) * SORT_BINS * (size_t)p.nb);
    p.totals = ws_take(c, sizeof(int) * SORT_BINS);
    p.head = ws_take(c, sizeof(float) * p.n_ranges * d->channels);
    p.tail = ws_take(c, sizeof(float) * p.n_ranges * d->channels);
  }
  p.total = (c + 255) & ~static_cast<size_t>(255);
  return p;
}

so2_status embed_checks(const so2conv_embed_desc *d, int64_t n, const int64_t *ids, void *ws,
                        size_t ws_bytes, int which, EmbedPlan &p) {
  if (!d) return SO2_ERR_INVALID_ARG;
  if (!embed_ok(d)) return SO2_ERR_UNSUPPORTED;
  if (n < 0 || n > (1ll << 30) || (n > 0 && !ids) || !aligned_to(ids, 8)) return SO2_ERR_INVALID_ARG;
  if (!ws || !aligned_to(ws, 256)) return SO2_ERR_WORKSPACE;
  p = embed_plan(d, n, which);
  if (ws_bytes < p.total) return SO2_ERR_WORKSPACE;
  return SO2_OK;
}

template <int V, typename TT, typename TO>
so2_status launch_embed(const so2conv_embed_desc *d, int64_t n, const int64_t *ids, const TT *table,
                        TO *out, int64_t ld, DevStatus *st, cudaStream_t s) {
  const int64_t row = (int64_t)d->n_comp * d->channels;
  const int shift = lane_shift(row / V);
  // one block, without a clearing launch before it, for what it does at once
  const bool one = n * row / V <= 4096;
  if (!one) MODEL_CK(cudaMemsetAsync(st, 0, sizeof(DevStatus), s));
  const int threads = one ? 1024 : 256;
  int64_t grid = one ? 1 : ceil_div(n << shift, threads);
  if (grid > 0x7fffffff) grid = 0x7fffffff;
  k_embed<V, TT, TO><<<(unsigned)grid, threads, 0, s>>>(n, ids, table, d->n_rows, d->channels, row,
                                                        d->scale, d->pad_id, out, ld, shift, st);
  MODEL_CKL();
  return SO2_OK;
}

template <typename TT, typename TO>
so2_status launch_embed(const so2conv_embed_desc *d, int64_t n, const int64_t *ids,
                        const void *table, void *out, int64_t ld, DevStatus *st, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(TO);  // 16-byte stores where every row allows them
  const TT *t = static_cast<const TT *>(table);
  TO *o = static_cast<TO *>(out);
  if (d->channels % V == 0 && ld % V == 0 && aligned_to(out, 16) &&
      aligned_to(table, V * sizeof(TT) < 16 ? V * sizeof(TT) : 16))
    return launch_embed<V>(d, n, ids, t, o, ld, st, s);
  return launch_embed<1>(d, n, ids, t, o, ld, st, s);
}

template <int V, typename TG>
so2_status embed_sums(const so2conv_embed_desc *d, int64_t n, const EmbedPlan &p, void *ws,
                      const uint32_t *keys, const int *perm, const TG *grad, int64_t ld,
                      float *table, cudaStream_t s) {
  const int shift = lane_shift(ceil_div(d->channels, V));
  float *head = ws_at<float>(ws, p.head), *tail = ws_at<float>(ws, p.tail);
  const dim3 grid((unsigned)ceil_div(p.n_ranges << shift, 256),
                  (unsigned)ceil_div(d->channels, (int64_t)V << shift));
  k_embed_runs<V, TG><<<grid, 256, 0, s>>>(n, p.n_ranges, p.len, keys, perm, (uint32_t)d->n_rows,
                                           grad, ld, d->channels, d->scale, shift, table, head, tail);
  MODEL_CKL();
  if (p.n_ranges > 1) {
    const dim3 g2((unsigned)ceil_div(p.n_ranges, JOIN_RANGES), (unsigned)ceil_div(d->channels, 32 * V));
    k_embed_join<V><<<g2, 32 * JOIN_WARPS, 0, s>>>(n, p.n_ranges, p.len, keys, (uint32_t)d->n_rows, d->channels,
                                       d->scale, table, head, tail);
    MODEL_CKL();
  }
  return SO2_OK;
}

template <int V, typename TG>
so2_status embed_grad(const so2conv_embed_desc *d, int64_t n, const int64_t *ids, const EmbedPlan &p,
                      void *ws, const TG *grad, int64_t ld, float *table, cudaStream_t s) {
  DevStatus *st = ws_at<DevStatus>(ws, p.status);
  if (embed_scans(d, n)) {
    const dim3 grid((unsigned)d->n_rows, (unsigned)ceil_div(d->channels, 32 * V));
    k_embed_scan<V, TG><<<grid, 256, 0, s>>>((int)n, ids, d->n_rows, d->pad_id, grad, ld,
                                             d->channels, d->scale, table, st);
    MODEL_CKL();
    return SO2_OK;
  }
  int *hist = ws_at<int>(ws, p.hist), *totals = ws_at<int>(ws, p.totals);
  const uint32_t mask = (1u << p.bits) - 1;
  const int64_t size = d->n_rows * d->channels;
  const int64_t zeroing = ceil_div(size, SORT_THREADS * 16);
  const unsigned extra = (unsigned)(zeroing < MODEL_SMS * 8 ? zeroing : MODEL_SMS * 8);
  for (int q = 0; q < p.passes; ++q) {
    const uint32_t *ki = ws_at<uint32_t>(ws, p.keys[(q + 1) & 1]);
    const int *pi = ws_at<int>(ws, p.perm[(q + 1) & 1]);
    uint32_t *ko = ws_at<uint32_t>(ws, p.keys[q & 1]);
    int *po = ws_at<int>(ws, p.perm[q & 1]);
    const int shift = q * p.bits;
    if (q == 0)
      k_sort_hist<true><<<p.nb + extra, SORT_THREADS, 0, s>>>(
          n, ids, d->n_rows, d->pad_id, nullptr, shift, mask, p.nb, hist, table, size, st);
    else
      k_sort_hist<false><<<p.nb, SORT_THREADS, 0, s>>>(n, nullptr, 0, 0, ki, shift, mask, p.nb, hist,
                                                       nullptr, 0, st);
    MODEL_CKL();
    if (!sort_direct(p.nb)) {
      k_sort_scan<<<SORT_BINS, SORT_THREADS, 0, s>>>(p.nb, hist, totals);
      MODEL_CKL();
    }
    if (q == 0)
      k_sort_scatter<true><<<p.nb, SORT_THREADS, 0, s>>>(n, ids, d->n_rows, d->pad_id, nullptr,
                                                         nullptr, shift, mask, hist, totals, ko, po, st);
    else
      k_sort_scatter<false><<<p.nb, SORT_THREADS, 0, s>>>(n, nullptr, 0, 0, ki, pi, shift, mask,
                                                          hist, totals, ko, po, st);
    MODEL_CKL();
  }
  return embed_sums<V, TG>(d, n, p, ws, ws_at<uint32_t>(ws, p.keys[(p.passes + 1) & 1]),
                           ws_at<int>(ws, p.perm[(p.passes + 1) & 1]), grad, ld, table, s);
}

template <typename TG>
so2_status embed_grad(const so2conv_embed_desc *d, int64_t n, const int64_t *ids, const EmbedPlan &p,
                      void *ws, const void *grad, int64_t ld, float *table, cudaStream_t s) {
  const TG *g = static_cast<const TG *>(grad);
  // rows in vectors of four where every row starts on one's boundary
  if (d->channels % 4 == 0 && ld % 4 == 0 && aligned_to(grad, 4 * sizeof(TG)) && aligned_to(table, 16))
    return embed_grad<4, TG>(d, n, ids, p, ws, g, ld, table, s);
  return embed_grad<1, TG>(d, n, ids, p, ws, g, ld, table, s);
}

}  // namespace

extern "C" {

size_t so2conv_embed_workspace_size(const so2conv_embed_desc *desc, int64_t n, int which) {
  if (!desc || !embed_ok(desc) || n < 0 || n > (1ll << 30) ||
      (which != SO2_WS_FORWARD && which != SO2_WS_BACKWARD))
    return 0;
  return embed_plan(desc, n, which).total;
}

so2_status so2conv_embed_forward(const so2conv_embed_desc *d, int64_t n, const int64_t *ids,
                                 const void *table, void *out, int64_t ld_out, void *ws,
                                 size_t ws_bytes, so2_stream_t stream) {
  EmbedPlan p;
  so2_status r = embed_checks(d, n, ids, ws, ws_bytes, SO2_WS_FORWARD, p);
  if (r != SO2_OK) return r;
  const int64_t row = (int64_t)d->n_comp * d->channels;
  if (ld_out < row || ld_out > (1ll << 40) || n > (1ll << 38) / row) return SO2_ERR_INVALID_ARG;
  if (n > 0 && (!table || !out || !aligned_to(table, dtype_size(d->table_dtype)) ||
                !aligned_to(out, dtype_size(d->out_dtype))))
    return SO2_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DevStatus *st = ws_at<DevStatus>(ws, p.status);
  if (n == 0) {
    MODEL_CK(cudaMemsetAsync(st, 0, sizeof(DevStatus), s));
    return SO2_OK;
  }
  typedef __nv_bfloat16 bf;
  if (d->table_dtype == SO2_F32 && d->out_dtype == SO2_F32)
    return launch_embed<float, float>(d, n, ids, table, out, ld_out, st, s);
  if (d->table_dtype == SO2_F32)
    return launch_embed<float, bf>(d, n, ids, table, out, ld_out, st, s);
  if (d->out_dtype == SO2_F32)
    return launch_embed<bf, float>(d, n, ids, table, out, ld_out, st, s);
  return launch_embed<bf, bf>(d, n, ids, table, out, ld_out, st, s);
}

so2_status so2conv_embed_backward(const so2conv_embed_desc *d, int64_t n, const int64_t *ids,
                                  const void *grad_out, int64_t ld_grad, float *grad_table,
                                  void *ws, size_t ws_bytes, so2_stream_t stream) {
  EmbedPlan p;
  so2_status r = embed_checks(d, n, ids, ws, ws_bytes, SO2_WS_BACKWARD, p);
  if (r != SO2_OK) return r;
  if (!grad_table || !aligned_to(grad_table, 4) || ld_grad < d->channels || ld_grad > (1ll << 40))
    return SO2_ERR_INVALID_ARG;
  const size_t es = dtype_size(d->out_dtype);
  if (n > 0 && (!grad_out || !aligned_to(grad_out, es))) return SO2_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n == 0) {
    MODEL_CK(cudaMemsetAsync(ws_at<DevStatus>(ws, p.status), 0, sizeof(DevStatus), s));
    MODEL_CK(cudaMemsetAsync(grad_table, 0, sizeof(float) * d->n_rows * d->channels, s));
    return SO2_OK;
  }
  if (d->out_dtype == SO2_F32)
    return embed_grad<float>(d, n, ids, p, ws, grad_out, ld_grad, grad_table, s);
  return embed_grad<__nv_bfloat16>(d, n, ids, p, ws, grad_out, ld_grad, grad_table, s);
}

}  // extern "C"
