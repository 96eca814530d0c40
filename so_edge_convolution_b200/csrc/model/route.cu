// route.cu -- routing to experts: scores, selection and the logits' gradient.
//
// One warp per token.  Experts are ranked by an integer key in the order of
// their selection scores: 0 for an expert that may not be chosen, 1 for NaN,
// then the numbers.  Without a bias the logits themselves give the order, in
// 32 bits exactly.  With one (or ranks of groups by two scores), c = s + bias
// is formed in f32 first, and a row in which two scores that meet at a place
// of the order lie closer than f32 can tell is ranked again in 64 bits.  That
// is rare (two scores within 40 * 2^-24 of each other), so the order of 64 bits
// costs what the order of f32 does.
#include <math.h>

#include "model_common.cuh"

namespace so2 {

struct RouteArgs {
  int K, top_k, n_groups, top_groups, group_top, per;
  int softmax, renorm;
  float scale;
};

__device__ __forceinline__ uint64_t order_key(double c, bool dead) {
  if (dead || c == -INFINITY) return 0;
  if (c != c) return 1;
  const long long b = __double_as_longlong(c + 0.0);  // -0 to +0
  return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float sigmoid_f(float x) { return 1.f / (1.f + expf(-x)); }

constexpr int ROUTE_WARPS = 4;

// The order of a row by scores (or logits) in 64 bits: rank[e] is K for the first expert
// down to 1, or 0 if it may not be chosen.  All lanes of the warp call; keys
// (K + n_groups words) and rank (K words) are the warp's shared memory, and
// nothing of the caller's is passed in registers, so that the usual path does
// not pay for this one.
template <bool BY_SCORE, typename T>
__device__ __noinline__ void rank_in_64_bits(const RouteArgs &a, const T *__restrict__ row, float m0,
                                             const float *__restrict__ bias, uint64_t *keys,
                                             uint32_t *rank) {
  const int lane = threadIdx.x & 31;
  uint64_t *gkeys = keys + a.K;
  double *cs = reinterpret_cast<double *>(keys);
  __syncwarp();
  double z = 0.0;
  if (BY_SCORE && a.softmax) {
    for (int e = lane; e < a.K; e += 32) z += exp((double)to_f32(row[e]) - m0);
    z = warp_sum(z);
  }
  for (int e = lane; e < a.K; e += 32) {
    const double x = to_f32(row[e]);
    double c = x;
    if (BY_SCORE) c = a.softmax ? exp(x - m0) / z : 1.0 / (1.0 + exp(-x));
    if (bias) c += bias[e];
    cs[e] = x == -INFINITY ? -INFINITY : c;
  }
  __syncwarp();
  const bool grouped = a.top_groups < a.n_groups;
  for (int g = lane; grouped && g < a.n_groups; g += 32) {
    double b0 = -INFINITY, b1 = -INFINITY;
    bool nan = false;
    for (int j = 0; j < a.per; ++j) {
      const double c = cs[g * a.per + j];
      if (c != c) nan = true;
      else if (c > b0) b1 = b0, b0 = c;
      else if (c > b1) b1 = c;
    }
    // NaN ranks below every number: it counts where too few numbers are left
    const bool two = a.group_top > 1;
    const bool few = b0 == -INFINITY || (two && b1 == -INFINITY);
    const double s = two && b1 != -INFINITY ? b0 + b1 : b0;
    gkeys[g] = nan && few ? 1 : order_key(s, b0 == -INFINITY);
  }
  __syncwarp();
  // keys in place of the scores, 0 outside the groups that stay
  for (int e = lane; e < a.K; e += 32) {
    const double x = to_f32(row[e]);
    uint64_t k = order_key(bias ? cs[e] : x, x == -INFINITY);
    if (grouped) {
      const int g = e / a.per;
      int before = 0;
      for (int h = 0; h < a.n_groups; ++h)
        before += gkeys[h] > gkeys[g] || (gkeys[h] == gkeys[g] && h < g);
      if (before >= a.top_groups) k = 0;
    }
    keys[e] = k;
  }
  __syncwarp();
  for (int e = lane; e < a.K; e += 32) {
    const uint64_t k = keys[e];
    int before = 0;
    for (int h = 0; h < a.K; ++h) before += keys[h] > k || (keys[h] == k && h < e);
    rank[e] = k ? (uint32_t)(a.K - before) : 0;
  }
  __syncwarp();
}

// 32-bit keys in the order of c; equal floats (+0 and -0 too) have equal keys.
__device__ __forceinline__ uint32_t order_key32(float c, bool dead = false) {
  const int b = __float_as_int(c + 0.f);
  const uint32_t k = (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
  return dead || c == -INFINITY ? 0u : c != c ? 1u : k;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// How far apart two f32 selection scores of a row have to be for their order to
// hold in 64 bits, relative to the row's largest score or |c|.  In units of
// u = 2^-24 of that, with expf within 2 steps (4 u):
// * each c on its own: the argument's rounding |y| e^-|y| <= 0.4, expf 4, the
//   division 1, c = s + bias 1: 6.4; a sigmoid's expf 4, sum 1, division 1, c 1: 7;
// * all softmax scores of a row together, by z: the terms' arguments 4.4 at most
//   (the solution v of v e^v = 1023 / e), expf 4, sum_exp 14, 1 / z 1: 23.4, which
//   moves a difference of two by no more than that once.
// So two of them are right beyond 23.4 + 2 * 6.4 = 36.2, and two groups, whose
// ranks add two scores and round by 2, beyond 2 * 36.2 + 4 = 76.4 = less than 2 * 40.
constexpr float ROUTE_NEAR = 40.f / (1 << 24);
// And in absolute terms, for scores that f32 loses: a sigmoid is 0 where e^-x
// overflows, below 2^-128, and denormal ones keep steps of 2^-149.
constexpr float ROUTE_LEAST = 1.f / (1ull << 63) / (1ull << 62);  // 2^-125

// A lane's share of softmax's denominator, in four sums side by side: at most
// 9 roundings for 32 values, and the 5 of the warp's tree.  (One sum would
// lose up to 31 terms just below half a step of the first.)
template <int NPL>
__device__ __forceinline__ float sum_exp(const float (&x)[NPL], float m0) {
  constexpr int P = NPL < 4 ? NPL : 4;
  float z[P];
#pragma unroll
  for (int i = 0; i < P; ++i) z[i] = expf(x[i] - m0);
#pragma unroll
  for (int i = P; i < NPL; ++i) z[i % P] += expf(x[i] - m0);
  if constexpr (P == 1) return z[0];
  else if constexpr (P == 2) return z[0] + z[1];
  else return (z[0] + z[1]) + (z[2] + z[3]);
}

// Shared memory per warp, in words of 8 bytes: the chosen experts (i32); by
// score also K + n_groups 64-bit keys and K 32-bit ranks, and the groups' f32
// scores and keys, which come before those, fit there.
__host__ __device__ constexpr int route_words(int K, int n_groups, int top_k, bool by_score) {
  return (top_k + 1) / 2 + (by_score ? K + n_groups + (K + 1) / 2 : n_groups > 1 ? (K + n_groups + 1) / 2 : 0);
}

// NPL consecutive experts' values of a row, those of lane `lane`; -inf beyond K.
template <int NPL, typename T>
__device__ __forceinline__ void load_experts(const T *__restrict__ row, int K, bool vec,
                                             float (&x)[NPL]) {
  const int e0 = (threadIdx.x & 31) * NPL;
  constexpr int V = NPL * sizeof(T) <= 16 ? NPL : 16 / (int)sizeof(T);
  if (NPL > 1 && vec) {
#pragma unroll
    for (int i = 0; i < NPL; i += V) {
      if (e0 + i < K) {
        if constexpr (V == 4 || V == 8) {
          float r[V];
          load_vec<V>(row + e0 + i, r);
#pragma unroll
          for (int v = 0; v < V; ++v) x[i + v] = r[v];
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) x[i + v] = to_f32(row[e0 + i + v]);
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[i + v] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) x[i] = e0 + i < K ? to_f32(row[e0 + i]) : -INFINITY;
  }
}

// Whether rows of K values can be read in the vectors of load_experts.
template <int NPL, typename T>
bool expert_vectors(int K, const T *logits) {
  constexpr int V = NPL * sizeof(T) <= 16 ? NPL : 16 / (int)sizeof(T);
  return K % V == 0 && aligned_to(logits, V * sizeof(T));
}

// NPL experts a lane: e = NPL lane + i, so that of equal keys the lowest lane
// holds the lowest index.  A round of the selection is one reduction of the
// lanes' largest keys and one vote for its lane, which notes its expert in
// shared memory and moves on; up to four keys a lane are sorted beforehand and
// shifted as they are taken, more are looked through in each round.  The
// instructions bound this kernel, not memory.
template <int NPL, bool BY_SCORE, typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
    k_route(RouteArgs a, int64_t n, const T *__restrict__ logits, bool vec,
            const float *__restrict__ bias, float *__restrict__ weights, int *__restrict__ index,
            int *__restrict__ counts) {
  extern __shared__ uint64_t sm[];
  constexpr bool SORTED = NPL <= 4;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int words = route_words(a.K, a.n_groups, a.top_k, BY_SCORE);
  int *chosen = reinterpret_cast<int *>(sm + w * words);
  uint64_t *keys = sm + w * words + (a.top_k + 1) / 2;
  float *cs = reinterpret_cast<float *>(keys);
  uint32_t *rank = reinterpret_cast<uint32_t *>(keys + a.K + a.n_groups);
  int *hist = reinterpret_cast<int *>(sm + ROUTE_WARPS * words);
  if (counts) {
    for (int e = threadIdx.x; e < a.K; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const bool grouped = a.top_groups < a.n_groups;
  const int64_t step = (int64_t)gridDim.x * ROUTE_WARPS;
  int64_t t = blockIdx.x * (int64_t)ROUTE_WARPS + w;
  float x[NPL], xn[NPL];
  if (t < n) load_experts<NPL>(logits + t * a.K, a.K, vec, xn);
  for (; t < n; t += step) {
    const T *row = logits + t * a.K;
#pragma unroll
    for (int i = 0; i < NPL; ++i) x[i] = xn[i];
    if (t + step < n)  // the next row's logits, under this row's work
      load_experts<NPL>(logits + (t + step) * a.K, a.K, vec, xn);
    float m0 = 0.f, z = 1.f;
    if (a.softmax && (BY_SCORE || !a.renorm)) {
      m0 = x[0];
#pragma unroll
      for (int i = 1; i < NPL; ++i) m0 = fmaxf(m0, x[i]);
      m0 = warp_max(m0);
      if (m0 == -INFINITY) m0 = 0.f;  // a row without any expert
      z = warp_sum(sum_exp(x, m0));
    }
    uint32_t key[NPL];
    float size = 0.f;  // BY_SCORE: the scores' largest magnitude, for what counts as near
    bool again = false;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane * NPL + i;
      const bool dead = x[i] == -INFINITY;  // beyond K too
      float c = x[i];
      if (BY_SCORE) {
        const float s = a.softmax ? expf(x[i] - m0) / z : sigmoid_f(x[i]);
        c = s + (bias && e < a.K ? bias[e] : 0.f);
        again |= !dead && c != c;  // NaN: let 64 bits sort it out
        // (a score counts where the bias takes its expert out too: the others' errors are relative to it)
        if (!dead) size = fmaxf(size, c == -INFINITY ? s : fmaxf(s, fabsf(c)));
      }
      key[i] = order_key32(bias || !BY_SCORE ? c : x[i], dead);
      if (grouped && e < a.K) cs[e] = dead ? -INFINITY : c;
    }
    float tol = 0.f;
    if (BY_SCORE) tol = warp_max(size) * ROUTE_NEAR + ROUTE_LEAST;
    if (grouped) {
      __syncwarp();
      uint32_t *gk = reinterpret_cast<uint32_t *>(cs + a.K);
      for (int g = lane; g < a.n_groups; g += 32) {
        float b0 = -INFINITY, b1 = -INFINITY;
        bool nan = false;
        for (int j = 0; j < a.per; ++j) {
          const float c = cs[g * a.per + j];
          nan |= c != c;
          b1 = fmaxf(b1, fminf(b0, c));
          b0 = fmaxf(b0, c);
        }
        // (fmaxf and fminf leave a NaN out; by score, 64 bits look at the row)
        uint32_t k = order_key32(a.group_top > 1 && b1 != -INFINITY ? b0 + b1 : b0, b0 == -INFINITY);
        if (nan && b0 == -INFINITY) k = 1;
        gk[g] = k;
      }
      __syncwarp();
      uint32_t floor_key = 0xffffffffu, next_key = 0;  // the last group that stays, the first that does not
      for (int g = lane; g < a.n_groups; g += 32) {
        const uint32_t k = gk[g];
        int before = 0;
        for (int h = 0; h < a.n_groups; ++h) before += gk[h] > k || (gk[h] == k && h < g);
        if (before == a.top_groups - 1) floor_key = k;
        if (before == a.top_groups) next_key = k;
        cs[g] = before < a.top_groups ? 1.f : 0.f;  // (the scores are not read any more)
      }
      __syncwarp();
      if (BY_SCORE) {
        floor_key = __reduce_min_sync(0xffffffffu, floor_key);
        next_key = __reduce_max_sync(0xffffffffu, next_key);
        if (next_key > 1) again |= !(key_value(floor_key) - key_value(next_key) > 2.f * tol);
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane * NPL + i;
        if (e < a.K && cs[e / a.per] == 0.f) key[i] = 0;
      }
      __syncwarp();
    }
    again = BY_SCORE && __any_sync(0xffffffffu, again);

    if (a.top_k == a.K) {  // nothing to select: slot e is expert e
      if (again) {  // (only to know which experts may not be chosen)
        rank_in_64_bits<true>(a, row, m0, bias, keys, rank);
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = lane * NPL + i < a.K ? rank[lane * NPL + i] : 0;
      }
      float mc = -INFINITY, total = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (key[i]) mc = fmaxf(mc, x[i]);
      mc = warp_max(mc);
      float s[NPL];
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        s[i] = 0.f;
        if (key[i])
          s[i] = !a.softmax ? sigmoid_f(x[i]) : a.renorm ? expf(x[i] - mc) : expf(x[i] - m0) / z;
        total += s[i];
      }
      if (a.renorm) total = warp_sum(total);
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane * NPL + i;
        if (e >= a.K) continue;
        float v = s[i];
        if (a.renorm) v = total == 0.f ? 0.f : v / total;
        weights[t * a.K + e] = key[i] ? v * a.scale : 0.f;
        index[t * a.K + e] = key[i] ? e : -1;
        if (counts && key[i]) atomicAdd(&hist[e], 1);
      }
      continue;
    }

    for (;;) {
      if (again) {
        rank_in_64_bits<true>(a, row, m0, bias, keys, rank);
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = lane * NPL + i < a.K ? rank[lane * NPL + i] : 0;
      }
      const bool look = BY_SCORE && !again && bias;
      uint32_t k[NPL];
      int id[NPL];
#pragma unroll
      for (int i = 0; i < NPL; ++i) k[i] = key[i], id[i] = lane * NPL + i;
      if constexpr (SORTED) {  // falling, equal keys by index: insertion
#pragma unroll
        for (int p = 1; p < NPL; ++p)
#pragma unroll
          for (int q = p; q > 0; --q) {
            const bool swap = k[q] > k[q - 1];
            const uint32_t kt = k[q];
            const int it = id[q];
            k[q] = swap ? k[q - 1] : kt, id[q] = swap ? id[q - 1] : it;
            k[q - 1] = swap ? kt : k[q - 1], id[q - 1] = swap ? it : id[q - 1];
          }
      }
      uint32_t prev = 0;
      int j = 0;
      bool near = false;
      for (; j < a.top_k; ++j) {
        uint32_t lk = k[0];
        int li = id[0];
        if constexpr (!SORTED) {
#pragma unroll
          for (int i = 1; i < NPL; ++i)
            if (k[i] > lk) lk = k[i], li = id[i];
        }
        const uint32_t bk = __reduce_max_sync(0xffffffffu, lk);
        if (bk == 0) break;  // uniform: nothing is left
        const int from = __ffs(__ballot_sync(0xffffffffu, lk == bk)) - 1;
        if (lane == from) {
          chosen[j] = li;
          if constexpr (SORTED) {
#pragma unroll
            for (int i = 0; i + 1 < NPL; ++i) k[i] = k[i + 1], id[i] = id[i + 1];
            k[NPL - 1] = 0;
          } else {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
              if (li == id[i]) k[i] = 0;
          }
        }
        if (BY_SCORE) {
          // scores this close may stand the other way round in 64 bits, unless
          // they come from the same numbers
          if (look && j > 0 && !(key_value(prev) - key_value(bk) > tol)) {
            __syncwarp();
            const int e = chosen[j], f = chosen[j - 1];
            near |= !(to_f32(row[e]) == to_f32(row[f]) && bias[e] == bias[f]);
          }
          prev = bk;
        }
      }
      for (j += lane; j < a.top_k; j += 32) chosen[j] = -1;
      __syncwarp();
      if (look && prev != 0) {  // the last one chosen and those left over
        bool close = false;
#pragma unroll
        for (int i = 0; i < NPL; ++i) close |= k[i] != 0 && !(key_value(prev) - key_value(k[i]) > tol);
        if (__any_sync(0xffffffffu, close)) {
          const int f = chosen[a.top_k - 1];  // (used: some are left over)
          const float px = f >= 0 ? to_f32(row[f]) : 0.f, pb = f >= 0 ? bias[f] : 0.f;
#pragma unroll
          for (int i = 0; i < NPL; ++i)
            if (k[i] != 0 && !(key_value(prev) - key_value(k[i]) > tol))
              near |= !(to_f32(row[id[i]]) == px && bias[id[i]] == pb);
          near = __any_sync(0xffffffffu, near);
        }
      }
      if (!near) break;
      again = true;
    }
    // weights: lane j takes the slots j, j + 32, ...
    float mc = 0.f, total = 0.f, v0 = 0.f, s0 = 0.f;  // v0, s0: of the first one
    const int e0 = lane < a.top_k ? chosen[lane] : -1;
    if (e0 >= 0) v0 = to_f32(row[e0]);
    if (a.softmax && a.renorm) {
      mc = e0 >= 0 ? v0 : -INFINITY;
      if (!BY_SCORE) {
        mc = __shfl_sync(0xffffffffu, mc, 0);  // the largest logit came first
      } else {
        for (int j = lane + 32; j < a.top_k; j += 32)
          if (chosen[j] >= 0) mc = fmaxf(mc, to_f32(row[chosen[j]]));
        mc = warp_max(mc);
      }
    }
    const float iz = a.softmax && !a.renorm ? 1.f / z : 1.f;
    auto score = [&](float v) {
      return !a.softmax ? sigmoid_f(v) : a.renorm ? expf(v - mc) : expf(v - m0) * iz;
    };
    if (e0 >= 0) s0 = score(v0);
    float f = a.scale;
    if (a.renorm) {
      total = s0;
      for (int j = lane + 32; j < a.top_k; j += 32)
        if (chosen[j] >= 0) total += score(to_f32(row[chosen[j]]));
      total = warp_sum(total);
      f = total == 0.f ? 0.f : a.scale / total;
    }
    for (int j = lane; j < a.top_k; j += 32) {
      const int e = j == lane ? e0 : chosen[j];
      if (counts && e >= 0) atomicAdd(&hist[e], 1);
      weights[t * a.top_k + j] = e < 0 ? 0.f : (j == lane ? s0 : score(to_f32(row[e]))) * f;
      index[t * a.top_k + j] = e;
    }
    __syncwarp();
  }
  if (counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.K; e += blockDim.x) {
      if (gridDim.x == 1) counts[e] = hist[e];
      else if (hist[e]) atomicAdd(&counts[e], hist[e]);
    }
  }
}

// ---- at most eight slots of at most 256 experts -----------------------------------
// A group of 2^SHIFT lanes a row, NPL experts a lane, so a warp takes several
// rows.  The expert's index replaces the low bits of its key, which makes the
// words distinct, ties in index order, and an exchange of a sorting network
// two instructions: each lane sorts its words, and SHIFT butterfly steps merge
// the lanes' best eight.  Keys that differ only in the replaced bits (2^-15 of
// a value at 256 experts) and, by score, scores that f32 cannot tell apart
// send the row to rank_in_64_bits.  Of 200,000 rows of normally distributed
// f32 logits the first were 0.07 % (8 of 128) and 0.2 % (8 of 256).  A bias of
// the type's lowest value makes all scores near beside it, so that every row
// goes there: 20,000 x 64, top 6, 30 -> 69 us, 20,000 x 128, top 8, 45 -> 171
// (-inf takes experts out without that).
__device__ __forceinline__ void exchange(uint32_t &a, uint32_t &b) {
  const uint32_t hi = a > b ? a : b;
  b = a > b ? b : a;
  a = hi;
}
// The order of numbers (NaN is looked for apart); -inf is the last below WORD_LIVE.
__device__ __forceinline__ uint32_t plain_key32(float c) {
  const int b = __float_as_int(c + 0.f);
  return (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}
constexpr uint32_t WORD_LIVE = 0x00800000u;  // the word of an expert that may be chosen is at least this
// Falling order of eight words that rise and fall, or fall and rise.
__device__ __forceinline__ void sort_bitonic8(uint32_t (&l)[8]) {
#pragma unroll
  for (int d = 4; d; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) exchange(l[i], l[i + d]);
}
// Falling order of N words (Batcher's odd-even merge sort).
template <int N>
__device__ __forceinline__ void sort_words(uint32_t *l) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p))
            exchange(l[i + j], l[i + j + k]);
}
// The eight best of two sorted lists, sorted, into the first.
__device__ __forceinline__ void merge8(uint32_t (&l)[8], const uint32_t (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) l[i] = l[i] > o[7 - i] ? l[i] : o[7 - i];
  sort_bitonic8(l);
}

__host__ __device__ constexpr int route_top_words(int K, int n_groups, int rows) {
  const int f32s = n_groups > 1 ? (rows * (K + n_groups) + 1) / 2 : 0;
  const int slow = K + n_groups + (K + 1) / 2;  // rank_in_64_bits
  return (f32s > slow ? f32s : slow) + rows * 4;
}

template <int SHIFT, int NPL, bool BY_SCORE, typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
    k_route_top(RouteArgs a, int64_t n, const T *__restrict__ logits, bool vec,
                const float *__restrict__ bias, float *__restrict__ weights,
                int *__restrict__ index, int *__restrict__ counts) {
  extern __shared__ uint64_t sm[];
  constexpr int LANES = 1 << SHIFT, ROWS = 32 >> SHIFT, IDX = LANES * NPL;  // indices of a word
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int sub = lane & (LANES - 1), r = lane >> SHIFT;
  const int words = route_top_words(a.K, a.n_groups, ROWS);
  uint64_t *keys = sm + w * words;
  int *chosen = reinterpret_cast<int *>(keys + words - ROWS * 4);  // [ROWS][8]
  float *cs = reinterpret_cast<float *>(keys) + r * (a.K + a.n_groups);
  uint32_t *rank = reinterpret_cast<uint32_t *>(keys + a.K + a.n_groups);
  int *hist = reinterpret_cast<int *>(sm + ROUTE_WARPS * words);
  if (counts) {
    for (int e = threadIdx.x; e < a.K; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  auto row_max = [&](float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  };
  auto row_sum = [&](float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  const unsigned row_lanes = (LANES == 32 ? 0xffffffffu : (1u << (LANES & 31)) - 1) << (r * LANES);
  auto row_any = [&](bool v) { return (__ballot_sync(0xffffffffu, v) & row_lanes) != 0; };
  const bool grouped = a.top_groups < a.n_groups;
  constexpr int V = NPL * sizeof(T) <= 16 ? NPL : 16 / (int)sizeof(T);
  auto load = [&](int64_t t, float(&x)[NPL]) {
    const T *p = logits + t * a.K;
#pragma unroll
    for (int i = 0; i < NPL; i += V) {
      const int e = sub * NPL + i;
      if (vec && t < n && e < a.K) {
        if constexpr (V >= 4) {
          float q[V];
          load_vec<V>(p + e, q);
#pragma unroll
          for (int v = 0; v < V; ++v) x[i + v] = q[v];
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[i + v] = t < n && e + v < a.K ? to_f32(p[e + v]) : -INFINITY;
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * ROUTE_WARPS * ROWS;
  int64_t t0 = (blockIdx.x * (int64_t)ROUTE_WARPS + w) * ROWS;
  float x[NPL], xn[NPL];
  load(t0 + r, xn);
  for (; t0 < n; t0 += step) {
    const int64_t t = t0 + r;
    const T *row = logits + t * a.K;
#pragma unroll
    for (int i = 0; i < NPL; ++i) x[i] = xn[i];
    load(t + step, xn);
    float m0 = 0.f, z = 1.f;
    if (a.softmax && (BY_SCORE || !a.renorm)) {
      m0 = x[0];
#pragma unroll
      for (int i = 1; i < NPL; ++i) m0 = fmaxf(m0, x[i]);
      m0 = row_max(m0);
      if (m0 == -INFINITY) m0 = 0.f;
      z = row_sum(sum_exp(x, m0));
    }
    // words, and by score the scores for a second look at what is near
    uint32_t l[NPL];
    float c[NPL];
    float size = 0.f;
    bool again = false;
    const float iz = BY_SCORE && a.softmax ? 1.f / z : 1.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = sub * NPL + i;
      const bool dead = x[i] == -INFINITY;
      c[i] = x[i];
      if (BY_SCORE) {
        const float s = a.softmax ? expf(x[i] - m0) * iz : sigmoid_f(x[i]);
        c[i] = s + (bias && e < a.K ? bias[e] : 0.f);
        if (dead) c[i] = -INFINITY;
        else size = fmaxf(size, c[i] == -INFINITY ? s : fmaxf(s, fabsf(c[i])));
      }
      again |= c[i] != c[i];  // NaN is left to the second look
      // (-inf maps below WORD_LIVE by itself)
      float v = bias || !BY_SCORE ? c[i] : x[i];
      if (BY_SCORE && !bias && c[i] == -INFINITY) v = -INFINITY;
      l[i] = (plain_key32(v) & ~(uint32_t)(IDX - 1)) | (uint32_t)(IDX - 1 - e);
      if (grouped && e < a.K) cs[e] = c[i];
    }
    float tol = 0.f;
    if (BY_SCORE) tol = row_max(size) * ROUTE_NEAR + ROUTE_LEAST;
    if (grouped) {
      __syncwarp();
      uint32_t *gk = reinterpret_cast<uint32_t *>(cs + a.K);
      for (int g = sub; g < a.n_groups; g += LANES) {
        float b0 = -INFINITY, b1 = -INFINITY;
        for (int j = 0; j < a.per; ++j) {
          const float v = cs[g * a.per + j];
          b1 = fmaxf(b1, fminf(b0, v));
          b0 = fmaxf(b0, v);
        }
        gk[g] = order_key32(a.group_top > 1 && b1 != -INFINITY ? b0 + b1 : b0, b0 == -INFINITY);
      }
      __syncwarp();
      uint32_t floor_key = 0xffffffffu, next_key = 0;  // the last group that stays, the first that does not
      for (int g = sub; g < a.n_groups; g += LANES) {
        const uint32_t k = gk[g];
        int before = 0;
        for (int h = 0; h < a.n_groups; ++h) before += gk[h] > k || (gk[h] == k && h < g);
        if (before == a.top_groups - 1) floor_key = k;
        if (before == a.top_groups) next_key = k;
        cs[g] = before < a.top_groups ? 1.f : 0.f;  // (the scores are not read any more)
      }
      __syncwarp();
      if (BY_SCORE) {
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) {
          const uint32_t f = __shfl_xor_sync(0xffffffffu, floor_key, o);
          const uint32_t m = __shfl_xor_sync(0xffffffffu, next_key, o);
          floor_key = f < floor_key ? f : floor_key;
          next_key = m > next_key ? m : next_key;
        }
        if (next_key > 1) again |= !(key_value(floor_key) - key_value(next_key) > 2.f * tol);
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = sub * NPL + i;
        if (e < a.K && cs[e / a.per] == 0.f) l[i] = 0, c[i] = -INFINITY;
      }
      __syncwarp();
    }
    // the row's eight best words, in every lane of the group
    uint32_t top[8];
    if constexpr (NPL == 16) {
      uint32_t o[8];
      uint32_t q[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) q[i] = l[i];
      sort_words<8>(q);
      sort_words<8>(q + 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = q[i], o[i] = q[8 + i];
      merge8(top, o);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = i < NPL ? l[i < NPL ? i : 0] : 0;
      sort_words<(NPL < 8 ? NPL : 8)>(top);
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) {
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __shfl_xor_sync(0xffffffffu, top[i], d);
      merge8(top, o);
    }
    // slot `sub` of the row, its logit and (by score) its c
    uint32_t word = 0, last = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i == sub) word = top[i];
      if (i == a.top_k - 1) last = top[i];
    }
    int e = sub < a.top_k && word >= WORD_LIVE ? IDX - 1 - (int)(word & (IDX - 1)) : -1;
    float v = e >= 0 ? to_f32(row[e]) : 0.f;
    const float b = BY_SCORE && bias && e >= 0 ? bias[e] : 0.f;
    {
      // neighbours whose words do not tell them apart, unless they are equal
      const uint32_t wn = __shfl_down_sync(0xffffffffu, word, 1);
      const float vn = __shfl_down_sync(0xffffffffu, v, 1), bn = __shfl_down_sync(0xffffffffu, b, 1);
      const uint32_t bits = ~(uint32_t)(IDX - 1);
      if (sub + 1 < a.top_k && e >= 0 && wn >= WORD_LIVE) {
        bool close = (word & bits) == (wn & bits);
        if (BY_SCORE && bias) close |= !(key_value(word & bits) - key_value((wn & bits) | (IDX - 1)) > tol);
        again |= close && !(v == vn && b == bn);
      }
      // the last one chosen and those left over
      const int from = r * LANES + a.top_k - 1;
      const float vl = __shfl_sync(0xffffffffu, v, from), bl = __shfl_sync(0xffffffffu, b, from);
      const bool scored = BY_SCORE && bias;
      const float cut = last >= WORD_LIVE ? key_value(last & bits) - tol : INFINITY;
      // a word less than IDX below the last one: the same bits, or nearly
      auto near_last = [&](int i) {
        return last - 1 - l[i] < IDX || (scored && l[i] < last && l[i] >= WORD_LIVE && !(c[i] < cut));
      };
      bool close = false;
#pragma unroll
      for (int i = 0; i < NPL; ++i) close |= near_last(i);
      if (close && last >= WORD_LIVE) {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (near_last(i) && l[i] >= WORD_LIVE)
            again |= !(x[i] == vl && (!scored || bias[sub * NPL + i] == bl));
      }
    }
    again = row_any(again) && t < n;
    for (unsigned m = __ballot_sync(0xffffffffu, again && sub == 0); m; m &= m - 1) {
      const int from = __ffs(m) - 1, rr = from >> SHIFT;
      const float mr = __shfl_sync(0xffffffffu, m0, from);
      rank_in_64_bits<BY_SCORE>(a, logits + (t0 + rr) * a.K, mr, bias, keys, rank);
      if (lane < 8) chosen[rr * 8 + lane] = -1;
      __syncwarp();
      for (int q = lane; q < a.K; q += 32)
        if (rank[q] != 0 && a.K - (int)rank[q] < a.top_k) chosen[rr * 8 + a.K - rank[q]] = q;
      __syncwarp();
    }
    if (again) {
      e = sub < a.top_k ? chosen[r * 8 + sub] : -1;
      v = e >= 0 ? to_f32(row[e]) : 0.f;
    }
    float s = 0.f;
    if (a.softmax && a.renorm) {
      const float mc = row_max(e >= 0 ? v : -INFINITY);
      if (e >= 0) s = expf(v - mc);
    } else if (e >= 0) {
      s = a.softmax ? expf(v - m0) / z : sigmoid_f(v);
    }
    if (a.renorm) {
      const float total = row_sum(s);
      s = total == 0.f ? 0.f : s / total;
    }
    if (t < n && sub < a.top_k) {
      weights[t * a.top_k + sub] = s * a.scale;
      index[t * a.top_k + sub] = e;
      if (counts && e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncwarp();
  }
  if (counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.K; e += blockDim.x) {
      if (gridDim.x == 1) counts[e] = hist[e];
      else if (hist[e]) atomicAdd(&counts[e], hist[e]);
    }
  }
}

// FULL: softmax without renormalisation, whose gradient reaches every logit;
// otherwise it reaches the chosen ones alone and the others are not read.
// Shared memory per warp: the row's gradient [32 NPL].
template <int NPL, bool FULL, typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
    k_route_grad(RouteArgs a, int64_t n, const T *__restrict__ logits, bool vec,
                 const int *__restrict__ index, const float *__restrict__ gw,
                 float *__restrict__ grad, bool vec_out) {
  __shared__ __align__(16) float rows[ROUTE_WARPS][32 * NPL];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float *gs = rows[w];
  constexpr int V = NPL >= 4 ? 4 : 1;
  const int64_t step = (int64_t)gridDim.x * ROUTE_WARPS;
  int64_t t = blockIdx.x * (int64_t)ROUTE_WARPS + w;
  // A lane's first slot, read ahead: its expert and gradient two rows, its
  // logit (and by FULL the row) one row before they are used, since the loads
  // depend on one another and the work between them is short.
  auto first = [&](int64_t r, int &e, float &g) {
    e = -1, g = 0.f;
    if (r < n && lane < a.top_k) {
      e = index[r * a.top_k + lane];
      g = gw[r * a.top_k + lane];
      if (e < 0 || e >= a.K) e = -1, g = 0.f;
    }
  };
  int e1, e2;
  float g1, g2, v1 = 0.f, xn[NPL];
  first(t, e1, g1);
  first(t + step, e2, g2);
  if (e1 >= 0) v1 = to_f32(logits[t * a.K + e1]);
  if (FULL && t < n) load_experts<NPL>(logits + t * a.K, a.K, vec, xn);
  for (; t < n; t += step) {
    const T *row = logits + t * a.K;
    auto slot = [&](int j, int &e, float &v, float &g) {
      e = j < a.top_k ? index[t * a.top_k + j] : -1;
      g = j < a.top_k ? gw[t * a.top_k + j] : 0.f;
      if (e < 0 || e >= a.K) e = -1, g = 0.f;
      v = e >= 0 ? to_f32(row[e]) : 0.f;
    };
    const int e0 = e1;  // slots beyond 32 are read below
    const float v0 = v1, g0 = g1;
    float x[NPL];
    if (FULL) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) x[i] = xn[i];
    }
    e1 = e2, g1 = g2, v1 = 0.f;
    if (e1 >= 0) v1 = to_f32(logits[(t + step) * a.K + e1]);
    first(t + 2 * step, e2, g2);
    if (FULL && t + step < n) load_experts<NPL>(logits + (t + step) * a.K, a.K, vec, xn);
    float m0 = 0.f, z = 1.f;
#pragma unroll
    for (int i = 0; i < NPL; i += V) {
      float zero[V] = {};
      store_vec<V>(gs + i * 32 + lane * V, zero);
    }
    if (FULL) {
      m0 = x[0];
#pragma unroll
      for (int i = 1; i < NPL; ++i) m0 = fmaxf(m0, x[i]);
      m0 = warp_max(m0);
      if (m0 == -INFINITY) m0 = 0.f;
      z = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        x[i] = expf(x[i] - m0);
        z += x[i];
      }
      z = warp_sum(z);
    }
    // renormalised: the chosen scores over their sum, and its product with the gradient
    float mc = 0.f, s0 = 0.f, p0 = 0.f, total = 1.f, dot = 0.f;
    auto score = [&](float v) { return a.softmax ? expf(v - mc) : sigmoid_f(v); };
    if (a.renorm) {
      if (a.softmax) {
        mc = e0 >= 0 ? v0 : -INFINITY;
        for (int j = lane + 32; j < a.top_k; j += 32) {
          int e;
          float v, g;
          slot(j, e, v, g);
          if (e >= 0) mc = fmaxf(mc, v);
        }
        mc = warp_max(mc);
        if (mc == -INFINITY) mc = 0.f;  // no slot in use
      }
      s0 = e0 < 0 ? 0.f : score(v0);
      total = s0;
      for (int j = lane + 32; j < a.top_k; j += 32) {
        int e;
        float v, g;
        slot(j, e, v, g);
        if (e >= 0) total += score(v);
      }
      total = warp_sum(total);
      if (total == 0.f) total = INFINITY;  // such scores weigh 0
      p0 = s0 / total;  // (1 for a single slot, whose gradient is then 0)
      dot = g0 * p0;
      for (int j = lane + 32; j < a.top_k; j += 32) {
        int e;
        float v, g;
        slot(j, e, v, g);
        if (e >= 0) dot += g * (score(v) / total);
      }
      dot = warp_sum(dot);
    }
    // Gradients of the scores (sigmoid, renormalised: of the logits), 32 slots
    // at a time.  An expert named twice, which its own tag then shows, adds up
    // in slot order.
    for (int j = 0; j < a.top_k; j += 32) {
      int e = e0;
      float v = v0, g = g0;
      if (j > 0) slot(j + lane, e, v, g);
      float d = (g - dot) * a.scale;
      if (a.softmax) {
        if (a.renorm) d *= j == 0 ? p0 : score(v) / total;
      } else {
        d *= sigmoid_f(v) * sigmoid_f(-v) / total;
      }
      __syncwarp();
      if (j == 0) {
        if (e >= 0) gs[e] = __int_as_float(lane);
        __syncwarp();
        const bool twice = e >= 0 && __float_as_int(gs[e]) != lane;
        const bool any = __any_sync(0xffffffffu, twice);
        if (e >= 0) gs[e] = any ? 0.f : d;
        __syncwarp();
        if (any)
          for (int l = 0; l < 32; ++l) {
            if (lane == l && e >= 0) gs[e] += d;
            __syncwarp();
          }
      } else {
        for (int l = 0; l < 32; ++l) {
          if (lane == l && e >= 0) gs[e] += d;
          __syncwarp();
        }
      }
    }
    __syncwarp();
    float sdot = 0.f;
    if (FULL) {
      const float iz = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        x[i] *= iz;  // the scores
        const float g = gs[lane * NPL + i];
        if (g != 0.f) sdot += x[i] * g;
      }
      sdot = warp_sum(sdot);
    }
    auto value = [&](int i, float g) { return !FULL ? g : z == 0.f ? 0.f : x[i] * (g - sdot); };
    if (vec_out) {
#pragma unroll
      for (int i = 0; i < NPL; i += V) {
        const int e = FULL ? lane * NPL + i : i * 32 + lane * V;
        if (e >= a.K) continue;
        float r[V];
        load_vec<V>(gs + e, r);
#pragma unroll
        for (int v = 0; v < V; ++v) r[v] = value(i + v, r[v]);
        store_vec<V>(grad + t * a.K + e, r);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = FULL ? lane * NPL + i : lane + 32 * i;
        if (e < a.K) grad[t * a.K + e] = value(i, gs[e]);
      }
    }
    __syncwarp();
  }
}

// The same without FULL and with at most 32 slots: a group of 2^SHIFT lanes a
// row, one slot a lane, so a warp takes 32 >> SHIFT consecutive rows, builds
// their gradients in shared memory (K each) and stores them in one piece.
template <int SHIFT, typename T>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
    k_route_grad_slots(RouteArgs a, int64_t n, const T *__restrict__ logits,
                       const int *__restrict__ index, const float *__restrict__ gw,
                       float *__restrict__ grad, bool vec) {
  extern __shared__ __align__(16) float gsm[];
  constexpr int LANES = 1 << SHIFT, ROWS = 32 >> SHIFT;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int sub = lane & (LANES - 1), r = lane >> SHIFT;
  const int size = (ROWS * a.K + 3) & ~3;
  float *gs = gsm + w * size;
  float *mine = gs + r * a.K;
  auto sum = [&](float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  const int64_t step = (int64_t)gridDim.x * ROUTE_WARPS * ROWS;
  int64_t t0 = (blockIdx.x * (int64_t)ROUTE_WARPS + w) * ROWS;
  // the next rows' slots are read under this step's work
  int en;
  float gn;
  auto read = [&](int64_t t) {
    en = -1, gn = 0.f;
    if (t < n && sub < a.top_k) {
      en = index[t * a.top_k + sub];
      gn = gw[t * a.top_k + sub];
    }
    if (en < 0 || en >= a.K) en = -1, gn = 0.f;
  };
  read(t0 + r);
  for (; t0 < n; t0 += step) {
    const int e = en;
    const float g = gn;
    const float v = e >= 0 ? to_f32(logits[(t0 + r) * a.K + e]) : 0.f;
    read(t0 + step + r);
    for (int i = lane * 4; i < size; i += 128)
      *reinterpret_cast<float4 *>(gs + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    float s = 0.f, total = 1.f, d = g;
    if (a.softmax) {  // renormalised
      float mc = e >= 0 ? v : -INFINITY;
#pragma unroll
      for (int o = LANES / 2; o; o >>= 1) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, o));
      if (e >= 0) s = expf(v - mc);
    } else if (e >= 0) {
      s = sigmoid_f(v);
    }
    if (a.renorm) {
      total = sum(s);
      if (total == 0.f) total = INFINITY;  // such scores weigh 0
      const float p = s / total;           // (1 for a single slot, whose gradient is then 0)
      d = g - sum(g * p);
      if (a.softmax) d *= p;
    }
    d *= a.scale;
    if (!a.softmax) d *= s * sigmoid_f(-v) / total;
    // an expert named twice shows by its tag, and adds up in slot order
    __syncwarp();
    if (e >= 0) mine[e] = __int_as_float(lane);
    __syncwarp();
    const bool any = __any_sync(0xffffffffu, e >= 0 && __float_as_int(mine[e]) != lane);
    __syncwarp();
    if (e >= 0) mine[e] = any ? 0.f : d;
    __syncwarp();
    if (any)
      for (int l = 0; l < LANES; ++l) {
        if (sub == l && e >= 0) mine[e] += d;
        __syncwarp();
      }
    const int64_t rows = n - t0 < ROWS ? n - t0 : ROWS;
    const int have = (int)rows * a.K;
    float *out = grad + t0 * a.K;
    if (vec && have % 4 == 0) {
      for (int i = lane * 4; i < have; i += 128)
        *reinterpret_cast<float4 *>(out + i) = *reinterpret_cast<const float4 *>(gs + i);
    } else {
      for (int i = lane; i < have; i += 32) out[i] = gs[i];
    }
    __syncwarp();
  }
}

}  // namespace so2

using namespace so2;

namespace {

bool route_ok(const so2conv_route_desc *d) {
  if (d->n_experts < 1 || d->n_experts > 1024) return false;
  if (d->top_k < 1 || d->top_k > d->n_experts) return false;
  if (d->n_groups < 1 || d->n_groups > d->n_experts || d->n_experts % d->n_groups) return false;
  if (d->top_groups < 1 || d->top_groups > d->n_groups) return false;
  const int per = d->n_experts / d->n_groups;
  if (d->group_top < 1 || d->group_top > 2 || d->group_top > per) return false;
  if (d->top_k > d->top_groups * per) return false;
  if (d->score != SO2_SCORE_SOFTMAX && d->score != SO2_SCORE_SIGMOID) return false;
  if (d->renormalise != 0 && d->renormalise != 1) return false;
  return dtype_ok(d->dtype);
}

RouteArgs route_args(const so2conv_route_desc *d) {
  RouteArgs a;
  a.K = d->n_experts;
  a.top_k = d->top_k;
  a.n_groups = d->n_groups;
  a.top_groups = d->top_groups;
  a.group_top = d->group_top;
  a.per = d->n_experts / d->n_groups;
  a.softmax = d->score == SO2_SCORE_SOFTMAX;
  a.renorm = d->renormalise;
  a.scale = d->scale;
  return a;
}

so2_status route_checks(const so2conv_route_desc *d, int64_t n, const void *logits) {
  if (!d) return SO2_ERR_INVALID_ARG;
  if (!route_ok(d)) return SO2_ERR_UNSUPPORTED;
  if (!(d->scale - d->scale == 0.f) || d->scale == 0.f) return SO2_ERR_INVALID_ARG;
  if (n < 0 || n > (1ll << 30)) return SO2_ERR_INVALID_ARG;
  if (n > 0 && (!logits || !aligned_to(logits, dtype_size(d->dtype)))) return SO2_ERR_INVALID_ARG;
  return SO2_OK;
}

// Experts a lane, as a compile-time power of two.
#define ROUTE_DISPATCH(K, ...)                                   \
  if ((K) <= 32) { constexpr int NPL = 1; __VA_ARGS__; }         \
  else if ((K) <= 64) { constexpr int NPL = 2; __VA_ARGS__; }    \
  else if ((K) <= 128) { constexpr int NPL = 4; __VA_ARGS__; }   \
  else if ((K) <= 256) { constexpr int NPL = 8; __VA_ARGS__; }   \
  else if ((K) <= 512) { constexpr int NPL = 16; __VA_ARGS__; }  \
  else { constexpr int NPL = 32; __VA_ARGS__; }

int route_grid(int64_t n) {
  const int64_t want = ceil_div(n, ROUTE_WARPS);
  return (int)(want < MODEL_SMS * 16 ? want : MODEL_SMS * 16);
}

template <int NPL, bool BY_SCORE, typename T>
so2_status run_route(const RouteArgs &a, int64_t n, const T *logits, const float *bias,
                     float *weights, int32_t *index, int32_t *counts, cudaStream_t s) {
  const int smem = ROUTE_WARPS * route_words(a.K, a.n_groups, a.top_k, BY_SCORE) * 8 + a.K * 4;
  constexpr int KM = 32 * NPL, most = ROUTE_WARPS * route_words(KM, KM, KM, BY_SCORE) * 8 + KM * 4;
  if (!allow_smem(k_route<NPL, BY_SCORE, T>, smem, most)) return SO2_ERR_CUDA;
  // up to 16 rows one block stores the counts itself, without a clearing launch
  const int grid = n <= 16 ? 1 : route_grid(n);
  if (counts && grid > 1) MODEL_CK(cudaMemsetAsync(counts, 0, sizeof(int32_t) * a.K, s));
  k_route<NPL, BY_SCORE, T><<<grid, 32 * ROUTE_WARPS, smem, s>>>(
      a, n, logits, expert_vectors<NPL>(a.K, logits), bias, weights, index, counts);
  MODEL_CKL();
  return SO2_OK;
}

template <int SHIFT, int NPL, bool BY_SCORE, typename T>
so2_status run_route_top(const RouteArgs &a, int64_t n, const T *logits, const float *bias,
                         float *weights, int32_t *index, int32_t *counts, cudaStream_t s) {
  constexpr int ROWS = 32 >> SHIFT;
  const int smem = ROUTE_WARPS * route_top_words(a.K, a.n_groups, ROWS) * 8 + a.K * 4;
  constexpr int KM = NPL << SHIFT;
  static_assert(ROUTE_WARPS * route_top_words(KM, KM, ROWS) * 8 + KM * 4 <= 48 * 1024, "");
  const int grid = n <= 16 ? 1 : route_grid(ceil_div(n, ROWS));
  if (counts && grid > 1) MODEL_CK(cudaMemsetAsync(counts, 0, sizeof(int32_t) * a.K, s));
  constexpr int V = NPL * sizeof(T) <= 16 ? NPL : 16 / (int)sizeof(T);
  const bool vec = V >= 4 && a.K % V == 0 && aligned_to(logits, V * sizeof(T));
  k_route_top<SHIFT, NPL, BY_SCORE, T><<<grid, 32 * ROUTE_WARPS, smem, s>>>(
      a, n, logits, vec, bias, weights, index, counts);
  MODEL_CKL();
  return SO2_OK;
}

template <bool BY_SCORE, typename T>
so2_status run_route_top(const RouteArgs &a, int64_t n, const T *x, const float *bias,
                         float *weights, int32_t *index, int32_t *counts, cudaStream_t s) {
  if (a.K <= 32) return run_route_top<3, 4, BY_SCORE, T>(a, n, x, bias, weights, index, counts, s);
  if (a.K <= 64) return run_route_top<3, 8, BY_SCORE, T>(a, n, x, bias, weights, index, counts, s);
  if (a.K <= 128) return run_route_top<3, 16, BY_SCORE, T>(a, n, x, bias, weights, index, counts, s);
  return run_route_top<4, 16, BY_SCORE, T>(a, n, x, bias, weights, index, counts, s);
}

template <typename T>
so2_status run_route(const RouteArgs &a, int64_t n, const void *logits, const float *bias,
                     float *weights, int32_t *index, int32_t *counts, cudaStream_t s) {
  const T *x = static_cast<const T *>(logits);
  const bool by_score = bias || (a.top_groups < a.n_groups && a.group_top > 1);
  if (a.top_k <= 8 && a.top_k < a.K && a.K <= 256)
    return by_score ? run_route_top<true, T>(a, n, x, bias, weights, index, counts, s)
                    : run_route_top<false, T>(a, n, x, bias, weights, index, counts, s);
  if (by_score)
    ROUTE_DISPATCH(a.K, return run_route<NPL, true, T>(a, n, x, bias, weights, index, counts, s))
  ROUTE_DISPATCH(a.K, return run_route<NPL, false, T>(a, n, x, bias, weights, index, counts, s))
}

template <int NPL, bool FULL, typename T>
so2_status run_route_grad(const RouteArgs &a, int64_t n, const T *logits, const int32_t *index,
                          const float *gw, float *grad, cudaStream_t s) {
  k_route_grad<NPL, FULL, T><<<route_grid(n), 32 * ROUTE_WARPS, 0, s>>>(
      a, n, logits, expert_vectors<NPL>(a.K, logits), index, gw, grad,
      NPL >= 4 && a.K % 4 == 0 && aligned_to(grad, 16));
  MODEL_CKL();
  return SO2_OK;
}

template <int SHIFT, typename T>
so2_status run_route_grad_slots(const RouteArgs &a, int64_t n, const T *logits,
                                const int32_t *index, const float *gw, float *grad, cudaStream_t s) {
  constexpr int ROWS = 32 >> SHIFT;
  const int smem = ROUTE_WARPS * ((ROWS * a.K + 3) & ~3) * 4;
  if (!allow_smem(k_route_grad_slots<SHIFT, T>, smem, ROUTE_WARPS * ROWS * 1024 * 4)) return SO2_ERR_CUDA;
  // a step's rows start on a vector's boundary if one row does, or four of them
  const bool vec = aligned_to(grad, 16) && (ROWS * a.K) % 4 == 0;
  k_route_grad_slots<SHIFT, T><<<route_grid(ceil_div(n, ROWS)), 32 * ROUTE_WARPS, smem, s>>>(
      a, n, logits, index, gw, grad, vec);
  MODEL_CKL();
  return SO2_OK;
}

template <typename T>
so2_status run_route_grad(const RouteArgs &a, int64_t n, const void *logits, const int32_t *index,
                          const float *gw, float *grad, cudaStream_t s) {
  const T *x = static_cast<const T *>(logits);
  if (a.softmax && !a.renorm)
    ROUTE_DISPATCH(a.K, return run_route_grad<NPL, true, T>(a, n, x, index, gw, grad, s))
  if (a.top_k <= 4) return run_route_grad_slots<2, T>(a, n, x, index, gw, grad, s);
  if (a.top_k <= 8) return run_route_grad_slots<3, T>(a, n, x, index, gw, grad, s);
  if (a.top_k <= 16) return run_route_grad_slots<4, T>(a, n, x, index, gw, grad, s);
  if (a.top_k <= 32) return run_route_grad_slots<5, T>(a, n, x, index, gw, grad, s);
  ROUTE_DISPATCH(a.K, return run_route_grad<NPL, false, T>(a, n, x, index, gw, grad, s))
}

}  // namespace

extern "C" {

so2_status so2conv_route_forward(const so2conv_route_desc *d, int64_t n, const void *logits,
                                 const float *bias, float *weights, int32_t *index,
                                 int32_t *counts, so2_stream_t stream) {
  so2_status r = route_checks(d, n, logits);
  if (r != SO2_OK) return r;
  if (n > 0 && (!weights || !index)) return SO2_ERR_INVALID_ARG;
  if (!aligned_to(weights, 4) || !aligned_to(index, 4) || !aligned_to(bias, 4) ||
      !aligned_to(counts, 4))
    return SO2_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (counts) MODEL_CK(cudaMemsetAsync(counts, 0, sizeof(int32_t) * d->n_experts, s));
    return SO2_OK;
  }
  const RouteArgs a = route_args(d);
  if (d->dtype == SO2_F32) return run_route<float>(a, n, logits, bias, weights, index, counts, s);
  return run_route<__nv_bfloat16>(a, n, logits, bias, weights, index, counts, s);
}

so2_status so2conv_route_backward(const so2conv_route_desc *d, int64_t n, const void *logits,
                                  const int32_t *index, const float *gw, float *grad,
                                  so2_stream_t stream) {
  so2_status r = route_checks(d, n, logits);
  if (r != SO2_OK) return r;
  if (n > 0 && (!index || !gw || !grad)) return SO2_ERR_INVALID_ARG;
  if (!aligned_to(index, 4) || !aligned_to(gw, 4) || !aligned_to(grad, 4)) return SO2_ERR_INVALID_ARG;
  if (n == 0) return SO2_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RouteArgs a = route_args(d);
  if (d->dtype == SO2_F32) return run_route_grad<float>(a, n, logits, index, gw, grad, s);
  return run_route_grad<__nv_bfloat16>(a, n, logits, index, gw, grad, s);
}

}  // extern "C"
