// Which drafted tokens stand, and the token after them, from given random numbers.
//
//     p = softmax(logits row / T) of a node (T = 0: all on the largest logit, the lowest index of equal ones)
//     chain with the drafter's q: token d stands if u q(d) < p(d); else the next token comes from max(p - q, 0)
//     tree of guesses: a node's children in the order of their indices, Z = 1 - the p of those rejected so far;
//       child d stands if u Z < p(d) (0 for a token that was rejected at this node before); the next
//       token comes from p without the rejected ones
//     a draw from weights r: the j with the largest r_j / e_j, e the given exponential numbers (the first to go off of
//       exponential clocks of rates r); nothing left of r: from p
//
// Both give the target's own distribution. A draw by clocks compares single ratios, so that its result does not hang on
// the last bits of a sum over the vocabulary, nor on the order in which that is added.
//
// Two kernels. The first reads every row once: running maximum and sum of exponentials, rows split over CTAs when
// they are few. The second has a cluster for each sequence: a thread for each token finds its parent and gathers p(d) and q(d); four
// threads for each token look at its siblings, so that every node knows the child that would stand there; the walk down the tree only
// follows these. Then the cluster's CTAs take a part of the vocabulary each, of the last node's row alone. A token's ratio costs an exponential and a division;
// whether it was rejected is only looked up by the few threads that meet a rejected one.
//
// Bound by memory in the first kernel, by the latency of its chain of small steps (sequence, statistics, tokens, logits of the
// drafted tokens, barriers) and then by loads in flight in the second. Measured: 64 sequences of up to 8 tokens, 128007 bf16 logits, with q:
// 38 us replayed from a graph, 17 us for the first kernel's 74 MB (5 TB/s while it streams) and 25 for the second's 81 MB; 8 trees of up to 64
// guesses, 65537 fp32 logits, 38 us; one chain of 5 tokens, 32003 logits, 9 us (11 to issue it); 64 single tokens sampled from 128007 logits 26, at temperature 0 9. Read by neighbouring threads, the three rows
// of the second kernel take 25 us where vectors of one of them took 26 and 33 with half as many loads in flight twice; the noise
// fetched into L2 while the last node is found delays that by more than it saves (40 us in all).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStatCtas = 4;   // on an SM
constexpr int kMaxQ = 64;
constexpr int kMaxSplits = 32;
constexpr float kLog2e = 1.4426950408889634f;

// Two fp32 numbers in one 64-bit register pair
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t x, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct F32 {};
template <class DT>
struct Elem {
  static constexpr int kBytes = 2, kVec = 8;
  static constexpr uint32_t kNone = DT::kBF16 ? 0xFF80FF80u : 0xFC00FC00u;  // -infinity
  // the largest of a word's (largest's) elements, element by element; NaN if one is NaN
  static __device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (DT::kBF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint64_t two(uint32_t w) {
    if constexpr (DT::kBF16) {
      return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
      return pair(f.x, f.y);
    }
  }
  static __device__ __forceinline__ uint64_t two(const uint4 &v, int i) { return two(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w); }
  template <int N>
  static __device__ __forceinline__ float top_of(const uint4 (&w)[N]) {
    uint32_t t = kNone;
#pragma unroll
    for (int i = 0; i < N; ++i) t = max_words(t, max_words(max_words(w[i].x, w[i].y), max_words(w[i].z, w[i].w)));
    float a, b;
    unpair(two(t), a, b);
    return max_nan(a, b);
  }
  static __device__ __forceinline__ float at(const void *p, int64_t i) {
    return bits_to_float(reinterpret_cast<const uint16_t *>(p)[i], DT::kBF16);
  }
};
template <>
struct Elem<F32> {
  static constexpr int kBytes = 4, kVec = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  static __device__ __forceinline__ uint64_t two(const uint4 &v, int i) {
    return i == 0 ? pair(__uint_as_float(v.x), __uint_as_float(v.y)) : pair(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  template <int N>
  static __device__ __forceinline__ float top_of(const uint4 (&w)[N]) {
    float t = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
      t = max_nan(max_nan(t, max_nan(__uint_as_float(w[i].x), __uint_as_float(w[i].y))),
                  max_nan(__uint_as_float(w[i].z), __uint_as_float(w[i].w)));
    return t;
  }
  static __device__ __forceinline__ float at(const void *p, int64_t i) { return reinterpret_cast<const float *>(p)[i]; }
};

struct Params {
  const uint8_t *logits;
  int64_t row_stride, total, vocab;
  const int64_t *tokens;
  const int32_t *q_start;  // null: one token for each sequence
  int64_t batch;
  int max_q;
  const uint64_t *tree_mask;
  const float *uniforms, *noise, *draft, *temperature;
  int64_t noise_stride, draft_stride;
  int32_t *accepted, *path;
  int64_t *out;
  float *probs;
  float2 *stats;  // [total][splits]: maximum, sum of exp((x - maximum) / T); T = 0: the index of the maximum in place of the sum
  int splits;
  int64_t share;  // elements of a split
  int csize;
  int64_t cshare;  // elements of a CTA of a sequence's cluster
};

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// log2(e) / T, kept so small that zero times it is zero (a tiny T is as good as none); NaN, and with it no probabilities, for a
// negative T
__device__ __forceinline__ float unit_of(float temp) {
  const float c = kLog2e / temp;
  return c > 1e30f ? 1e30f : temp > 0.f ? c : __int_as_float(0x7FFFFFFF);
}
// exp2((a - m) c) of a running maximum a that grows to m. (No bound on the difference: at a high temperature elements far below the
// largest count too, and one that leaves fp32's range is -infinity, whose exponential is zero. A maximum of +infinity gives NaN.)
__device__ __forceinline__ float shrink(float a, float m, float c) {
  return a == -INFINITY ? 0.f : exp2_approx((a - m) * c);
}
__device__ __forceinline__ void join(float &m, float &s, float om, float os, float c) {
  const float top = max_nan(m, om);
  s = s * shrink(m, top, c) + os * shrink(om, top, c);
  m = top;
}
// the larger value, the lower index of equal ones; a NaN stays
__device__ __forceinline__ void join_index(float &m, int &i, float om, int oi) {
  if (om > m || (om == m && oi < i) || !(om == om)) m = om, i = oi;
}

// A row as head (up to the first 16-byte boundary), whole vectors, tail
template <class DT>
struct Span {
  const uint4 *vec;
  int64_t lo;
  int head, n_vec, tail;
  __device__ __forceinline__ Span(const uint8_t *row, int64_t lo_, int64_t hi) : lo(lo_) {
    using E = Elem<DT>;
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + lo * E::kBytes);
    head = static_cast<int>(min(int64_t((16 - (at & 15)) & 15) / E::kBytes, hi - lo));
    n_vec = static_cast<int>((hi - lo - head) / E::kVec);
    tail = static_cast<int>(hi - lo - head - int64_t(n_vec) * E::kVec);
    vec = reinterpret_cast<const uint4 *>(row + (lo + head) * E::kBytes);
  }
  // index of the i-th element that is in no vector
  __device__ __forceinline__ int64_t loose(int i) const {
    return i < head ? lo + i : lo + head + int64_t(n_vec) * Elem<DT>::kVec + (i - head);
  }
};

template <class DT>
__global__ void __launch_bounds__(kThreads, kStatCtas) verify_stats_kernel(const Params p) {
  using E = Elem<DT>;
  constexpr int kVec = E::kVec, U = 4;
  __shared__ float ms[kWarps], ss[kWarps];
  __shared__ int is[1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / p.splits;
  const int split = static_cast<int>(blockIdx.x % p.splits);
  griddep_wait();
  griddep_launch_dependents();

  float temp = 1.f;
  if (p.temperature) {
    int64_t seq = row;
    if (p.q_start) {  // sequences that end at or before the row
      seq = 0;
      for (int64_t b0 = 0; b0 < p.batch; b0 += kThreads) seq += __syncthreads_count(b0 + tid < p.batch && p.q_start[b0 + tid + 1] <= row);
    }
    if (seq < p.batch) temp = p.temperature[seq];
  }
  const float c = temp == 0.f ? 0.f : unit_of(temp);
  const uint8_t *x = p.logits + row * p.row_stride * E::kBytes;
  const int64_t lo = min(p.share * split, p.vocab), hi = min(lo + p.share, p.vocab);
  const Span<DT> span(x, lo, hi);
  float m = -INFINITY, s = 0.f;
  int first = 0x7FFFFFFF;
  uint4 w[U], ahead[U];
  auto fetch = [&](uint4 (&v)[U], int j0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * kThreads + tid;
      v[u] = make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
      if (j < span.n_vec) v[u] = __ldg(span.vec + j);
    }
  };
  if (span.n_vec > 0) fetch(w, 0);
  float loose = -INFINITY;  // an element that is in no vector (there are fewer than two vectors of them)
  if (tid < span.head + span.tail) loose = E::at(x, span.loose(tid));
  if (temp == 0.f) {
    int where = 0;  // the first step of this thread's largest element; its index is looked up at the end
    for (int j0 = 0; j0 < span.n_vec; j0 += kThreads * U) {
      if (j0 + kThreads * U < span.n_vec) fetch(ahead, j0 + kThreads * U);
      const float top = E::top_of(w);
      if (!(top <= m)) m = max_nan(m, top), where = j0;
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = ahead[u];
    }
    float all = max_nan(m, loose);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all = max_nan(all, __shfl_xor_sync(0xFFFFFFFFu, all, o));
    if (lane == 0) ms[warp] = all;
    if (tid == 0) is[0] = 0x7FFFFFFF;
    __syncthreads();
    all = ms[0];
    for (int i = 1; i < kWarps; ++i) all = max_nan(all, ms[i]);
    if (loose == all && tid < span.head + span.tail) first = static_cast<int>(span.loose(tid));
    if (m == all && span.n_vec > 0) {
      fetch(w, where);
#pragma unroll
      for (int u = U - 1; u >= 0; --u)
#pragma unroll
        for (int e = kVec / 2 - 1; e >= 0; --e) {
          float x0, x1;
          unpair(E::two(w[u], e), x0, x1);
          const int i = static_cast<int>(lo) + span.head + (where + u * kThreads + tid) * kVec + 2 * e;
          if (x1 == all && i + 1 < hi) first = min(first, i + 1);
          if (x0 == all && i < hi) first = min(first, i);
        }
    }
    if (first != 0x7FFFFFFF) atomicMin(&is[0], first);
    __syncthreads();
    if (tid == 0) p.stats[row * p.splits + split] = make_float2(all, __int_as_float(is[0]));
    return;
  }
  m = loose;
  if (m > -INFINITY || !(m == m)) s = m - m + 1.f;  // NaN for a NaN or an infinity
  {
    uint64_t s2 = 0;  // the sums of the even and the odd elements
    const uint64_t unit = pair(c, c);
    for (int j0 = 0; j0 < span.n_vec; j0 += kThreads * U) {
      if (j0 + kThreads * U < span.n_vec) fetch(ahead, j0 + kThreads * U);  // in flight while this step is computed
      const float top = max_nan(m, E::top_of(w));
      const float f = shrink(m, top, c);
      s2 = mul2(s2, pair(f, f));
      s *= f;
      m = top;
      const float minus = m == -INFINITY ? 0.f : -m;
      const uint64_t shift = pair(minus, minus);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e) {
          float x0, x1;
          unpair(mul2(add2(E::two(w[u], e), shift), unit), x0, x1);
          s2 = add2(s2, pair(exp2_approx(x0), exp2_approx(x1)));
        }
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = ahead[u];
    }
    float se, so;
    unpair(s2, se, so);
    s += se + so;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xFFFFFFFFu, m, o), os = __shfl_xor_sync(0xFFFFFFFFu, s, o);
    join(m, s, om, os, c);
  }
  if (lane == 0) ms[warp] = m, ss[warp] = s;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kWarps; ++i) join(m, s, ms[i], ss[i], c);
    p.stats[row * p.splits + split] = make_float2(m, s);
  }
}

// score and index as a number that grows with the score and falls with the index; 0: none
__device__ __forceinline__ uint64_t key_of(float score, uint32_t i) {
  return uint64_t(__float_as_uint(score) + 1u) << 32 | (0xFFFFFFFFu - i);
}

template <class DT>
__global__ void __launch_bounds__(kThreads, 4) verify_walk_kernel(const Params p) {
  using E = Elem<DT>;
  __shared__ float row_m[kMaxQ], row_s[kMaxQ];  // s: 1 / sum, or the index of the maximum
  __shared__ float pd[kMaxQ], qd[kMaxQ], us[kMaxQ];
  __shared__ int64_t tok[kMaxQ];
  __shared__ int parent[kMaxQ];  // -1: a token that cannot stand
  __shared__ float weight[kMaxQ];  // p(d), 0 for a token that an earlier sibling has
  __shared__ bool passed[kMaxQ];
  __shared__ int next[kMaxQ];      // the child that stands, -1: none
  __shared__ int chosen[kMaxQ];
  __shared__ int64_t rejected[kMaxQ];
  __shared__ int s_accepted, s_rejected;
  __shared__ uint64_t warp_key[kWarps];
  __shared__ uint64_t cta_key;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int csize = p.csize;
  const int crank = csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t b = blockIdx.x / csize;
  const int64_t lo = min(p.cshare * crank, p.vocab), hi = min(lo + p.cshare, p.vocab);
  griddep_wait();
  griddep_launch_dependents();
  int64_t start = b, end = b + 1;
  if (p.q_start) start = max(p.q_start[b], 0), end = min(int64_t(p.q_start[b + 1]), p.total);
  const int n = static_cast<int>(min(int64_t(p.max_q), end - start));
  if (n <= 0) {  // (the same for the whole cluster)
    if (crank == 0) {
      if (tid == 0) p.accepted[b] = 0;
      for (int i = tid; i < p.max_q; i += kThreads) p.path[b * p.max_q + i] = -1, p.out[b * p.max_q + i] = -1, p.probs[b * p.max_q + i] = 0.f;
    }
    return;
  }
  const float temp = p.temperature ? p.temperature[b] : 1.f;
  const bool greedy = temp == 0.f;
  const float c = greedy ? 0.f : unit_of(temp);
  const int64_t my_token = tid < n ? p.tokens[start + tid] : 0;
  const float my_uniform = tid < n ? p.uniforms[start + tid] : 0.f;
  const uint64_t my_word = tid < n && p.tree_mask ? p.tree_mask[start + tid] : ~0ull;
  // the rows' statistics, four threads a row
  {
    const int i = tid >> 2;
    if (i < n) {
      const float2 *st = p.stats + (start + i) * p.splits;
      float m = -INFINITY, s = 0.f;
      int at = 0x7FFFFFFF;
      for (int k = tid & 3; k < p.splits; k += 4) {
        const float2 o = st[k];
        if (greedy) join_index(m, at, o.x, __float_as_int(o.y));
        else join(m, s, o.x, o.y, c);
      }
      const unsigned four = 0xFu << (lane & 28);
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        const float om = __shfl_xor_sync(four, m, o);
        if (greedy) {
          const int oi = __shfl_xor_sync(four, at, o);
          join_index(m, at, om, oi);
        } else {
          const float os = __shfl_xor_sync(four, s, o);
          join(m, s, om, os, c);
        }
      }
      if ((tid & 3) == 0) {
        // a row without probabilities (NaN, +infinity, nothing finite): NaN, and every comparison with it fails
        const bool ok = fabsf(m) < INFINITY && (greedy || s < INFINITY);
        row_m[i] = ok ? m : __int_as_float(0x7FFFFFFF);
        row_s[i] = greedy ? __int_as_float(at) : 1.f / s;
      }
    }
    if (tid < n) {
      tok[tid] = my_token;
      us[tid] = my_uniform;
    }
  }
  __syncthreads();
  // the target's probability of a token under a node's row
  auto prob = [&](int node, int64_t token) {
    const float m = row_m[node];
    if (!(m == m)) return m;
    if (greedy) return token == __float_as_int(row_s[node]) ? 1.f : 0.f;
    return exp2f((E::at(p.logits + (start + node) * p.row_stride * E::kBytes, token) - m) * c) * row_s[node];
  };
  if (tid < n) {
    const uint64_t below = my_word & ((1ull << tid) - 1);
    const int up = below == 0 || my_token < 0 || my_token >= p.vocab ? -1 : 63 - __clzll(static_cast<long long>(below));
    parent[tid] = up;
    if (up >= 0) {
      qd[tid] = p.draft ? p.draft[(start + up) * p.draft_stride + my_token] : 0.f;
      pd[tid] = prob(up, my_token);
    }
  }
  __syncthreads();
  // four threads for each token look at its siblings
  const int own = tid >> 2, part = tid & 3;
  const unsigned quad = 0xFu << (lane & 28);
  if (own < n) {
    bool dup = false;
    if (p.tree_mask)
      for (int j = 1 + part; j < own; j += 4) dup |= parent[j] == parent[own] && tok[j] == tok[own];
    dup = __any_sync(quad, dup);
    if (part == 0) {
      weight[own] = dup || parent[own] < 0 ? 0.f : pd[own];
      next[own] = -1;
    }
  }
  __syncthreads();
  if (own < n) {
    float gone = 0.f;
    if (!p.draft && p.tree_mask)
      for (int j = 1 + part; j < own; j += 4)
        if (parent[j] == parent[own]) gone += weight[j];
    gone += __shfl_xor_sync(quad, gone, 1);
    gone += __shfl_xor_sync(quad, gone, 2);
    // (rejected siblings may add up to more than 1 by rounding: a token of no weight does not stand for that)
    if (part == 0) passed[own] = parent[own] >= 0 && us[own] * (p.draft ? qd[own] : fmaxf(1.f - gone, 0.f)) < weight[own];
  }
  __syncthreads();
  if (own < n) {
    bool before = false;  // an earlier sibling stands
    if (p.tree_mask)
      for (int j = 1 + part; j < own; j += 4) before |= passed[j] && parent[j] == parent[own];
    before = __any_sync(quad, before);
    if (part == 0 && own > 0 && passed[own] && !before) next[parent[own]] = own;
  }
  __syncthreads();
  if (warp == 0) {
    int node = 0, k = 0;
    while (true) {  // (a child's index is larger than its parent's)
      if (lane == 0) chosen[k] = node;
      const int to = next[node];
      if (to < 0) break;
      node = to, ++k;
    }
    // its children, none of which stands
    int nr = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      const bool kid = i > 0 && i < n && parent[i] == node;
      const unsigned vote = __ballot_sync(0xFFFFFFFFu, kid);
      if (kid) rejected[nr + __popc(vote & ((1u << lane) - 1))] = tok[i];
      nr += __popc(vote);
    }
    if (lane == 0) s_accepted = k, s_rejected = nr;
  }
  __syncthreads();
  const int k = s_accepted, last = chosen[k];
  int nr = s_rejected;
  const float m = row_m[last];
  const bool valid = m == m;
  uint64_t best = 0;
  if (valid && greedy) {
    best = key_of(1.f, static_cast<uint32_t>(__float_as_int(row_s[last])));
  } else if (valid) {
    const uint8_t *x = p.logits + (start + last) * p.row_stride * E::kBytes;
    const float *e = p.noise + b * p.noise_stride;
    const float *q = p.draft && nr ? p.draft + (start + last) * p.draft_stride : nullptr;
    const float inv = row_s[last];
    if (q) nr = 0;
    // The threads that come across a rejected token (few of them, and only these look a ratio's token up)
    bool meets = false;
    if (nr) {
      for (int j = 0; j < nr; ++j) {
        const int64_t d = rejected[j];
        meets |= d >= lo && d < hi && static_cast<int>((d - lo) % kThreads) == tid;
      }
    }
    while (true) {
      float top = -1.f;
      uint32_t top_i = 0;
      // neighbouring elements in neighbouring threads: the three rows start at different offsets from 16 bytes
      constexpr int U = 8;
      auto pass = [&](auto with_q) {
        for (int64_t i0 = lo + tid; i0 < hi; i0 += kThreads * U) {
          float xv[U], ev[U], qv[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kThreads;
            const bool in = i < hi;
            xv[u] = in ? E::at(x, i) : -INFINITY;
            ev[u] = in ? __ldcs(e + i) : 1.f;
            if constexpr (decltype(with_q)::value) qv[u] = in ? __ldcs(q + i) : 0.f;
            else qv[u] = 0.f;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float r = fmaxf(exp2_approx((xv[u] - m) * c) * inv - qv[u], 0.f);
            const float score = __fdividef(r, ev[u]);
            // (ascending indices within a thread, so that the first of equal ratios stays)
            if (r > 0.f && score > top) {
              const uint32_t i = static_cast<uint32_t>(i0) + u * kThreads;
              bool gone = false;
              if (meets)
                for (int j = 0; j < nr; ++j) gone |= rejected[j] == i;
              if (!gone) top = score, top_i = i;
            }
          }
        }
      };
      if (q) pass(std::true_type{});
      else pass(std::false_type{});
      best = top >= 0.f ? key_of(top, top_i) : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
      if (lane == 0) warp_key[warp] = best;
      __syncthreads();
      best = warp_key[0];
      for (int w = 1; w < kWarps; ++w) best = max(best, warp_key[w]);
      if (csize > 1) {
        if (tid == 0) cta_key = best;
        cluster_sync_all();
        for (int r = 0; r < csize; ++r) {
          uint64_t o;
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(o) : "r"(map_to_rank(smem_u32(&cta_key), r)));
          best = max(best, o);
        }
        cluster_sync_all();  // read by all, before it is written again or its CTA leaves
      } else {
        __syncthreads();
      }
      if (best != 0 || (!q && nr == 0)) break;
      q = nullptr, nr = 0;  // nothing is left: from p itself
    }
  }
  if (crank != 0) return;
  if (tid < p.max_q) {
    const int64_t at = b * p.max_q + tid;
    int64_t token = -1;
    float pr = 0.f;
    if (tid < k) {
      token = tok[chosen[tid + 1]];
      pr = pd[chosen[tid + 1]];
    } else if (tid == k) {
      token = best ? static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
      pr = token >= 0 ? prob(last, token) : __int_as_float(0x7FFFFFFF);
    }
    p.path[at] = tid <= k ? chosen[tid] : -1;
    p.out[at] = token;
    p.probs[at] = pr;
  }
  if (tid == 0) p.accepted[b] = k;
}

// CTAs of a row: while all are resident at once and each keeps 4096 elements
int splits_of(int64_t total, int64_t vocab, int num_sms) {
  int s = 1;
  while (s < kMaxSplits && total * s * 2 <= int64_t(kStatCtas) * num_sms && vocab / (s * 2) >= 4096) s *= 2;
  return s;
}

template <class DT>
cudaError_t go(const Params &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.total * p.splits), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.total > 0) {
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_stats_kernel<DT>, p);
    if (e != cudaSuccess) return e;
    note_launch();
  }
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch * p.csize), 1, 1);
  if (p.csize > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.csize);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_walk_kernel<DT>, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

size_t verify_workspace_bytes(int64_t total, int64_t vocab, int num_sms) {
  return 4096 + static_cast<size_t>(total) * splits_of(total, vocab, num_sms) * sizeof(float2);
}

cudaError_t launch_verify(const VerifyArgs &a, const DeviceInfo &dev) {
  Params p{};
  p.logits = static_cast<const uint8_t *>(a.logits);
  p.row_stride = a.row_stride;
  p.total = a.total;
  p.vocab = a.vocab;
  p.tokens = a.tokens;
  p.q_start = a.q_start;
  p.batch = a.batch;
  p.max_q = a.max_q;
  p.tree_mask = a.tree_mask;
  p.uniforms = a.uniforms;
  p.noise = a.noise;
  p.noise_stride = a.noise_stride;
  p.draft = a.draft;
  p.draft_stride = a.draft_stride;
  p.temperature = a.temperature;
  p.accepted = a.accepted;
  p.path = a.path;
  p.out = a.out;
  p.probs = a.probs;
  p.stats = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a.workspace) + 4096);  // (past the counters of other calls)
  p.splits = splits_of(a.total, a.vocab, dev.num_sms);
  p.share = ((a.vocab + p.splits - 1) / p.splits + 63) / 64 * 64;
  int c = 1;
  while (c < 8 && a.vocab / (c * 2) >= 2048) c *= 2;
  p.csize = c;
  p.cshare = ((a.vocab + c - 1) / c + 63) / 64 * 64;
  if (a.dtype == W4A16_F32) return go<F32>(p, a.stream);
  return a.dtype == W4A16_BF16 ? go<BF16>(p, a.stream) : go<F16>(p, a.stream);
}

}  // namespace w4a16
