// Log probabilities of given tokens, the entropy and the most probable alternatives of rows of logits.
//
//     d_j = x_j - m, m = max x;   S = sum exp d_j;   log p_t = d_t - log S
//     H = -sum p_j log p_j = log S - (sum d_j exp d_j) / S
//     alternatives: the k largest logits, equal ones in the order of their indices
//
// Bound by memory: the row is read once. Each thread keeps a running maximum m and the two sums over
// its elements, rescaled when m grows (exp(m - m') once for each step of 64 bytes a thread, not for each
// element); the threads' triples are joined at the end, the CTAs of a row (a thread-block cluster, when
// there are few rows) through distributed shared memory, in a fixed order.
//
// The alternatives come from the same pass. After the first step every group of four threads knows its
// largest element; the k-th largest of these 64 is a bound that at least k elements reach, so only
// elements that reach it can be among the k largest. They go to a list in shared memory, whose members are ranked
// by counting; after 1, 2, 4, .. steps only the k largest are kept and the last of them is the new bound (so about
// k of them are added while the elements seen double). Elements are ordered
// by (value, lower index), a total order, so equal logits, and masked rows in which most elements are the
// same, neither overflow the list nor make the result depend on timing. A row that rises along its length
// can overflow it; it is then read again k times.
//
// Measured: 1024 rows of 128007 bf16 logits, 20 alternatives: 72 us for 262 MB, 3.6 TB/s, 0.54 of the device's copy
// rate. 1024 rows are 1.7 waves of four CTAs on an SM; in them the schedulers issue in 64 % of the cycles
// (conversion, subtraction, exponential, two sums and the comparison with the bound for each element).
// 512 rows of fp32: 50 us, 5.3 TB/s (0.78); 1024 of fp16 70 us. 5 rows of 32003: 12.5 to 15 us a call, the host's time to issue
// it (four output tensors); replayed from a graph 6.0.
#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4;  // on an SM
constexpr int kWarps = kThreads / 32;
constexpr int kGroupLanes = 4;
constexpr int kGroups = kThreads / kGroupLanes;
constexpr int kMaxTopK = 32;
constexpr int kList = 1280;  // at least 1024 + 14: a segment in which fewer than k groups have elements fits
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -1.0e4f;  // exp(kFar) is zero; keeps -inf and the type's lowest value out of products

struct Params {
  const void *logits;
  int64_t row_stride, vocab;
  const int64_t *tokens;
  int n_tokens, top_k;
  int csize;       // CTAs of a row
  int64_t share;   // elements of one CTA
  float *logprobs, *entropy, *top_logprobs;
  int64_t *top_ids;
};

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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

struct F32 {};
template <class DT>
struct Elem {
  static constexpr int kBytes = 2, kVec = 8;
  static constexpr uint32_t kNone = DT::kBF16 ? 0xFF80FF80u : 0xFC00FC00u;  // -infinity
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

  static __device__ __forceinline__ float at(const void *p, int64_t i) {
    return bits_to_float(reinterpret_cast<const uint16_t *>(p)[i], DT::kBF16);
  }
};
template <>
struct Elem<F32> {
  static constexpr int kBytes = 4, kVec = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  static __device__ __forceinline__ float at(const void *p, int64_t i) { return reinterpret_cast<const float *>(p)[i]; }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The largest element of N vectors, NaN if one is NaN.
template <class DT, int N>
__device__ __forceinline__ float top_of(const uint4 (&w)[N]) {
  if constexpr (Elem<DT>::kVec == 4) {
    float t = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
      t = max_nan(max_nan(t, max_nan(__uint_as_float(w[i].x), __uint_as_float(w[i].y))),
                  max_nan(__uint_as_float(w[i].z), __uint_as_float(w[i].w)));
    return t;
  } else {
    using E = Elem<DT>;
    uint32_t t = E::max_words(E::max_words(w[0].x, w[0].y), E::max_words(w[0].z, w[0].w));
#pragma unroll
    for (int i = 1; i < N; ++i) t = E::max_words(t, E::max_words(E::max_words(w[i].x, w[i].y), E::max_words(w[i].z, w[i].w)));
    float a, b;
    unpair(E::two(t), a, b);
    return max_nan(a, b);
  }
}
// Elements 2 i and 2 i + 1 of a vector (F32: i = 0, 1; else 0 .. 3)
template <class DT>
__device__ __forceinline__ uint64_t two_of(const uint4 &w, int i) {
  if constexpr (Elem<DT>::kVec == 4) return i == 0 ? pair(__uint_as_float(w.x), __uint_as_float(w.y)) : pair(__uint_as_float(w.z), __uint_as_float(w.w));
  else return Elem<DT>::two(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w);
}
// A whole number that orders by value, then by the lower index. -0 counts as +0.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return 0xFFFFFFFFu - static_cast<uint32_t>(key); }

// Running maximum and sums over some elements: s = sum exp(x - m), t = sum (x - m) exp(x - m).
struct Stats {
  float m, s, t;
};
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ void rescale(Stats &a, float m) {  // to the maximum m >= a.m
  const float d = a.m == -INFINITY ? kFar : max_nan(a.m - shift_of(m), kFar);
  const float f = exp2_approx(d * kLog2e);
  a.t = f * (a.t + d * a.s);
  a.s *= f;
  a.m = m;
}
__device__ __forceinline__ void join(Stats &a, Stats b) {
  const float m = max_nan(a.m, b.m);
  rescale(a, m);
  rescale(b, m);
  a.s += b.s;
  a.t += b.t;
}

template <class DT, int U>
__global__ void __launch_bounds__(kThreads, kCtas) logprobs_kernel(const Params p) {
  using E = Elem<DT>;
  constexpr int kVec = E::kVec;
  __shared__ uint64_t list[kList];
  __shared__ uint64_t best[kMaxTopK];        // this CTA's alternatives, in order
  __shared__ uint64_t group_key[kGroups];
  __shared__ Stats warp_stats[kWarps];
  __shared__ Stats cta_stats;
  __shared__ uint64_t bound;
  __shared__ unsigned int count;
  __shared__ uint64_t found[kWarps];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = p.csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t row = blockIdx.x / p.csize;
  const int k = p.top_k;
  if (tid == 0) count = 0;
  griddep_wait();
  griddep_launch_dependents();

  const uint8_t *x_row = static_cast<const uint8_t *>(p.logits) + row * p.row_stride * E::kBytes;
  const int64_t lo = min(p.share * rank, p.vocab), hi = min(lo + p.share, p.vocab);
  // [lo, hi) = head (up to the first 16-byte boundary), whole vectors, tail
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(x_row + lo * E::kBytes);
  const int head = static_cast<int>(min(int64_t((16 - (a0 & 15)) & 15) / E::kBytes, hi - lo));
  const int n_vec = static_cast<int>((hi - lo - head) / kVec);
  const int tail = static_cast<int>(hi - lo - head - int64_t(n_vec) * kVec);
  const uint4 *vec = reinterpret_cast<const uint4 *>(x_row + (lo + head) * E::kBytes);
  const uint32_t first = static_cast<uint32_t>(lo) + head;  // index of the first whole vector's first element

  Stats st{-INFINITY, 0.f, 0.f};
  float tau_v = INFINITY;
  uint32_t tau_i = 0;
  float xe = -INFINITY;  // a head or tail element, held by one of the first threads
  uint32_t xe_i = 0;
  bool has_e = tid < head + tail;
  if (has_e) {
    xe_i = tid < head ? static_cast<uint32_t>(lo) + tid : static_cast<uint32_t>(hi) - tail + (tid - head);
    xe = E::at(x_row, xe_i);
  }
  auto push = [&](float v, uint32_t i) {
    if (v > tau_v || (v == tau_v && i <= tau_i) || !(v == v)) {
      const unsigned int at = atomicAdd(&count, 1u);
      if (at < kList) list[at] = key_of(v, i);
    }
  };

  uint4 w[U], ahead[U];
  auto fetch = [&](uint4 (&v)[U], int j0) {
    if (j0 + U * kThreads <= n_vec) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = __ldcs(vec + j0 + u * kThreads + tid);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * kThreads + tid;
        v[u] = make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
        if (j < n_vec) v[u] = __ldcs(vec + j);
      }
    }
  };
  fetch(w, 0);
  uint64_t s2 = 0, t2 = 0;  // the sums of the even and the odd elements
  for (int j0 = 0; j0 == 0 || j0 < n_vec; j0 += kThreads * U) {
    if (j0 + kThreads * U < n_vec) fetch(ahead, j0 + kThreads * U);  // in flight while this step is computed
    float sm = top_of<DT>(w);
    if (j0 == 0) sm = max_nan(sm, xe);
    {
      // to the new maximum (as rescale(), for both halves of the sums)
      const float m = max_nan(st.m, sm);
      const float d = st.m == -INFINITY ? kFar : max_nan(st.m - shift_of(m), kFar);
      const float f = exp2_approx(d * kLog2e);
      t2 = mul2(pair(f, f), fma2(pair(d, d), s2, t2));
      s2 = mul2(pair(f, f), s2);
      st.m = m;
    }
    const float shift = shift_of(st.m);
    const uint64_t minus = pair(-shift, -shift), unit = pair(kLog2e, kLog2e);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < kVec / 2; ++e) {
        float d0, d1, a0, a1;
        unpair(add2(two_of<DT>(w[u], e), minus), d0, d1);
        const uint64_t d = pair(max_nan(d0, kFar), max_nan(d1, kFar));
        unpair(mul2(d, unit), a0, a1);
        const uint64_t y = pair(exp2_approx(a0), exp2_approx(a1));
        s2 = add2(s2, y);
        t2 = fma2(d, y, t2);
      }
    }
    if (j0 == 0 && has_e) {
      const float d = max_nan(xe - shift, kFar);
      const float y = exp2_approx(d * kLog2e);
      s2 = add2(s2, pair(y, 0.f));
      t2 = add2(t2, pair(d * y, 0.f));
    }
    if (k > 0) {
      if (j0 == 0) {
        // the k-th largest of the groups' largest elements bounds the k-th largest element
        uint32_t at = 0x80000000u + tid;  // no element: behind every real one
#pragma unroll
        for (int u = U - 1; u >= 0; --u) {
          const int j = u * kThreads + tid;
          if (j < n_vec) {
#pragma unroll
            for (int e = kVec / 2 - 1; e >= 0; --e) {
              float a, b;
              unpair(two_of<DT>(w[u], e), a, b);
              const uint32_t i = first + static_cast<uint32_t>(j) * kVec + 2 * e;
              if (b == sm) at = i + 1;
              if (a == sm) at = i;
            }
          }
        }
        if (has_e && xe == sm && (tid < head || at >= 0x80000000u)) at = xe_i;
        uint64_t key = key_of(sm, at);
#pragma unroll
        for (int o = kGroupLanes / 2; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, o));
        if ((lane & (kGroupLanes - 1)) == 0) group_key[tid / kGroupLanes] = key;
        __syncthreads();
        // four lanes rank one group
        const uint64_t mine = group_key[tid / 4];
        int above = 0;
#pragma unroll
        for (int g = 0; g < kGroups / 4; ++g) above += group_key[(lane & 3) + 4 * g] > mine;
#pragma unroll
        for (int o = 2; o > 0; o >>= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
        if (above == k - 1 && (lane & 3) == 0) bound = mine;
        __syncthreads();
        tau_v = value_of(bound);
        tau_i = index_of(bound);
        if (has_e) push(xe, xe_i);
      }
      if (!(sm < tau_v)) {
        uint32_t hits = 0;  // bit u * kVec + e: elements that may be among the k largest
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint4 one[1] = {w[u]};
          if (j0 + u * kThreads + tid < n_vec && !(top_of<DT>(one) < tau_v)) {
#pragma unroll
            for (int e = 0; e < kVec / 2; ++e) {
              float a, b;
              unpair(two_of<DT>(w[u], e), a, b);
              if (!(a < tau_v)) hits |= 1u << (u * kVec + 2 * e);
              if (!(b < tau_v)) hits |= 1u << (u * kVec + 2 * e + 1);
            }
          }
        }
#pragma unroll 1
        while (hits) {  // (compact code, for one element in a thousand: the element is read again)
          const int at = __ffs(hits) - 1;
          hits &= hits - 1;
          const uint32_t i = first + static_cast<uint32_t>(j0 + at / kVec * kThreads + tid) * kVec + at % kVec;
          push(E::at(x_row, i), i);
        }
      }
      // after 1, 2, 4, 8 .. steps: the k largest so far, in order, and their last as the bound
      const int step = j0 / (kThreads * U) + 1;
      if ((step & (step - 1)) == 0 && j0 + kThreads * U < n_vec) {
        __syncthreads();
        const unsigned int n = count;
        if (n <= kThreads) {  // (more: leave it to the end)
          const uint64_t mine = tid < n ? list[tid] : 0;
          int above = kThreads;
          if (tid < n) {
            above = 0;
#pragma unroll 4
            for (unsigned int j = 0; j < n; ++j) above += list[j] > mine;
          }
          __syncthreads();
          if (above < k) list[above] = mine;
          if (tid == 0) count = min(n, static_cast<unsigned int>(k));
          __syncthreads();
          if (n >= static_cast<unsigned int>(k)) {
            const uint64_t key = list[k - 1];
            tau_v = value_of(key);
            tau_i = index_of(key);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = ahead[u];
  }
  {
    float a, b;
    unpair(s2, a, b);
    st.s = a + b;
    unpair(t2, a, b);
    st.t = a + b;
  }

  // join the statistics: lanes, warps (warp 0), then the CTAs of the row
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stats b{__shfl_xor_sync(0xFFFFFFFFu, st.m, o), __shfl_xor_sync(0xFFFFFFFFu, st.s, o),
            __shfl_xor_sync(0xFFFFFFFFu, st.t, o)};
    join(st, b);
  }
  if (lane == 0) warp_stats[warp] = st;
  __syncthreads();
  if (warp == 0) {
    st = lane < kWarps ? warp_stats[lane] : Stats{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      Stats b{__shfl_xor_sync(0xFFFFFFFFu, st.m, o), __shfl_xor_sync(0xFFFFFFFFu, st.s, o),
              __shfl_xor_sync(0xFFFFFFFFu, st.t, o)};
      join(st, b);
    }
    if (lane == 0) cta_stats = st;
  }
  if (k > 0) {
    const unsigned int n = count;
    if (tid < k) best[tid] = 0;
    __syncthreads();
    if (n <= kList) {
      for (unsigned int i = tid; i < n; i += kThreads) {
        const uint64_t mine = list[i];
        int above = 0;
        for (unsigned int j = 0; j < n; ++j) above += list[j] > mine;
        if (above < k) best[above] = mine;
      }
    } else {
      uint64_t last = ~0ull;  // keys below this one are left
      for (int r = 0; r < k; ++r) {
        uint64_t top = 0;
        for (int64_t i = lo + tid; i < hi; i += kThreads) {
          const uint64_t key = key_of(E::at(x_row, i), static_cast<uint32_t>(i));
          if (key < last) top = max(top, key);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (lane == 0) found[warp] = top;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) top = max(top, found[w]);
        if (tid == 0) best[r] = top;
        last = top;
        __syncthreads();
      }
    }
  }
  __syncthreads();
  if (p.csize > 1) {
    cluster_sync_all();
    if (rank == 0) {
      // the other CTAs' lists and statistics, in the order of their ranks
      for (int i = tid; i < p.csize * k; i += kThreads) {
        const uint32_t src = map_to_rank(smem_u32(&best[i % k]), i / k);
        uint64_t key;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(key) : "r"(src));
        list[i] = key;
      }
      __syncthreads();
      if (tid == 0) {
        Stats a = cta_stats;
        for (int r = 1; r < p.csize; ++r) {
          const uint32_t src = map_to_rank(smem_u32(&cta_stats), r);
          join(a, Stats{ld_dsmem_f32(src), ld_dsmem_f32(src + 4), ld_dsmem_f32(src + 8)});
        }
        warp_stats[0] = a;
      }
      uint64_t mine = 0;
      int above = kMaxTopK;
      if (tid < p.csize * k) {  // (at most 8 * 32)
        mine = list[tid];
        above = 0;
        for (int j = 0; j < p.csize * k; ++j) above += list[j] > mine;
      }
      __syncthreads();
      if (tid < k) best[tid] = 0;
      __syncthreads();
      if (mine != 0 && above < k) best[above] = mine;
      if (tid == 0) cta_stats = warp_stats[0];
      __syncthreads();
    }
    cluster_sync_all();  // the other CTAs' shared memory was read
    if (rank != 0) return;
  }
  const float m = cta_stats.m, log_s = logf(cta_stats.s);
  for (int i = tid; i < p.n_tokens; i += kThreads) {
    const int64_t tok = p.tokens[row * p.n_tokens + i];
    const bool in = tok >= 0 && tok < p.vocab;
    p.logprobs[row * p.n_tokens + i] = in ? (E::at(x_row, tok) - m) - log_s : __int_as_float(0x7FFFFFFF);
  }
  if (tid == 0 && p.entropy) p.entropy[row] = log_s - cta_stats.t / cta_stats.s;
  if (tid < k) {
    const uint64_t key = best[tid];
    p.top_ids[row * k + tid] = key ? static_cast<int64_t>(index_of(key)) : -1;
    p.top_logprobs[row * k + tid] = key ? (value_of(key) - m) - log_s : __int_as_float(0x7FFFFFFF);
  }
}

template <class DT>
cudaError_t go(const Params &p, int64_t rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * p.csize), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.csize > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.csize);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, 4>, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs &a, const DeviceInfo &dev) {
  Params p{};
  p.logits = a.logits;
  p.row_stride = a.row_stride;
  p.vocab = a.vocab;
  p.tokens = a.tokens;
  p.n_tokens = a.n_tokens;
  p.top_k = a.top_k;
  p.logprobs = a.logprobs;
  p.entropy = a.entropy;
  p.top_ids = a.top_ids;
  p.top_logprobs = a.top_logprobs;
  // Few rows: up to eight CTAs (one cluster) share a row, while each keeps at least 4096 elements and all are resident
  // at once. 256 x 128007 with 20 alternatives: clusters of two 29 us (one CTA a row about as long, its times from 27 to
  // 68 between 160 and 400 rows); 1024 rows, past the residency: one CTA 73 us, two 90, four 121.
  int c = 1;
  while (c < 8 && a.rows * c * 2 <= kCtas * dev.num_sms && a.vocab / (c * 2) >= 4096) c *= 2;
  p.csize = c;
  p.share = ((a.vocab + c - 1) / c + 63) / 64 * 64;
  if (a.dtype == W4A16_F32) return go<F32>(p, a.rows, a.stream);
  return a.dtype == W4A16_BF16 ? go<BF16>(p, a.rows, a.stream) : go<F16>(p, a.rows, a.stream);
}

}  // namespace w4a16
