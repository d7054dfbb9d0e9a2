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
// The alternatives come from the same pass. After the first step every group of eight threads knows its
// largest element; the k-th largest of these 64 is a bound that at least k elements reach, so only
// elements that reach it can be among the k largest. They go to a list in shared memory (about 1.5 k of
// 128000 normal logits for k = 20), whose members are ranked by counting at the end. Elements are ordered
// by (value, lower index), a total order, so equal logits, and masked rows in which most elements are the
// same, neither overflow the list nor make the result depend on timing. A row that rises along its length
// can overflow it; it is then read again k times.
#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = kThreads / 8;
constexpr int kMaxTopK = 32;
constexpr int kList = 2560;  // at least 2048 + 14: a segment in which fewer than k groups have elements fits
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

struct F32 {};
template <class DT>
struct Elem {
  static constexpr int kBytes = 2, kVec = 8;
  static __device__ __forceinline__ float at(const void *p, int64_t i) {
    return bits_to_float(reinterpret_cast<const uint16_t *>(p)[i], DT::kBF16);
  }
  static __device__ __forceinline__ void unpack(const uint4 &w, float *x) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT::kBF16) {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
};
template <>
struct Elem<F32> {
  static constexpr int kBytes = 4, kVec = 4;
  static __device__ __forceinline__ float at(const void *p, int64_t i) { return reinterpret_cast<const float *>(p)[i]; }
  static __device__ __forceinline__ void unpack(const uint4 &w, float *x) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
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
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(const Params p) {
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

  for (int j0 = 0; j0 == 0 || j0 < n_vec; j0 += kThreads * U) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * kThreads + tid;
      if (j < n_vec) w[u] = __ldcs(vec + j);
    }
    float x[U * kVec];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j0 + u * kThreads + tid < n_vec) {
        E::unpack(w[u], x + u * kVec);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[u * kVec + e] = -INFINITY;
      }
    }
    float sm = j0 == 0 ? xe : -INFINITY;
#pragma unroll
    for (int e = 0; e < U * kVec; ++e) sm = max_nan(sm, x[e]);
    rescale(st, max_nan(st.m, sm));
    const float shift = shift_of(st.m);
#pragma unroll
    for (int e = 0; e < U * kVec; ++e) {
      const float d = max_nan(x[e] - shift, kFar);
      const float y = exp2_approx(d * kLog2e);
      st.s += y;
      st.t += d * y;
    }
    if (j0 == 0 && has_e) {
      const float d = max_nan(xe - shift, kFar);
      const float y = exp2_approx(d * kLog2e);
      st.s += y;
      st.t += d * y;
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
            for (int e = kVec - 1; e >= 0; --e)
              if (x[u * kVec + e] == sm) at = first + static_cast<uint32_t>(j) * kVec + e;
          }
        }
        if (has_e && xe == sm && (tid < head || at >= 0x80000000u)) at = xe_i;
        uint64_t key = key_of(sm, at);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, o));
        if ((lane & 7) == 0) group_key[tid >> 3] = key;
        __syncthreads();
        // warp w ranks groups 4 w .. 4 w + 3, eight lanes each
        const uint64_t mine = group_key[warp * 4 + (lane >> 3)];
        int above = 0;
#pragma unroll
        for (int g = 0; g < kGroups / 8; ++g) above += group_key[(lane & 7) + 8 * g] > mine;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
        if (above == k - 1 && (lane & 7) == 0) bound = mine;
        __syncthreads();
        tau_v = value_of(bound);
        tau_i = index_of(bound);
        if (has_e) push(xe, xe_i);
      }
      if (!(sm < tau_v)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * kThreads + tid;
          if (j < n_vec) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) push(x[u * kVec + e], first + static_cast<uint32_t>(j) * kVec + e);
          }
        }
      }
    }
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
      if (tid < p.csize * k) {
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
  // few rows: up to eight CTAs (one cluster) share a row, while each keeps at least 4096 elements
  int c = 1;
  while (c < 8 && a.rows * c * 2 <= 2 * dev.num_sms && a.vocab / (c * 2) >= 4096) c *= 2;
  p.csize = c;
  p.share = ((a.vocab + c - 1) / c + 63) / 64 * 64;
  if (a.dtype == W4A16_F32) return go<F32>(p, a.rows, a.stream);
  return a.dtype == W4A16_BF16 ? go<BF16>(p, a.rows, a.stream) : go<F16>(p, a.rows, a.stream);
}

}  // namespace w4a16
