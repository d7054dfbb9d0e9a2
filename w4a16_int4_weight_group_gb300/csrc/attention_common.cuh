// Shared by the attention kernels: the work split, queries, results and the joining of split sequences.
#pragma once

#include <atomic>

#include "attention.h"
#include "common.cuh"

namespace w4a16 {
namespace attention {

constexpr uint64_t kDefaultWaitNs = 2000000000ull;  // 2 s
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 3.f;        // how far (powers of two) scores may exceed the running maximum
constexpr float kProbExp = 12.f;     // probabilities are held times 2^12: at most 2^15 with the slack, under 65504
constexpr float kProbUnit = 4096.f;
constexpr float kSmall = 6.103515625e-05f;  // 2^-14, the smallest normal fp16 number
constexpr float kPlane = 268435456.f;       // 2^28
constexpr int kPlanes = 5;                  // 2^-14 - 4 * 28 = 2^-126

// Position in the list of units, and what of the sequence it takes to walk on.
struct Cursor {
  int b, h, rt, blk;
  int nb, nrt;  // of the sequence: units of a segment, row tiles
  int len;      // cached tokens
};
// What a segment takes beyond that.
struct Queries {
  int64_t q0;    // row of the first query token
  int n, first;  // query tokens, cache position of the first of them
};

__device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ __forceinline__ int length_of(const Params &p, int b) {
  const int64_t cap = p.max_pages * p.page_tiles * 16;
  const int len = p.kv_lens[b];
  return len < 0 ? 0 : static_cast<int>(min(int64_t(len), cap));
}
__device__ __forceinline__ Queries queries_of(const Params &p, int b, int len) {
  const int64_t q0 = p.q_start ? p.q_start[b] : b, q1 = p.q_start ? p.q_start[b + 1] : b + 1;
  int64_t n = q1 - q0;
  if (n < 0 || q0 < 0 || q1 > p.total_q) n = 0;
  return Queries{q0, static_cast<int>(min(n, int64_t(p.max_q))), static_cast<int>(len - n)};
}

// Loads sequence b into the cursor; units of the sequence (0: nothing to do).
template <class L>
__device__ __forceinline__ int64_t load_sequence(const Params &p, int b, Cursor &c) {
  c.b = b;
  c.h = c.rt = c.blk = 0;
  c.len = length_of(p, b);
  c.nrt = static_cast<int>((int64_t(queries_of(p, b, c.len).n) * p.group + L::R - 1) / L::R);
  c.nb = c.len > 0 ? (c.len + L::kUnit - 1) / L::kUnit : 1;
  return int64_t(c.nb) * c.nrt * p.kv_heads;
}

// The first unit of the next segment (the caller knows that there is one).
template <class L>
__device__ __forceinline__ void next_segment(const Params &p, Cursor &c) {
  c.blk = 0;
  if (++c.rt < c.nrt) return;
  c.rt = 0;
  if (++c.h < p.kv_heads) return;
  int b = c.b + 1;
  while (b < p.batch && load_sequence<L>(p, b, c) == 0) ++b;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) { return sub2_rn<false>(a, b); }
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Writes a finished value group of four elements of a row.
__device__ __forceinline__ void store_out4(const Params &p, int64_t at, float4 v) {
  uint2 w;
  if (p.bf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  } else {
    w = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
  }
  *reinterpret_cast<uint2 *>(p.out + at) = w;
}

// ... of eight elements (16 bytes).
__device__ __forceinline__ void store_out8(const Params &p, int64_t at, const float *v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.bf16) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&a);
    } else {
      w[i] = pack_half2(v[2 * i], v[2 * i + 1]);
    }
  }
  *reinterpret_cast<uint4 *>(p.out + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// N elements from d on of row `row` of a segment's row tile of `height` rows (zeros past its `rows`).
template <int N>
__device__ __forceinline__ void load_query(const Params &p, const Cursor &seg, const Queries &qu, int row, int rows, int height, int d,
                                           float (&x)[N]) {
  static_assert(N == 8, "16 bytes");
  uint4 w = make_uint4(0, 0, 0, 0);
  if (row < rows) {
    const int gr = seg.rt * height + row;
    const int i = gr / p.group;
    const int h = seg.h * p.group + (gr - i * p.group);
    w = *reinterpret_cast<const uint4 *>(p.q + (qu.q0 + i) * p.q_ts + h * p.q_hs + d);
  }
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = bits_to_float(static_cast<uint16_t>(ww[j >> 1] >> (16 * (j & 1))), p.bf16 != 0);
}
// Drafted tokens that query token i of the sequence sees, a bit each.
__device__ __forceinline__ uint64_t mask_word(const Params &p, const Queries &qu, int i) {
  return p.tree_mask ? p.tree_mask[qu.q0 + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
}
// A row with largest magnitude `top` times `up` (a power of two, with the sign of the softmax scale) has its
// largest element near 2^12; `unit` turns its products with keys into powers of two of the softmax.
__device__ __forceinline__ void query_unit(const Params &p, float top, float &up, float &unit) {
  int e = top > 0.f ? 12 - (static_cast<int>((__float_as_uint(top) >> 23) & 0xFFu) - 127) : 0;
  e = min(e, 100);
  up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23) * (p.scale < 0.f ? -1.f : 1.f);
  unit = fabsf(p.scale) * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// This CTA's share of the units: an equal part of the list over all sequences (total units over ctas CTAs; it
// starts at cur, has `units` units and ends before unit u1). False when there is nothing for it. Without a
// workspace the share is the segments that start in that part, whole. Called by all threads; scan_s has a
// word for each of the W warps, share_s two words.
template <class L, int W>
__device__ __forceinline__ bool share_of(const Params &p, int64_t *scan_s, volatile int64_t *share_s, Cursor &cur, int64_t &u1,
                                         int64_t &total, int64_t &ctas, int64_t &units) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slice = (p.batch + 32 * W - 1) / (32 * W);
  int64_t mine = 0;
  for (int b = tid * slice; b < min(p.batch, (tid + 1) * slice); ++b) mine += load_sequence<L>(p, b, cur);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) scan_s[warp] = upto;
  __syncthreads();
  int64_t before = upto - mine;
  total = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += scan_s[w];
    total += scan_s[w];
  }
  ctas = total < gridDim.x ? total : gridDim.x;
  const int64_t cta = blockIdx.x;
  if (cta >= ctas) return false;
  const int64_t u0 = cta * total / ctas;
  u1 = (cta + 1) * total / ctas;
  if (u0 >= before && u0 < before + mine) {
    int64_t at = u0 - before;
    for (int b = tid * slice;; ++b) {
      const int64_t n = load_sequence<L>(p, b, cur);
      if (at < n) {
        share_s[0] = b;
        share_s[1] = at;
        break;
      }
      at -= n;
    }
  }
  __syncthreads();
  load_sequence<L>(p, static_cast<int>(share_s[0]), cur);
  {
    int64_t at = share_s[1];
    cur.h = static_cast<int>(at / (int64_t(cur.nb) * cur.nrt));
    at -= int64_t(cur.h) * cur.nb * cur.nrt;
    cur.rt = static_cast<int>(at / cur.nb);
    cur.blk = static_cast<int>(at - int64_t(cur.rt) * cur.nb);
  }
  units = u1 - u0;
  if (!p.flags) {
    if (cur.blk != 0) {
      units -= min(int64_t(cur.nb - cur.blk), units);
      if (units == 0) return false;
      next_segment<L>(p, cur);
    }
    Cursor c = cur;
    int64_t left = units, whole = 0;
    while (true) {
      whole += c.nb;
      left -= c.nb;
      if (left <= 0) break;
      next_segment<L>(p, c);
    }
    units = whole;
  }
  return true;
}

// Adds the parts of a split segment and writes its rows: THREADS threads, the parts in the order of the CTAs.
// The maxima first, side by side (the parts of one long sequence are many), then CHUNK parts at a time their
// weights and their weighted sums. scratch: THREADS + CHUNK * R floats.
template <int R, int D, int THREADS, int CHUNK, class Slot, class Sync>
__device__ __forceinline__ void join_parts(const Params &p, const Cursor &seg, const Queries &qu, int rows, int parts, Slot slot_of,
                                           float *scratch, int tid, Sync sync) {
  float *red = scratch;            // [THREADS / R][R]
  float *wgt = scratch + THREADS;  // [CHUNK][R]
  constexpr int kLanes = THREADS / R;
  const int row_t = tid % R, lane_t = tid / R;
  float top = -INFINITY;
#pragma unroll 4
  for (int c = lane_t; c < parts; c += kLanes) top = fmaxf(top, __ldcg(slot_of(c) + R * D + row_t));
  red[tid] = top;
  sync();
#pragma unroll
  for (int x = 0; x < kLanes; ++x) top = fmaxf(top, red[x * R + row_t]);
  sync();
  constexpr int kPer = (R * D / 4 + THREADS - 1) / THREADS;  // groups of four elements of a thread
  constexpr int kPass = kPer < 4 ? kPer : 4;                 // of them at a time
  const bool works = R * D / 4 >= THREADS || tid < R * D / 4;
  float sum = 0.f;
#pragma unroll 1
  for (int x0 = 0; x0 < kPer; x0 += kPass) {
    float4 v[kPass];
#pragma unroll
    for (int x = 0; x < kPass; ++x) v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int cc = 0; cc < parts; cc += CHUNK) {
      const int now = min(CHUNK, parts - cc);
      for (int c = lane_t; c < now; c += kLanes) {
        const float mc = __ldcg(slot_of(cc + c) + R * D + row_t), lc = __ldcg(slot_of(cc + c) + R * (D + 1) + row_t);
        const float f = mc == -INFINITY ? (lc == 0.f ? 0.f : 1.f) : exp2_approx(mc - top);
        wgt[c * R + row_t] = f;
        if (x0 == 0) sum += lc * f;
      }
      sync();
#pragma unroll 4
      for (int c = 0; c < now; ++c) {
        const float4 *src = reinterpret_cast<const float4 *>(slot_of(cc + c)) + tid + x0 * THREADS;
#pragma unroll
        for (int x = 0; x < kPass; ++x) {
          if (!works) continue;
          const float4 y = __ldcg(src + x * THREADS);
          const float f = wgt[c * R + (tid + (x0 + x) * THREADS) / (D / 4)];
          v[x] = make_float4(fmaf(y.x, f, v[x].x), fmaf(y.y, f, v[x].y), fmaf(y.z, f, v[x].z), fmaf(y.w, f, v[x].w));
        }
      }
      sync();
    }
    if (x0 == 0) {
      red[tid] = sum;
      sync();
    }
#pragma unroll
    for (int x = 0; x < kPass; ++x) {
      const int i = tid + (x0 + x) * THREADS, row = i / (D / 4), d = (i % (D / 4)) * 4;
      if (works && row < rows) {
        float s = 0.f;
#pragma unroll
        for (int y = 0; y < kLanes; ++y) s += red[y * R + row];
        const int gr = seg.rt * R + row, qi = gr / p.group;
        const int64_t at = (qu.q0 + qi) * p.q_heads + seg.h * p.group + (gr - qi * p.group);
        const float inv = s == 0.f ? 0.f : 1.f / s;
        store_out4(p, at * D + d, make_float4(v[x].x * inv, v[x].y * inv, v[x].z * inv, v[x].w * inv));
      }
    }
  }
  if (p.lse) {
    if (lane_t == 0) wgt[row_t] = top;
    sync();
    if (tid < rows) {
      float s = 0.f;
#pragma unroll
      for (int y = 0; y < kLanes; ++y) s += red[y * R + tid];
      const int gr = seg.rt * R + tid, qi = gr / p.group;
      const int64_t at = (qu.q0 + qi) * p.q_heads + seg.h * p.group + (gr - qi * p.group);
      const float t = wgt[tid];
      p.lse[at] = s == 0.f ? -INFINITY : (t == -INFINITY ? s : (t + log2f(s)) * kLn2);
    }
  }
  sync();
}

// Launches `ctas` CTAs of a kernel with its layout's shared memory, programmatic stream serialisation on.
template <class L>
cudaError_t start_kernel(void (*kernel)(Params), int ctas, const Params &p, cudaStream_t stream) {
  static std::atomic<uint64_t> raised{0};  // devices on which its limit of dynamic shared memory has been raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(raised.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) raised.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < kMaxCtas ? ctas : kMaxCtas), 1, 1);
  cfg.blockDim = dim3(L::kThreads, 1, 1);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace attention
}  // namespace w4a16
