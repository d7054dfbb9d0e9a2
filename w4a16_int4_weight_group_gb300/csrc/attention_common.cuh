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

// a / b of numbers that are not negative, in 32 bits where they fit (a 64-bit division takes hundreds of cycles).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// The list of `total` units cut into `ctas` contiguous shares, the first `extra` of them one unit longer.
struct Shares {
  int64_t total, ctas, each, extra;
  __device__ __forceinline__ int64_t begin(int64_t c) const { return c * each + (c < extra ? c : extra); }
  // the CTA whose share holds unit u
  __device__ __forceinline__ int64_t owner(int64_t u) const {
    const int64_t longer = extra * (each + 1);
    return u < longer ? quotient(u, each + 1) : extra + quotient(u - longer, each);
  }
};
__device__ __forceinline__ unsigned int add_acq_rel(unsigned int *p, unsigned int v) {
  unsigned int old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// Cached tokens of a sequence: its length, at least zero, at most what its row of the page table holds, and at most
// 2^31 - 256, so that the positions of its last unit (64 to 256 tokens) are still 32-bit numbers.
constexpr int kMaxLength = 0x7FFFFF00;
__device__ __forceinline__ int length_of(const Params &p, int b) {
  const int64_t pages = p.max_pages * p.page_tiles * 16;
  const int len = p.kv_lens[b];
  return len < 0 ? 0 : static_cast<int>(min(int64_t(min(len, kMaxLength)), pages));
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
__device__ __forceinline__ void store_out4(uint16_t *out, bool bf16, int64_t at, float4 v) {
  uint2 w;
  if (bf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  } else {
    w = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
  }
  *reinterpret_cast<uint2 *>(out + at) = w;
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

// This CTA's share of the units: an equal part of the list over all sequences (it starts at cur, has `units` units
// and ends before unit u1). False when there is nothing for it. Without a workspace the share is the segments that
// start in that part, whole. Called by all threads; scan_s has a word for each of the W warps, share_s two words.
template <class L, int W>
__device__ __forceinline__ bool share_of(const Params &p, int64_t *scan_s, volatile int64_t *share_s, Cursor &cur, Shares &sh,
                                         int64_t &u1, int64_t &units) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t cta = blockIdx.x;
  auto scan = [&](int64_t x) {  // over the warp's lanes, this one's included
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += v;
    }
    return x;
  };
  auto cut = [&](int64_t total) {
    sh.total = total;
    sh.ctas = total < gridDim.x ? total : gridDim.x;
    if (cta >= sh.ctas) return false;
    sh.each = quotient(total, sh.ctas);
    sh.extra = total - sh.each * sh.ctas;
    u1 = sh.begin(cta + 1);
    return true;
  };
  int64_t u0, at;  // the share's first unit, among all and in its sequence
  if (p.batch <= 32) {
    // a lane for each sequence, every warp for itself: no barrier, and no second look at the lengths
    int64_t mine = 0;
    if (lane < p.batch) mine = load_sequence<L>(p, lane, cur);
    const int64_t upto = scan(mine);
    if (!cut(__shfl_sync(0xFFFFFFFFu, upto, 31))) return false;
    u0 = sh.begin(cta);
    const int b = __popc(__ballot_sync(0xFFFFFFFFu, upto <= u0));
    at = u0 - __shfl_sync(0xFFFFFFFFu, upto - mine, b);
    cur.b = b;
    cur.nb = __shfl_sync(0xFFFFFFFFu, cur.nb, b);
    cur.nrt = __shfl_sync(0xFFFFFFFFu, cur.nrt, b);
    cur.len = __shfl_sync(0xFFFFFFFFu, cur.len, b);
  } else {
    const int slice = (p.batch + 32 * W - 1) / (32 * W);
    int64_t mine = 0;
    for (int b = tid * slice; b < min(p.batch, (tid + 1) * slice); ++b) mine += load_sequence<L>(p, b, cur);
    const int64_t upto = scan(mine);
    if (lane == 31) scan_s[warp] = upto;
    __syncthreads();
    int64_t before = upto - mine, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int64_t v = scan_s[w];
      if (w < warp) before += v;
      total += v;
    }
    if (!cut(total)) return false;
    u0 = sh.begin(cta);
    if (u0 >= before && u0 < before + mine) {
      int64_t rest = u0 - before;
      for (int b = tid * slice;; ++b) {
        const int64_t n = load_sequence<L>(p, b, cur);
        if (rest < n) {
          share_s[0] = b;
          share_s[1] = rest;
          break;
        }
        rest -= n;
      }
    }
    __syncthreads();
    load_sequence<L>(p, static_cast<int>(share_s[0]), cur);
    at = share_s[1];
  }
  cur.h = static_cast<int>(quotient(at, int64_t(cur.nb) * cur.nrt));
  at -= int64_t(cur.h) * cur.nb * cur.nrt;
  cur.rt = static_cast<int>(quotient(at, cur.nb));
  cur.blk = static_cast<int>(at - int64_t(cur.rt) * cur.nb);
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

// NaN into the rows that are not computed, where the caller asks for it: those of a sequence past its first max_q (a CTA
// for each sequence, from the last one on: in small calls these have no share), those before the first sequence and after
// the last, and those of a sequence whose ends are no rows of q. One look at two words a sequence where there are none.
// (Streaming kernel: at its start, since behind the loops over the cache it adds up to 70 bytes of spills to those. Tiles: at
// its end; at the start it held up every role, 2 us of a call of 352.)
template <int D, int THREADS>
__device__ __forceinline__ void fill_unowned(const Params &p, int tid) {
  if (!p.fill) return;
  auto nan_rows = [&](int64_t from, int64_t to) {
    from = from > 0 ? from : 0;
    to = to < p.total_q ? to : p.total_q;
    if (from >= to) return;
    const int64_t each = int64_t(p.q_heads) * (D / 8);  // 16-byte vectors of a row
    if (p.fill & 1)
      for (int64_t i = from * each + tid; i < to * each; i += THREADS)
        reinterpret_cast<uint4 *>(p.out)[i] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
    if ((p.fill & 2) && p.lse)
      for (int64_t i = from * p.q_heads + tid; i < to * p.q_heads; i += THREADS) p.lse[i] = __int_as_float(0x7FFFFFFF);
  };
  for (int64_t b = gridDim.x - 1 - blockIdx.x; b <= p.batch; b += gridDim.x) {
    if (b == p.batch) {
      nan_rows(0, p.q_start[0]);
      nan_rows(p.q_start[b], p.total_q);
    } else {
      const int64_t q0 = p.q_start[b], q1 = p.q_start[b + 1];
      const bool valid = q0 >= 0 && q0 <= q1 && q1 <= p.total_q;
      nan_rows(valid ? q0 + (q1 - q0 < p.max_q ? q1 - q0 : p.max_q) : q0, q1);
    }
  }
}

// Barrier of THREADS threads: the CTA's own (BAR 0) or a named one.
template <int BAR, int THREADS>
__device__ __forceinline__ void sync_threads() {
  if constexpr (BAR == 0) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"n"(BAR), "n"(THREADS) : "memory");
}

// A split segment's parts and where its rows go.
struct Parts {
  const float *slot0, *slot1;  // of the first part and of the second; those after it are two slots apart each
  int count;
  int rows;              // of the row tile in use
  int first_row;         // of the row tile among the cache head's
  int group, q_heads, head0;  // query heads of a cache head, of all, and the first of this cache head
  int64_t q0;            // row of the sequence's first query token
  uint16_t *out;
  float *lse;
  bool bf16;
  float *scratch;        // THREADS + CHUNK * R floats
};
__device__ __forceinline__ Parts parts_of(const Params &p, const Cursor &seg, const Queries &qu, int rows, int height, int64_t c0, int count,
                                          int64_t slot_floats, float *scratch) {
  return Parts{p.partials + (2 * c0 + 1) * slot_floats, p.partials + 2 * (c0 + 1) * slot_floats, count, rows, seg.rt * height, p.group,
               p.q_heads, seg.h * p.group, qu.q0, p.out, p.lse, p.bf16 != 0, scratch};
}

// The split segments that this CTA was the last to finish: at most two (the share's first and last). They are joined
// after the share: inside it the joining's registers would push the loops over the cache into local memory.
struct Pending {
  Parts parts[2];
  int count;
};
// Counts this CTA's part of a segment (units seg_u .. seg_u + nb - 1 of the list) in, its partial result being
// written by the threads that `sync` joins; the last one to come is to join them.
template <int BAR, int THREADS>
__device__ __forceinline__ void count_in(const Params &p, const Shares &sh, const Cursor &seg, const Queries &qu, int rows, int height,
                                         int64_t seg_u, int64_t slot_floats, float *scratch, Pending *pending, int tid) {
  sync_threads<BAR, THREADS>();
  if (tid == 0) {
    const int64_t c0 = sh.owner(seg_u);
    const int parts = static_cast<int>(sh.owner(seg_u + seg.nb - 1) - c0) + 1;
    if (add_acq_rel(p.flags + c0, 1u) == static_cast<unsigned int>(parts - 1)) {
      p.flags[c0] = 0u;
      pending->parts[pending->count++] = parts_of(p, seg, qu, rows, height, c0, parts, slot_floats, scratch);
    }
  }
}

// Adds the parts of a split segment and writes its rows: THREADS threads, the parts in the order of the CTAs. The
// maxima and denominators first, side by side (the parts of one long sequence are many), then the weighted sums with
// many loads in flight: with one part after the other this took 11000 of the 36000 cycles of a call over 8192 tokens
// (131073 tokens 76.5 us, joined this way 67.7).
template <int R, int D, int THREADS, int CHUNK, int BAR>
__device__ __forceinline__ void join_parts(const Parts &g, const int tid) {
  auto sync = [] { sync_threads<BAR, THREADS>(); };
  const int parts = g.count, rows = g.rows;
  float *scratch = g.scratch;
  float *red = scratch;            // [THREADS / R][R]
  float *wgt = scratch + THREADS;  // [CHUNK][R]
  constexpr int kLanes = THREADS / R;
  const int row_t = tid % R, lane_t = tid / R;
  constexpr int kFloats = R * (D + 2);
  auto slot = [&](int c) { return c == 0 ? g.slot0 : g.slot1 + int64_t(c - 1) * (2 * kFloats); };
  auto place = [&](int row) {  // of a row among all query heads of all tokens
    const int gr = g.first_row + row, qi = gr / g.group;
    return (g.q0 + qi) * g.q_heads + g.head0 + (gr - qi * g.group);
  };
  constexpr int kPer = (R * D / 4 + THREADS - 1) / THREADS;  // groups of four elements of a thread
  constexpr int kPass = kPer < 4 ? kPer : 4;                 // of them at a time
  constexpr int kFlight = kPass == 1 ? 16 : kPass == 2 ? 8 : 4;  // parts whose loads are in flight
  auto mine = [&](int x) { return R * D / 4 % THREADS == 0 || tid + x * THREADS < R * D / 4; };  // this thread has group x
  float4 y[kFlight][kPass];
  auto fetch = [&](int c0, int end, int x0) {
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (c0 + f < end) {
        const float4 *src = reinterpret_cast<const float4 *>(slot(c0 + f)) + tid + x0 * THREADS;
#pragma unroll
        for (int x = 0; x < kPass; ++x)
          if (mine(x0 + x)) y[f][x] = __ldcg(src + x * THREADS);
      }
    }
  };
  fetch(0, min(parts, CHUNK), 0);  // (in flight while the weights are made)
  // the first parts' maxima and denominators, kept for the weights
  constexpr int kKeep = 4;
  float mc[kKeep], lc[kKeep], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int c = lane_t + i * kLanes;
    mc[i] = -INFINITY;
    lc[i] = 0.f;
    if (c < parts) {
      const float *s = slot(c);
      mc[i] = __ldcg(s + R * D + row_t);
      lc[i] = __ldcg(s + R * (D + 1) + row_t);
    }
  }
#pragma unroll
  for (int i = 0; i < kKeep; ++i) top = fmaxf(top, mc[i]);
  for (int c = lane_t + kKeep * kLanes; c < parts; c += kLanes) top = fmaxf(top, __ldcg(slot(c) + R * D + row_t));
  red[tid] = top;
  sync();
#pragma unroll
  for (int x = 0; x < kLanes; ++x) top = fmaxf(top, red[x * R + row_t]);
  sync();
  auto weight = [&](float m, float l) { return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2_approx(m - top); };
  float sum = 0.f;
#pragma unroll 1
  for (int x0 = 0; x0 < kPer; x0 += kPass) {
    float4 v[kPass];
#pragma unroll
    for (int x = 0; x < kPass; ++x) v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int cc = 0; cc < parts; cc += CHUNK) {
      const int now = min(CHUNK, parts - cc);
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int c = lane_t + i * kLanes;
        if (c < parts && c >= cc && c < cc + now) {
          const float f = weight(mc[i], lc[i]);
          wgt[(c - cc) * R + row_t] = f;
          if (x0 == 0) sum += lc[i] * f;
        }
      }
      // (parts past the kept ones: the same threads, read again)
      for (int c = lane_t + kKeep * kLanes; c < cc + now; c += kLanes) {
        if (c < cc) continue;
        const float m = __ldcg(slot(c) + R * D + row_t), l = __ldcg(slot(c) + R * (D + 1) + row_t);
        const float f = weight(m, l);
        wgt[(c - cc) * R + row_t] = f;
        if (x0 == 0) sum += l * f;
      }
      sync();
      {
#pragma unroll 1
        for (int c = 0; c < now; c += kFlight) {
          if (c + cc + x0 > 0) fetch(cc + c, cc + now, x0);
#pragma unroll
          for (int f = 0; f < kFlight; ++f) {
            if (c + f < now) {
#pragma unroll
              for (int x = 0; x < kPass; ++x) {
                if (!mine(x0 + x)) continue;
                const float k = wgt[(c + f) * R + (tid + (x0 + x) * THREADS) / (D / 4)];
                v[x] = make_float4(fmaf(y[f][x].x, k, v[x].x), fmaf(y[f][x].y, k, v[x].y), fmaf(y[f][x].z, k, v[x].z),
                                   fmaf(y[f][x].w, k, v[x].w));
              }
            }
          }
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
      if (mine(x0 + x) && row < rows) {
        float s = 0.f;
#pragma unroll
        for (int y = 0; y < kLanes; ++y) s += red[y * R + row];
        const float inv = s == 0.f ? 0.f : 1.f / s;
        store_out4(g.out, g.bf16, place(row) * D + d, make_float4(v[x].x * inv, v[x].y * inv, v[x].z * inv, v[x].w * inv));
      }
    }
  }
  if (g.lse) {
    if (lane_t == 0) wgt[row_t] = top;
    sync();
    if (tid < rows) {
      float s = 0.f;
#pragma unroll
      for (int y = 0; y < kLanes; ++y) s += red[y * R + tid];
      const float t = wgt[tid];
      g.lse[place(tid)] = s == 0.f ? -INFINITY : (t == -INFINITY ? s : (t + log2f(s)) * kLn2);
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
