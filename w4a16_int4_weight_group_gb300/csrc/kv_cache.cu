// Rotary positions and the quantised paged cache of keys and values.
//
// Rotation of the pair (x1, x2) at position p, frequency i:
//     y1 = x1 cos - x2 sin,   y2 = x1 sin + x2 cos,   cos and sin = table[p][i], table[p][rot / 2 + i]
// in fp32 without contraction (each product and sum rounded by itself, so that the result does not
// depend on how the compiler pairs them), rounded once to the dtype. Half layout: the pair is
// (i, i + rot / 2); interleaved: (2 i, 2 i + 1). Elements from rot on are copied.
//
// Quantisation of one (token, head) row of keys or of values, L = 255 (8 bits) or 15 (4 bits):
//     lo = min(0, min x), hi = max(0, max x), s = RNE_dtype(hi / L - lo / L), z = rint(-lo / s),
//     u = clamp(rint(x / s) + z, 0, L),   value = (u - z) s
// i.e. the weights' own dequantisation rule, one group per row. 1 / L and 1 / s are rounded to fp32
// first and multiplied. A scale under the smallest normal fp32 number is zero (the row reads back as
// zeros); a row with an infinity or a NaN gets the scale NaN and reads back as NaN.
//
// Layout: a tile holds 16 tokens of one head in one contiguous piece (K codes, V codes, K parameters, V
// parameters), so that the attention fetches a tile with one bulk copy.
//
// All three kernels are bound by memory: a lane handles 8 elements (16 bytes), so that the lanes of a
// row are 8, 16 or 32 neighbours and its minimum and maximum are a few shuffles. A thread takes up to four heads (the
// write: two) of one token: their loads are in flight together, and the token's cosines and sines (four times the bytes of a
// 16-bit vector), its slot and its place in the cache are fetched once for them. With little work it takes one.
//
// Measured (share of the device's 6782 GB/s copy rate):
//  * rotation of 8191 tokens x 48 heads of 128, 64 rotated, interleaved: 36.5 us for 203 MB, 5.6 TB/s (0.82; one head a
//    thread: 44), 128 rotated 38; half layout (92 to 94 registers, where the other has 52) 41 with 128 rotated, 52 with 64.
//    Parts that do not divide into 16-byte vectors go element by element: 40 of 128 rotated 132 us, 20 of 80 90 us for 127 MB
//  * write with rotation of 8192 tokens, 40 q and 8 cached heads, 8 bits: 57 us with the
//    read of the same tokens after it, 274 MB in all, 4.8 TB/s (0.71); in the write (50 us with a cold cache) the
//    schedulers issue in 73 % of the cycles (the reductions and conversions of each row); interleaved 54, 4 bits 59 for
//    257 MB; 40 of 128 rotated, element by element, 99 (that kernel spills 380 bytes a thread at its 40 registers)
//  * read of 50001 tokens of 8 heads, 4 bits: 41 us for 260 MB, 6.3 TB/s (0.93); 8 bits 49 for 311 MB (0.93)
//  * 5 tokens turned, 16 tokens written and read: 7.5 to 10 and 20 to 24 us, the host's time to issue one and two calls;
//    replayed from a graph 1.6 and 3.5
#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads whose loads a thread has in flight together
constexpr int kRows = 2;   // rows of the cache write (6 CTAs of 40 registers an SM: 57 us for 8192 tokens; 4 rows at 64 registers: 59)
constexpr float kSmallest = 1.17549435e-38f;  // smallest normal fp32 number

template <class DT>
__device__ __forceinline__ float lo16(uint32_t w) {
  if constexpr (DT::kBF16) return __uint_as_float(w << 16);
  else return __half2float(__ushort_as_half(static_cast<unsigned short>(w & 0xFFFFu)));
}
template <class DT>
__device__ __forceinline__ float hi16(uint32_t w) {
  if constexpr (DT::kBF16) return __uint_as_float(w & 0xFFFF0000u);
  else return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16)));
}
template <class DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (DT::kBF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}
template <class DT>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  x[0] = lo16<DT>(w.x); x[1] = hi16<DT>(w.x);
  x[2] = lo16<DT>(w.y); x[3] = hi16<DT>(w.y);
  x[4] = lo16<DT>(w.z); x[5] = hi16<DT>(w.z);
  x[6] = lo16<DT>(w.w); x[7] = hi16<DT>(w.w);
}
template <class DT>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack16<DT>(x[0], x[1]), pack16<DT>(x[2], x[3]), pack16<DT>(x[4], x[5]), pack16<DT>(x[6], x[7]));
}

// The two results of one pair, each product and sum rounded by itself.
__device__ __forceinline__ float turn_first(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_second(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
}

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

struct RopeParams {
  const uint16_t *x;
  uint16_t *out;
  int64_t x_ts, x_hs, o_ts, o_hs;
  const int64_t *positions;
  const float *table;
  int64_t table_rows;
  uint32_t threads;  // tokens * head_groups * units
  int heads, rot;
  uint32_t units;        // pieces of a row that one thread each handles
  uint32_t head_groups;  // threads that share a (token, unit): each takes every head_groups-th head
  bool copy_rest;   // out is not x: elements from rot on are copied
};

// V: elements of a vector (8: 16-byte accesses; 1: any size, stride and alignment). Half layout: a unit
// below rot / (2 V) is the pair of vectors (u, u + rot / (2 V)); the rest are copied vectors.
// Interleaved: V = 8: a unit is a vector; V = 1: a unit below rot / 2 is the pair (2 u, 2 u + 1).
template <class DT, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t idx = blockIdx.x * kThreads + threadIdx.x;
  if (idx >= p.threads) return;
  const uint32_t row = idx / p.units;
  const int u = static_cast<int>(idx - row * p.units);
  const int64_t t = row / p.head_groups;
  const int h0 = static_cast<int>(row - static_cast<uint32_t>(t) * p.head_groups);
  const int step = static_cast<int>(p.head_groups);
  const int64_t pos = p.positions[t];
  const bool known = pos >= 0 && pos < p.table_rows;
  const float *row_c = p.table + (known ? pos : 0) * p.rot;
  const int half = p.rot / 2;
  const float nan = __int_as_float(0x7FFFFFFF);
  const uint16_t *x_t = p.x + t * p.x_ts;
  uint16_t *o_t = p.out + t * p.o_ts;
  if constexpr (V == 8) {
    const int pairs = half / 8;
    const bool turned = INTER ? u * 8 < p.rot : u < pairs;
    if (!turned && !p.copy_rest) return;
    const int d = INTER || turned ? u * 8 : p.rot + (u - pairs) * 8;
    float c[8], s[8];
    if (turned) {
      if constexpr (INTER) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(row_c + u * 4));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(row_c + half + u * 4));
        c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
        s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
      } else {
        load8(row_c + u * 8, c);
        load8(row_c + half + u * 8, s);
      }
    }
    for (int hb = h0; hb < p.heads; hb += kHeads * step) {
      uint4 w[kHeads], w2[kHeads];  // all loads first: the stores might, as far as the compiler knows, touch them
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int h = hb + i * step;
        if (h < p.heads) {
          w[i] = *reinterpret_cast<const uint4 *>(x_t + h * p.x_hs + d);
          if (!INTER && turned) w2[i] = *reinterpret_cast<const uint4 *>(x_t + h * p.x_hs + d + half);
        }
      }
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int h = hb + i * step;
        if (h >= p.heads) continue;
        uint16_t *dst = o_t + h * p.o_hs + d;
        if (!turned) {
          *reinterpret_cast<uint4 *>(dst) = w[i];
        } else if constexpr (INTER) {
          float x[8], y[8];
          unpack8<DT>(w[i], x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[2 * j] = known ? turn_first(x[2 * j], x[2 * j + 1], c[j], s[j]) : nan;
            y[2 * j + 1] = known ? turn_second(x[2 * j], x[2 * j + 1], c[j], s[j]) : nan;
          }
          *reinterpret_cast<uint4 *>(dst) = pack8<DT>(y);
        } else {
          float a[8], b[8], y1[8], y2[8];
          unpack8<DT>(w[i], a);
          unpack8<DT>(w2[i], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            y1[j] = known ? turn_first(a[j], b[j], c[j], s[j]) : nan;
            y2[j] = known ? turn_second(a[j], b[j], c[j], s[j]) : nan;
          }
          *reinterpret_cast<uint4 *>(dst) = pack8<DT>(y1);
          *reinterpret_cast<uint4 *>(dst + half) = pack8<DT>(y2);
        }
      }
    }
  } else {
    if (u >= half) {
      if (!p.copy_rest) return;
      const int d = p.rot + (u - half);
      for (int h = h0; h < p.heads; h += step) o_t[h * p.o_hs + d] = x_t[h * p.x_hs + d];
      return;
    }
    const int d1 = INTER ? 2 * u : u, d2 = INTER ? 2 * u + 1 : u + half;
    const float c = row_c[u], s = row_c[half + u];
    for (int h = h0; h < p.heads; h += step) {
      const uint16_t *src = x_t + h * p.x_hs;
      const float a = lo16<DT>(src[d1]), b = lo16<DT>(src[d2]);
      uint16_t *dst = o_t + h * p.o_hs;
      dst[d1] = static_cast<uint16_t>(pack16<DT>(known ? turn_first(a, b, c, s) : nan, 0.f));
      dst[d2] = static_cast<uint16_t>(pack16<DT>(known ? turn_second(a, b, c, s) : nan, 0.f));
    }
  }
}

// A cache as the kernels see it.
struct CacheView {
  uint8_t *data;
  int64_t slots_total, tile_bytes;
  int kv_heads, page_tiles;
  int page_shift;  // log2 of page_tiles, or -1
};
// Tile of cache head 0 that holds a slot (the tile of head h: h * page_tiles further), and the row in it.
__device__ __forceinline__ int64_t tile_of(const CacheView &c, int64_t slot, int &row) {
  const uint32_t tile = static_cast<uint32_t>(slot / kTileTokens);  // the cache holds fewer than 2^31 tiles
  row = static_cast<int>(slot % kTileTokens);
  const uint32_t page = c.page_shift >= 0 ? tile >> c.page_shift : tile / static_cast<uint32_t>(c.page_tiles);
  return int64_t(page) * c.kv_heads * c.page_tiles + (tile - page * c.page_tiles);
}

struct WriteParams {
  CacheView cache;
  const uint16_t *k, *v, *q;
  uint16_t *q_out;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs;
  const int64_t *slots, *positions;
  const float *table;
  int64_t table_rows;
  uint32_t groups;      // tokens * row_groups
  uint32_t row_groups;  // groups of up to ROWS rows of a token: heads of q (q_groups of them), then of k and v
  int q_groups, q_heads, rot, bits;
  bool interleaved;
};

// Minimum or maximum that keeps a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// How a row's elements turn: not at all; in the half layout with whole vectors (rot / 2 a multiple of 8); interleaved
// (rot a multiple of 8); any other layout, element by element.
enum Mode { kNone, kHalf, kInterleaved, kElements };

// The cosines and sines of a lane's 8 elements (d0 = 8 * lane) at its token's position, so that an element x with its
// pair's other element o becomes x c + o s (the sign of the pair's first element is in s).
struct Turn {
  float c[8], s[8];
};
template <int MODE>
__device__ __forceinline__ void load_turn(const WriteParams &p, int64_t t, int d0, Turn &w) {
  const int64_t pos = p.positions[t];
  const bool known = pos >= 0 && pos < p.table_rows;
  const float *row = p.table + (known ? pos : 0) * p.rot;
  const int half = p.rot / 2;
  if constexpr (MODE == kHalf) {
    const bool first = d0 < half;
    const int i0 = first ? d0 : d0 - half;
    load8(row + i0, w.c);
    load8(row + half + i0, w.s);
#pragma unroll
    for (int j = 0; j < 8; ++j) w.s[j] = first ? -w.s[j] : w.s[j];
  } else if constexpr (MODE == kInterleaved) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(row + d0 / 2));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(row + half + d0 / 2));
    const float c[4] = {a.x, a.y, a.z, a.w}, s[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w.c[j] = c[j / 2];
      w.s[j] = j & 1 ? s[j / 2] : -s[j / 2];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = d0 + j;
      const bool in = d < p.rot, first = p.interleaved ? (d & 1) == 0 : d < half;
      const int i = p.interleaved ? d >> 1 : (first ? d : d - half);
      w.c[j] = in ? __ldg(row + i) : 1.f;
      w.s[j] = in ? (first ? -__ldg(row + half + i) : __ldg(row + half + i)) : 0.f;
    }
  }
  if (!known) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (MODE != kElements || d0 + j < p.rot) w.c[j] = __int_as_float(0x7FFFFFFF);
  }
}
// x: the lane's elements of the row at src; other: their pairs' other elements (kHalf).
template <class DT, int MODE>
__device__ __forceinline__ void turn8(const WriteParams &p, const uint16_t *src, int d0, const Turn &w, const uint4 &other, float (&x)[8]) {
  float o[8];
  if constexpr (MODE == kHalf) {
    unpack8<DT>(other, o);
  } else if constexpr (MODE == kInterleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = x[j ^ 1];
  } else {
    const int half = p.rot / 2;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = d0 + j;
      o[j] = d < p.rot ? lo16<DT>(src[p.interleaved ? d ^ 1 : (d < half ? d + half : d - half)]) : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float y = __fadd_rn(__fmul_rn(x[j], w.c[j]), __fmul_rn(o[j], w.s[j]));
    if (MODE != kElements || d0 + j < p.rot) x[j] = y;
  }
}

// Up to ROWS consecutive rows of a token for each group of LANES = head_dim / 8 lanes: heads of q, or of k and then
// v. The rows' reductions go side by side (a row's alone would wait for each of its shuffles).
template <class DT, int LANES, int MODE, int ROWS>
__global__ void __launch_bounds__(kThreads, 6) kv_write_kernel(const WriteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int D = LANES * 8;
  const uint32_t idx = (blockIdx.x * kThreads + threadIdx.x) / LANES;
  const int lane = threadIdx.x % LANES, d0 = lane * 8;
  if (idx >= p.groups) return;  // the whole group leaves together
  const uint32_t t = idx / p.row_groups;
  const int g = static_cast<int>(idx - t * p.row_groups);
  const int half = p.rot / 2, pair_at = d0 < half ? d0 + half : d0 - half;
  if (MODE != kNone && g < p.q_groups) {
    const int r0 = g * ROWS;
    const uint16_t *src = p.q + t * p.q_ts + r0 * p.q_hs;
    const bool turns = d0 < p.rot;
    uint4 w[ROWS], other[MODE == kHalf ? ROWS : 1];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (r0 + i < p.q_heads) {
        w[i] = *reinterpret_cast<const uint4 *>(src + i * p.q_hs + d0);
        if (MODE == kHalf && turns) other[i] = *reinterpret_cast<const uint4 *>(src + i * p.q_hs + pair_at);
      }
    }
    Turn turn;
    if (turns) load_turn<MODE>(p, t, d0, turn);
    uint16_t *dst = p.q_out + (int64_t(t) * p.q_heads + r0) * D + d0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (r0 + i < p.q_heads) {
        float x[8];
        unpack8<DT>(w[i], x);
        if (turns) turn8<DT, MODE>(p, src + i * p.q_hs, d0, turn, other[MODE == kHalf ? i : 0], x);
        *reinterpret_cast<uint4 *>(dst + i * D) = pack8<DT>(x);
      }
    }
    return;
  }
  const int kv = p.cache.kv_heads, r0 = (g - p.q_groups) * ROWS;
  const int64_t slot = p.slots[t];
  if (slot < 0 || slot >= p.cache.slots_total) return;
  const uint32_t mask = LANES == 32 ? 0xFFFFFFFFu : ((1u << (LANES & 31)) - 1u) << ((threadIdx.x & 31) / LANES * LANES);
  const bool turns = MODE != kNone && d0 < p.rot && r0 < kv;
  uint4 w[ROWS], other[MODE == kHalf ? ROWS : 1];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + i;
    w[i] = make_uint4(0, 0, 0, 0);
    if (r < 2 * kv) {
      const uint16_t *src = r < kv ? p.k + t * p.k_ts + r * p.k_hs : p.v + t * p.v_ts + (r - kv) * p.v_hs;
      w[i] = *reinterpret_cast<const uint4 *>(src + d0);
      if (MODE == kHalf && turns && r < kv) other[i] = *reinterpret_cast<const uint4 *>(src + pair_at);
    }
  }
  if (turns) {
    Turn turn;
    load_turn<MODE>(p, t, d0, turn);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (r0 + i < kv) {
        float x[8];
        unpack8<DT>(w[i], x);
        turn8<DT, MODE>(p, p.k + t * p.k_ts + (r0 + i) * p.k_hs, d0, turn, other[MODE == kHalf ? i : 0], x);
        w[i] = pack8<DT>(x);  // the key as a dtype tensor would hold it
      }
    }
  }
  float lo[ROWS], hi[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    float x[8];
    unpack8<DT>(w[i], x);
    lo[i] = hi[i] = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      lo[i] = min_nan(lo[i], x[j]);
      hi[i] = max_nan(hi[i], x[j]);
    }
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      lo[i] = min_nan(lo[i], __shfl_xor_sync(mask, lo[i], o));
      hi[i] = max_nan(hi[i], __shfl_xor_sync(mask, hi[i], o));
    }
  }
  int row = 0;
  uint8_t *tile0 = p.cache.data + tile_of(p.cache, slot, row) * p.cache.tile_bytes;
  const float top = p.bits == 8 ? 255.f : 15.f, inv_top = p.bits == 8 ? 1.f / 255.f : 1.f / 15.f;
  const int row_bytes = D * p.bits / 8;  // of its codes
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + i;
    if (r >= 2 * kv) break;
    const int kind = r < kv ? 0 : 1;  // keys, values
    const bool finite = fabsf(lo[i]) <= 3.402823466e38f && fabsf(hi[i]) <= 3.402823466e38f;
    const float low = fminf(lo[i], 0.f), high = fmaxf(hi[i], 0.f);
    const uint16_t sbits = static_cast<uint16_t>(pack16<DT>(__fsub_rn(__fmul_rn(high, inv_top), __fmul_rn(low, inv_top)), 0.f));
    float s = lo16<DT>(sbits);
    if (s < kSmallest) s = 0.f;
    const float inv = (finite && s > 0.f) ? __frcp_rn(s) : 0.f;
    const float z = finite ? fminf(fmaxf(rintf(__fmul_rn(-low, inv)), 0.f), top) : 0.f;
    float x[8];
    unpack8<DT>(w[i], x);
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = finite ? __fmul_rn(x[j], inv) : 0.f;
      u[j] = static_cast<uint32_t>(fminf(fmaxf(__fadd_rn(rintf(v), z), 0.f), top));
    }
    uint8_t *dst = tile0 + int64_t(r - kind * kv) * p.cache.page_tiles * p.cache.tile_bytes;
    uint8_t *codes = dst + (kind * kTileTokens + row) * row_bytes;
    if (p.bits == 8) {
      const uint32_t a = u[0] | (u[1] << 8) | (u[2] << 16) | (u[3] << 24);
      const uint32_t b = u[4] | (u[5] << 8) | (u[6] << 16) | (u[7] << 24);
      *reinterpret_cast<uint2 *>(codes + lane * 8) = make_uint2(a, b);
    } else {
      uint32_t a = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) a |= u[j] << (4 * j);
      *reinterpret_cast<uint32_t *>(codes + lane * 4) = a;
    }
    if (lane == 0) {
      const uint32_t bits16 = finite ? static_cast<uint16_t>(pack16<DT>(s, 0.f)) : 0x7FFFu;
      *reinterpret_cast<uint32_t *>(dst + 2 * kTileTokens * row_bytes + kind * 64 + row * 4) = bits16 | (static_cast<uint32_t>(z) << 16);
    }
  }
}

struct ReadParams {
  CacheView cache;
  const int64_t *slots;
  uint16_t *k_out, *v_out;
  uint32_t groups;       // tokens * head_groups
  uint32_t head_groups;  // groups of up to HEADS consecutive heads
};

// Eight values from their codes (4 bits: in w.x).
template <class DT, int BITS>
__device__ __forceinline__ uint4 decode8(uint2 w, uint32_t param) {
  const float s = lo16<DT>(param & 0xFFFFu);
  const int z = static_cast<int>(param >> 16);
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = BITS == 8 ? ((j < 4 ? w.x : w.y) >> (8 * (j & 3))) & 0xFFu : (w.x >> (4 * j)) & 0xFu;
    x[j] = static_cast<float>(static_cast<int>(u) - z) * s;
  }
  return pack8<DT>(x);
}
template <int BITS>
__device__ __forceinline__ uint2 load_codes(const uint8_t *codes, int lane) {
  if constexpr (BITS == 8) return __ldg(reinterpret_cast<const uint2 *>(codes) + lane);
  else return make_uint2(__ldg(reinterpret_cast<const uint32_t *>(codes) + lane), 0u);
}

// The keys and values of up to HEADS consecutive heads of a token for each group of LANES lanes.
template <class DT, int LANES, int BITS, int HEADS>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int D = LANES * 8, RB = D * BITS / 8;
  const uint32_t idx = (blockIdx.x * kThreads + threadIdx.x) / LANES;
  const int lane = threadIdx.x % LANES;
  if (idx >= p.groups) return;
  const uint32_t t = idx / p.head_groups;
  const int h0 = static_cast<int>(idx - t * p.head_groups) * HEADS;
  const int64_t slot = p.slots[t];
  uint2 k[HEADS], v[HEADS];
  uint32_t pk[HEADS], pv[HEADS];
  const bool stored = slot >= 0 && slot < p.cache.slots_total;
  int row = 0;
  const int64_t tile0 = stored ? tile_of(p.cache, slot, row) : 0;
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    k[i] = v[i] = make_uint2(0, 0);
    pk[i] = pv[i] = 0;
    if (stored && h0 + i < p.cache.kv_heads) {
      const uint8_t *src = p.cache.data + (tile0 + int64_t(h0 + i) * p.cache.page_tiles) * p.cache.tile_bytes;
      const uint32_t *par = reinterpret_cast<const uint32_t *>(src + 2 * kTileTokens * RB) + row;
      k[i] = load_codes<BITS>(src + row * RB, lane);
      v[i] = load_codes<BITS>(src + (kTileTokens + row) * RB, lane);
      pk[i] = __ldg(par);
      pv[i] = __ldg(par + kTileTokens);
    }
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    if (h0 + i >= p.cache.kv_heads) break;
    const int64_t at = (int64_t(t) * p.cache.kv_heads + h0 + i) * D + lane * 8;
    *reinterpret_cast<uint4 *>(p.k_out + at) = decode8<DT, BITS>(k[i], pk[i]);
    *reinterpret_cast<uint4 *>(p.v_out + at) = decode8<DT, BITS>(v[i], pv[i]);
  }
}

// Launch with programmatic stream serialisation (the kernels wait for their predecessor themselves).
template <class P>
cudaError_t launch(void (*fn)(P), int64_t threads, const P &p, cudaStream_t stream) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

bool vec_ok(const HeadsView &x) { return aligned(x.ptr, 16) && x.token_stride % 8 == 0 && x.head_stride % 8 == 0; }

// Threads of one launch (32-bit indices): calls with more run as several launches over their tokens.
constexpr int64_t kMaxThreads = int64_t(1) << 31;
// Threads of a call, one head each, below which a thread takes one head. One tuned value for the three kernels (heads
// of 128, 152 SMs, replayed; one / several heads a thread): rotation of 48 heads, 128 tokens 2.0 / 2.3 us, 512 tokens 4.4 / 3.2, 4096
// tokens 42 / 19; write of 40 + 2 x 8 heads with the read after it, 128 tokens 3.9 / 4.9, 512 tokens 7.0 / 7.4, 1024 tokens
// 10.6 / 10.0, 4096 tokens 39 / 31; read of 8 heads at 4 bits, 512 tokens 1.75 / 2.05, 1024 tokens 2.3 / 2.1.
constexpr int64_t kFill = 303104;

CacheView view_of(const w4a16_kv_cache_t &c) {
  CacheView v{static_cast<uint8_t *>(c.data), c.num_pages * c.page_size, kv_tile_bytes(c.head_dim, c.bits), c.kv_heads,
              c.page_size / kTileTokens, -1};
  for (int i = 0; i < 20; ++i)
    if (v.page_tiles == 1 << i) v.page_shift = i;
  return v;
}

template <class DT>
cudaError_t rope_for(const RopeParams &p, bool vec, bool inter, cudaStream_t stream) {
  if (vec) return launch(inter ? rope_kernel<DT, 8, true> : rope_kernel<DT, 8, false>, p.threads, p, stream);
  return launch(inter ? rope_kernel<DT, 1, true> : rope_kernel<DT, 1, false>, p.threads, p, stream);
}

// Work items of a token in groups of up to `most` (1 when all of them one by one are fewer than kFill).
int items_a_group(int64_t tokens, int items, int lanes, int most) { return tokens * items * lanes < kFill ? 1 : most; }

template <class DT, int LANES, int ROWS>
cudaError_t write_rows(const WriteParams &p, int mode, cudaStream_t stream) {
  const int64_t threads = int64_t(p.groups) * LANES;
  switch (mode) {
    case kNone: return launch(kv_write_kernel<DT, LANES, kNone, ROWS>, threads, p, stream);
    case kHalf: return launch(kv_write_kernel<DT, LANES, kHalf, ROWS>, threads, p, stream);
    case kInterleaved: return launch(kv_write_kernel<DT, LANES, kInterleaved, ROWS>, threads, p, stream);
    default: return launch(kv_write_kernel<DT, LANES, kElements, ROWS>, threads, p, stream);
  }
}
template <class DT, int LANES>
cudaError_t write_for(WriteParams p, int64_t tokens, int mode, cudaStream_t stream) {
  const int rows = p.q_heads + 2 * p.cache.kv_heads;
  const int each = items_a_group(tokens, rows, LANES, kRows);
  p.q_groups = (p.q_heads + each - 1) / each;
  p.row_groups = static_cast<uint32_t>(p.q_groups + (2 * p.cache.kv_heads + each - 1) / each);
  const int64_t most = kMaxThreads / (int64_t(p.row_groups) * LANES) - 1;
  for (int64_t done = 0; done < tokens; done += most) {
    const int64_t n = tokens - done < most ? tokens - done : most;
    WriteParams c = p;
    c.groups = static_cast<uint32_t>(n * p.row_groups);
    c.k += done * p.k_ts;
    c.v += done * p.v_ts;
    if (c.q) c.q += done * p.q_ts, c.q_out += done * p.q_heads * (LANES * 8);
    c.slots += done;
    if (c.positions) c.positions += done;
    const cudaError_t e = each == 1 ? write_rows<DT, LANES, 1>(c, mode, stream) : write_rows<DT, LANES, kRows>(c, mode, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <class DT>
cudaError_t write_for(const WriteParams &p, int64_t tokens, int head_dim, int mode, cudaStream_t stream) {
  if (head_dim == 64) return write_for<DT, 8>(p, tokens, mode, stream);
  if (head_dim == 128) return write_for<DT, 16>(p, tokens, mode, stream);
  return write_for<DT, 32>(p, tokens, mode, stream);
}
template <class DT, int LANES, int BITS>
cudaError_t read_for(ReadParams p, int64_t tokens, cudaStream_t stream) {
  const int each = items_a_group(tokens, p.cache.kv_heads, LANES, kHeads);
  p.head_groups = static_cast<uint32_t>((p.cache.kv_heads + each - 1) / each);
  const int64_t most = kMaxThreads / (int64_t(p.head_groups) * LANES) - 1;
  for (int64_t done = 0; done < tokens; done += most) {
    const int64_t n = tokens - done < most ? tokens - done : most;
    ReadParams c = p;
    c.groups = static_cast<uint32_t>(n * p.head_groups);
    c.slots += done;
    c.k_out += done * p.cache.kv_heads * (LANES * 8);
    c.v_out += done * p.cache.kv_heads * (LANES * 8);
    const int64_t threads = int64_t(c.groups) * LANES;
    const cudaError_t e = launch(each == 1 ? kv_read_kernel<DT, LANES, BITS, 1> : kv_read_kernel<DT, LANES, BITS, kHeads>, threads, c, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <class DT, int BITS>
cudaError_t read_for(const ReadParams &p, int64_t tokens, int head_dim, cudaStream_t stream) {
  if (head_dim == 64) return read_for<DT, 8, BITS>(p, tokens, stream);
  if (head_dim == 128) return read_for<DT, 16, BITS>(p, tokens, stream);
  return read_for<DT, 32, BITS>(p, tokens, stream);
}

}  // namespace

cudaError_t launch_rope(const HeadsView &x, const HeadsView &out, int64_t tokens, int heads, int head_dim, int dtype,
                        const RopeArgs &rope, cudaStream_t stream) {
  RopeParams p{};
  p.x_ts = x.token_stride;
  p.x_hs = x.head_stride;
  p.o_ts = out.token_stride;
  p.o_hs = out.head_stride;
  p.table = rope.table;
  p.table_rows = rope.table_rows;
  p.heads = heads;
  p.rot = rope.rot_dim;
  p.copy_rest = x.ptr != out.ptr;
  const bool inter = rope.interleaved;
  const bool vec = vec_ok(x) && vec_ok(out) && head_dim % 8 == 0 && rope.rot_dim % (inter ? 8 : 16) == 0 && aligned(rope.table, 16);
  p.units = static_cast<uint32_t>(vec ? (inter ? head_dim / 8 : p.rot / 16 + (head_dim - p.rot) / 8) : p.rot / 2 + (head_dim - p.rot));
  const int each = items_a_group(tokens, heads, static_cast<int>(p.units), kHeads);
  p.head_groups = static_cast<uint32_t>((heads + each - 1) / each);
  const int64_t most = kMaxThreads / (int64_t(p.units) * p.head_groups) - 1;
  for (int64_t done = 0; done < tokens; done += most) {
    const int64_t n = tokens - done < most ? tokens - done : most;
    p.x = static_cast<const uint16_t *>(x.ptr) + done * x.token_stride;
    p.out = static_cast<uint16_t *>(const_cast<void *>(out.ptr)) + done * out.token_stride;
    p.positions = rope.positions + done;
    p.threads = static_cast<uint32_t>(n * p.units * p.head_groups);
    const cudaError_t e = dtype == W4A16_BF16 ? rope_for<BF16>(p, vec, inter, stream) : rope_for<F16>(p, vec, inter, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_kv_write(const w4a16_kv_cache_t &cache, const HeadsView &k, const HeadsView &v, const int64_t *slots,
                            int64_t tokens, int dtype, const RopeArgs &rope, const HeadsView &q, int q_heads, void *q_out,
                            cudaStream_t stream) {
  WriteParams p{};
  p.cache = view_of(cache);
  p.k = static_cast<const uint16_t *>(k.ptr);
  p.v = static_cast<const uint16_t *>(v.ptr);
  p.q = static_cast<const uint16_t *>(q.ptr);
  p.q_out = static_cast<uint16_t *>(q_out);
  p.k_ts = k.token_stride;
  p.k_hs = k.head_stride;
  p.v_ts = v.token_stride;
  p.v_hs = v.head_stride;
  p.q_ts = q.token_stride;
  p.q_hs = q.head_stride;
  p.slots = slots;
  p.positions = rope.positions;
  p.table = rope.table;
  p.table_rows = rope.table_rows;
  p.q_heads = q.ptr ? q_heads : 0;
  p.rot = rope.rot_dim;
  p.interleaved = rope.interleaved;
  p.bits = cache.bits;
  int mode = kNone;
  if (rope.positions) {
    mode = kElements;
    if (aligned(rope.table, 16)) {
      if (!rope.interleaved && rope.rot_dim % 16 == 0) mode = kHalf;
      if (rope.interleaved && rope.rot_dim % 8 == 0) mode = kInterleaved;
    }
  }
  return dtype == W4A16_BF16 ? write_for<BF16>(p, tokens, cache.head_dim, mode, stream)
                             : write_for<F16>(p, tokens, cache.head_dim, mode, stream);
}

cudaError_t launch_kv_read(const w4a16_kv_cache_t &cache, const int64_t *slots, int64_t tokens, void *k_out, void *v_out,
                           int dtype, cudaStream_t stream) {
  ReadParams p{};
  p.cache = view_of(cache);
  p.slots = slots;
  p.k_out = static_cast<uint16_t *>(k_out);
  p.v_out = static_cast<uint16_t *>(v_out);
  if (dtype == W4A16_BF16)
    return cache.bits == 8 ? read_for<BF16, 8>(p, tokens, cache.head_dim, stream)
                           : read_for<BF16, 4>(p, tokens, cache.head_dim, stream);
  return cache.bits == 8 ? read_for<F16, 8>(p, tokens, cache.head_dim, stream)
                         : read_for<F16, 4>(p, tokens, cache.head_dim, stream);
}

}  // namespace w4a16
