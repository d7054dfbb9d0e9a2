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
// row are 8, 16 or 32 neighbours and its minimum and maximum are a few shuffles.
#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
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
  int64_t tokens;
  int heads, head_dim, rot;
  int units;        // pieces of a row that one thread each handles
  int head_groups;  // threads that share a (token, unit): each takes every head_groups-th head
  bool copy_rest;   // out is not x: elements from rot on are copied
};

// V: elements of a vector (8: 16-byte accesses; 1: any size, stride and alignment). Half layout: a unit
// below rot / (2 V) is the pair of vectors (u, u + rot / (2 V)); the rest are copied vectors.
// Interleaved: V = 8: a unit is a vector; V = 1: a unit below rot / 2 is the pair (2 u, 2 u + 1).
template <class DT, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t idx = blockIdx.x * int64_t(kThreads) + threadIdx.x;
  const int64_t row = idx / p.units;
  const int u = static_cast<int>(idx - row * p.units);
  const int64_t t = row / p.head_groups;
  const int h0 = static_cast<int>(row - t * p.head_groups);
  if (t >= p.tokens) return;
  const int64_t pos = p.positions[t];
  const bool known = pos >= 0 && pos < p.table_rows;
  const float *row_c = p.table + (known ? pos : 0) * p.rot;
  const int half = p.rot / 2;
  const float nan = __int_as_float(0x7FFFFFFF);
  if constexpr (V == 8) {
    if constexpr (INTER) {
      const bool turned = u * 8 < p.rot;
      if (!turned && !p.copy_rest) return;
      float c[4], s[4];
      if (turned) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(row_c + u * 4));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(row_c + half + u * 4));
        c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
        s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
      }
#pragma unroll 4
      for (int h = h0; h < p.heads; h += p.head_groups) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p.x + t * p.x_ts + h * p.x_hs + u * 8);
        uint4 r = w;
        if (turned) {
          float x[8], y[8];
          unpack8<DT>(w, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[2 * j] = known ? turn_first(x[2 * j], x[2 * j + 1], c[j], s[j]) : nan;
            y[2 * j + 1] = known ? turn_second(x[2 * j], x[2 * j + 1], c[j], s[j]) : nan;
          }
          r = pack8<DT>(y);
        }
        *reinterpret_cast<uint4 *>(p.out + t * p.o_ts + h * p.o_hs + u * 8) = r;
      }
    } else {
      const int pairs = half / 8;
      if (u >= pairs) {  // a vector that is not turned
        if (!p.copy_rest) return;
        const int d = p.rot + (u - pairs) * 8;
        for (int h = h0; h < p.heads; h += p.head_groups)
          *reinterpret_cast<uint4 *>(p.out + t * p.o_ts + h * p.o_hs + d) =
              *reinterpret_cast<const uint4 *>(p.x + t * p.x_ts + h * p.x_hs + d);
        return;
      }
      float c[8], s[8];
      load8(row_c + u * 8, c);
      load8(row_c + half + u * 8, s);
#pragma unroll 4
      for (int h = h0; h < p.heads; h += p.head_groups) {
        const uint16_t *src = p.x + t * p.x_ts + h * p.x_hs + u * 8;
        float a[8], b[8], y1[8], y2[8];
        unpack8<DT>(*reinterpret_cast<const uint4 *>(src), a);
        unpack8<DT>(*reinterpret_cast<const uint4 *>(src + half), b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y1[j] = known ? turn_first(a[j], b[j], c[j], s[j]) : nan;
          y2[j] = known ? turn_second(a[j], b[j], c[j], s[j]) : nan;
        }
        uint16_t *dst = p.out + t * p.o_ts + h * p.o_hs + u * 8;
        *reinterpret_cast<uint4 *>(dst) = pack8<DT>(y1);
        *reinterpret_cast<uint4 *>(dst + half) = pack8<DT>(y2);
      }
    }
  } else {
    if (u >= half) {
      if (!p.copy_rest) return;
      const int d = p.rot + (u - half);
      for (int h = h0; h < p.heads; h += p.head_groups) p.out[t * p.o_ts + h * p.o_hs + d] = p.x[t * p.x_ts + h * p.x_hs + d];
      return;
    }
    const int d1 = INTER ? 2 * u : u, d2 = INTER ? 2 * u + 1 : u + half;
    const float c = row_c[u], s = row_c[half + u];
    for (int h = h0; h < p.heads; h += p.head_groups) {
      const uint16_t *src = p.x + t * p.x_ts + h * p.x_hs;
      const float a = lo16<DT>(src[d1]), b = lo16<DT>(src[d2]);
      uint16_t *dst = p.out + t * p.o_ts + h * p.o_hs;
      dst[d1] = static_cast<uint16_t>(pack16<DT>(known ? turn_first(a, b, c, s) : nan, 0.f));
      dst[d2] = static_cast<uint16_t>(pack16<DT>(known ? turn_second(a, b, c, s) : nan, 0.f));
    }
  }
}

struct WriteParams {
  uint8_t *cache;
  const uint16_t *k, *v, *q;
  uint16_t *q_out;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs;
  const int64_t *slots, *positions;
  const float *table;
  int64_t table_rows, tokens, slots_total;
  int q_heads, kv_heads, rot;
  int page_tiles;
  int64_t tile_bytes;
  bool interleaved;
  bool pair_vectors;  // rot / 2 is a multiple of 8 and the table's rows are 16-byte aligned
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

// One lane's 8 elements x (d0 = 8 * chunk) turned; src points at the row (the pair's other half is read
// from it again: it is in the first-level cache).
template <class DT>
__device__ __forceinline__ void turn8(const WriteParams &p, const uint16_t *src, int d0, int64_t t, float (&x)[8]) {
  if (d0 >= p.rot) return;
  const int64_t pos = p.positions[t];
  const bool known = pos >= 0 && pos < p.table_rows;
  const float *row = p.table + (known ? pos : 0) * p.rot;
  const int half = p.rot / 2;
  float y[8];
  if (p.pair_vectors && !p.interleaved) {
    const bool first = d0 < half;
    const int i0 = first ? d0 : d0 - half;
    float o[8], c[8], s[8];
    unpack8<DT>(*reinterpret_cast<const uint4 *>(src + (first ? d0 + half : d0 - half)), o);
    load8(row + i0, c);
    load8(row + half + i0, s);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = first ? turn_first(x[j], o[j], c[j], s[j]) : turn_second(o[j], x[j], c[j], s[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = d0 + j;
      const bool first = p.interleaved ? (d & 1) == 0 : d < half;
      const int i = p.interleaved ? d >> 1 : (first ? d : d - half);
      const bool in = d < p.rot;
      const int od = p.interleaved ? d ^ 1 : (first ? d + half : d - half);
      const float o = in ? lo16<DT>(src[od]) : 0.f;
      const float c = in ? __ldg(row + i) : 0.f, s = in ? __ldg(row + half + i) : 0.f;
      y[j] = !in ? x[j] : (first ? turn_first(x[j], o, c, s) : turn_second(o, x[j], c, s));
    }
  }
  const float nan = __int_as_float(0x7FFFFFFF);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (known || d0 + j >= p.rot) ? y[j] : nan;
}

// A row (token, head of q, k or v) for each group of LANES = head_dim / 8 lanes.
template <class DT, int LANES, int BITS, bool ROPE>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const WriteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int D = LANES * 8;
  const int64_t idx = (blockIdx.x * int64_t(kThreads) + threadIdx.x) / LANES;
  const int lane = threadIdx.x % LANES;
  const int rows = p.q_heads + 2 * p.kv_heads;
  const int64_t t = idx / rows;
  const int r = static_cast<int>(idx - t * rows);
  if (t >= p.tokens) return;
  const uint32_t mask = LANES == 32 ? 0xFFFFFFFFu : ((1u << (LANES & 31)) - 1u) << ((threadIdx.x & 31) / LANES * LANES);
  const bool is_q = r < p.q_heads;
  const int kind = is_q ? 0 : (r - p.q_heads) / p.kv_heads;  // of the cached rows: 0 keys, 1 values
  const int h = is_q ? r : r - p.q_heads - kind * p.kv_heads;
  const uint16_t *src = is_q ? p.q + t * p.q_ts + h * p.q_hs
                             : (kind == 0 ? p.k + t * p.k_ts + h * p.k_hs : p.v + t * p.v_ts + h * p.v_hs);
  const uint4 w = *reinterpret_cast<const uint4 *>(src + lane * 8);
  float x[8];
  unpack8<DT>(w, x);
  if constexpr (ROPE) {
    if (is_q || kind == 0) turn8<DT>(p, src, lane * 8, t, x);
  }
  if (is_q) {
    *reinterpret_cast<uint4 *>(p.q_out + (t * p.q_heads + h) * D + lane * 8) = pack8<DT>(x);
    return;
  }
  const int64_t slot = p.slots[t];
  if (slot < 0 || slot >= p.slots_total) return;  // the whole group leaves together
  if constexpr (ROPE) {
    const uint4 y = pack8<DT>(x);  // the key as a dtype tensor would hold it
    unpack8<DT>(y, x);
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    lo = min_nan(lo, x[j]);
    hi = max_nan(hi, x[j]);
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(mask, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(mask, hi, o));
  }
  constexpr float top = BITS == 8 ? 255.f : 15.f;
  constexpr float inv_top = 1.f / top;
  const bool finite = fabsf(lo) <= 3.402823466e38f && fabsf(hi) <= 3.402823466e38f;
  lo = fminf(lo, 0.f);
  hi = fmaxf(hi, 0.f);
  const uint16_t sbits = static_cast<uint16_t>(pack16<DT>(__fsub_rn(__fmul_rn(hi, inv_top), __fmul_rn(lo, inv_top)), 0.f));
  float s = lo16<DT>(sbits);
  if (s < kSmallest) s = 0.f;
  const float inv = (finite && s > 0.f) ? __frcp_rn(s) : 0.f;
  const float z = finite ? fminf(fmaxf(rintf(__fmul_rn(-lo, inv)), 0.f), top) : 0.f;
  uint32_t u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = finite ? __fmul_rn(x[j], inv) : 0.f;
    u[j] = static_cast<uint32_t>(fminf(fmaxf(__fadd_rn(rintf(v), z), 0.f), top));
  }
  const int64_t tile = slot / kTileTokens;
  const int row = static_cast<int>(slot % kTileTokens);
  const int64_t page = tile / p.page_tiles;
  uint8_t *dst = p.cache + ((page * p.kv_heads + h) * p.page_tiles + (tile - page * p.page_tiles)) * p.tile_bytes;
  constexpr int RB = D * BITS / 8;  // bytes of a row's codes
  uint8_t *codes = dst + kind * (kTileTokens * RB) + row * RB;
  if constexpr (BITS == 8) {
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
    *reinterpret_cast<uint32_t *>(dst + 2 * kTileTokens * RB + kind * 64 + row * 4) = bits16 | (static_cast<uint32_t>(z) << 16);
  }
}

struct ReadParams {
  const uint8_t *cache;
  const int64_t *slots;
  uint16_t *k_out, *v_out;
  int64_t tokens, slots_total;
  int kv_heads, page_tiles;
  int64_t tile_bytes;
};

template <class DT, int BITS>
__device__ __forceinline__ uint4 decode8(const uint8_t *codes, int lane, uint32_t param) {
  const float s = lo16<DT>(param & 0xFFFFu);
  const int z = static_cast<int>(param >> 16);
  float x[8];
  if constexpr (BITS == 8) {
    const uint2 w = *reinterpret_cast<const uint2 *>(codes + lane * 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = static_cast<float>(static_cast<int>(((j < 4 ? w.x : w.y) >> (8 * (j & 3))) & 0xFFu) - z) * s;
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + lane * 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = static_cast<float>(static_cast<int>((w >> (4 * j)) & 0xFu) - z) * s;
  }
  return pack8<DT>(x);
}

// A (token, head) for each group of LANES lanes: its key and its value.
template <class DT, int LANES, int BITS>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int D = LANES * 8, RB = D * BITS / 8;
  const int64_t idx = (blockIdx.x * int64_t(kThreads) + threadIdx.x) / LANES;
  const int lane = threadIdx.x % LANES;
  const int64_t t = idx / p.kv_heads;
  const int h = static_cast<int>(idx - t * p.kv_heads);
  if (t >= p.tokens) return;
  const int64_t slot = p.slots[t];
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  if (slot >= 0 && slot < p.slots_total) {
    const int64_t tile = slot / kTileTokens;
    const int row = static_cast<int>(slot % kTileTokens);
    const int64_t page = tile / p.page_tiles;
    const uint8_t *src = p.cache + ((page * p.kv_heads + h) * p.page_tiles + (tile - page * p.page_tiles)) * p.tile_bytes;
    const uint8_t *par = src + 2 * kTileTokens * RB + row * 4;
    k = decode8<DT, BITS>(src + row * RB, lane, *reinterpret_cast<const uint32_t *>(par));
    v = decode8<DT, BITS>(src + kTileTokens * RB + row * RB, lane, *reinterpret_cast<const uint32_t *>(par + 64));
  }
  const int64_t at = (t * p.kv_heads + h) * D + lane * 8;
  *reinterpret_cast<uint4 *>(p.k_out + at) = k;
  *reinterpret_cast<uint4 *>(p.v_out + at) = v;
}

// Launch with programmatic stream serialisation (the kernels wait for their predecessor themselves).
template <class P>
cudaError_t launch(void (*fn)(P), int64_t threads, const P &p, cudaStream_t stream) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
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

template <class DT>
cudaError_t rope_for(RopeParams &p, bool vec, bool inter, cudaStream_t stream) {
  p.units = vec ? (inter ? p.head_dim / 8 : p.rot / 16 + (p.head_dim - p.rot) / 8) : p.rot / 2 + (p.head_dim - p.rot);
  // four heads a thread (the table's row is read once for them), fewer when there is little work
  const int64_t full = int64_t(p.tokens) * p.units * p.heads;
  p.head_groups = full < 148 * 2048 ? p.heads : (p.heads + 3) / 4;
  const int64_t threads = p.tokens * p.head_groups * p.units;
  if (vec) return launch(inter ? rope_kernel<DT, 8, true> : rope_kernel<DT, 8, false>, threads, p, stream);
  return launch(inter ? rope_kernel<DT, 1, true> : rope_kernel<DT, 1, false>, threads, p, stream);
}

template <class DT, int LANES, int BITS>
cudaError_t write_for(const WriteParams &p, bool rope, cudaStream_t stream) {
  const int64_t threads = p.tokens * (p.q_heads + 2 * p.kv_heads) * LANES;
  return launch(rope ? kv_write_kernel<DT, LANES, BITS, true> : kv_write_kernel<DT, LANES, BITS, false>, threads, p, stream);
}
template <class DT, int BITS>
cudaError_t write_for(const WriteParams &p, int head_dim, bool rope, cudaStream_t stream) {
  if (head_dim == 64) return write_for<DT, 8, BITS>(p, rope, stream);
  if (head_dim == 128) return write_for<DT, 16, BITS>(p, rope, stream);
  return write_for<DT, 32, BITS>(p, rope, stream);
}
template <class DT, int BITS>
cudaError_t read_for(const ReadParams &p, int head_dim, cudaStream_t stream) {
  const int64_t threads = p.tokens * p.kv_heads * (head_dim / 8);
  if (head_dim == 64) return launch(kv_read_kernel<DT, 8, BITS>, threads, p, stream);
  if (head_dim == 128) return launch(kv_read_kernel<DT, 16, BITS>, threads, p, stream);
  return launch(kv_read_kernel<DT, 32, BITS>, threads, p, stream);
}

}  // namespace

cudaError_t launch_rope(const HeadsView &x, const HeadsView &out, int64_t tokens, int heads, int head_dim, int dtype,
                        const RopeArgs &rope, cudaStream_t stream) {
  RopeParams p{};
  p.x = static_cast<const uint16_t *>(x.ptr);
  p.out = static_cast<uint16_t *>(const_cast<void *>(out.ptr));
  p.x_ts = x.token_stride;
  p.x_hs = x.head_stride;
  p.o_ts = out.token_stride;
  p.o_hs = out.head_stride;
  p.positions = rope.positions;
  p.table = rope.table;
  p.table_rows = rope.table_rows;
  p.tokens = tokens;
  p.heads = heads;
  p.head_dim = head_dim;
  p.rot = rope.rot_dim;
  p.copy_rest = x.ptr != out.ptr;
  const bool vec = vec_ok(x) && vec_ok(out) && head_dim % 8 == 0 && rope.rot_dim % (rope.interleaved ? 8 : 16) == 0 &&
                   aligned(rope.table, 16);
  return dtype == W4A16_BF16 ? rope_for<BF16>(p, vec, rope.interleaved, stream)
                             : rope_for<F16>(p, vec, rope.interleaved, stream);
}

cudaError_t launch_kv_write(const w4a16_kv_cache_t &cache, const HeadsView &k, const HeadsView &v, const int64_t *slots,
                            int64_t tokens, int dtype, const RopeArgs &rope, const HeadsView &q, int q_heads, void *q_out,
                            cudaStream_t stream) {
  WriteParams p{};
  p.cache = static_cast<uint8_t *>(cache.data);
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
  p.tokens = tokens;
  p.slots_total = cache.num_pages * cache.page_size;
  p.q_heads = q.ptr ? q_heads : 0;
  p.kv_heads = cache.kv_heads;
  p.rot = rope.rot_dim;
  p.page_tiles = cache.page_size / kTileTokens;
  p.tile_bytes = kv_tile_bytes(cache.head_dim, cache.bits);
  p.interleaved = rope.interleaved;
  p.pair_vectors = rope.rot_dim % 16 == 0 && aligned(rope.table, 16);
  const bool turn = rope.positions != nullptr;
  if (dtype == W4A16_BF16)
    return cache.bits == 8 ? write_for<BF16, 8>(p, cache.head_dim, turn, stream)
                           : write_for<BF16, 4>(p, cache.head_dim, turn, stream);
  return cache.bits == 8 ? write_for<F16, 8>(p, cache.head_dim, turn, stream)
                         : write_for<F16, 4>(p, cache.head_dim, turn, stream);
}

cudaError_t launch_kv_read(const w4a16_kv_cache_t &cache, const int64_t *slots, int64_t tokens, void *k_out, void *v_out,
                           int dtype, cudaStream_t stream) {
  ReadParams p{};
  p.cache = static_cast<const uint8_t *>(cache.data);
  p.slots = slots;
  p.k_out = static_cast<uint16_t *>(k_out);
  p.v_out = static_cast<uint16_t *>(v_out);
  p.tokens = tokens;
  p.slots_total = cache.num_pages * cache.page_size;
  p.kv_heads = cache.kv_heads;
  p.page_tiles = cache.page_size / kTileTokens;
  p.tile_bytes = kv_tile_bytes(cache.head_dim, cache.bits);
  if (dtype == W4A16_BF16)
    return cache.bits == 8 ? read_for<BF16, 8>(p, cache.head_dim, stream) : read_for<BF16, 4>(p, cache.head_dim, stream);
  return cache.bits == 8 ? read_for<F16, 8>(p, cache.head_dim, stream) : read_for<F16, 4>(p, cache.head_dim, stream);
}

}  // namespace w4a16
