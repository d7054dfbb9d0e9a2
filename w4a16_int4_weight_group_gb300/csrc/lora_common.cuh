// What the two forms of the low-rank adapters share: tiles of sorted tokens and the parts of h.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace lora {

struct Tile {
  int adapter, first, count;  // of the sorted tokens
};

// A number of h as the sum of this many of the dtype: all 24 bits for bfloat16, 22 below the token's largest for float16 (scaled before)
template <class DT>
constexpr int kParts = DT::kBF16 ? 3 : 2;

// The next part of two numbers, as a pair of the dtype; the numbers become what is left of them
template <class DT>
__device__ __forceinline__ uint32_t take_part(float &a, float &b) {
  uint32_t w;
  float ha, hb;
  if constexpr (DT::kBF16) {  // truncated, so that a finite number's part is finite; the third one is exact
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    w = prmt(ua, ub, 0x7632);
    ha = __uint_as_float(ua & 0xFFFF0000u), hb = __uint_as_float(ub & 0xFFFF0000u);
    if (!(a == a)) w |= 0x7FFFu;  // a NaN's payload may lie in the lost bits
    if (!(b == b)) w |= 0x7FFF0000u;
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    w = *reinterpret_cast<const uint32_t *>(&h);
    ha = __low2float(h), hb = __high2float(h);
  }
  // an infinite or NaN number has no rest
  a = fabsf(a) < INFINITY ? a - ha : 0.f, b = fabsf(b) < INFINITY ? b - hb : 0.f;
  return w;
}

// The power of two that brings a token's largest number to [2^13, 2^14), as what its sums are multiplied by in the end (float16)
__device__ __forceinline__ float unit_of_largest(float top) {
  const int e = static_cast<int>(__float_as_uint(top) >> 23);  // 0: zero or subnormal; 255: infinite
  const int d = e == 0 || e == 255 ? 0 : max(-126, min(126, e - 127 - 13));
  return __uint_as_float(static_cast<uint32_t>(127 + d) << 23);
}

// a pair of the dtype plus two sums (times a power of two), each rounded once
template <class DT>
__device__ __forceinline__ void add2(uint32_t &w, float a, float b, float f) {
  if constexpr (DT::kBF16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(__uint_as_float(w << 16) + a, __uint_as_float(w & 0xFFFF0000u) + b);
    w = *reinterpret_cast<const uint32_t *>(&r);
  } else {
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    const __half2 r = __floats2half2_rn(fmaf(a, f, x.x), fmaf(b, f, x.y));
    w = *reinterpret_cast<const uint32_t *>(&r);
  }
}

// The form for many tokens (sorted tiles of kLongTile tokens, lists in `order`, `tiles` and `num_tiles`; h: workspace)
constexpr int kLongTile = 128;
cudaError_t launch_long(const LoraArgs &a, const DeviceInfo &dev, const int32_t *order, const Tile *tiles, const int32_t *num_tiles, float *h);
size_t long_workspace_bytes(int64_t tokens, int rank);

}  // namespace lora
}  // namespace w4a16
