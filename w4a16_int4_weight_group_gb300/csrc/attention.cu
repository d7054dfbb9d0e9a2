// Attention of drafted tokens over the quantised paged cache.
//
//     s_t = scale (q . k_t),  k_t = (u_t - z_t) s^k_t over the positions t that the query may see,
//     out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),   lse = m + log sum_t exp(s_t - m)
//
// A sequence's cache holds kv_len tokens, the last n of them the drafted ones. Query i sees every token
// before the drafted ones and the drafted tokens whose bits are set in its mask word (without masks:
// the drafted tokens up to itself).
//
// One warp for each (query, head): one pass with the running maximum and sum.
#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

struct Params {
  const uint8_t *cache;
  const uint16_t *q;
  int64_t q_ts, q_hs;
  const int32_t *q_start, *kv_lens, *page_table;
  int64_t max_pages, num_pages, tile_bytes;
  const uint64_t *tree_mask;
  float scale;
  uint16_t *out;
  float *lse;
  int64_t batch, total_q;
  int q_heads, kv_heads, page_size, max_q;
};

template <class DT, int D, int BITS>
__global__ void __launch_bounds__(128) attend_simple(const Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t w = blockIdx.x * 4ll + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  const int h = static_cast<int>(w % p.q_heads);
  const int i = static_cast<int>(w / p.q_heads % p.max_q);
  const int64_t b = w / p.q_heads / p.max_q;
  if (b >= p.batch) return;
  const int64_t q0 = p.q_start ? p.q_start[b] : b, q1 = p.q_start ? p.q_start[b + 1] : b + 1;
  const int n = static_cast<int>(q1 - q0);
  if (i >= n) return;
  const int64_t row = q0 + i;
  if (row < 0 || row >= p.total_q) return;
  constexpr int E = D / 32, RB = D * BITS / 8;
  const uint16_t *qp = p.q + row * p.q_ts + h * p.q_hs + lane * E;
  float q[E], o[E];
  for (int e = 0; e < E; ++e) q[e] = bits_to_float(qp[e], DT::kBF16) * p.scale, o[e] = 0.f;
  const int64_t cap = p.max_pages * p.page_size;
  const int len = static_cast<int>(p.kv_lens[b] < cap ? p.kv_lens[b] : cap);
  const int first = len - n;
  const int hk = h / (p.q_heads / p.kv_heads);
  const uint64_t word = p.tree_mask ? p.tree_mask[row] : (i >= 63 ? ~0ull : (2ull << i) - 1);
  const int page_tiles = p.page_size / kTileTokens;
  float m = -INFINITY, sum = 0.f;
  for (int t = 0; t < len; ++t) {
    if (t >= first && !((word >> (t - first)) & 1)) continue;
    const int page = p.page_table[b * p.max_pages + t / p.page_size];
    if (page < 0 || page >= p.num_pages) continue;
    const uint8_t *tile = p.cache + ((int64_t(page) * p.kv_heads + hk) * page_tiles + t % p.page_size / kTileTokens) * p.tile_bytes;
    const int r = t % kTileTokens;
    const uint32_t pk = *reinterpret_cast<const uint32_t *>(tile + 32 * RB + 4 * r);
    const uint32_t pv = *reinterpret_cast<const uint32_t *>(tile + 32 * RB + 64 + 4 * r);
    float dot = 0.f, v[E];
    for (int e = 0; e < E; ++e) {
      const int d = lane * E + e;
      int uk, uv;
      if (BITS == 8) {
        uk = tile[r * RB + d];
        uv = tile[16 * RB + r * RB + d];
      } else {
        uk = (tile[r * RB + d / 2] >> (4 * (d & 1))) & 15;
        uv = (tile[16 * RB + r * RB + d / 2] >> (4 * (d & 1))) & 15;
      }
      dot += q[e] * static_cast<float>(uk - static_cast<int>(pk >> 16));
      v[e] = static_cast<float>(uv - static_cast<int>(pv >> 16)) * bits_to_float(pv & 0xFFFF, DT::kBF16);
    }
    for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, x);
    const float s = dot * bits_to_float(pk & 0xFFFF, DT::kBF16);
    const float m2 = fmaxf(m, s);
    const float f = m == m2 ? 1.f : expf(m - m2), e1 = s == m2 ? 1.f : expf(s - m2);
    m = m2;
    sum = sum * f + e1;
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + e1 * v[e];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int e = 0; e < E; ++e) {
    const float y = sum == 0.f ? 0.f : o[e] * inv;
    reinterpret_cast<typename DT::T *>(p.out)[(row * p.q_heads + h) * D + lane * E + e] = DT::from_float_rn(y);
  }
  if (p.lse && lane == 0) p.lse[row * p.q_heads + h] = sum == 0.f ? -INFINITY : m + logf(sum);
}

template <class DT, int D, int BITS>
cudaError_t go(const Params &p, cudaStream_t stream) {
  const int64_t warps = p.batch * p.max_q * p.q_heads;
  attend_simple<DT, D, BITS><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}
template <class DT, int BITS>
cudaError_t go(const Params &p, int head_dim, cudaStream_t stream) {
  if (head_dim == 64) return go<DT, 64, BITS>(p, stream);
  if (head_dim == 128) return go<DT, 128, BITS>(p, stream);
  return go<DT, 256, BITS>(p, stream);
}

}  // namespace

cudaError_t launch_tree_attention(const AttentionArgs &a, const DeviceInfo &) {
  Params p{};
  p.cache = static_cast<const uint8_t *>(a.cache.data);
  p.q = static_cast<const uint16_t *>(a.q.ptr);
  p.q_ts = a.q.token_stride;
  p.q_hs = a.q.head_stride;
  p.q_start = a.q_start;
  p.kv_lens = a.kv_lens;
  p.page_table = a.page_table;
  p.max_pages = a.max_pages;
  p.num_pages = a.cache.num_pages;
  p.tile_bytes = kv_tile_bytes(a.cache.head_dim, a.cache.bits);
  p.tree_mask = a.tree_mask;
  p.scale = a.scale;
  p.out = static_cast<uint16_t *>(a.out);
  p.lse = a.lse;
  p.batch = a.batch;
  p.total_q = a.total_q;
  p.q_heads = a.q_heads;
  p.kv_heads = a.cache.kv_heads;
  p.page_size = a.cache.page_size;
  p.max_q = a.max_q;
  if (a.dtype == W4A16_BF16)
    return a.cache.bits == 8 ? go<BF16, 8>(p, a.cache.head_dim, a.stream) : go<BF16, 4>(p, a.cache.head_dim, a.stream);
  return a.cache.bits == 8 ? go<F16, 8>(p, a.cache.head_dim, a.stream) : go<F16, 4>(p, a.cache.head_dim, a.stream);
}

size_t tree_attention_workspace_bytes(int, int, int, int, int) { return 0; }

}  // namespace w4a16
