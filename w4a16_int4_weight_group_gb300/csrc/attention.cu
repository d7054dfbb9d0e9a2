// Attention of drafted tokens over the quantised paged cache: dispatch, workspace and failure detection
// (the kernels: attention_stream.cuh and attention_tiles.cuh).
#include <mutex>

#include "attention.h"

namespace w4a16 {
namespace attention {
namespace {

__device__ Control g_control;

// Address of the control block on the current device, looked up once for each device.
cudaError_t control_of(int device, Control **out) {
  static std::mutex mu;
  static Control *known[64] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (device >= 0 && device < 64 && known[device]) {
    *out = known[device];
    return cudaSuccess;
  }
  void *ptr = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&ptr, g_control);
  if (e != cudaSuccess) return e;
  *out = static_cast<Control *>(ptr);
  if (device >= 0 && device < 64) known[device] = *out;
  return cudaSuccess;
}

}  // namespace
}  // namespace attention

using namespace attention;

cudaError_t launch_tree_attention(const AttentionArgs &a, const DeviceInfo &dev) {
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
  p.tree_mask = a.tree_mask;
  p.scale = a.scale;
  p.out = static_cast<uint16_t *>(a.out);
  p.lse = a.lse;
  p.fill = a.q_start ? a.fill : 0;  // without q_start every row is a sequence's
  p.total_q = a.total_q;
  p.batch = static_cast<int>(a.batch);
  p.q_heads = a.q_heads;
  p.kv_heads = a.cache.kv_heads;
  p.group = a.q_heads / a.cache.kv_heads;
  p.page_tiles = a.cache.page_size / kTileTokens;
  p.max_q = a.max_q;
  p.page_shift = -1;
  for (int i = 0; i < 20; ++i)
    if (p.page_tiles == 1 << i) p.page_shift = i;
  p.bf16 = a.dtype == W4A16_BF16;
  if (a.workspace && a.workspace_bytes >= tree_attention_workspace_bytes(a.max_q, a.q_heads, p.kv_heads, a.cache.head_dim, dev.num_sms)) {
    p.flags = static_cast<unsigned int *>(a.workspace);
    p.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kFlagBytes);
  }
  const cudaError_t e = control_of(dev.device, &p.control);
  if (e != cudaSuccess) return e;
  if (use_tiles(a.max_q * p.group, a.cache.head_dim))
    return a.cache.head_dim == 64 ? launch_tiles<64>(p, a.cache.bits, dev.num_sms, a.stream)
                                  : launch_tiles<128>(p, a.cache.bits, dev.num_sms, a.stream);
  const int rows = stream_rows(a.max_q * p.group, a.cache.head_dim);
  const bool wide = a.cache.bits == 8;
  switch (a.cache.head_dim) {
    case 64: return wide ? launch_stream<64, 8>(p, rows, dev.num_sms, a.stream) : launch_stream<64, 4>(p, rows, dev.num_sms, a.stream);
    case 128: return wide ? launch_stream<128, 8>(p, rows, dev.num_sms, a.stream) : launch_stream<128, 4>(p, rows, dev.num_sms, a.stream);
    default: return wide ? launch_stream<256, 8>(p, rows, dev.num_sms, a.stream) : launch_stream<256, 4>(p, rows, dev.num_sms, a.stream);
  }
}

size_t tree_attention_workspace_bytes(int max_q, int q_heads, int kv_heads, int head_dim, int num_sms) {
  const int max_rows = max_q * (q_heads / kv_heads);
  const bool tiles = use_tiles(max_rows, head_dim);
  const int rows = tiles ? kTileRows : stream_rows(max_rows, head_dim);
  const int64_t want = tiles ? num_sms : 2 * num_sms, ctas = want < kMaxCtas ? want : kMaxCtas;
  return kFlagBytes + static_cast<size_t>(2 * ctas * partial_floats(rows, head_dim) * 4);
}

cudaError_t attention_take_device_error(uint32_t *err) {
  Control c;
  cudaError_t e = cudaMemcpyFromSymbol(&c, g_control, sizeof(c));
  if (e != cudaSuccess) return e;
  *err = c.error;
  c.error = 0;
  return *err ? cudaMemcpyToSymbol(g_control, &c, sizeof(c)) : cudaSuccess;
}
cudaError_t attention_set_wait_limit_ns(uint64_t ns) {
  const unsigned long long v = ns;
  return cudaMemcpyToSymbol(g_control, &v, sizeof(v), offsetof(Control, limit_ns));
}
cudaError_t attention_set_stall(bool on) {
  const unsigned int v = on ? 1u : 0u;
  return cudaMemcpyToSymbol(g_control, &v, sizeof(v), offsetof(Control, stall));
}

}  // namespace w4a16
