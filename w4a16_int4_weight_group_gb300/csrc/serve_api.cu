// C ABI of the serving operators next to the linear layer: argument validation and launches.
#include <cmath>

#include "internal.h"

using namespace w4a16;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 31;
constexpr int kMaxHeads = 1024;
constexpr int kMaxTopK = 32;

w4a16_status check_dtype(int dtype) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16)
    return fail(W4A16_ERR_UNSUPPORTED, "Only float16/bfloat16 tensors are supported (dtype %d)", dtype);
  return W4A16_OK;
}

w4a16_status check_cache(const w4a16_kv_cache_t *c, int dtype) {
  if (!c) return fail(W4A16_ERR_INVALID_ARG, "cache must not be NULL");
  const w4a16_status st = check_dtype(dtype);
  if (st != W4A16_OK) return st;
  if (c->bits != 4 && c->bits != 8) return fail(W4A16_ERR_UNSUPPORTED, "cache bits %d not supported; supported: [4, 8]", c->bits);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(W4A16_ERR_UNSUPPORTED, "cache head_dim %d not supported; supported: [64, 128, 256]", c->head_dim);
  if (c->page_size <= 0 || c->page_size % kTileTokens != 0 || c->page_size > (1 << 20))
    return fail(W4A16_ERR_INVALID_ARG, "page_size (%d) must be a positive multiple of 16, at most 2^20", c->page_size);
  if (c->kv_heads <= 0 || c->kv_heads > kMaxHeads)
    return fail(W4A16_ERR_INVALID_ARG, "kv_heads (%d) must be in [1, %d]", c->kv_heads, kMaxHeads);
  if (c->num_pages <= 0 || c->num_pages >= (int64_t(1) << 31) || c->num_pages * (c->page_size / kTileTokens) >= (int64_t(1) << 31))
    return fail(W4A16_ERR_INVALID_ARG, "num_pages (%lld) must be positive and the cache hold fewer than 2^31 tiles of 16 tokens",
                (long long)c->num_pages);
  if (!c->data) return fail(W4A16_ERR_INVALID_ARG, "cache data must not be NULL");
  if (!aligned(c->data, 128)) return fail(W4A16_ERR_MISALIGNED, "cache data must be 128-byte aligned");
  return W4A16_OK;
}

int64_t cache_bytes(const w4a16_kv_cache_t &c) {
  return c.num_pages * c.kv_heads * (c.page_size / kTileTokens) * kv_tile_bytes(c.head_dim, c.bits);
}

// Bytes from the first to the last element of a strided [tokens, heads, head_dim] tensor of 16-bit elements.
Range view_range(const HeadsView &v, int64_t tokens, int heads, int head_dim) {
  const int64_t last = (tokens - 1) * v.token_stride + int64_t(heads - 1) * v.head_stride + head_dim;
  return range(v.ptr, last * 2);
}

// A strided tensor as the kernels get it: a dimension of one element has no stride that counts.
HeadsView view(const void *ptr, int64_t token_stride, int64_t head_stride, int64_t tokens, int heads) {
  return HeadsView{ptr, tokens == 1 ? 0 : token_stride, heads == 1 ? 0 : head_stride};
}

w4a16_status check_view(const HeadsView &v, int64_t tokens, int heads, int head_dim, const char *name, bool vectors) {
  if (!v.ptr) return fail(W4A16_ERR_INVALID_ARG, "%s must not be NULL", name);
  if ((heads > 1 && v.head_stride < head_dim) || (tokens > 1 && v.token_stride < 1) || v.head_stride < 0 || v.token_stride < 0)
    return fail(W4A16_ERR_INVALID_ARG, "%s: head stride %lld and token stride %lld do not hold rows of %d elements", name,
                (long long)v.head_stride, (long long)v.token_stride, head_dim);
  if (!aligned(v.ptr, vectors ? 16 : 2) || (vectors && (v.head_stride % 8 != 0 || v.token_stride % 8 != 0)))
    return fail(W4A16_ERR_MISALIGNED, vectors ? "%s must be 16-byte aligned, its strides multiples of 8 elements"
                                              : "%s must be 2-byte aligned", name);
  return W4A16_OK;
}

// Whether two rows (token, head) of a checked view share elements: |dt token_stride - dh head_stride| < head_dim for some dt and
// dh that are not both zero. (Both signs of dh: only equal ones can come near, since strides are not negative.)
bool rows_overlap(const HeadsView &v, int64_t tokens, int heads, int head_dim) {
  if (tokens == 1) return false;  // (the heads of a token are apart: check_view)
  if (v.token_stride < head_dim) return true;
  if (v.token_stride >= int64_t(heads - 1) * v.head_stride + head_dim) return false;
  for (int64_t dh = 1; dh < heads; ++dh) {
    const int64_t at = dh * v.head_stride, dt = at / v.token_stride;  // the tokens before and after that offset
    if ((dt < tokens && at - dt * v.token_stride < head_dim) || (dt + 1 < tokens && (dt + 1) * v.token_stride - at < head_dim)) return true;
  }
  return false;
}

w4a16_status check_rope(const w4a16_rope_t *r, int head_dim, RopeArgs *out) {
  if (!r->positions || !r->table) return fail(W4A16_ERR_INVALID_ARG, "positions and table must not be NULL");
  if (!aligned(r->positions, 8) || !aligned(r->table, 4))
    return fail(W4A16_ERR_MISALIGNED, "positions must be 8-byte and the table 4-byte aligned");
  if (r->rot_dim <= 0 || r->rot_dim % 2 != 0 || r->rot_dim > head_dim)
    return fail(W4A16_ERR_INVALID_ARG, "rot_dim (%d) must be even and in [2, head_dim = %d]", r->rot_dim, head_dim);
  if (r->table_rows <= 0 || r->table_rows >= kMaxTokens)
    return fail(W4A16_ERR_INVALID_ARG, "table_rows (%lld) must be in [1, 2^31)", (long long)r->table_rows);
  *out = RopeArgs{r->positions, r->table, r->table_rows, r->rot_dim, r->interleaved != 0};
  return W4A16_OK;
}

}  // namespace

extern "C" {

size_t w4a16_kv_tile_bytes(int head_dim, int bits) {
  if ((bits != 4 && bits != 8) || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return 0;
  return static_cast<size_t>(kv_tile_bytes(head_dim, bits));
}

w4a16_status w4a16_rope(const w4a16_rope_t *rope, const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out,
                        int64_t out_token_stride, int64_t out_head_stride, int64_t tokens, int heads, int head_dim,
                        w4a16_dtype dtype, w4a16_stream_t stream) {
  w4a16_status st = check_dtype(dtype);
  if (st != W4A16_OK) return st;
  if (!rope) return fail(W4A16_ERR_INVALID_ARG, "rope must not be NULL");
  if (tokens < 0 || tokens >= kMaxTokens) return fail(W4A16_ERR_INVALID_ARG, "tokens (%lld) must be in [0, 2^31)", (long long)tokens);
  if (heads < 0 || heads > kMaxHeads || head_dim < 2 || head_dim > 1024)
    return fail(W4A16_ERR_INVALID_ARG, "heads (%d) must be in [0, %d] and head_dim (%d) in [2, 1024]", heads, kMaxHeads, head_dim);
  if (tokens == 0 || heads == 0) return ok();
  RopeArgs ra;
  if ((st = check_rope(rope, head_dim, &ra)) != W4A16_OK) return st;
  const HeadsView xv = view(x, x_token_stride, x_head_stride, tokens, heads), ov = view(out, out_token_stride, out_head_stride, tokens, heads);
  if ((st = check_view(xv, tokens, heads, head_dim, "x", false)) != W4A16_OK) return st;
  if ((st = check_view(ov, tokens, heads, head_dim, "out", false)) != W4A16_OK) return st;
  if (rows_overlap(ov, tokens, heads, head_dim)) return fail(W4A16_ERR_INVALID_ARG, "out: rows of different tokens or heads share elements");
  if (x == out ? (xv.token_stride != ov.token_stride || xv.head_stride != ov.head_stride)
               : overlaps(view_range(xv, tokens, heads, head_dim), view_range(ov, tokens, heads, head_dim)))
    return fail(W4A16_ERR_INVALID_ARG, "out overlaps x (in place: the same pointer and strides)");
  const Range o = view_range(ov, tokens, heads, head_dim);
  if (overlaps(o, range(rope->positions, tokens * 8)) || overlaps(o, range(rope->table, rope->table_rows * rope->rot_dim * 4)))
    return fail(W4A16_ERR_INVALID_ARG, "out overlaps positions or the table");
  const cudaError_t e = launch_rope(xv, ov, tokens, heads, head_dim, dtype, ra, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_rope launch");
  return ok();
}

w4a16_status w4a16_kv_write(const w4a16_kv_cache_t *cache, const void *k, int64_t k_token_stride, int64_t k_head_stride,
                            const void *v, int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                            int64_t tokens, const w4a16_rope_t *rope, const void *q, int64_t q_token_stride,
                            int64_t q_head_stride, int q_heads, void *q_out, w4a16_dtype dtype, w4a16_stream_t stream) {
  w4a16_status st = check_cache(cache, dtype);
  if (st != W4A16_OK) return st;
  if (tokens < 0 || tokens >= kMaxTokens) return fail(W4A16_ERR_INVALID_ARG, "tokens (%lld) must be in [0, 2^31)", (long long)tokens);
  if (tokens == 0) return ok();
  const int D = cache->head_dim;
  if (!slots) return fail(W4A16_ERR_INVALID_ARG, "slots must not be NULL");
  if (!aligned(slots, 8)) return fail(W4A16_ERR_MISALIGNED, "slots must be 8-byte aligned");
  const HeadsView kv = view(k, k_token_stride, k_head_stride, tokens, cache->kv_heads);
  const HeadsView vv = view(v, v_token_stride, v_head_stride, tokens, cache->kv_heads);
  HeadsView qv{nullptr, 0, 0};
  if ((st = check_view(kv, tokens, cache->kv_heads, D, "k", true)) != W4A16_OK) return st;
  if ((st = check_view(vv, tokens, cache->kv_heads, D, "v", true)) != W4A16_OK) return st;
  RopeArgs ra{};
  if (rope && (st = check_rope(rope, D, &ra)) != W4A16_OK) return st;
  const Range data = range(cache->data, cache_bytes(*cache));
  if (overlaps(data, view_range(kv, tokens, cache->kv_heads, D)) || overlaps(data, view_range(vv, tokens, cache->kv_heads, D)) ||
      overlaps(data, range(slots, tokens * 8)))
    return fail(W4A16_ERR_INVALID_ARG, "the cache overlaps k, v or slots");
  if (rope && (overlaps(data, range(rope->positions, tokens * 8)) ||
               overlaps(data, range(rope->table, rope->table_rows * rope->rot_dim * 4))))
    return fail(W4A16_ERR_INVALID_ARG, "the cache overlaps positions or the table");
  if (q) {
    if (!rope) return fail(W4A16_ERR_INVALID_ARG, "q is only taken with rope (it is turned, not cached)");
    if (q_heads <= 0 || q_heads > kMaxHeads) return fail(W4A16_ERR_INVALID_ARG, "q_heads (%d) must be in [1, %d]", q_heads, kMaxHeads);
    qv = view(q, q_token_stride, q_head_stride, tokens, q_heads);
    if ((st = check_view(qv, tokens, q_heads, D, "q", true)) != W4A16_OK) return st;
    const HeadsView qo{q_out, int64_t(q_heads) * D, D};
    if ((st = check_view(qo, tokens, q_heads, D, "q_out", true)) != W4A16_OK) return st;
    const Range o = view_range(qo, tokens, q_heads, D);
    if (overlaps(o, view_range(qv, tokens, q_heads, D)) || overlaps(o, view_range(kv, tokens, cache->kv_heads, D)) ||
        overlaps(o, view_range(vv, tokens, cache->kv_heads, D)) || overlaps(o, data) || overlaps(o, range(slots, tokens * 8)) ||
        overlaps(o, range(rope->positions, tokens * 8)) || overlaps(o, range(rope->table, rope->table_rows * rope->rot_dim * 4)) ||
        overlaps(data, view_range(qv, tokens, q_heads, D)))
      return fail(W4A16_ERR_INVALID_ARG, "q_out overlaps an input or the cache, or the cache overlaps q");
  }
  const cudaError_t e = launch_kv_write(*cache, kv, vv, slots, tokens, dtype, ra, qv, q_heads, q_out,
                                        reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_kv_write launch");
  return ok();
}

w4a16_status w4a16_kv_read(const w4a16_kv_cache_t *cache, const int64_t *slots, int64_t tokens, void *k_out, void *v_out,
                           w4a16_dtype dtype, w4a16_stream_t stream) {
  w4a16_status st = check_cache(cache, dtype);
  if (st != W4A16_OK) return st;
  if (tokens < 0 || tokens >= kMaxTokens) return fail(W4A16_ERR_INVALID_ARG, "tokens (%lld) must be in [0, 2^31)", (long long)tokens);
  if (tokens == 0) return ok();
  if (!slots || !k_out || !v_out) return fail(W4A16_ERR_INVALID_ARG, "slots, k_out and v_out must not be NULL");
  if (!aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(W4A16_ERR_MISALIGNED, "slots must be 8-byte, k_out and v_out 16-byte aligned");
  const int64_t bytes = tokens * cache->kv_heads * cache->head_dim * 2;
  const Range ko = range(k_out, bytes), vo = range(v_out, bytes), data = range(cache->data, cache_bytes(*cache));
  if (overlaps(ko, vo) || overlaps(ko, data) || overlaps(vo, data) || overlaps(ko, range(slots, tokens * 8)) ||
      overlaps(vo, range(slots, tokens * 8)))
    return fail(W4A16_ERR_INVALID_ARG, "k_out, v_out, the cache and slots overlap");
  const cudaError_t e = launch_kv_read(*cache, slots, tokens, k_out, v_out, dtype, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_kv_read launch");
  return ok();
}

w4a16_status w4a16_tree_attention(const w4a16_kv_cache_t *cache, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                  int q_heads, int64_t total_q, const int32_t *q_start, int64_t batch, int max_q,
                                  const int32_t *kv_lens, const int32_t *page_table, int64_t max_pages,
                                  const uint64_t *tree_mask, float softmax_scale, void *out, float *lse, w4a16_dtype dtype,
                                  void *workspace, size_t workspace_bytes, w4a16_stream_t stream) {
  return w4a16_tree_attention_fill(cache, q, q_token_stride, q_head_stride, q_heads, total_q, q_start, batch, max_q, kv_lens, page_table,
                                   max_pages, tree_mask, softmax_scale, out, lse, 0, dtype, workspace, workspace_bytes, stream);
}

w4a16_status w4a16_tree_attention_fill(const w4a16_kv_cache_t *cache, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                       int q_heads, int64_t total_q, const int32_t *q_start, int64_t batch, int max_q,
                                       const int32_t *kv_lens, const int32_t *page_table, int64_t max_pages,
                                       const uint64_t *tree_mask, float softmax_scale, void *out, float *lse, int fill, w4a16_dtype dtype,
                                       void *workspace, size_t workspace_bytes, w4a16_stream_t stream) {
  w4a16_status st = check_cache(cache, dtype);
  if (st != W4A16_OK) return st;
  if (batch < 0 || batch > (1 << 20) || total_q < 0 || total_q >= kMaxTokens)
    return fail(W4A16_ERR_INVALID_ARG, "batch (%lld) must be in [0, 2^20] and total_q (%lld) in [0, 2^31)", (long long)batch,
                (long long)total_q);
  if (max_q < 1 || max_q > 64) return fail(W4A16_ERR_UNSUPPORTED, "max_q (%d) must be in [1, 64]", max_q);
  if (q_heads <= 0 || q_heads > kMaxHeads || q_heads % cache->kv_heads != 0)
    return fail(W4A16_ERR_INVALID_ARG, "q_heads (%d) must be a positive multiple of kv_heads (%d), at most %d", q_heads,
                cache->kv_heads, kMaxHeads);
  if (!std::isfinite(softmax_scale)) return fail(W4A16_ERR_INVALID_ARG, "softmax_scale must be finite");
  if (max_pages < 0 || max_pages >= (int64_t(1) << 31))
    return fail(W4A16_ERR_INVALID_ARG, "max_pages (%lld) must be in [0, 2^31)", (long long)max_pages);
  if (!q_start && total_q != batch)
    return fail(W4A16_ERR_INVALID_ARG, "without q_start there is one query token for each sequence: total_q (%lld), batch (%lld)",
                (long long)total_q, (long long)batch);
  if (fill < 0 || fill > 3) return fail(W4A16_ERR_INVALID_ARG, "fill (%d) must be in [0, 3]", fill);
  if (total_q == 0) return ok();
  if (batch == 0) {  // no row is a sequence's: all bits set are a NaN of every dtype
    cudaError_t e = cudaSuccess;
    if ((fill & 1) && out) e = cudaMemsetAsync(out, 0xFF, static_cast<size_t>(total_q) * q_heads * cache->head_dim * 2, reinterpret_cast<cudaStream_t>(stream));
    if (e == cudaSuccess && (fill & 2) && lse)
      e = cudaMemsetAsync(lse, 0xFF, static_cast<size_t>(total_q) * q_heads * 4, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ok() : cuda_fail(e, "w4a16_tree_attention fill");
  }
  if (!kv_lens || (!page_table && max_pages > 0) || !out)
    return fail(W4A16_ERR_INVALID_ARG, "kv_lens, page_table and out must not be NULL");
  const int D = cache->head_dim;
  const HeadsView qv = view(q, q_token_stride, q_head_stride, total_q, q_heads);
  if ((st = check_view(qv, total_q, q_heads, D, "q", true)) != W4A16_OK) return st;
  if (!aligned(kv_lens, 4) || !aligned(page_table, 4) || !aligned(q_start, 4) || !aligned(tree_mask, 8) || !aligned(lse, 4) ||
      !aligned(out, 16))
    return fail(W4A16_ERR_MISALIGNED, "out must be 16-byte, tree_mask 8-byte, kv_lens, page_table, q_start and lse 4-byte aligned");
  if (workspace && !aligned(workspace, 256)) return fail(W4A16_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  const Range in[] = {view_range(qv, total_q, q_heads, D), range(cache->data, cache_bytes(*cache)), range(kv_lens, batch * 4),
                      range(page_table, page_table ? batch * max_pages * 4 : 0), range(q_start, q_start ? (batch + 1) * 4 : 0),
                      range(tree_mask, tree_mask ? total_q * 8 : 0)};
  const Range written[] = {range(out, total_q * q_heads * D * 2), range(lse, lse ? total_q * q_heads * 4 : 0),
                           range(workspace, workspace ? static_cast<int64_t>(workspace_bytes) : 0)};
  for (int i = 0; i < 3; ++i) {
    for (const Range &r : in)
      if (overlaps(written[i], r)) return fail(W4A16_ERR_INVALID_ARG, "out, lse or the workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(written[i], written[j])) return fail(W4A16_ERR_INVALID_ARG, "out, lse and the workspace overlap");
  }
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  AttentionArgs a{*cache, qv, q_heads, total_q, q_start, batch, max_q, kv_lens, page_table, max_pages, tree_mask, softmax_scale,
                  out, lse, fill, static_cast<int>(dtype), workspace, workspace ? workspace_bytes : 0,
                  reinterpret_cast<cudaStream_t>(stream)};
  e = launch_tree_attention(a, dev);
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_tree_attention launch");
  return ok();
}

size_t w4a16_tree_attention_workspace_size(int max_q, int q_heads, int kv_heads, int head_dim) {
  if (max_q < 1 || max_q > 64 || kv_heads <= 0 || q_heads <= 0 || q_heads % kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  DeviceInfo dev;
  if (current_device_info(&dev) != cudaSuccess) return 0;
  return tree_attention_workspace_bytes(max_q, q_heads, kv_heads, head_dim, dev.num_sms);
}

w4a16_status w4a16_token_logprobs(const void *logits, int64_t row_stride, int64_t rows, int64_t vocab, w4a16_dtype dtype,
                                  const int64_t *tokens, int n_tokens, int top_k, float *logprobs, float *entropy,
                                  int64_t *top_ids, float *top_logprobs, w4a16_stream_t stream) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16 && dtype != W4A16_F32)
    return fail(W4A16_ERR_UNSUPPORTED, "Only float16/bfloat16/float32 logits are supported (dtype %d)", static_cast<int>(dtype));
  if (rows < 0 || rows >= (int64_t(1) << 27) || vocab < 1 || vocab >= (int64_t(1) << 30))
    return fail(W4A16_ERR_INVALID_ARG, "rows (%lld) must be in [0, 2^27) and vocab (%lld) in [1, 2^30)", (long long)rows,
                (long long)vocab);
  if (row_stride < 0 || (rows > 1 && row_stride < vocab))
    return fail(W4A16_ERR_INVALID_ARG, "row_stride (%lld) must be at least vocab (%lld)", (long long)row_stride, (long long)vocab);
  if (n_tokens < 0 || n_tokens > 1024) return fail(W4A16_ERR_INVALID_ARG, "n_tokens (%d) must be in [0, 1024]", n_tokens);
  if (top_k < 0 || top_k > kMaxTopK || top_k > vocab)
    return fail(W4A16_ERR_UNSUPPORTED, "top_k (%d) must be in [0, %d] and at most vocab (%lld)", top_k, kMaxTopK, (long long)vocab);
  if (rows == 0) return ok();
  if (!logits || (n_tokens > 0 && (!tokens || !logprobs)) || (top_k > 0 && (!top_ids || !top_logprobs)))
    return fail(W4A16_ERR_INVALID_ARG, "logits, tokens, logprobs, top_ids and top_logprobs must not be NULL");
  const int e_bytes = dtype == W4A16_F32 ? 4 : 2;
  if (!aligned(logits, e_bytes) || !aligned(tokens, 8) || !aligned(top_ids, 8) || !aligned(logprobs, 4) || !aligned(entropy, 4) ||
      !aligned(top_logprobs, 4))
    return fail(W4A16_ERR_MISALIGNED, "tensors must be naturally aligned");
  const Range in[] = {range(logits, ((rows - 1) * row_stride + vocab) * e_bytes), range(tokens, tokens ? rows * n_tokens * 8 : 0)};
  const Range written[] = {range(logprobs, logprobs ? rows * n_tokens * 4 : 0), range(entropy, entropy ? rows * 4 : 0),
                           range(top_ids, top_ids ? rows * top_k * 8 : 0), range(top_logprobs, top_logprobs ? rows * top_k * 4 : 0)};
  for (int i = 0; i < 4; ++i) {
    for (const Range &r : in)
      if (overlaps(written[i], r)) return fail(W4A16_ERR_INVALID_ARG, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(written[i], written[j])) return fail(W4A16_ERR_INVALID_ARG, "outputs overlap");
  }
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const LogprobArgs a{logits, row_stride, rows, vocab, static_cast<int>(dtype), tokens, n_tokens, top_k, logprobs, entropy,
                      top_ids, top_logprobs, reinterpret_cast<cudaStream_t>(stream)};
  e = launch_token_logprobs(a, dev);
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_token_logprobs launch");
  return ok();
}

}  // extern "C"
