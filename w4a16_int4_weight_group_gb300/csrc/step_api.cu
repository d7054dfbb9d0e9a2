// C ABI of the operators around a step of many users: argument validation and launches.
#include "internal.h"

using namespace w4a16;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 31;
constexpr int64_t kMaxBatch = 1 << 20;
constexpr int kMaxRank = 128;

// Bytes from the first to the last element of a [rows, cols] tensor
Range rows_range(const void *p, int64_t rows, int64_t stride, int64_t cols, int elem) {
  return range(p, rows > 0 ? ((rows - 1) * stride + cols) * elem : 0);
}

// A matrix of 16-bit elements that the kernels read in vectors: contiguous rows that share no elements
w4a16_status check_rows(const void *p, int64_t rows, int64_t stride, int64_t cols, const char *name) {
  if (!p) return fail(W4A16_ERR_INVALID_ARG, "%s must not be NULL", name);
  if (rows > 1 && (stride < cols || stride >= (int64_t(1) << 35) / rows))
    return fail(W4A16_ERR_INVALID_ARG, "%s: a row stride of %lld does not hold rows of %lld elements, or all rows span 2^35 elements and more", name,
                (long long)stride, (long long)cols);
  if (!aligned(p, 16) || (rows > 1 && stride % 8 != 0))
    return fail(W4A16_ERR_MISALIGNED, "%s must be 16-byte aligned, its row stride a multiple of 8 elements", name);
  return W4A16_OK;
}

w4a16_status check_pool(const int32_t *refs, int64_t num_pages, int page_size, const int32_t *table, int64_t max_pages, int64_t batch) {
  if (num_pages <= 0 || num_pages >= (int64_t(1) << 30))
    return fail(W4A16_ERR_INVALID_ARG, "num_pages (%lld) must be in [1, 2^30)", (long long)num_pages);
  if (page_size <= 0 || page_size > (1 << 20)) return fail(W4A16_ERR_INVALID_ARG, "page_size (%d) must be in [1, 2^20]", page_size);
  if (batch < 0 || batch > kMaxBatch) return fail(W4A16_ERR_INVALID_ARG, "batch (%lld) must be in [0, 2^20]", (long long)batch);
  if (max_pages < 0 || max_pages >= (int64_t(1) << 29) || batch * max_pages >= (int64_t(1) << 29))
    return fail(W4A16_ERR_INVALID_ARG, "the page table must have fewer than 2^29 entries (%lld x %lld)", (long long)batch, (long long)max_pages);
  if (!refs || (!table && batch * max_pages > 0)) return fail(W4A16_ERR_INVALID_ARG, "refs and page_table must not be NULL");
  if (!aligned(refs, 4) || !aligned(table, 4)) return fail(W4A16_ERR_MISALIGNED, "refs and page_table must be 4-byte aligned");
  return W4A16_OK;
}

w4a16_status check_layers(const w4a16_kv_cache_t *c, int64_t layers) {
  if (!c) return fail(W4A16_ERR_INVALID_ARG, "cache must not be NULL");
  if (c->bits != 4 && c->bits != 8) return fail(W4A16_ERR_UNSUPPORTED, "cache bits %d not supported; supported: [4, 8]", c->bits);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(W4A16_ERR_UNSUPPORTED, "cache head_dim %d not supported; supported: [64, 128, 256]", c->head_dim);
  if (c->page_size <= 0 || c->page_size % kTileTokens != 0 || c->page_size > (1 << 20))
    return fail(W4A16_ERR_INVALID_ARG, "page_size (%d) must be a positive multiple of 16, at most 2^20", c->page_size);
  if (c->kv_heads <= 0 || c->kv_heads > 1024) return fail(W4A16_ERR_INVALID_ARG, "kv_heads (%d) must be in [1, 1024]", c->kv_heads);
  if (c->num_pages <= 0 || c->num_pages >= (int64_t(1) << 30) || c->num_pages * (c->page_size / kTileTokens) >= (int64_t(1) << 31))
    return fail(W4A16_ERR_INVALID_ARG, "num_pages (%lld) must be in [1, 2^30) and a layer hold fewer than 2^31 tiles of 16 tokens",
                (long long)c->num_pages);
  if (layers < 1 || layers > 65535) return fail(W4A16_ERR_INVALID_ARG, "layers (%lld) must be in [1, 65535]", (long long)layers);
  if (!c->data) return fail(W4A16_ERR_INVALID_ARG, "cache data must not be NULL");
  if (!aligned(c->data, 128)) return fail(W4A16_ERR_MISALIGNED, "cache data must be 128-byte aligned");
  return W4A16_OK;
}
Range layers_range(const w4a16_kv_cache_t &c, int64_t layers) {
  return range(c.data, layers * c.num_pages * c.kv_heads * (c.page_size / kTileTokens) * kv_tile_bytes(c.head_dim, c.bits));
}

// Whether an output overlaps an input or another output.
template <int W, int I>
bool conflict(const Range (&written)[W], const Range (&in)[I]) {
  for (int i = 0; i < W; ++i) {
    for (const Range &r : in)
      if (overlaps(written[i], r)) return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(written[i], written[j])) return true;
  }
  return false;
}

cudaStream_t as_stream(w4a16_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

size_t w4a16_lora_workspace_size(int64_t tokens, int rank, int64_t adapters) {
  if (tokens < 0 || tokens >= kMaxTokens || rank < 1 || rank > kMaxRank || adapters < 1 || adapters > lora_most_adapters()) return 0;
  return lora_workspace_bytes(tokens, rank, adapters);
}

w4a16_status w4a16_lora(const void *x, int64_t x_stride, const void *a, const void *b, const int32_t *ids, const float *scales, const void *base,
                        int64_t base_stride, void *out, int64_t out_stride, int64_t tokens, int64_t k, int64_t n, int rank, int64_t adapters,
                        w4a16_dtype dtype, void *workspace, size_t workspace_bytes, w4a16_stream_t stream) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16)
    return fail(W4A16_ERR_UNSUPPORTED, "Only float16/bfloat16 tensors are supported (dtype %d)", static_cast<int>(dtype));
  if (tokens < 0 || tokens >= (int64_t(1) << 30)) return fail(W4A16_ERR_INVALID_ARG, "tokens (%lld) must be in [0, 2^30)", (long long)tokens);
  if (k < 8 || n < 8 || k % 8 != 0 || n % 8 != 0 || k >= (int64_t(1) << 24) || n >= (int64_t(1) << 24))
    return fail(W4A16_ERR_UNSUPPORTED, "k (%lld) and n (%lld) must be multiples of 8 in [8, 2^24)", (long long)k, (long long)n);
  if (rank < 8 || rank > kMaxRank || rank % 8 != 0)
    return fail(W4A16_ERR_UNSUPPORTED, "rank (%d) must be a multiple of 8 in [8, %d] (pad smaller ones with zeros)", rank, kMaxRank);
  if (adapters < 1 || adapters > lora_most_adapters())
    return fail(W4A16_ERR_UNSUPPORTED, "adapters (%lld) must be in [1, %d]", (long long)adapters, lora_most_adapters());
  if (tokens == 0) return ok();
  w4a16_status st;
  if (tokens == 1) x_stride = base_stride = out_stride = 0;
  if ((st = check_rows(x, tokens, x_stride, k, "x")) != W4A16_OK) return st;
  if ((st = check_rows(base, tokens, base_stride, n, "base")) != W4A16_OK) return st;
  if ((st = check_rows(out, tokens, out_stride, n, "out")) != W4A16_OK) return st;
  if (!a || !b || !ids) return fail(W4A16_ERR_INVALID_ARG, "a, b and ids must not be NULL");
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(ids, 4) || !aligned(scales, 4))
    return fail(W4A16_ERR_MISALIGNED, "a and b must be 16-byte, ids and scales 4-byte aligned");
  const size_t need = lora_workspace_bytes(tokens, rank, adapters);
  if (need && (!workspace || workspace_bytes < need))
    return fail(W4A16_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : size_t(0), need);
  if (workspace && !aligned(workspace, 256)) return fail(W4A16_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  const Range o = rows_range(out, tokens, out_stride, n, 2), ws = range(workspace, workspace ? static_cast<int64_t>(workspace_bytes) : 0);
  const Range bs = rows_range(base, tokens, base_stride, n, 2);
  const Range in[] = {rows_range(x, tokens, x_stride, k, 2), range(a, adapters * rank * k * 2), range(b, adapters * n * rank * 2), range(ids, tokens * 4),
                      range(scales, scales ? adapters * 4 : 0)};
  const Range written[] = {o, ws};
  if (conflict(written, in) || overlaps(ws, bs)) return fail(W4A16_ERR_INVALID_ARG, "out or the workspace overlaps an input");
  if (base == out ? base_stride != out_stride : overlaps(o, bs))
    return fail(W4A16_ERR_INVALID_ARG, "out overlaps base (in place: the same pointer and stride)");
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const LoraArgs args{x, a, b, base, out, ids, scales, x_stride, base_stride, out_stride, tokens, k, n, rank, adapters, static_cast<int>(dtype),
                      workspace, as_stream(stream)};
  e = launch_lora(args, dev);
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_lora launch");
  return ok();
}

size_t w4a16_verify_drafts_workspace_size(int64_t total, int64_t vocab) {
  if (total < 0 || total >= (int64_t(1) << 24) || vocab < 1 || vocab >= (int64_t(1) << 30)) return 0;
  DeviceInfo dev;
  if (current_device_info(&dev) != cudaSuccess) return 0;
  return verify_workspace_bytes(total, vocab, dev.num_sms);
}

w4a16_status w4a16_verify_drafts(const void *logits, int64_t row_stride, int64_t total, int64_t vocab, w4a16_dtype dtype, const int64_t *tokens,
                                 const int32_t *q_start, int64_t batch, int max_q, const uint64_t *tree_mask, const float *uniforms,
                                 const float *noise, int64_t noise_stride, const float *draft_probs, int64_t draft_stride,
                                 const float *temperature, int32_t *accepted, int32_t *path, int64_t *out_tokens, float *out_probs,
                                 void *workspace, size_t workspace_bytes, w4a16_stream_t stream) {
  if (dtype != W4A16_F16 && dtype != W4A16_BF16 && dtype != W4A16_F32)
    return fail(W4A16_ERR_UNSUPPORTED, "Only float16/bfloat16/float32 logits are supported (dtype %d)", static_cast<int>(dtype));
  if (batch < 0 || batch > kMaxBatch || total < 0 || total >= (int64_t(1) << 24))
    return fail(W4A16_ERR_INVALID_ARG, "batch (%lld) must be in [0, 2^20] and total (%lld) in [0, 2^24)", (long long)batch, (long long)total);
  if (vocab < 1 || vocab >= (int64_t(1) << 30)) return fail(W4A16_ERR_INVALID_ARG, "vocab (%lld) must be in [1, 2^30)", (long long)vocab);
  if (max_q < 1 || max_q > 64) return fail(W4A16_ERR_UNSUPPORTED, "max_q (%d) must be in [1, 64]", max_q);
  if (!q_start && total != batch)
    return fail(W4A16_ERR_INVALID_ARG, "without q_start there is one token for each sequence: total (%lld), batch (%lld)", (long long)total,
                (long long)batch);
  if (draft_probs && tree_mask)
    return fail(W4A16_ERR_UNSUPPORTED, "draft_probs are taken for chains only: the tokens of a tree are guesses");
  if (total == 1) row_stride = draft_stride = vocab;
  if (batch == 1) noise_stride = vocab;
  if ((total > 0 && row_stride < vocab) || (batch > 0 && noise_stride < vocab) || (draft_probs && draft_stride < vocab))
    return fail(W4A16_ERR_INVALID_ARG, "row strides (%lld, %lld, %lld) must be at least vocab (%lld)", (long long)row_stride,
                (long long)noise_stride, (long long)draft_stride, (long long)vocab);
  if (batch == 0) return ok();
  if (!accepted || !path || !out_tokens || !out_probs || !noise || (total > 0 && (!logits || !tokens || !uniforms)))
    return fail(W4A16_ERR_INVALID_ARG, "logits, tokens, uniforms, noise, accepted, path, out_tokens and out_probs must not be NULL");
  if (!aligned(logits, dtype == W4A16_F32 ? 4 : 2) || !aligned(tokens, 8) || !aligned(out_tokens, 8) || !aligned(tree_mask, 8) ||
      !aligned(q_start, 4) || !aligned(uniforms, 4) || !aligned(noise, 4) || !aligned(draft_probs, 4) || !aligned(temperature, 4) ||
      !aligned(accepted, 4) || !aligned(path, 4) || !aligned(out_probs, 4))
    return fail(W4A16_ERR_MISALIGNED, "tensors must be naturally aligned");
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const size_t need = verify_workspace_bytes(total, vocab, dev.num_sms);
  if (!workspace || workspace_bytes < need)
    return fail(W4A16_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : size_t(0), need);
  if (!aligned(workspace, 256)) return fail(W4A16_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  const Range in[] = {rows_range(logits, total, row_stride, vocab, dtype == W4A16_F32 ? 4 : 2), range(tokens, total * 8), range(uniforms, total * 4),
                      range(q_start, q_start ? (batch + 1) * 4 : 0), range(tree_mask, tree_mask ? total * 8 : 0),
                      rows_range(noise, batch, noise_stride, vocab, 4), rows_range(draft_probs, draft_probs ? total : 0, draft_stride, vocab, 4),
                      range(temperature, temperature ? batch * 4 : 0)};
  const Range written[] = {range(accepted, batch * 4), range(path, batch * max_q * 4), range(out_tokens, batch * max_q * 8),
                           range(out_probs, batch * max_q * 4), range(workspace, static_cast<int64_t>(workspace_bytes))};
  if (conflict(written, in)) return fail(W4A16_ERR_INVALID_ARG, "an output or the workspace overlaps an input or another output");
  const VerifyArgs args{logits, row_stride, total, vocab, static_cast<int>(dtype), tokens, q_start, batch, max_q, tree_mask, uniforms, noise,
                        noise_stride, draft_probs, draft_stride, temperature, accepted, path, out_tokens, out_probs, workspace, as_stream(stream)};
  e = launch_verify(args, dev);
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_verify_drafts launch");
  return ok();
}

w4a16_status w4a16_kv_fork(int32_t *refs, int64_t num_pages, int page_size, const int32_t *page_table, int64_t max_pages, const int32_t *kv_lens,
                           int64_t batch, const int32_t *parents, int64_t rows, int32_t *new_table, int32_t *new_lens, w4a16_stream_t stream) {
  w4a16_status st = check_pool(refs, num_pages, page_size, page_table, max_pages, batch);
  if (st != W4A16_OK) return st;
  if (rows < 0 || rows > kMaxBatch || rows * max_pages >= (int64_t(1) << 29))
    return fail(W4A16_ERR_INVALID_ARG, "rows (%lld) must be in [0, 2^20] and the new table have fewer than 2^29 entries", (long long)rows);
  if (rows == 0) return ok();
  if (!parents || !new_lens || (!new_table && max_pages > 0) || (!kv_lens && batch > 0))
    return fail(W4A16_ERR_INVALID_ARG, "kv_lens, parents, new_table and new_lens must not be NULL");
  if (!aligned(parents, 4) || !aligned(new_lens, 4) || !aligned(new_table, 4) || !aligned(kv_lens, 4))
    return fail(W4A16_ERR_MISALIGNED, "tensors must be 4-byte aligned");
  const Range in[] = {range(page_table, batch * max_pages * 4), range(kv_lens, batch * 4), range(parents, rows * 4)};
  const Range written[] = {range(refs, num_pages * 4), range(new_table, rows * max_pages * 4), range(new_lens, rows * 4)};
  if (conflict(written, in)) return fail(W4A16_ERR_INVALID_ARG, "refs or an output overlaps an input or another output");
  const cudaError_t e = launch_kv_fork(PoolArgs{refs, num_pages, page_size, max_pages}, page_table, kv_lens, batch, parents, rows, new_table, new_lens,
                                       as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_kv_fork launch");
  return ok();
}

w4a16_status w4a16_kv_reserve(int32_t *refs, int64_t num_pages, int page_size, int32_t *page_table, int64_t max_pages, const int32_t *kv_lens,
                              const int32_t *new_lens, int64_t batch, int32_t *held, int32_t *copies, w4a16_stream_t stream) {
  w4a16_status st = check_pool(refs, num_pages, page_size, page_table, max_pages, batch);
  if (st != W4A16_OK) return st;
  if (batch > kv_reserve_most_sequences())
    return fail(W4A16_ERR_UNSUPPORTED, "batch (%lld) must be at most %d in one call", (long long)batch, kv_reserve_most_sequences());
  if (batch == 0) return ok();
  if (!kv_lens || !new_lens || !held || !copies) return fail(W4A16_ERR_INVALID_ARG, "kv_lens, new_lens, held and copies must not be NULL");
  if (!aligned(kv_lens, 4) || !aligned(new_lens, 4) || !aligned(held, 4) || !aligned(copies, 8))
    return fail(W4A16_ERR_MISALIGNED, "copies must be 8-byte, the other tensors 4-byte aligned");
  const Range in[] = {range(kv_lens, batch * 4), range(new_lens, batch * 4)};
  const Range written[] = {range(refs, num_pages * 4), range(page_table, batch * max_pages * 4), range(held, batch * 4), range(copies, batch * 8)};
  if (conflict(written, in)) return fail(W4A16_ERR_INVALID_ARG, "refs, page_table or an output overlaps an input or another output");
  const cudaError_t e = launch_kv_reserve(PoolArgs{refs, num_pages, page_size, max_pages}, page_table, kv_lens, new_lens, batch, held, copies,
                                          as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_kv_reserve launch");
  return ok();
}

w4a16_status w4a16_kv_free(int32_t *refs, int64_t num_pages, int page_size, int32_t *page_table, int64_t max_pages, const int32_t *kv_lens,
                           const int32_t *keep, int64_t batch, w4a16_stream_t stream) {
  w4a16_status st = check_pool(refs, num_pages, page_size, page_table, max_pages, batch);
  if (st != W4A16_OK) return st;
  if (batch == 0) return ok();
  if (!kv_lens) return fail(W4A16_ERR_INVALID_ARG, "kv_lens must not be NULL");
  if (!aligned(kv_lens, 4) || !aligned(keep, 4)) return fail(W4A16_ERR_MISALIGNED, "kv_lens and keep must be 4-byte aligned");
  const Range in[] = {range(kv_lens, batch * 4), range(keep, keep ? batch * 4 : 0)};
  const Range written[] = {range(refs, num_pages * 4), range(page_table, batch * max_pages * 4)};
  if (conflict(written, in)) return fail(W4A16_ERR_INVALID_ARG, "refs or page_table overlaps an input, or each other");
  const cudaError_t e = launch_kv_free(PoolArgs{refs, num_pages, page_size, max_pages}, page_table, kv_lens, keep, batch, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_kv_free launch");
  return ok();
}

w4a16_status w4a16_kv_copy(const w4a16_kv_cache_t *cache, int64_t layers, const int32_t *copies, int64_t n, w4a16_stream_t stream) {
  w4a16_status st = check_layers(cache, layers);
  if (st != W4A16_OK) return st;
  if (n < 0 || n >= kMaxTokens) return fail(W4A16_ERR_INVALID_ARG, "n (%lld) must be in [0, 2^31)", (long long)n);
  if (n == 0) return ok();
  if (!copies) return fail(W4A16_ERR_INVALID_ARG, "copies must not be NULL");
  if (!aligned(copies, 8)) return fail(W4A16_ERR_MISALIGNED, "copies must be 8-byte aligned");
  if (overlaps(layers_range(*cache, layers), range(copies, n * 8))) return fail(W4A16_ERR_INVALID_ARG, "the cache overlaps copies");
  const cudaError_t e = launch_kv_copy(*cache, layers, copies, n, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_kv_copy launch");
  return ok();
}

w4a16_status w4a16_kv_compact(const w4a16_kv_cache_t *cache, int64_t layers, const int32_t *page_table, int64_t max_pages, const int32_t *kv_lens,
                              const int32_t *q_start, int64_t batch, const int32_t *path, int max_q, int32_t *new_lens, w4a16_stream_t stream) {
  w4a16_status st = check_layers(cache, layers);
  if (st != W4A16_OK) return st;
  if (batch < 0 || batch > kMaxBatch) return fail(W4A16_ERR_INVALID_ARG, "batch (%lld) must be in [0, 2^20]", (long long)batch);
  if (max_q < 1 || max_q > 64) return fail(W4A16_ERR_UNSUPPORTED, "max_q (%d) must be in [1, 64]", max_q);
  if (max_pages < 0 || max_pages >= (int64_t(1) << 31))
    return fail(W4A16_ERR_INVALID_ARG, "max_pages (%lld) must be in [0, 2^31)", (long long)max_pages);
  if (batch == 0) return ok();
  if ((!page_table && max_pages > 0) || !kv_lens || !path || !new_lens)
    return fail(W4A16_ERR_INVALID_ARG, "page_table, kv_lens, path and new_lens must not be NULL");
  if (!aligned(page_table, 4) || !aligned(kv_lens, 4) || !aligned(q_start, 4) || !aligned(path, 4) || !aligned(new_lens, 4))
    return fail(W4A16_ERR_MISALIGNED, "page_table, kv_lens, q_start, path and new_lens must be 4-byte aligned");
  const Range in[] = {range(page_table, batch * max_pages * 4), range(kv_lens, batch * 4), range(q_start, q_start ? (batch + 1) * 4 : 0),
                      range(path, batch * max_q * 4)};
  const Range written[] = {layers_range(*cache, layers), range(new_lens, batch * 4)};
  if (conflict(written, in)) return fail(W4A16_ERR_INVALID_ARG, "the cache or new_lens overlaps an input, or each other");
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  e = launch_kv_compact(CompactArgs{*cache, layers, page_table, max_pages, kv_lens, q_start, path, batch, max_q, new_lens}, dev.num_sms,
                        as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w4a16_kv_compact launch");
  return ok();
}

}  // extern "C"
