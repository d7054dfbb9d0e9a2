// Shared between the translation units of the attention (one for each head size, compiled in parallel).
#pragma once

#include "internal.h"

namespace w4a16 {
namespace attention {

// Failure detection: error word, limit of the bounded waits (0: the default) and the test hook.
struct Control {
  unsigned int error;
  unsigned int stall;  // the workers first wait on a barrier that nothing arrives on
  unsigned long long limit_ns;
};

struct Params {
  const uint8_t *cache;
  const uint16_t *q;
  int64_t q_ts, q_hs;
  const int32_t *q_start, *kv_lens, *page_table;
  int64_t max_pages, num_pages;
  const uint64_t *tree_mask;
  float scale;
  uint16_t *out;
  float *lse;
  int fill;  // outputs (1: out, 2: lse) whose rows that are not computed get NaN
  int64_t total_q;
  int batch, q_heads, kv_heads, group, page_tiles, max_q;
  int page_shift;  // log2 of page_tiles, or -1
  int bf16;
  unsigned int *flags;  // one counter for each CTA, zero before and after; null: no sequence is split
  float *partials;
  Control *control;
};

// Workspace: the counters first (the area that calls leave zero), then two partial results for each CTA.
constexpr size_t kFlagBytes = 4096;
constexpr int kMaxCtas = kFlagBytes / 4;
// Floats of one partial result of `rows` rows: the sums, the maxima, the denominators.
inline int64_t partial_floats(int rows, int head_dim) { return int64_t(rows) * (head_dim + 2); }

// Rows of a row tile of the streaming kernel for sequences of max_rows query rows on a cache head: as few as hold
// them, since each 8 rows add products and exponentials to every tile (131072 tokens of 8 heads of 128 elements at 4
// bits: 8 rows 63 us, 16 rows 89, 32 rows 161). Heads of 256 elements have registers for the sums of 16 rows only.
inline int stream_rows(int max_rows, int head_dim) { return max_rows <= 8 ? 8 : max_rows <= 16 || head_dim == 256 ? 16 : 32; }

// Query rows of a cache head from which the kernel on the fifth-generation tensor cores takes over, and its row tile.
// Past 32 rows the streaming kernel would go over the cache once more for every 32. One sequence of 131072 tokens, 8
// cache heads of 128 (64) elements: 30 rows on the streaming kernel 161 us at 4 bits, 176 at 8 (144, 148), 35 to 125
// rows on the other 172 to 179 and 224 to 230 (132 to 144). Heads of 256 elements leave no room for two stages of
// operands of 128 tokens beside Q (tiles of fewer tokens were not tried): they stay on the streaming kernel (35 rows 448 us, 125
// rows 1174 to 1207).
constexpr int kTileRows = 128;
inline bool use_tiles(int max_rows, int head_dim) { return max_rows > 32 && head_dim <= 128; }

template <int D>
cudaError_t launch_tiles(const Params &p, int bits, int num_sms, cudaStream_t stream);  // head_dim 64 and 128
template <int D, int BITS>
cudaError_t launch_stream(const Params &p, int rows, int num_sms, cudaStream_t stream);

}  // namespace attention
}  // namespace w4a16
