// Pages of a quantised paged cache: forked, reserved, copied, given back, and the accepted tokens of a drafted tree put
// together.
//
// refs[page] counts the sequences that hold a page; a page with none is free. fork and free only add and subtract, and
// reserve hands out the free pages in ascending order to the sequences in theirs: there is no list whose order could depend on
// timing. A sequence that is to write into a page that others hold too gets a copy (the last holder in the call keeps the
// page, once the others have theirs): reserve says which pages, copy moves them in all layers. Nothing comes back to the host.
//
// All of it is bytes moved or integers counted. reserve is one CTA, bound by the latency of its steps (holders of the
// same page counted against each other in shared memory, sums over the sequences, free pages counted 4096 at a time); copy is
// bound by memory; compact by the latency of load, barrier, store: a CTA reads all tokens of a sequence that move, for one
// head and some layers, before it writes one, so that a place may be read and written in any order.
//
// Measured: 128 pages of 128 tokens, 8 heads of 128 at 8 bits, in 8 layers copied in 62 us (553 MB, 8.9 TB/s with part of the writes left in
// L2; the step of fork, reserve, copy, free and two copies of the tables 86 us replayed); reserve 8 to 12 us alone, 5 replayed in a pool of 400 pages and 27
// in one of 100000 whose free pages are the last; fork and free 4 to 6, free 2 replayed.
// compact: 64 sequences of up to 16 tokens in 16 layers 6.5 us replayed (a layer a CTA: 19 us a call), 4 of 8 in one layer 3.0.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kMaxQ = 64;  // drafted tokens of a sequence
constexpr int kMaxSequences = 4096;  // of one reserve: their tables are in shared memory
constexpr int kReserveThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyVectors = 4;  // of 16 bytes, a thread

struct Pool {
  int32_t *refs;
  int pages, page_size;
  int64_t cols;  // entries of a sequence in the page table
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, const Pool &p) {
  return min((max(tokens, int64_t(0)) + p.page_size - 1) / p.page_size, p.cols);
}

__global__ void __launch_bounds__(256) fork_kernel(const Pool p, const int32_t *table, const int32_t *lens, int64_t batch, const int32_t *parents,
                                                   int32_t *new_table, int32_t *new_lens) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int from = parents[row];
  const bool has = from >= 0 && from < batch;
  const int len = has ? max(lens[from], 0) : 0;
  const int64_t have = pages_of(len, p);
  for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const int page = c < have ? table[from * p.cols + c] : -1;
    new_table[row * p.cols + c] = page;
    if (page >= 0 && page < p.pages) atomicAdd(p.refs + page, 1);
  }
  if (threadIdx.x == 0) new_lens[row] = len;
}

__global__ void __launch_bounds__(256) free_kernel(const Pool p, int32_t *table, const int32_t *lens, const int32_t *keep) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int64_t have = pages_of(lens[row], p);
  for (int64_t c = pages_of(keep ? keep[row] : 0, p) + threadIdx.x; c < have; c += blockDim.x) {
    const int page = table[row * p.cols + c];
    table[row * p.cols + c] = -1;
    // (a page that nobody holds stays at zero)
    if (page >= 0 && page < p.pages && atomicSub(p.refs + page, 1) <= 0) atomicAdd(p.refs + page, 1);
  }
}

// Exclusive sum over the CTA's threads, and the total.
__device__ __forceinline__ int block_sum(int v, int *sums, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int a = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, a, o);
    if (lane >= o) a += u;
  }
  if (lane == 31) sums[warp] = a;
  __syncthreads();
  const int s = lane < kReserveThreads / 32 ? sums[lane] : 0;
  int w = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, w - s, warp);
  __syncthreads();
  return before + a - v;
}

__global__ void __launch_bounds__(kReserveThreads) reserve_kernel(const Pool p, int32_t *table, const int32_t *lens, const int32_t *new_lens,
                                                                  int batch, int32_t *held, int2 *copies) {
  __shared__ __align__(16) int tail[kMaxSequences];  // the shared page that a sequence is about to write into, or -1 - b
  __shared__ int first[kMaxSequences + 1];           // pages wanted by the sequences before
  __shared__ int sums[kReserveThreads / 32];
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int padded = (batch + 3) / 4 * 4;
  auto old_len = [&](int b) { return int64_t(max(lens[b], 0)); };
  for (int b = tid; b < padded; b += kReserveThreads) {
    int page = -1 - b;
    if (b < batch) {
      const int64_t len = old_len(b), have = pages_of(len, p);
      if (new_lens[b] > len && len % p.page_size != 0 && len < p.cols * p.page_size) {
        const int last = table[b * p.cols + have - 1];
        if (last >= 0 && last < p.pages && p.refs[last] > 1) page = last;
      }
      copies[b] = make_int2(-1, -1);
    }
    tail[b] = page;
  }
  __syncthreads();
  int wanted = 0;
  for (int b0 = 0; b0 < batch; b0 += kReserveThreads) {
    const int b = b0 + tid;
    int need = 0;
    if (b < batch) {
      const int64_t len = old_len(b), have = pages_of(len, p), want = pages_of(new_lens[b], p);
      need = static_cast<int>(max(want - have, int64_t(0)));
      const int page = tail[b];
      if (page >= 0) {
        int earlier = 0;
        const int4 *all = reinterpret_cast<const int4 *>(tail);
        for (int j = 0; j * 4 < b; ++j) {
          const int4 v = all[j];
          earlier += (v.x == page) + (v.y == page && j * 4 + 1 < b) + (v.z == page && j * 4 + 2 < b) + (v.w == page && j * 4 + 3 < b);
        }
        // (the top bit of `first` is free: the page table has fewer than 2^29 entries)
        if (earlier < p.refs[page] - 1) need = (need + 1) | 0x40000000;
      }
    }
    const bool copy = need & 0x40000000;
    need &= 0x3FFFFFFF;
    int total;
    const int before = block_sum(need, sums, total);
    if (b < batch) first[b] = (wanted + before) | (copy ? 0x40000000 : 0);
    wanted += total;
  }
  if (tid == 0) first[batch] = wanted;
  __syncthreads();
  // the free pages, in ascending order, to their takers
  auto start_of = [&](int b) { return first[b] & 0x3FFFFFFF; };
  int found = 0;
  for (int q0 = 0; q0 < p.pages && found < wanted; q0 += kReserveThreads * 4) {
    const int q = q0 + tid * 4;
    bool free_page[4];
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      free_page[i] = q + i < p.pages && p.refs[q + i] == 0;
      n += free_page[i];
    }
    int total;
    int at = found + block_sum(n, sums, total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!free_page[i] || at >= wanted) continue;
      int lo = 0, hi = batch;  // the last sequence whose pages start at or before `at`
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start_of(mid) <= at) lo = mid;
        else hi = mid;
      }
      const int page = q + i, j = at - start_of(lo);
      const bool copy = first[lo] & 0x40000000;
      const int64_t have = pages_of(old_len(lo), p);
      int64_t col = have + j;
      if (copy) {
        --col;  // its copy comes first, in the place of the shared page
        if (j == 0) {
          copies[lo] = make_int2(tail[lo], page);
          atomicSub(p.refs + tail[lo], 1);  // (stays above zero: fewer copies than holders)
        }
      }
      table[lo * p.cols + col] = page;
      p.refs[page] = 1;
      ++at;
    }
    found += total;
  }
  __syncthreads();  // the copies are counted
  for (int b = tid; b < batch; b += kReserveThreads) {
    const int64_t len = old_len(b);
    int64_t now = len;
    if (new_lens[b] > len) {
      const bool copy = first[b] & 0x40000000;
      const int got = min(start_of(b + 1), found) - min(start_of(b), found);
      // (A page kept in place is the sequence's own only if every earlier holder got its copy; one that did not used up the free pages,
      // so that this one got none either.)
      const bool own = copy ? got > 0 : tail[b] < 0 || __ldcg(p.refs + tail[b]) <= 1;
      if (own) now = max(len, min(int64_t(new_lens[b]), (pages_of(len, p) + got - copy) * p.page_size));
    }
    held[b] = static_cast<int32_t>(now);
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(uint8_t *cache, int64_t layer_bytes, int64_t page_bytes, int pages, const int2 *pairs) {
  griddep_wait();
  griddep_launch_dependents();
  const int2 pair = pairs[blockIdx.y];
  if (pair.x < 0 || pair.x >= pages || pair.y < 0 || pair.y >= pages || pair.x == pair.y) return;
  uint8_t *layer = cache + blockIdx.z * layer_bytes;
  const uint4 *src = reinterpret_cast<const uint4 *>(layer + pair.x * page_bytes);
  uint4 *dst = reinterpret_cast<uint4 *>(layer + pair.y * page_bytes);
  const int64_t n = page_bytes / 16, at = int64_t(blockIdx.x) * (kCopyThreads * kCopyVectors) + threadIdx.x;
  uint4 v[kCopyVectors];
#pragma unroll
  for (int i = 0; i < kCopyVectors; ++i)
    if (at + i * kCopyThreads < n) v[i] = __ldcs(src + at + i * kCopyThreads);
#pragma unroll
  for (int i = 0; i < kCopyVectors; ++i)
    if (at + i * kCopyThreads < n) dst[at + i * kCopyThreads] = v[i];
}

struct CompactParams {
  uint8_t *cache;
  int64_t layer_bytes;
  int pages, heads, page_size, code_bytes;  // code_bytes: of a token's K (or V) codes
  int64_t cols;
  const int32_t *table, *lens, *q_start, *path;
  int max_q;
  int32_t *new_lens;
  int layers, each;  // each: layers of a CTA
};
constexpr int kCompactThreads = 128;
constexpr int kCompactSmem = 34 * 1024;  // 64 tokens of 512 + 8 bytes: one layer always fits

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p) {
  extern __shared__ __align__(16) uint8_t rows[];  // codes [layer][token][2 code_bytes], then parameters [layer][token][2]
  __shared__ int64_t src[kMaxQ], dst[kMaxQ];  // tiles' first bytes, within a layer
  __shared__ int src_row[kMaxQ], dst_row[kMaxQ];
  __shared__ int moved, kept;
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.y;
  const int head = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int n = p.q_start ? max(p.q_start[b + 1] - p.q_start[b], 0) : 1;
  const int64_t len = min(int64_t(max(p.lens[b], 0)), p.cols * p.page_size);
  const int64_t place0 = len - n;  // of the sequence's first drafted token
  const int64_t tile_bytes = 32 * p.code_bytes + 128, head_bytes = p.page_size / 16 * tile_bytes, page_bytes = p.heads * head_bytes;
  if (tid == 0) moved = 0;
  if (tid < 32) {  // the path ends at its first negative entry
    unsigned ends = __ballot_sync(0xFFFFFFFFu, tid >= p.max_q || p.path[b * p.max_q + tid] < 0);
    int k = ends ? __ffs(ends) - 1 : 32;
    if (k == 32) {
      ends = __ballot_sync(0xFFFFFFFFu, tid + 32 >= p.max_q || p.path[b * p.max_q + tid + 32] < 0);
      k += ends ? __ffs(ends) - 1 : 32;
    }
    if (tid == 0) kept = k;
  }
  __syncthreads();
  const int count = kept;
  if (tid < count) {
    const int from = p.path[b * p.max_q + tid];
    const int64_t a = place0 + from, z = place0 + tid;
    // (a place past the cached tokens, in front of the first or on a page outside the cache is not moved)
    if (from != tid && from < n && tid < n && a >= 0 && z >= 0) {
      const int pa = p.table[b * p.cols + a / p.page_size], pz = p.table[b * p.cols + z / p.page_size];
      if (pa >= 0 && pa < p.pages && pz >= 0 && pz < p.pages) {
        const int i = atomicAdd(&moved, 1);  // (in any order: each has its own places)
        src[i] = pa * page_bytes + head * head_bytes + a % p.page_size / 16 * tile_bytes;
        dst[i] = pz * page_bytes + head * head_bytes + z % p.page_size / 16 * tile_bytes;
        src_row[i] = static_cast<int>(a % 16), dst_row[i] = static_cast<int>(z % 16);
      }
    }
  }
  __syncthreads();
  const int units = 2 * p.code_bytes / 16, half = p.code_bytes / 16;
  const int m = moved, first = blockIdx.z * p.each, layers = min(p.each, p.layers - first);
  uint8_t *cache = p.cache + first * p.layer_bytes;
  uint4 *codes = reinterpret_cast<uint4 *>(rows);
  uint32_t *params = reinterpret_cast<uint32_t *>(rows + p.each * p.max_q * 2 * p.code_bytes);
  auto code_at = [&](int e, const int64_t *tile, const int *row) {  // of vector e: layer, token, unit
    const int u = e % units, i = e / units % m, kind = u >= half;
    return reinterpret_cast<uint4 *>(cache + e / units / m * p.layer_bytes + tile[i] + (kind * 16 + row[i]) * p.code_bytes + (u - kind * half) * 16);
  };
  auto param_at = [&](int e, const int64_t *tile, const int *row) {
    const int i = e / 2 % m;
    return reinterpret_cast<uint32_t *>(cache + e / 2 / m * p.layer_bytes + tile[i] + 32 * p.code_bytes + (e & 1) * 64 + row[i] * 4);
  };
  for (int e = tid; e < layers * m * units; e += kCompactThreads) codes[e] = *code_at(e, src, src_row);
  for (int e = tid; e < layers * m * 2; e += kCompactThreads) params[e] = *param_at(e, src, src_row);
  __syncthreads();
  for (int e = tid; e < layers * m * units; e += kCompactThreads) *code_at(e, dst, dst_row) = codes[e];
  for (int e = tid; e < layers * m * 2; e += kCompactThreads) *param_at(e, dst, dst_row) = params[e];
  if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) p.new_lens[b] = static_cast<int32_t>(max(place0 + min(count, n), int64_t(0)));
}

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e == cudaSuccess) note_launch();
  return e;
}

Pool pool_of(const PoolArgs &a) { return Pool{a.refs, static_cast<int>(a.num_pages), a.page_size, a.max_pages}; }

}  // namespace

int kv_reserve_most_sequences() { return kMaxSequences; }

cudaError_t launch_kv_fork(const PoolArgs &a, const int32_t *table, const int32_t *lens, int64_t batch, const int32_t *parents, int64_t rows,
                           int32_t *new_table, int32_t *new_lens, cudaStream_t stream) {
  return launch(fork_kernel, dim3(static_cast<unsigned>(rows)), 256, 0, stream, pool_of(a), table, lens, batch, parents, new_table, new_lens);
}
cudaError_t launch_kv_free(const PoolArgs &a, int32_t *table, const int32_t *lens, const int32_t *keep, int64_t batch, cudaStream_t stream) {
  return launch(free_kernel, dim3(static_cast<unsigned>(batch)), 256, 0, stream, pool_of(a), table, lens, keep);
}
cudaError_t launch_kv_reserve(const PoolArgs &a, int32_t *table, const int32_t *lens, const int32_t *new_lens, int64_t batch, int32_t *held,
                              int32_t *copies, cudaStream_t stream) {
  return launch(reserve_kernel, dim3(1), kReserveThreads, 0, stream, pool_of(a), table, lens, new_lens, static_cast<int>(batch), held,
                reinterpret_cast<int2 *>(copies));
}
cudaError_t launch_kv_copy(const w4a16_kv_cache_t &c, int64_t layers, const int32_t *pairs, int64_t n, cudaStream_t stream) {
  const int64_t page_bytes = int64_t(c.kv_heads) * (c.page_size / kTileTokens) * kv_tile_bytes(c.head_dim, c.bits);
  const int64_t parts = (page_bytes / 16 + kCopyThreads * kCopyVectors - 1) / (kCopyThreads * kCopyVectors);
  for (int64_t done = 0; done < n; done += 65535) {
    const int64_t m = std::min<int64_t>(n - done, 65535);
    const cudaError_t e = launch(copy_kernel, dim3(static_cast<unsigned>(parts), static_cast<unsigned>(m), static_cast<unsigned>(layers)),
                                 kCopyThreads, 0, stream, static_cast<uint8_t *>(c.data), c.num_pages * page_bytes, page_bytes,
                                 static_cast<int>(c.num_pages), reinterpret_cast<const int2 *>(pairs) + done);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
cudaError_t launch_kv_compact(const CompactArgs &a, int num_sms, cudaStream_t stream) {
  const w4a16_kv_cache_t &c = a.cache;
  CompactParams p{};
  p.cache = static_cast<uint8_t *>(c.data);
  p.pages = static_cast<int>(c.num_pages);
  p.heads = c.kv_heads;
  p.page_size = c.page_size;
  p.code_bytes = c.head_dim * c.bits / 8;
  p.layer_bytes = c.num_pages * c.kv_heads * (c.page_size / kTileTokens) * kv_tile_bytes(c.head_dim, c.bits);
  p.cols = a.max_pages;
  p.table = a.page_table;
  p.lens = a.kv_lens;
  p.q_start = a.q_start;
  p.path = a.path;
  p.max_q = a.max_q;
  p.new_lens = a.new_lens;
  // Several layers a CTA, which share the look-up of the places and have their loads in flight together, while the rows fit and
  // the CTAs fill the device (eight of 128 threads on an SM)
  const int row_bytes = 2 * p.code_bytes + 8;
  const int64_t ctas = a.batch * c.kv_heads;
  p.layers = static_cast<int>(a.layers);
  p.each = 1;
  while (p.each < p.layers && p.each * 2 * a.max_q * row_bytes <= kCompactSmem && ctas * (p.layers / (p.each * 2)) >= 8 * num_sms) p.each *= 2;
  const size_t smem = static_cast<size_t>(p.each) * a.max_q * row_bytes;
  const unsigned parts = static_cast<unsigned>((p.layers + p.each - 1) / p.each);
  for (int64_t done = 0; done < a.batch; done += 65535) {
    const int64_t m = std::min<int64_t>(a.batch - done, 65535);
    const cudaError_t e = launch(compact_kernel, dim3(static_cast<unsigned>(c.kv_heads), static_cast<unsigned>(m), parts),
                                 kCompactThreads, smem, stream, p);
    if (e != cudaSuccess) return e;
    p.table += m * a.max_pages;
    p.lens += m;
    if (p.q_start) p.q_start += m;
    p.path += m * a.max_q;
    p.new_lens += m;
  }
  return cudaSuccess;
}

}  // namespace w4a16
