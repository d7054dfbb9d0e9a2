// Low-rank adapters of many requests beside a shared projection.
//
//     out_t = base_t + s_i (x_t A_i^T) B_i^T,   i = ids[t];  A_i [r, K], B_i [N, r]
//
// One kernel does both products; h = x A^T (r numbers a token) never leaves the SMs. A cluster of CTAs takes a tile of tokens
// of one adapter. First product: the CTAs and their warps split K, so that A and x are read once a tile, as fragments of
// mma.m16n8k16 (adapter rows on the M side, tokens on the N side). The order of k within a sum is free, so a lane's 16
// contiguous bytes of a row serve as its elements of two MMAs, for both operands alike: asynchronous copies bring them into slots that
// only this thread reads, a stage ahead of the MMAs, with no barrier and no bank conflict. The slices' partial sums are added in shared
// memory, the CTAs' through distributed shared memory, in a fixed order. Second product: the CTAs and warps split N, tokens on the M
// side, h as the A operand from shared memory; the columns of four n-tiles are dealt out so that a lane ends up with eight
// contiguous columns of a token: 16-byte copies of base and stores of out. (Steps of 128 instead of 64 bytes a row, in a ring that a warp
// shares: the first product alone 3 us faster, the second 7 slower, since half the warps fit.)
//
// h is fp32 and goes into the second product whole, as a sum of numbers of the dtype: three for bfloat16, which hold all 24 bits (with
// two, 16 of them, 3 of 1000 elements of out were rounded the other way, and what cancels between the products was off), two for
// float16, 22 bits below the token's largest (whose range its sums may leave: each token's h is scaled by a power
// of two). The rounding of out is then the only one that shows. The third part costs 7 to 9 % at ranks 17 to 64 of long prompts (8191 tokens 5120 -> 7168, rank 32:
// 74.6 -> 81.3 us); up to rank 16, and for few tokens, the parts share a pass whose half was empty, and it costs nothing or 2 %.
//
// Tiles: tokens of the same adapter wherever they stand. Up to kFewTokens tokens every CTA ranks the tokens among
// those of their adapter by itself, up to kCountTokens it counts them by adapter in shared memory (one launch); more are sorted by a
// kernel before this one (counting sort). The composition of a tile does not change a token's result: the rows of an MMA do not mix
// and K is split in the same way.
//
// Bound by memory for long prompts (base read and out written are most of the bytes), by the chain of copies, barriers and sums for few tokens. Measured, replayed from a graph: 8191 tokens 5120 -> 7168 of rank
// 32 81 us for 328 MB, 4.0 TB/s, 0.60 of the device's copy rate (9 us of them the sort and the launch; the same tiles copied without
// an adapter 0.85 of it while they stream); DRAM 49 %, tensor pipe 39 %, schedulers 40 % of the cycles. 520 tokens 2560 -> 3840 of rank 64 19.1
// us in float16, 20.0 in bfloat16; 48 tokens 5120 -> 7168 of rank 16 8.9; one token 2112 -> 1152 4.2.
#include <algorithm>
#include <atomic>

#include "lora_common.cuh"

namespace w4a16 {
using namespace lora;
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
// One thread for each. Ranked against counted, 5120 -> 7168, 256 tokens of 32 adapters: 15.1 against 16.1 us (rank 16), 22.4 against
// 25.1 (rank 64); 64 tokens: 9.2 against 12.9, 19.8 against 23.5.
constexpr int kFewTokens = 256;
constexpr int kFewTile = 8;      // tokens of a tile then
// Up to this many tokens of this many adapters (and ranks that stay with this form) a CTA counts the tokens of each adapter in shared memory. On the GPU as long as sorted by
// a kernel before (2560 -> 3840, rank 64: 400 tokens 20.0 against 19.3 us, 1000 tokens 19.4 against 19.2), with a launch less to
// issue (3.8 against 14 us, a workspace among it).
constexpr int kCountTokens = 1024, kCountAdapters = 512;
constexpr int kSortThreads = 1024;
constexpr int kMaxAdapters = 8191;  // counters of the sort in shared memory

struct Params {
  const uint16_t *x, *a, *b, *base;
  uint16_t *out;
  const int32_t *ids;
  const float *scales;
  int64_t x_stride, base_stride, out_stride;
  int64_t tokens, K, N;
  int rank, adapters;
  int csize;
  bool copy;  // out is not base: tokens without an adapter are copied
  int32_t *order;     // sorted tokens (null: few tokens, ranked here)
  const Tile *tiles;
  const int32_t *num_tiles;
};

// MR, NT: m-tiles (adapter rows) and n-tiles (tokens) of a warp's first product; RS: parts of the rank, each with its warps
template <int MR_, int NT_, int RS_, int STAGES, int CTAS>
struct Shape {
  static constexpr int MR = MR_, NT = NT_, RS = RS_, kCtas = CTAS;
  static constexpr int kRanks = 16 * MR * RS, kTokens = 8 * NT;
  static constexpr int kSlices = kWarps / RS;       // parts of K in a CTA
  static constexpr int kMT = (NT + 1) / 2;          // m-tiles of the second product
  static constexpr int kHalves = NT == 1 ? 1 : 2;   // (one n-tile fills half an m-tile)
  static constexpr int kChunks = (MR * RS + 1) / 2; // its k, in steps of 32
  static constexpr int kHStride = kRanks + 4;
  // 16-byte slots of a thread in a stage of each product's ring
  static constexpr int kSlots1 = 2 * MR + NT, kSlots2 = kMT * kHalves + 4 * kChunks;
  static constexpr int kSlots = STAGES * (kSlots1 > kSlots2 ? kSlots1 : kSlots2);
  static constexpr int kStages1 = kSlots / kSlots1, kStages2 = kSlots / kSlots2;
  static constexpr int kRing = kSlots * kThreads * 16;  // bytes
  static constexpr int kSums = MR * RS * NT * 32;       // float4 of a K slice's sums
  static constexpr int kH = kMT * 16 * kHStride;        // floats
  static_assert(kSlices * kSums * 16 + kH * 4 <= kRing, "the partial sums and h lie in the ring");
  static_assert(kSums % kMaxCluster == 0, "equal shares of the sums for the CTAs of a cluster");
  static_assert(kStages1 >= 2 && kStages2 >= 2, "one stage is in flight while another is used");
  // The parts of h that one pass of the second product takes: where a rank of 16 leaves half of a chunk's k empty, and a single n-tile half of
  // the m-tile's rows, these hold further parts (their B again, their sums added)
  static constexpr int kKParts = MR * RS == 1 ? 2 : 1, kMParts = NT == 1 ? 2 : 1;
  template <int PARTS>
  static constexpr int kPasses = (PARTS + kKParts * kMParts - 1) / (kKParts * kMParts);
  static constexpr int kFrag = kMT * kChunks * 2 * 32 * 16;  // bytes of a pass: [m-tile][chunk][step][pass][lane]
};

__device__ __forceinline__ void st_dsmem_f32(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

// How a CTA comes to its tiles
enum Tiling {
  kRanked,   // few tokens: each compared with those before it
  kCounted,  // more: counted by adapter in shared memory
  kListed    // sorted by a kernel before this one
};

template <class DT, class S, int TILING>
__global__ void __launch_bounds__(kThreads, S::kCtas) lora_kernel(const Params p) {
  constexpr int MR = S::MR, NT = S::NT;
  extern __shared__ __align__(16) uint8_t smem[];
  uint4 *ring = reinterpret_cast<uint4 *>(smem) + threadIdx.x;           // this thread's slots, kThreads apart
  float4 *part = reinterpret_cast<float4 *>(smem);                       // [slice][m-tile][n-tile][lane], in the ring's place
  float *h = reinterpret_cast<float *>(part + S::kSlices * S::kSums);    // [token][rank], behind it
  constexpr int kP = kParts<DT>, kPasses = S::template kPasses<kP>;
  uint4 *frag = reinterpret_cast<uint4 *>(smem + S::kRing);
  __shared__ int tok[S::kTokens];
  __shared__ float back[S::kMT * 16];  // what a token's h was divided by (float16)
  constexpr int kIds = TILING == kRanked ? kFewTokens : 4, kCodes = TILING == kCounted ? kCountTokens : 4;
  __shared__ __align__(16) int ids_s[kIds];
  // counted: each token's tile (adapter << 5 | the tile's number in it) and place there, in 3 KB, which lets two CTAs of rank 64 on an SM
  __shared__ uint16_t codes[kCodes];
  __shared__ uint8_t places[kCodes];
  __shared__ uint16_t leaders[TILING == kCounted ? kCountTokens / S::kTokens + kCountAdapters + 1 : kIds];  // counted: the tiles
  __shared__ int warp_count[kWarps];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int slice = warp / S::RS, ranks = warp % S::RS;  // part of K, part of the rank
  const int csize = p.csize;
  const int crank = csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster = blockIdx.x / csize, clusters = gridDim.x / csize;
  griddep_wait();

  int my_id = -2, my_rank = 0, ntiles;
  if constexpr (TILING == kListed) {
    ntiles = *p.num_tiles;
  } else if constexpr (TILING == kCounted) {
    static_assert(kCountTokens / S::kTokens <= 32 && kCountAdapters < 2048 && S::kTokens <= 256, "a tile in 16 bits, a place in 8");
    static_assert(((kWarps + 1) * (kCountAdapters + 1)) * 4 <= S::kRing, "the counters lie in the ring");
    constexpr int kEach = kCountTokens / kThreads;
    int *counts = reinterpret_cast<int *>(smem);  // [warp][adapter], tokens without one last; then the sums
    const int na = p.adapters + 1, tokens = static_cast<int>(p.tokens);
    // each warp has consecutive tokens, so that ranks follow the tokens' order whatever the timing
    const int per = (tokens + kThreads - 1) / kThreads * 32;
    int *mine = counts + warp * na;
    int id[kEach], rank[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = warp * per + j * 32 + lane;
      id[j] = -1;
      if (j * 32 < per && i < tokens) {
        id[j] = p.ids[i];
        if (id[j] < 0 || id[j] >= p.adapters) id[j] = p.adapters;
      }
    }
    for (int i = tid; i < kWarps * na; i += kThreads) counts[i] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const unsigned same = __match_any_sync(0xFFFFFFFFu, id[j]);
      const int before = id[j] >= 0 ? mine[id[j]] : 0;
      __syncwarp();
      rank[j] = before + __popc(same & ((1u << lane) - 1));
      if (id[j] >= 0 && lane == __ffs(same) - 1) mine[id[j]] = before + __popc(same);
      __syncwarp();
    }
    __syncthreads();
    for (int a = tid; a < na; a += kThreads) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int v = counts[w * na + a];
        counts[w * na + a] = sum;
        sum += v;
      }
      counts[kWarps * na + a] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (id[j] >= 0) {
        const int i = warp * per + j * 32 + lane, r = mine[id[j]] + rank[j];
        codes[i] = static_cast<uint16_t>(id[j] << 5 | r / S::kTokens), places[i] = static_cast<uint8_t>(r % S::kTokens);
      }
    if (warp == 0) {
      int listed = 0;
      for (int a0 = 0; a0 < na; a0 += 32) {
        const int a = a0 + lane;
        const int n = a < na && (a < p.adapters || p.copy) ? (counts[kWarps * na + a] + S::kTokens - 1) / S::kTokens : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
          if (lane >= o) sum += u;
        }
        for (int i = 0; i < n; ++i) leaders[listed + sum - n + i] = static_cast<uint16_t>(a << 5 | i);
        listed += __shfl_sync(0xFFFFFFFFu, sum, 31);
      }
      if (lane == 0) warp_count[0] = listed;
    }
    __syncthreads();
    ntiles = warp_count[0];
  } else {
    if (tid < p.tokens) {
      my_id = p.ids[tid];
      if (my_id < 0 || my_id >= p.adapters) my_id = -1;
    }
    ids_s[tid] = my_id;
    __syncthreads();
    const int4 *all = reinterpret_cast<const int4 *>(ids_s);
    for (int j = 0; j * 4 < p.tokens; ++j) {
      const int4 v = all[j];
      my_rank += (v.x == my_id && j * 4 < tid) + (v.y == my_id && j * 4 + 1 < tid) + (v.z == my_id && j * 4 + 2 < tid) +
                 (v.w == my_id && j * 4 + 3 < tid);
    }
    const bool lead = tid < p.tokens && my_rank % S::kTokens == 0 && (my_id >= 0 || p.copy);
    const unsigned vote = __ballot_sync(0xFFFFFFFFu, lead);
    if (lane == 0) warp_count[warp] = __popc(vote);
    __syncthreads();
    int at = __popc(vote & ((1u << lane) - 1));
    ntiles = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) at += ntiles;
      ntiles += warp_count[w];
    }
    if (lead) leaders[at] = static_cast<uint16_t>(tid);
    __syncthreads();
  }

  for (int tile = cluster; tile < ntiles; tile += clusters) {
    int adapter, count;
    if constexpr (TILING == kListed) {
      const Tile d = p.tiles[tile];
      adapter = d.adapter, count = d.count;
      if (tid < count) tok[tid] = p.order[d.first + tid];
    } else if constexpr (TILING == kCounted) {
      const int d = leaders[tile], a = d >> 5;
      adapter = a == p.adapters ? -1 : a;
      count = 0;
      for (int i0 = 0; i0 < p.tokens; i0 += kThreads) {
        const int i = i0 + tid;
        const bool in = i < p.tokens && codes[i] == d;
        if (in) tok[places[i]] = i;
        count += __syncthreads_count(in);
      }
    } else {
      const int leader = leaders[tile];
      adapter = ids_s[leader];
      // (the leader's rank is counted by its own thread only)
      const bool same = my_id == adapter && tid < p.tokens;
      int lead_rank = 0;
      for (int j = lane; j < leader; j += 32) lead_rank += ids_s[j] == adapter;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) lead_rank += __shfl_xor_sync(0xFFFFFFFFu, lead_rank, o);
      const int at = my_rank - lead_rank;
      const bool in = same && at >= 0 && at < S::kTokens;
      if (in) tok[at] = tid;
      count = __syncthreads_count(in);
    }
    __syncthreads();

    // ---- first product: h^T = A x^T, K split over the cluster's warps
    const uint16_t *ap = nullptr, *bp = nullptr;
    if (adapter >= 0) {
      ap = p.a + int64_t(adapter) * p.rank * p.K;
      bp = p.b + int64_t(adapter) * p.N * p.rank;
      float acc[MR][NT][4];
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
      // rows in units of 16 bytes
      uint32_t xr[NT], ar[MR][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) xr[n] = static_cast<uint32_t>(tok[min(n * 8 + g, count - 1)] * p.x_stride >> 3);
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) ar[m][i] = static_cast<uint32_t>((ranks * MR + m) * 16 + i * 8 + g) * static_cast<uint32_t>(p.K >> 3);
      const uint4 *x16 = reinterpret_cast<const uint4 *>(p.x), *a16 = reinterpret_cast<const uint4 *>(ap);
      const uint32_t units = static_cast<uint32_t>(p.K >> 3);  // of 8 elements
      const uint32_t u0 = (crank * S::kSlices + slice) * 4, step = csize * S::kSlices * 4;
      const int steps = u0 < units ? static_cast<int>((units - u0 + step - 1) / step) : 0;
      // loads of step i, into this thread's own slots: no barrier between them and their use
      // (Tokens past the tile's last and eights of rows past the rank are left out, and so are the sums with what lies in their slots.
      // The last row read once more in their place was a line that many asked for: 86 tokens 7960 -> 512 of rank 72 took 22 us, 11
      // without.)
      auto fetch = [&](int i) {
        const uint32_t k = u0 + i * step + t;
        const bool in = k < units;
        const uint32_t kk = in ? k : 0;
        const uint32_t at = smem_u32(ring + (i % S::kStages1) * S::kSlots1 * kThreads);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n * 8 + g < count) cp_async_16(at + n * (kThreads * 16), x16 + (xr[n] + kk), in);
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2)
            if ((ranks * MR + m) * 16 + i2 * 8 < p.rank) cp_async_16(at + (NT + m * 2 + i2) * (kThreads * 16), a16 + (ar[m][i2] + kk), in);
      };
#pragma unroll
      for (int i = 0; i < S::kStages1 - 1; ++i) {
        if (i < steps) fetch(i);
        cp_async_commit();
      }
      for (int i = 0; i < steps; ++i) {
        // (into the slots that the step before this one has read)
        if (i + S::kStages1 - 1 < steps) fetch(i + S::kStages1 - 1);
        cp_async_commit();
        cp_async_wait<S::kStages1 - 1>();
        const uint4 *at = ring + (i % S::kStages1) * S::kSlots1 * kThreads;
        uint4 av[MR][2];
#pragma unroll
        for (int m = 0; m < MR; ++m) av[m][0] = at[(NT + m * 2) * kThreads], av[m][1] = at[(NT + m * 2 + 1) * kThreads];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (NT > 1 && n * 8 >= count) break;
          const uint4 xv = at[n * kThreads];
#pragma unroll
          for (int m = 0; m < MR; ++m) {
            const uint4 v0 = av[m][0], v1 = av[m][1];
            const uint32_t f0[4] = {v0.x, v1.x, v0.y, v1.y}, f1[4] = {v0.z, v1.z, v0.w, v1.w};
            mma_16816<DT::kBF16>(acc[m][n], f0, xv.x, xv.y);
            mma_16816<DT::kBF16>(acc[m][n], f1, xv.z, xv.w);
          }
        }
      }
      __syncthreads();  // the ring is not read any more (every load of it was waited for)
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          part[slice * S::kSums + ((ranks * MR + m) * NT + n) * 32 + lane] = make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
    }
    __syncthreads();
    const float s = adapter >= 0 ? (p.scales ? p.scales[adapter] : 1.f) : 0.f;
    if (adapter >= 0) {
      // the slices' sums, then the CTAs', each in order
      for (int e = tid; e < S::kSums; e += kThreads) {
        float4 v = part[e];
#pragma unroll
        for (int w = 1; w < S::kSlices; ++w) {
          const float4 o = part[w * S::kSums + e];
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        part[e] = v;
      }
      if (csize > 1) {
        // Each CTA adds an equal share of the sums and writes the result into every CTA's h: a lane for each destination, so
        // that a warp's remote loads are of few addresses. (All CTAs reading all sums: 2.2 to 4.2 us for eight of them.)
        cluster_sync_all();
        const int share = S::kSums / csize;
        for (int i = tid; i < S::kSums; i += kThreads) {
          const int e = crank * share + i / csize, to = i % csize;
          const uint32_t mine = smem_u32(&part[e]);
          float4 o[kMaxCluster];  // all loads in flight together
#pragma unroll
          for (int c = 0; c < kMaxCluster; ++c) o[c] = ld_dsmem_v4(map_to_rank(mine, min(c, csize - 1)));
          float4 v = o[0];
#pragma unroll
          for (int c = 1; c < kMaxCluster; ++c)
            if (c < csize) v.x += o[c].x, v.y += o[c].y, v.z += o[c].z, v.w += o[c].w;
          const int l = e & 31, n = (e >> 5) % NT, m = (e >> 5) / NT;
          const uint32_t at = map_to_rank(smem_u32(h + (n * 8 + 2 * (l & 3)) * S::kHStride + m * 16 + (l >> 2)), to);
          st_dsmem_f32(at, v.x * s), st_dsmem_f32(at + S::kHStride * 4, v.y * s);
          st_dsmem_f32(at + 32, v.z * s), st_dsmem_f32(at + S::kHStride * 4 + 32, v.w * s);
        }
        cluster_sync_all();
      } else {
        for (int e = tid; e < S::kSums; e += kThreads) {  // (each thread's own elements)
          const float4 v = part[e];
          const int l = e & 31, n = (e >> 5) % NT, m = (e >> 5) / NT;
          float *at = h + (n * 8 + 2 * (l & 3)) * S::kHStride + m * 16 + (l >> 2);
          at[0] = v.x * s, at[S::kHStride] = v.y * s, at[8] = v.z * s, at[S::kHStride + 8] = v.w * s;
        }
        __syncthreads();
      }
      if constexpr (!DT::kBF16) {  // each token's power of two
        for (int i = tid >> 3; i < S::kTokens; i += kThreads / 8) {  // eight threads a token
          float top = 0.f;
          for (int r = tid & 7; r < p.rank; r += 8) top = fmaxf(top, fabsf(h[i * S::kHStride + r]));  // (a NaN does not count)
          const unsigned eight = 0xFFu << (lane & 24);
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(eight, top, o));
          if ((tid & 7) == 0) back[i] = unit_of_largest(top);
        }
        __syncthreads();
      }
      // a thread's words: of a lane's fragment of a step those of row g (i = 0) or g + 8
      uint32_t *words = reinterpret_cast<uint32_t *>(frag);
      for (int e = tid; e < S::kMT * S::kChunks * 128; e += kThreads) {
        const int i = e & 1, l = e >> 1 & 31, st = e >> 6 & 1, c = (e >> 7) % S::kChunks, m = (e >> 7) / S::kChunks;
        const int row = m * 16 + (S::kMParts == 1 ? i * 8 : 0) + (l >> 2);
        const int r0 = (S::kKParts == 1 ? c * 32 + (l & 3) * 8 : (l & 1) * 8) + 4 * st;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 < p.rank) v = *reinterpret_cast<const float4 *>(h + row * S::kHStride + r0);  // (the rank is a multiple of 8)
        if constexpr (!DT::kBF16) {
          const float unit = 1.f / back[row];  // (exact: a power of two)
          v.x *= unit, v.y *= unit, v.z *= unit, v.w *= unit;
        }
        uint32_t part[2][kP];
#pragma unroll
        for (int q = 0; q < kP; ++q) part[0][q] = take_part<DT>(v.x, v.y), part[1][q] = take_part<DT>(v.z, v.w);
        const int first = (S::kMParts == 1 ? 0 : i) * S::kKParts + (S::kKParts == 1 ? 0 : l >> 1 & 1);  // of the first pass
        uint32_t *at = words + (((m * S::kChunks + c) * 2 + st) * kPasses * 32 + l) * 4 + i;
#pragma unroll
        for (int q = 0; q < kPasses; ++q) {
          uint2 w = make_uint2(0, 0);  // the part first + q kMParts kKParts, if there is one
#pragma unroll
          for (int k = 0; k < kP; ++k)
            if (k == first + q * S::kMParts * S::kKParts) w = make_uint2(part[0][k], part[1][k]);
          at[q * 128] = w.x, at[q * 128 + 2] = w.y;
        }
      }
      // (the ring takes the second product's loads: the partial sums in its place were read by the whole cluster)
      __syncthreads();
    }

    // ---- second product: out = base + h B^T, N split over the cluster's warps in groups of 32 columns
    const uint32_t n_units = static_cast<uint32_t>(p.N >> 3), r_units = p.rank >> 3;
    const uint4 *b16 = reinterpret_cast<const uint4 *>(bp), *base16 = reinterpret_cast<const uint4 *>(p.base);
    uint4 *out16 = reinterpret_cast<uint4 *>(p.out);
    const uint32_t c0 = (crank * kWarps + warp) * 4, cstep = csize * kWarps * 4;  // in units of 8 columns
    const int groups = c0 < n_units ? static_cast<int>((n_units - c0 + cstep - 1) / cstep) : 0;
    auto fetch = [&](int i) {
      const uint32_t n0 = c0 + i * cstep, col = n0 + t;
      const uint32_t at = smem_u32(ring + (i % S::kStages2) * S::kSlots2 * kThreads);
#pragma unroll
      for (int m = 0; m < S::kMT; ++m)
#pragma unroll
        for (int i2 = 0; i2 < S::kHalves; ++i2) {
          const int row = m * 16 + i2 * 8 + g;
          if (col < n_units && row < count)
            cp_async_16(at + (m * S::kHalves + i2) * (kThreads * 16), base16 + ((tok[row] * p.base_stride >> 3) + col), true);
        }
      if (adapter >= 0) {
        const bool has = n0 + (g >> 1) < n_units;
        const uint32_t brow = has ? n0 * 8 + (g >> 1) * 8 + (g & 1) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < S::kChunks; ++c) {
            const uint32_t unit = S::kKParts == 1 ? c * 4 + t : t & 1;
            const bool in = has && unit < r_units;
            cp_async_16(at + (S::kMT * S::kHalves + j * S::kChunks + c) * (kThreads * 16),
                        b16 + (in ? uint64_t(brow + 2 * j) * r_units + unit : 0), in);
          }
      }
    };
#pragma unroll
    for (int i = 0; i < S::kStages2 - 1; ++i) {
      if (i < groups) fetch(i);
      cp_async_commit();
    }
    for (int i = 0; i < groups; ++i) {
      if (i + S::kStages2 - 1 < groups) fetch(i + S::kStages2 - 1);
      cp_async_commit();
      cp_async_wait<S::kStages2 - 1>();
      const uint32_t col = c0 + i * cstep + t;
      const bool in = col < n_units;
      const uint4 *at = ring + (i % S::kStages2) * S::kSlots2 * kThreads;
      uint4 bv[4][S::kChunks];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < S::kChunks; ++c) bv[j][c] = at[(S::kMT * S::kHalves + j * S::kChunks + c) * kThreads];
#pragma unroll
      for (int m = 0; m < S::kMT; ++m) {
        if (m * 16 >= count) break;
        const int i0 = m * 16 + g, i1 = i0 + 8;
        uint4 o0 = at[m * S::kHalves * kThreads], o1 = at[(m * S::kHalves + S::kHalves - 1) * kThreads];
        if (adapter >= 0) {
          float acc[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
          for (int c = 0; c < S::kChunks; ++c)
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              const uint4 *f = frag + ((m * S::kChunks + c) * 2 + st) * kPasses * 32 + lane;
#pragma unroll
              for (int q = kPasses - 1; q >= 0; --q) {  // the smallest parts first
                const uint4 v = f[q * 32];
                const uint32_t fr[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_16816<DT::kBF16>(acc[j], fr, st ? bv[j][c].z : bv[j][c].x, st ? bv[j][c].w : bv[j][c].y);
              }
            }
          if constexpr (S::kMParts == 2)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j][0] += acc[j][2], acc[j][1] += acc[j][3];
          float f0 = 1.f, f1 = 1.f;
          if constexpr (!DT::kBF16) f0 = back[i0 < S::kTokens ? i0 : 0], f1 = back[i1 < S::kTokens ? i1 : 0];
          add2<DT>(o0.x, acc[0][0], acc[0][1], f0), add2<DT>(o1.x, acc[0][2], acc[0][3], f1);
          add2<DT>(o0.y, acc[1][0], acc[1][1], f0), add2<DT>(o1.y, acc[1][2], acc[1][3], f1);
          add2<DT>(o0.z, acc[2][0], acc[2][1], f0), add2<DT>(o1.z, acc[2][2], acc[2][3], f1);
          add2<DT>(o0.w, acc[3][0], acc[3][1], f0), add2<DT>(o1.w, acc[3][2], acc[3][3], f1);
        }
        if (in && i0 < count) __stcs(out16 + (tok[i0] * p.out_stride >> 3) + col, o0);
        if (S::kHalves == 2 && in && i1 < count) __stcs(out16 + (tok[i1] * p.out_stride >> 3) + col, o1);
      }
    }
    __syncthreads();  // done with the tile's tables and the ring
  }
  // Only now: CTAs of the next kernel that start while this one runs all go to the SMs that it leaves free, two on one while others
  // have none (1000 tokens of rank 64, call after call: 28 us, 19 with this)
  griddep_launch_dependents();
}

// Counting sort of the tokens by adapter (those without one last), and the list of tiles. One CTA.
__global__ void __launch_bounds__(kSortThreads) lora_sort_kernel(const int32_t *ids, int tokens, int adapters, int tile_tokens, bool copy,
                                                                 int32_t *order, Tile *tiles, int32_t *num_tiles) {
  extern __shared__ int counts[];  // [adapters + 1], then the next place of each
  __shared__ int sums[2][kSortThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();  // the kernel before this one may still read the lists
  griddep_launch_dependents();
  for (int i = tid; i <= adapters; i += kSortThreads) counts[i] = 0;
  __syncthreads();
  auto key = [&](int i) {
    const int id = ids[i];
    return id < 0 || id >= adapters ? adapters : id;
  };
  // (the loads of eight steps are in flight together)
  constexpr int kBatch = 8;
  for (int i0 = tid; i0 - lane < tokens; i0 += kSortThreads * kBatch) {
    int k[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) k[j] = i0 + j * kSortThreads < tokens ? key(i0 + j * kSortThreads) : -1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      // a run of one request's tokens fills most warps; else each lane adds for itself
      const bool one = __all_sync(0xFFFFFFFFu, k[j] == __shfl_sync(0xFFFFFFFFu, k[j], 0));
      if (k[j] >= 0 && (!one || lane == 0)) atomicAdd(&counts[k[j]], one ? 32 : 1);
    }
  }
  __syncthreads();
  // places of each adapter's tokens and tiles: exclusive sums over the adapters, in chunks of one a thread
  int tokens_before = 0, tiles_before = 0;
  for (int k0 = 0; k0 <= adapters; k0 += kSortThreads) {
    const int k = k0 + tid;
    const int n = k <= adapters ? counts[k] : 0;
    const int nt = k == adapters && !copy ? 0 : (n + tile_tokens - 1) / tile_tokens;
    int a = n, b = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ua = __shfl_up_sync(0xFFFFFFFFu, a, o), ub = __shfl_up_sync(0xFFFFFFFFu, b, o);
      if (lane >= o) a += ua, b += ub;
    }
    if (lane == 31) sums[0][warp] = a, sums[1][warp] = b;
    __syncthreads();
    static_assert(kSortThreads == 1024, "a lane for each warp's sums");
    const int sa = sums[0][lane], sb = sums[1][lane];
    int ta = sa, tb = sb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ua = __shfl_up_sync(0xFFFFFFFFu, ta, o), ub = __shfl_up_sync(0xFFFFFFFFu, tb, o);
      if (lane >= o) ta += ua, tb += ub;
    }
    const int wa = __shfl_sync(0xFFFFFFFFu, ta - sa, warp), wb = __shfl_sync(0xFFFFFFFFu, tb - sb, warp);
    ta = __shfl_sync(0xFFFFFFFFu, ta, 31), tb = __shfl_sync(0xFFFFFFFFu, tb, 31);
    const int first = tokens_before + wa + a - n;
    int at = tiles_before + wb + b - nt;
    if (k <= adapters) {
      counts[k] = first;
      for (int i = 0; i < nt; ++i)
        tiles[at++] = Tile{k == adapters ? -1 : k, first + i * tile_tokens, min(tile_tokens, n - i * tile_tokens)};
    }
    tokens_before += ta, tiles_before += tb;
    __syncthreads();
  }
  if (tid == 0) *num_tiles = tiles_before;
  for (int i0 = tid; i0 - lane < tokens; i0 += kSortThreads * kBatch) {
    int k[kBatch], at[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) k[j] = i0 + j * kSortThreads < tokens ? key(i0 + j * kSortThreads) : -1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const bool one = __all_sync(0xFFFFFFFFu, k[j] == __shfl_sync(0xFFFFFFFFu, k[j], 0));
      at[j] = 0;
      if (k[j] >= 0 && (!one || lane == 0)) at[j] = atomicAdd(&counts[k[j]], one ? 32 : 1);
      if (one) at[j] = __shfl_sync(0xFFFFFFFFu, at[j], 0) + lane;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (k[j] >= 0) order[at[j]] = i0 + j * kSortThreads;
  }
}

// Tokens of a sorted tile: 32 while there are few of them or the rank is past 32 (the sums of 64 do not fit beside its h), else 64 (A and B
// are read half as often, for fewer and larger shares of work). 2560 -> 3840, 16 adapters, rank 16: 1500 tokens 18.1 us with 32 and 19.2 with 64, 2000 tokens 18.7 and 19.5. 5120 -> 7168, 8191 tokens
// of 12 adapters: rank 16 83 and 77, rank 32 84 and 80.
constexpr int64_t kMidTokens = 2048;
// Which calls go to the form on tcgen05: ranks past 32, in layers of some size (three launches show: 512 -> 512, 2000 tokens of rank 128 16.8 us
// warp-level, 22.6 on tcgen05; at 8000 tokens as long), and where its tiles of 128 tokens are not nearly empty, since each has A and B
// read and multiplied in full. Warp-level against tcgen05, 5120 -> 7168, bfloat16, replayed:
//   rank 40: 1000 tokens of 12 adapters 28.2 against 31.6; 1300 of 12 39.4 against 34.5; 1500 of 23 39.7 against 41.4; 4000 of 62 106 against 86, of
//     120 113 against 111 (float16 100 against 106); 8000 of 3 117 against 83, of 400 175 against 304
//   rank 72 (one CTA on an SM warp-level): 300 tokens of 3 30.1 against 26.7; 1000 of 40 72 against 59; 1100 of 120 104 against 124; 3000 of 120
//     115 against 132; 4000 of 120 216 against 134; 8000 of 3 221 against 94
// and for ranks to 32: 4000 tokens of rank 32 49.6 against 54.9, 8191 82.2 against 79.6; 2560 -> 3840 4000 tokens 33.5 against 36.9, 16000 tokens 87.6 against 86.3.
constexpr int kMidRank = 32, kWideRank = 64;
constexpr int64_t kLongLayer = 4096, kLongTokens = 1280, kWideTokens = 640, kWideAdapters = 48;
bool may_be_long(int64_t tokens, int rank, int64_t adapters) {
  if (rank <= kMidRank) return false;
  if (rank <= kWideRank) return tokens > kLongTokens && tokens >= 64 * adapters;
  return tokens > kFewTokens && (tokens >= 32 * adapters || (adapters <= kWideAdapters && (tokens > kWideTokens || tokens >= 24 * adapters)));
}
bool is_long(const LoraArgs &a) { return a.K + a.N >= kLongLayer && may_be_long(a.tokens, a.rank, a.adapters); }
bool can_count(int64_t tokens, int64_t adapters) { return tokens <= kCountTokens && adapters <= kCountAdapters; }
int sorted_tile(int64_t tokens, int rank) { return tokens <= kMidTokens || rank > kMidRank ? 32 : 64; }
int64_t most_tiles(int64_t tokens, int64_t adapters, int rank) { return tokens / sorted_tile(tokens, rank) + std::min<int64_t>(tokens, adapters + 1); }

template <class DT, class S, int TILING>
cudaError_t go(Params p, int64_t tiles, int64_t most, const DeviceInfo &dev, cudaStream_t stream) {
  constexpr int kDevices = 64;
  auto kernel = lora_kernel<DT, S, TILING>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  constexpr int kSmem = S::kRing + S::kFrag * S::template kPasses<kParts<DT>>;
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // Clusters of 1, 2, 4 and 8 CTAs that are resident at once (asked for once a device, with the shared memory past 48 KB): fewer
  // than the SMs' CTAs divided by the size, since a cluster stays within a group of SMs (36 of eight at two CTAs on each of 152 SMs)
  static std::atomic<int> resident[kDevices][4];
  int room[4];
  const bool kept = dev.device < kDevices;
  for (int i = 0; i < 4; ++i) room[i] = kept ? resident[dev.device][i].load(std::memory_order_acquire) : 0;
  if (room[0] == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    for (int i = 3; i >= 0 && e == cudaSuccess; --i) {  // (the first entry, which says that all are there, last)
      attr[0].val.clusterDim.x = 1u << i;
      cfg.gridDim = dim3(8, 1, 1);
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&room[i], kernel, &cfg);
      if (e == cudaSuccess && room[i] < 1) e = cudaErrorInvalidConfiguration;
      if (e == cudaSuccess && kept) resident[dev.device][i].store(room[i], std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
  }
  // CTAs of a tile: up to eight, while all tiles are resident together and the split pays for the cluster's barriers and sums. With 1, 2, 4 and
  // 8 CTAs, us: 48 tokens of rank 16, K + N = 512 3.9, 4.8, 5.0, 6.0; 2048 5.8, 5.3, 5.0, 6.0; 4096 8.4, 6.8, 5.8, 6.2; 7680 17.8, 11.5, 8.2, 8.4;
  // 300 of rank 32: 512 5.8, 7.2, 7.5, 9.4; 2048 12.0, 9.4, 7.7, 9.6; 5632 21.4, 14.3, 10.9, 12.1; 12288 48.6, 28.8, 18.1, 16.8.
  // 6 tokens of as many adapters, K + N = 6400: rank 16 11.6, 8.4, 6.2, 5.1; rank 64 16.6, 11.6, 8.2, 6.5. One tile alone, 1 token of rank 16: 512
  // 3.3, 4.1, 4.1, 4.3; 4096 7.7, 6.2, 4.8, 4.4. Ranks past 64 do about twice as much in a step: 6 tokens of rank 128, 512 4.8, 5.9, 6.2, 6.3.
  const int64_t both = (p.K + p.N) * (S::RS > 1 ? 2 : 1);
  const int most_c = both < 1536 ? 0 : tiles > 2 && both < (tiles > 12 ? 7168 : 5120) ? 2 : 3;
  int c = 0;
  while (c < most_c && tiles <= room[c + 1]) ++c;
  p.csize = 1 << c;
  attr[0].val.clusterDim.x = 1u << c;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(most, room[c]) << c), 1, 1);
  if (c > 0) cfg.numAttrs = 2;
  else cfg.attrs = attr + 1, cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <class DT>
cudaError_t run(const Params &p, bool few, int64_t tiles, int64_t most, const DeviceInfo &dev, cudaStream_t stream) {
  const int r = p.rank;
  if (few) {
    if (r <= 16) return go<DT, Shape<1, 1, 1, 3, 3>, kRanked>(p, tiles, most, dev, stream);
    if (r <= 32) return go<DT, Shape<2, 1, 1, 3, 3>, kRanked>(p, tiles, most, dev, stream);
    if (r <= 64) return go<DT, Shape<4, 1, 1, 2, 2>, kRanked>(p, tiles, most, dev, stream);
    return go<DT, Shape<4, 1, 2, 2, 1>, kRanked>(p, tiles, most, dev, stream);
  }
  if (!p.tiles) {
    if (r <= 16) return go<DT, Shape<1, 4, 1, 3, 2>, kCounted>(p, tiles, most, dev, stream);
    if (r <= 32) return go<DT, Shape<2, 4, 1, 3, 2>, kCounted>(p, tiles, most, dev, stream);
    if (r <= 64) return go<DT, Shape<4, 4, 1, 2, 2>, kCounted>(p, tiles, most, dev, stream);
    return go<DT, Shape<4, 4, 2, 2, 1>, kCounted>(p, tiles, most, dev, stream);
  }
  if (p.tokens <= kMidTokens || r > kMidRank) {
    if (r <= 16) return go<DT, Shape<1, 4, 1, 3, 2>, kListed>(p, tiles, most, dev, stream);
    if (r <= 32) return go<DT, Shape<2, 4, 1, 3, 2>, kListed>(p, tiles, most, dev, stream);
    if (r <= 64) return go<DT, Shape<4, 4, 1, 2, 2>, kListed>(p, tiles, most, dev, stream);
    return go<DT, Shape<4, 4, 2, 2, 1>, kListed>(p, tiles, most, dev, stream);
  }
  if (r <= 16) return go<DT, Shape<1, 8, 1, 2, 2>, kListed>(p, tiles, most, dev, stream);
  return go<DT, Shape<2, 8, 1, 2, 2>, kListed>(p, tiles, most, dev, stream);
}

}  // namespace

// The workspace past the first 4 KiB (the counters of other calls): the number of tiles, the sorted tokens, the tiles, h
static size_t tiles_at(int64_t tokens) { return 256 + static_cast<size_t>((tokens * 4 + 255) / 256 * 256); }
static size_t h_at(int64_t tokens, int64_t adapters, int rank) {
  return tiles_at(tokens) + (static_cast<size_t>(most_tiles(tokens, adapters, rank)) * sizeof(Tile) + 255) / 256 * 256;
}
size_t lora_workspace_bytes(int64_t tokens, int rank, int64_t adapters) {
  const bool maybe = may_be_long(tokens, rank, adapters);
  if (tokens <= kFewTokens || (can_count(tokens, adapters) && !maybe)) return 0;
  return 4096 + h_at(tokens, adapters, rank) + (maybe ? long_workspace_bytes(tokens, rank) : 0);
}
int lora_most_adapters() { return kMaxAdapters; }

cudaError_t launch_lora(const LoraArgs &a, const DeviceInfo &dev) {
  Params p{};
  p.x = static_cast<const uint16_t *>(a.x);
  p.a = static_cast<const uint16_t *>(a.a);
  p.b = static_cast<const uint16_t *>(a.b);
  p.base = static_cast<const uint16_t *>(a.base);
  p.out = static_cast<uint16_t *>(a.out);
  p.ids = a.ids;
  p.scales = a.scales;
  p.x_stride = a.x_stride;
  p.base_stride = a.base_stride;
  p.out_stride = a.out_stride;
  p.tokens = a.tokens;
  p.K = a.K;
  p.N = a.N;
  p.rank = a.rank;
  p.adapters = static_cast<int>(a.adapters);
  p.copy = a.base != a.out;
  const bool few = a.tokens <= kFewTokens, long_form = !few && is_long(a);
  // tiles, as far as can be told here, and at most
  int64_t tiles = std::min<int64_t>(a.tokens, a.tokens / kFewTile + a.adapters), most = a.tokens;
  if (!few) {
    tiles = (a.tokens + sorted_tile(a.tokens, a.rank) - 1) / sorted_tile(a.tokens, a.rank) + std::min<int64_t>(a.adapters, a.tokens / 2) / 2;
    most = most_tiles(a.tokens, a.adapters, a.rank);
  }
  if (!few && (long_form || !can_count(a.tokens, a.adapters))) {
    uint8_t *ws = static_cast<uint8_t *>(a.workspace) + 4096;
    int32_t *num = reinterpret_cast<int32_t *>(ws);
    p.order = reinterpret_cast<int32_t *>(ws + 256);
    Tile *list = reinterpret_cast<Tile *>(ws + tiles_at(a.tokens));
    p.num_tiles = num;
    p.tiles = list;
    const int per = long_form ? kLongTile : sorted_tile(a.tokens, a.rank);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(kSortThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.adapters + 1) * 4;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, lora_sort_kernel, a.ids, static_cast<int>(a.tokens), p.adapters, per, p.copy, p.order, list, num);
    if (e != cudaSuccess) return e;
    note_launch();
    if (long_form) return launch_long(a, dev, p.order, list, num, reinterpret_cast<float *>(ws + h_at(a.tokens, a.adapters, a.rank)));
  }
  return a.dtype == W4A16_BF16 ? run<BF16>(p, few, tiles, most, dev, a.stream) : run<F16>(p, few, tiles, most, dev, a.stream);
}

}  // namespace w4a16
