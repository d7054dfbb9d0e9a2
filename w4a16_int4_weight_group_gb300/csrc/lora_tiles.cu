// Low-rank adapters of many tokens: both products on tcgen05, for sorted tiles of 128 tokens of one adapter.
//
//     h = x A^T,   out = base + s h B^T
//
// Two kernels. The first multiplies 128 gathered rows of x by A, 64 elements of K a step, K split over the CTAs of a cluster where the tiles
// do not fill the device; their fp32 sums are added through distributed shared memory, in order, and go to a workspace (r numbers a
// token). The second multiplies them by s, puts h as a sum of numbers of the dtype (three for bfloat16, which hold all of its bits, two for float16: scaled by a
// power of two a token) into tensor memory, and multiplies it by columns of B, all parts' products into the
// same accumulators; each thread adds a row of base to a row of these, and the rows go out in pieces of 128 bytes and more.
//
// All copies are asynchronous 16-byte ones (rows are gathered, so there is no box to describe) into the 128-byte swizzle, a stage
// or more ahead of the MMAs that one thread issues; waits for MMAs are bounded, and the threads of a CTA vote before each
// barrier, so that all give up together.
//
// Taken instead of the warp-level form where that is bound by mma.sync: for many tokens of ranks past 32 (its second product takes two for
// each, and one m16n8k16 takes about 16 cycles on a quarter of an SM), a good part of a tile for each adapter. Bound by what the SMs read and write through L2: base, out, and B
// once a tile, 6.2 to 6.5 TB/s in the second kernel. Measured: 8191 tokens 5120 -> 7168 of 12 adapters, rank 64 23 + 53 us and 7 for the sort (90 a
// call out of L2), rank 128 26 + 69 (109). Replayed, bfloat16's three parts
// and, at rank 128, one accumulator against float16's two of each: rank 64 85 and 82 us, rank 128 103 and 97.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "lora_common.cuh"

namespace w4a16 {
namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;  // of a step of the second product
template <int RA>
constexpr int kSecondStages = RA == 1 ? 4 : 3;  // of 24 and 32 KB

struct Control {
  unsigned int error;
  unsigned int stall;  // no MMA is issued: the waits run out
  unsigned long long limit_ns;
};
__device__ Control g_lora_control = {0u, 0u, 2000000000ull};

struct Params {
  const uint4 *x, *a, *b, *base;
  uint4 *out;
  const float *scales;
  int64_t x_stride, base_stride, out_stride;  // in units of 16 bytes
  int64_t tokens;
  uint32_t k_units, n_units, r_units;  // of 8 elements
  int r16;                             // the rank, rounded up to 16
  int csize, per_split;                // CTAs of a tile in the first product, and blocks of 64 elements of K for each
  int slices;                          // of N
  bool copy;
  const int32_t *order;
  const Tile *tiles;
  const int32_t *num_tiles;
  float *h;  // [sorted token][r16]
  Control *control;
};

// ---- tcgen05 and its shared-memory operands (K-major, 128-byte swizzle, eight rows in 1024 bytes)
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// the same with A in tensor memory: a lane a row, two elements of k a column
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
               "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]),
        "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// start >> 4 in bits 0-13, leading byte offset >> 4 in 16-29, stride byte offset >> 4 in 32-45, the fixed 0b001 in 46-48, swizzle mode
// in 61-63 (2: 128 bytes)
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(16u >> 4) << 16) | (static_cast<uint64_t>(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
template <class DT>
__device__ __forceinline__ uint32_t idesc_of(int n) {  // D fp32, A and B of the dtype, both K-major, 128 x n
  constexpr uint32_t t = DT::kBF16 ? 1u : 0u;
  return (1u << 4) | (t << 7) | (t << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kLongTile >> 4) << 24);
}
// Byte offset of unit c (16 bytes) of a row in a tile of `rows` rows: pieces of 64 elements one after another, swizzled
__device__ __forceinline__ uint32_t place(int row, int c, int rows) {
  return static_cast<uint32_t>((c >> 3) * rows * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

// What a CTA's threads share, in front of its tiles
struct Shared {
  uint64_t stage_bar[4], done_bar, drain_bar;
  uint32_t tmem, abort;
  float back[2][kLongTile];  // of each half of a token's ranks: the largest; then what its h was divided by (float16)
};
constexpr int kShared = 2048;
static_assert(sizeof(Shared) <= kShared, "");

// The start and the end of both kernels: barriers and tensor memory
__device__ __forceinline__ void begin(Shared *sh, uint32_t cols) {
  if (threadIdx.x == 0) {
    for (uint64_t &b : sh->stage_bar) mbar_init(smem_u32(&b), 1);
    mbar_init(smem_u32(&sh->done_bar), 1);
    mbar_init(smem_u32(&sh->drain_bar), 1);
    sh->abort = 0;
    mbar_init_fence();
  }
  if (threadIdx.x < 32) tmem_alloc(smem_u32(&sh->tmem), cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}
__device__ __forceinline__ void finish(Shared *sh, uint32_t cols, bool ok, Control *control) {
  cp_async_wait<0>();
  if (!ok && threadIdx.x == 0) {  // MMAs that are still under way
    umma_commit(smem_u32(&sh->drain_bar));
    drain_phase(smem_u32(&sh->drain_bar), 0, &control->error);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x < 32) tmem_dealloc(sh->tmem, cols);
  griddep_launch_dependents();
}

// First product. RA: pieces of 64 of the rank
template <class DT, int RA>
__global__ void __launch_bounds__(kThreads, 2) long_first_kernel(const Params p) {
  constexpr int kX = kLongTile * 128, kA = RA * 64 * 128, kStage = kX + kA, S = RA == 1 ? 4 : 3;
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Shared *sh = reinterpret_cast<Shared *>(smem);
  const uint32_t stages = smem_u32(smem) + kShared;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  begin(sh, 128);
  const uint32_t tmem = sh->tmem, abort_flag = smem_u32(&sh->abort);
  const uint64_t limit = p.control->limit_ns;
  const bool stall = p.control->stall != 0;
  const int csize = p.csize, crank = csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int ntiles = *p.num_tiles;
  const int blocks = static_cast<int>((p.k_units + 7) / 8);
  const uint32_t idesc = idesc_of<DT>(p.r16);
  uint32_t t = 0, done = 0;  // blocks and items so far
  bool ok = true;
  // (a CTA that gave up a wait goes on without MMAs: the others of its cluster meet it at the barriers and read its shared memory)
  for (int tile = blockIdx.x / csize; tile < ntiles; tile += gridDim.x / csize) {
    const Tile d = p.tiles[tile];
    if (d.adapter < 0) continue;  // (the same for the cluster)
    const int b0 = crank * p.per_split, nb = ok ? max(min(b0 + p.per_split, blocks) - b0, 0) : 0;
    const uint4 *a = p.a + int64_t(d.adapter) * p.r_units * 8 * p.k_units;
    const int c = tid & 7;
    uint32_t xr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) xr[j] = static_cast<uint32_t>(p.order[d.first + min(j * 32 + (tid >> 3), d.count - 1)] * p.x_stride);
    auto fetch = [&](int i, uint32_t at) {  // block i of the item into the stage of the at-th block
      const uint32_t k = static_cast<uint32_t>(b0 + i) * 8 + c;
      const bool in = k < p.k_units;
      const uint32_t kk = in ? k : 0, to = stages + at % S * kStage;
#pragma unroll
      for (int j = 0; j < 4; ++j)  // rows past the tile's last are zeros (the last row again: a line that many ask for)
        cp_async_16(to + place(j * 32 + (tid >> 3), c, kLongTile), p.x + (xr[j] + kk), in && j * 32 + (tid >> 3) < d.count);
#pragma unroll
      for (int j = 0; j < 2 * RA; ++j) {  // rows past the rank are zeros
        const uint32_t row = j * 32 + (tid >> 3);
        const bool has = in && row < p.r_units * 8;
        cp_async_16(to + kX + row * 128 + ((c ^ (row & 7)) << 4), a + (has ? row * p.k_units + kk : 0), has);
      }
    };
    // the stage of the at-th block is free: its last MMAs are done
    auto freed = [&](uint32_t at) {
      return at < S || wait_phase(smem_u32(&sh->stage_bar[at % S]), (at / S - 1) & 1, abort_flag, limit, &p.control->error);
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i < nb && ok) ok = freed(t + i);
      if (i < nb && ok) fetch(i, t + i);
      cp_async_commit();
    }
    for (int i = 0; i < nb; ++i) {
      if (i + S - 1 < nb && ok) ok = freed(t + i + S - 1);
      if (i + S - 1 < nb && ok) fetch(i + S - 1, t + i + S - 1);
      cp_async_commit();
      cp_async_wait<S - 1>();
      fence_proxy_async_smem();
      ok = __syncthreads_and(ok);
      if (!ok) break;
      if (tid == 0 && !stall) {
        tc_fence_after();
        const uint32_t at = stages + (t + i) % S * kStage;
        const uint64_t xd = smem_desc(at), ad = smem_desc(at + kX);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma(tmem, xd + 2 * kk, ad + 2 * kk, idesc, i > 0 || kk > 0);
        umma_commit(smem_u32(&sh->stage_bar[(t + i) % S]));
        if (i == nb - 1) umma_commit(smem_u32(&sh->done_bar));
      }
    }
    if (ok && nb > 0) {
      t += nb;
      ok = wait_phase(smem_u32(&sh->done_bar), done & 1, abort_flag, limit, &p.control->error);
      ++done;
      ok = __syncthreads_and(ok);
    }
    tc_fence_after();
    // the sums of this CTA's part of K, in the ring's place, then an equal share of the tokens added over the cluster, in order
    const int stride = p.r16 + 4;
    float *sums = reinterpret_cast<float *>(smem + kShared);
    cp_async_wait<0>();
    __syncthreads();
    {
      const int row = (warp & 3) * 32 + lane;
      for (int c0 = (warp >> 2) * 16; c0 < p.r16; c0 += 32) {
        float v[16] = {};
        if (ok && nb > 0) {
          tmem_ld16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0, v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4 *>(sums + row * stride + c0 + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    }
    tc_fence_before();
    if (csize > 1) cluster_sync_all();
    else __syncthreads();
    const int quads = p.r16 / 4, rows = kLongTile / csize;
    for (int e = tid; e < rows * quads; e += kThreads) {
      const int row = crank * rows + e / quads, q = e % quads;
      const uint32_t mine = smem_u32(sums + row * stride + 4 * q);
      float4 o[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < csize) o[c] = csize > 1 ? ld_dsmem_v4(map_to_rank(mine, c)) : *reinterpret_cast<const float4 *>(sums + row * stride + 4 * q);
      float4 v = o[0];
#pragma unroll
      for (int c = 1; c < 8; ++c)
        if (c < csize) v.x += o[c].x, v.y += o[c].y, v.z += o[c].z, v.w += o[c].w;
      if (row < d.count) *reinterpret_cast<float4 *>(p.h + int64_t(d.first + row) * p.r16 + 4 * q) = v;
    }
    if (csize > 1) cluster_sync_all();
    else __syncthreads();
  }
  finish(sh, 128, ok, p.control);
}

// Second product, 64 columns a step: a ring of copies (base, whose place the results take, and B), two accumulators, so that copies and
// MMAs of the next steps run while this one's results are added and stored. h is in tensor memory, which leaves shared memory to the
// ring of two CTAs on an SM (h in shared memory, rank 128: one CTA with two stages of 128 columns 70 us, three of 64 93). Three parts of 128
// ranks leave room for one accumulator beside them: the next step's MMAs are issued once it has been read.
template <class DT, int RA>
__global__ void __launch_bounds__(kThreads, 2) long_second_kernel(const Params p) {
  constexpr int NC = kCols, S = kSecondStages<RA>, kHalf = 32 * RA;  // kHalf: columns of tensor memory of a part of h
  constexpr int kP = kParts<DT>, kAccs = kP * kHalf + 2 * NC <= 256 ? 2 : 1;
  static_assert(kP * kHalf + kAccs * NC <= 256, "two CTAs on an SM");
  constexpr int kB = RA * NC * 128, kBase = kLongTile * NC * 2, kRow = NC / 8;  // kRow: units of a row of base
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  Shared *sh = reinterpret_cast<Shared *>(smem);
  uint8_t *bs = smem + kShared, *os = bs + S * kB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  begin(sh, 256);
  const uint32_t ht = sh->tmem, tmem = ht + kP * kHalf, abort_flag = smem_u32(&sh->abort);
  const uint64_t limit = p.control->limit_ns;
  const bool stall = p.control->stall != 0;
  const int64_t items = int64_t(*p.num_tiles) * p.slices;
  const int chunks = static_cast<int>((p.n_units + kRow - 1) / kRow), per = (chunks + p.slices - 1) / p.slices;
  uint32_t g = 0;  // steps with products so far: their accumulators and barriers take turns
  bool ok = true;
  for (int64_t item = blockIdx.x; item < items && ok; item += gridDim.x) {
    const Tile d = p.tiles[item / p.slices];
    const int j0 = static_cast<int>(item % p.slices) * per, n = min(j0 + per, chunks) - j0;
    if (n <= 0 || (d.adapter < 0 && !p.copy)) continue;
    const uint4 *b = p.b + int64_t(max(d.adapter, 0)) * p.n_units * 8 * p.r_units;
    const int32_t *tok = p.order + d.first;
    const int c = tid % kRow;  // this thread's unit of the rows that it copies
    constexpr int kRows = kLongTile * kRow / kThreads, kStep = kThreads / kRow;
    int my[kRows];  // their tokens, -1 past the tile's last
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int row = j * kStep + tid / kRow;
      my[j] = row < d.count ? tok[row] : -1;
    }
    auto fetch = [&](int i) {
      const uint32_t n0 = static_cast<uint32_t>(j0 + i) * kRow;
      const uint32_t to = smem_u32(os) + i % S * kBase, bt = smem_u32(bs) + i % S * kB;
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (my[j] >= 0 && n0 + c < p.n_units) cp_async_16(to + place(j * kStep + tid / kRow, c, kLongTile), p.base + (my[j] * p.base_stride + n0 + c), true);
      if (d.adapter >= 0) {
        const uint32_t cols = (p.n_units - n0) * 8;
#pragma unroll
        for (int j = 0; j < NC * RA * 8 / kThreads; ++j) {  // columns and ranks past the ends are zeros
          const uint32_t u = j * kThreads + tid, col = u / (RA * 8), cu = u % (RA * 8);
          const bool in = col < cols && cu < p.r_units;
          cp_async_16(bt + place(col, cu, NC), b + (in ? uint64_t(n0 * 8 + col) * p.r_units + cu : 0), in);
        }
      }
    };
    // step i's MMAs, by one thread, once its copies have landed for all
    auto multiply = [&](int i) {
      cp_async_wait<S - 2>();
      fence_proxy_async_smem();
      __syncthreads();
      if (d.adapter < 0 || tid != 0 || stall) return;
      tc_fence_after();
      const uint64_t bd = smem_desc(smem_u32(bs) + i % S * kB);
      const uint32_t idesc = idesc_of<DT>(NC), to = tmem + (g + i) % kAccs * NC;
      for (int kk = 0; kk < p.r16 / 16; ++kk) {
        const uint64_t bo = ((kk >> 2) * NC * 128 + (kk & 3) * 32) >> 4;
#pragma unroll
        for (int q = kP - 1; q >= 0; --q) umma_ts(to, ht + q * kHalf + 8 * kk, bd + bo, idesc, kk > 0 || q < kP - 1);  // the smallest part first
      }
      umma_commit(smem_u32(&sh->stage_bar[(g + i) % kAccs]));
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i < n) fetch(i);
      cp_async_commit();
    }
    if (d.adapter >= 0) {
      // h, times s: half of a token's ranks a thread
      const int row = (warp & 3) * 32 + lane, half = warp >> 2;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const float s = p.scales ? p.scales[d.adapter] : 1.f;
      float v[kHalf];
#pragma unroll
      for (int e = 0; e < kHalf; ++e) v[e] = 0.f;
      if (row < d.count) {
        const float *from = p.h + int64_t(d.first + row) * p.r16 + half * kHalf;
#pragma unroll
        for (int e = 0; e < kHalf; e += 4)
          if (half * kHalf + e < p.r16) {
            const float4 q = *reinterpret_cast<const float4 *>(from + e);
            v[e] = q.x, v[e + 1] = q.y, v[e + 2] = q.z, v[e + 3] = q.w;
          }
      }
      float f = s;
      if constexpr (!DT::kBF16) {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < kHalf; ++e) top = fmaxf(top, fabsf(v[e] * s));  // (a NaN does not count)
        sh->back[half][row] = top;
        __syncthreads();
        const float unit = unit_of_largest(fmaxf(sh->back[0][row], sh->back[1][row]));
        __syncthreads();
        if (half == 0) sh->back[0][row] = unit;
#pragma unroll
        for (int e = 0; e < kHalf; ++e) v[e] *= s;
        f = 1.f / unit;  // (exact: a power of two)
      }
#pragma unroll
      for (int e = 0; e < kHalf; ++e) v[e] *= f;
#pragma unroll
      for (int e0 = 0; e0 < kHalf; e0 += 32)
#pragma unroll
        for (int q = 0; q < kP; ++q) {
          uint32_t part[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) part[e] = take_part<DT>(v[e0 + 2 * e], v[e0 + 2 * e + 1]);
          tmem_st16(ht + q * kHalf + lanes + (half * kHalf + e0) / 2, part);
        }
      tmem_wait_st();
      tc_fence_before();
    }
    multiply(0);
    for (int i = 0; i < n; ++i) {
      if (i + S - 1 < n) fetch(i + S - 1);  // (where step i - 1 was: its results have been stored)
      cp_async_commit();
      if (i + 1 < n && (kAccs > 1 || d.adapter < 0)) multiply(i + 1);
      uint8_t *ot = os + i % S * kBase;
      if (d.adapter >= 0) {
        ok = wait_phase(smem_u32(&sh->stage_bar[(g + i) % kAccs]), (g + i) / kAccs & 1, abort_flag, limit, &p.control->error);
        ok = __syncthreads_and(ok);
        if (!ok) break;
        tc_fence_after();
        // a thread's row, half of its columns
        const int row = (warp & 3) * 32 + lane;
        float f = 1.f;
        if constexpr (!DT::kBF16) f = sh->back[0][row];
        const uint32_t from = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (g + i) % kAccs * NC + (warp >> 2) * (NC / 2);
        float v[NC / 32][16];
        if constexpr (kAccs == 1) {
#pragma unroll
          for (int k = 0; k < NC / 32; ++k) tmem_ld16(from + 16 * k, v[k]);
          tmem_wait_ld();
          tc_fence_before();
          if (i + 1 < n) multiply(i + 1);
        }
#pragma unroll
        for (int k = 0; k < NC / 32; ++k) {
          if constexpr (kAccs > 1) {
            tmem_ld16(from + 16 * k, v[k]);
            tmem_wait_ld();
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint4 *at = reinterpret_cast<uint4 *>(ot + place(row, (warp >> 2) * (NC / 16) + 2 * k + u, kLongTile));
            uint4 w = *at;
            add2<DT>(w.x, v[k][8 * u], v[k][8 * u + 1], f), add2<DT>(w.y, v[k][8 * u + 2], v[k][8 * u + 3], f);
            add2<DT>(w.z, v[k][8 * u + 4], v[k][8 * u + 5], f), add2<DT>(w.w, v[k][8 * u + 6], v[k][8 * u + 7], f);
            *at = w;
          }
        }
        tc_fence_before();
        __syncthreads();
      }
      const uint32_t n0 = static_cast<uint32_t>(j0 + i) * kRow;
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (my[j] >= 0 && n0 + c < p.n_units)
          __stcs(p.out + (my[j] * p.out_stride + n0 + c), *reinterpret_cast<const uint4 *>(ot + place(j * kStep + tid / kRow, c, kLongTile)));
      __syncthreads();  // the stage may be filled again
    }
    if (d.adapter >= 0) g += n;
  }
  finish(sh, 256, ok, p.control);
}

// Every adapter may leave a tile that is not full: more than it turns out to be rather than less, which costs a second wave
int64_t tiles_about(int64_t tokens, int64_t adapters) { return tokens / kLongTile + std::min<int64_t>(adapters, tokens / 4) + 1; }
int rounded(int rank) { return (rank + 15) / 16 * 16; }

template <class K>
cudaError_t prepare(K kernel, int smem, int device, std::atomic<bool> (&asked)[64]) {
  if (device < 64 && asked[device].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && device < 64) asked[device].store(true, std::memory_order_release);
  return e;
}

template <class DT, int RA>
cudaError_t go(Params p, int64_t about, const DeviceInfo &dev, cudaStream_t stream) {
  constexpr int kFirst = kShared + 1024 + (RA == 1 ? 4 : 3) * (kLongTile * 128 + RA * 64 * 128);
  constexpr int kSecond = kShared + 1024 + kSecondStages<RA> * (RA * kCols * 128 + kLongTile * kCols * 2);
  static std::atomic<bool> asked_first[64], asked_second[64];
  cudaError_t e = prepare(long_first_kernel<DT, RA>, kFirst, dev.device, asked_first);
  if (e == cudaSuccess) e = prepare(long_second_kernel<DT, RA>, kSecond, dev.device, asked_second);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.csize);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.csize > 1 ? 2 : 1;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(about * p.csize, 2 * dev.num_sms / p.csize * p.csize)), 1, 1);
  cfg.dynamicSmemBytes = kFirst;
  e = cudaLaunchKernelEx(&cfg, long_first_kernel<DT, RA>, p);
  if (e != cudaSuccess) return e;
  note_launch();
  // slices of N: the number whose last wave costs least, a slice's h counting as much as two of its steps
  const int resident = 2 * dev.num_sms;
  const int64_t chunks = (p.n_units + kCols / 8 - 1) / (kCols / 8);
  double best = 0;
  for (int64_t s = 1; s <= std::min<int64_t>(chunks, 32); ++s) {
    const double waves = static_cast<double>((about * s + resident - 1) / resident), cost = waves * (2.0 + static_cast<double>((chunks + s - 1) / s));
    if (s == 1 || cost < best) best = cost, p.slices = static_cast<int>(s);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(resident), 1, 1);
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = kSecond;
  e = cudaLaunchKernelEx(&cfg, long_second_kernel<DT, RA>, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t control_of(int device, Control **out) {
  static std::mutex mu;
  static Control *known[64] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 64 && known[device]) {
    *out = known[device];
    return cudaSuccess;
  }
  void *ptr = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&ptr, g_lora_control);
  if (e != cudaSuccess) return e;
  *out = static_cast<Control *>(ptr);
  if (device < 64) known[device] = *out;
  return cudaSuccess;
}

}  // namespace

size_t long_workspace_bytes(int64_t tokens, int rank) { return static_cast<size_t>(tokens) * rounded(rank) * 4; }

cudaError_t launch_long(const LoraArgs &a, const DeviceInfo &dev, const int32_t *order, const Tile *tiles, const int32_t *num_tiles, float *h) {
  Params p{};
  p.x = static_cast<const uint4 *>(a.x);
  p.a = static_cast<const uint4 *>(a.a);
  p.b = static_cast<const uint4 *>(a.b);
  p.base = static_cast<const uint4 *>(a.base);
  p.out = static_cast<uint4 *>(a.out);
  p.scales = a.scales;
  p.x_stride = a.x_stride / 8;
  p.base_stride = a.base_stride / 8;
  p.out_stride = a.out_stride / 8;
  p.tokens = a.tokens;
  p.k_units = static_cast<uint32_t>(a.K / 8);
  p.n_units = static_cast<uint32_t>(a.N / 8);
  p.r_units = static_cast<uint32_t>(a.rank / 8);
  p.r16 = rounded(a.rank);
  const int blocks = static_cast<int>((a.K + 63) / 64);
  // CTAs of a tile: while all are resident (a cluster stays within a group of SMs: of eight there are 36 at two CTAs on each of 152
  // SMs, not 38) and each keeps four blocks
  const int64_t about = tiles_about(a.tokens, a.adapters);
  p.csize = 1;
  while (p.csize < 8 && about * p.csize * 2 <= (p.csize == 4 ? 36 * dev.num_sms / 19 : 2 * dev.num_sms) && blocks / (p.csize * 2) >= 4) p.csize *= 2;
  p.per_split = (blocks + p.csize - 1) / p.csize;
  p.copy = a.base != a.out;
  p.order = order;
  p.tiles = tiles;
  p.num_tiles = num_tiles;
  p.h = h;
  const cudaError_t e = control_of(dev.device, &p.control);
  if (e != cudaSuccess) return e;
  if (a.dtype == W4A16_BF16)
    return a.rank <= 64 ? go<BF16, 1>(p, about, dev, a.stream) : go<BF16, 2>(p, about, dev, a.stream);
  return a.rank <= 64 ? go<F16, 1>(p, about, dev, a.stream) : go<F16, 2>(p, about, dev, a.stream);
}

}  // namespace lora

cudaError_t lora_take_device_error(uint32_t *err) {
  lora::Control c;
  cudaError_t e = cudaMemcpyFromSymbol(&c, lora::g_lora_control, sizeof(c));
  if (e != cudaSuccess) return e;
  *err = c.error;
  c.error = 0;
  return *err ? cudaMemcpyToSymbol(lora::g_lora_control, &c, sizeof(c)) : cudaSuccess;
}
cudaError_t lora_set_wait_limit_ns(uint64_t ns) {
  const unsigned long long v = ns ? ns : 2000000000ull;
  return cudaMemcpyToSymbol(lora::g_lora_control, &v, sizeof(v), offsetof(lora::Control, limit_ns));
}
cudaError_t lora_set_stall(bool on) {
  const unsigned int v = on ? 1u : 0u;
  return cudaMemcpyToSymbol(lora::g_lora_control, &v, sizeof(v), offsetof(lora::Control, stall));
}

}  // namespace w4a16
