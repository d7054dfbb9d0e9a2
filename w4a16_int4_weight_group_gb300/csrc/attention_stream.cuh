// Attention of a few query rows (up to 32 of one cache head) over the quantised paged cache: the kernel
// that streams the cache.
//
//     s_t = scale (q . k_t),  k_t = (u_t - z_t) s^k_t over the positions t that the query may see,
//     out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),   lse = m + log sum_t exp(s_t - m)
//
// Bound by the cache's bytes ((2 D bits / 8 + 8) a token and cache head) and, with 4-bit codes, nearly as
// much by the instructions that turn codes into operands. So:
//
//  * Work split. The units are (sequence, cache head, row tile, 64 to 256 tokens), in this order; every CTA of a
//    resident grid takes an equal, contiguous share of them, whatever the lengths are. A CTA that holds all of
//    a segment (sequence, head, row tile) writes its result; otherwise it leaves its sums in the workspace
//    and the last one to finish adds them in the order of the CTAs (so results do not depend on timing).
//  * Every warp streams its own tokens: a ring of bulk copies of whole tiles (16 tokens of one head are one
//    contiguous piece), issued by the warp itself, so no warp waits for another until its CTA's segment ends.
//  * Products (mma.sync m16n8k16, fp16 operands, fp32 sums) with the codes on the M side: S^T = K Q^T and
//    O^T = V^T P^T, so that 8 query rows fill the N side and the codes' operands are reused for up to four
//    row groups. A lane's elements of the reduced (or output) dimension may be any, as long as Q (or the
//    output) uses the same order: each lane takes contiguous bytes of a token's row, so that codes come
//    by 4- to 16-byte loads without a transposition.
//  * Operands. A code u becomes the half 1024 + u by a byte permutation (8 bits) or one LOP3 (4 bits; the high
//    nibble of a byte gives 1024 + 16 u, and 1/16 is folded into Q or taken out of the result); one exact
//    subtraction of 1024 + z leaves u - z. So the products are of exact integers; the key's scale multiplies
//    the fp32 score, the value's scale goes into the probability.
//  * Ranges. A query row is scaled by a power of two to a largest element near 2^12. The probabilities times
//    the values' scales are kept relative to a running power of two sref above every scale seen, times 2^12:
//    fp16 holds them with 11 bits down to 2^-26 of the largest. A step that has smaller ones (a value's code
//    may be its zero point at every larger one) takes them in further products of 28 powers of two each, so
//    that every probability counts with 11 bits over the range of fp32.
//  * The running maximum is raised only when a score exceeds it by more than 3 (in powers of two), so most
//    steps need neither the reduction across lanes nor the rescaling of the sums.
//
// Measured (HBM: share of the device's 6782 GB/s copy rate):
//  * 131073 tokens of 8 heads of 128 elements, 8 bits, 5 rows a head: 64 to 71 us = 4.1 TB/s, 0.60 of it. Each further
//    131072 tokens take 45 us (0.90): about 15 us are the call's start, first loads and the joining of the parts.
//  * 48 sequences of up to 6001 tokens, 4 bits: 75 to 82 us = 2.1 TB/s (0.31). A 4-bit code costs the instructions of an
//    8-bit one for half of the bytes; the schedulers issue in half of the cycles.
//  * 12 sequences of up to 8200 tokens, heads of 256 elements, 8 bits, 13 drafted tokens: 77 us. 26 rows are two row
//    tiles, so every code is decoded twice, by eight warps on an SM (255 registers a thread).
//  * 517 tokens of one sequence: 12 to 15 us a call; 10.3 replayed from a graph, for 0.36 MB: fixed time (the search for
//    the share, the first copies and the joining of the parts, one after the other), not bytes.
//  * One token over 131073 tokens of 64 elements at 8 bits 55 us, of 128 at 4 bits 70 us, over 65537 of 256 elements 71 (8 bits)
//    and 68 us (4 bits).
// Registers: all but the 8-row layouts for 256 elements spill (bytes stored and loaded a thread): 8 rows of 128 elements at 4 bits
// 316 and 368 (128 registers), of 64 and of 128 at 8 bits 40 to 124 and 56 to 160; 16 rows 24 to 120 and 24 to 168; 32 rows of
// 64 elements 180 and 244, of 128 64 to 72 and 100 to 116.
#pragma once

#include "attention.h"
#include "attention_common.cuh"
#include "common.cuh"

namespace w4a16 {
namespace attention {

template <int D_, int BITS_, int NT_, bool BF_>
struct StreamLayout {
  static constexpr int D = D_, BITS = BITS_, NT = NT_;
  static constexpr bool BF = BF_;
  static constexpr int R = 8 * NT;              // query rows of a row tile
  static constexpr int RB = D * BITS / 8;       // bytes of a token's codes
  static constexpr int kTile = 16 * (2 * RB + 8);
  static constexpr int TPS = kTile <= 2176 && NT == 1 ? 2 : 1;  // tiles of a warp's step
  static constexpr int W = D == 256 ? 4 : NT * D == 256 ? 12 : 8;  // warps
  static constexpr int kThreads = 32 * W;
  static constexpr int kStage = TPS * kTile;
  static constexpr int kUnit = W * TPS * 16;    // tokens of a unit
  static constexpr int MB = W / 2;              // sums kept in shared memory when the warps join
  static constexpr int kPad = D + 4;            // floats of a row of them
  static constexpr bool kQSmem = NT * D >= 256; // Q's operands stay in shared memory, not in registers
  static constexpr int kCtas = NT * D >= 256 && D < 256 ? 1 : 2;  // on an SM (one: 168 or 255 registers a thread, not 128)
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kFixed = kQBytes + MB * R * kPad * 4 + R * (8 + 4) + 2 * W * R * 4 + 768;
  static constexpr int kBudget = (kCtas == 2 ? 113 : 226) * 1024;
  static constexpr int kFit = (kBudget - kFixed) / (W * kStage);
  static constexpr int S = kFit > 4 ? 4 : kFit;  // stages of a warp's ring
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = kOffQ + kQBytes;
  static constexpr int kOffO = kOffRing + W * S * kStage;
  static constexpr int kOffMask = kOffO + MB * R * kPad * 4;  // uint64 a row
  static constexpr int kOffQs = kOffMask + R * 8;             // float a row: score unit
  static constexpr int kOffM = kOffQs + R * 4;                // [W][R] maxima, then denominators
  static constexpr int kOffBar = (kOffM + 2 * W * R * 4 + 7) / 8 * 8;
  static constexpr int kOffMisc = kOffBar + 8 * (W * S + 1);  // abort flag, start, scan, split segments to join
  static constexpr int kSmem = kOffMisc + 32 + 8 * W + sizeof(Pending);
  static_assert(S >= 2, "a ring of two stages at least");
  static_assert(kUnit <= 256, "positions past the longest sequence's end");
  static_assert(kSmem <= kBudget, "shared memory");
  static_assert(MB * R * kPad >= kThreads + 64 * R, "scratch of the joining of parts");
  static_assert(kOffRing % 128 == 0 && kOffO % 16 == 0 && kTile % 128 == 0, "alignment");
};

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {  // 8 x 8 matrix of 16-bit elements
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// N 32-bit words from shared memory
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) w[0] = lds32(addr);
  else if constexpr (N == 2) lds64(addr, w[0], w[1]);
  else {
#pragma unroll
    for (int i = 0; i < N; i += 4) lds128(addr + 4 * i, w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}
// Adds up `v` over the lanes that share lane % 4.
__device__ __forceinline__ float sum_over_tokens(float v) {
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 16);
}
__device__ __forceinline__ float max_over_tokens(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
}

// acc += A B, or acc += unit * (A B)
__device__ __forceinline__ void add_product(float (&acc)[4], const uint32_t (&a)[4], const uint32_t (&b)[2], bool straight, float unit) {
  if (straight) {
    mma_16816<false>(acc, a, b[0], b[1]);
  } else {
    float t[4];
    mma_16816_z<false>(t, a, b[0], b[1]);
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = fmaf(t[c], unit, acc[c]);
  }
}

template <class L>
__global__ void __launch_bounds__(L::kThreads, L::kCtas) stream_kernel(const Params p) {
  constexpr int D = L::D, BITS = L::BITS, NT = L::NT, R = L::R, RB = L::RB, W = L::W, S = L::S, TPS = L::TPS;
  constexpr int KS = D / 16;       // k steps of the scores, and 16-row tiles of the values' product
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, r = lane & 3;

  uint64_t *mask_s = reinterpret_cast<uint64_t *>(smem + L::kOffMask);
  float *qs_s = reinterpret_cast<float *>(smem + L::kOffQs);
  float *m_s = reinterpret_cast<float *>(smem + L::kOffM);
  float *l_s = m_s + W * R;
  float *o_s = reinterpret_cast<float *>(smem + L::kOffO);
  const uint32_t bars = base + L::kOffBar + 8u * S * warp;  // this warp's ring
  const uint32_t stall_bar = base + L::kOffBar + 8u * S * W;
  const uint32_t abort_flag = base + L::kOffMisc;
  Pending *pending = reinterpret_cast<Pending *>(smem + L::kOffMisc + 32 + 8 * W);
  volatile int64_t *share_s = reinterpret_cast<volatile int64_t *>(smem + L::kOffMisc + 8);
  int64_t *scan_s = reinterpret_cast<int64_t *>(smem + L::kOffMisc + 32);
  const uint32_t ring = base + L::kOffRing + static_cast<uint32_t>(warp * S * L::kStage);

  if (lane == 0)
    for (int s = 0; s < S; ++s) mbar_init(bars + 8u * s, 1);
  if (tid == 0) {
    mbar_init(stall_bar, 1);
    st_flag(abort_flag, 0u);
    pending->count = 0;
  }
  mbar_init_fence();
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const uint64_t lim = p.control->limit_ns;
  const uint64_t limit_ns = lim ? lim : kDefaultWaitNs;
  unsigned int *error = &p.control->error;

  fill_unowned<D, L::kThreads>(p, tid);
  Cursor cur;
  Shares sh;
  int64_t u1, units;
  if (!share_of<L, W>(p, scan_s, share_s, cur, sh, u1, units)) return;  // nothing for this CTA
  const int64_t cta = blockIdx.x;

  // ---- the ring: copies are issued S steps ahead, across segments
  Cursor ahead = cur;
  int64_t to_issue = units;
  uint32_t valid = 0;   // TPS bits for each stage: tiles that are there
  uint32_t phases = 0;  // parity of each stage's next completion
  auto issue = [&](int s) {
    if (to_issue == 0) return;
    const int tile0 = (ahead.blk * W + warp) * TPS;
    uint32_t v = 0;
    int64_t from[TPS];
#pragma unroll
    for (int j = 0; j < TPS; ++j) {
      const int tile = tile0 + j;
      from[j] = 0;
      if (tile * 16 < ahead.len) {
        const int page_i = p.page_shift >= 0 ? tile >> p.page_shift : tile / p.page_tiles;
        const int page = __ldg(p.page_table + ahead.b * p.max_pages + page_i);
        if (page >= 0 && page < p.num_pages) {
          v |= 1u << j;
          from[j] = ((int64_t(page) * p.kv_heads + ahead.h) * p.page_tiles + (tile - page_i * p.page_tiles)) * L::kTile;
        }
      }
    }
    if (v != 0 && lane == 0) {
      const uint32_t dst = ring + static_cast<uint32_t>(s * L::kStage);
      mbar_arrive_expect_tx(bars + 8u * s, static_cast<uint32_t>(__popc(v)) * L::kTile);
      if (TPS == 2 && v == 3 && from[TPS - 1] == from[0] + L::kTile) {
        bulk_load(dst, p.cache + from[0], 2 * L::kTile, bars + 8u * s);
      } else {
#pragma unroll
        for (int j = 0; j < TPS; ++j)
          if (v & (1u << j)) bulk_load(dst + j * L::kTile, p.cache + from[j], L::kTile, bars + 8u * s);
      }
    }
    valid |= v << (TPS * s);
    if (--to_issue > 0 && ++ahead.blk == ahead.nb) next_segment<L>(p, ahead);
  };
#pragma unroll
  for (int s = 0; s < S; ++s) issue(s);

  bool ok = true;
  if (p.control->stall) ok = __all_sync(0xFFFFFFFFu, wait_phase(stall_bar, 0, abort_flag, limit_ns, error));

  int stage = 0;
  uint32_t qreg[L::kQSmem ? 1 : KS * NT * 2];
  float o[KS][NT][4];
  float m[NT][2], l[NT][2], qs[NT][2];  // rows 8 nt + 2 r, + 1
  float sref = 0.f, isref = 0.f;

  while (units > 0) {
    // ---------------------------------------------------------------- segment: (sequence, head, row tile)
    const Cursor seg = cur;
    const Queries qu = queries_of(p, seg.b, seg.len);
    const int count = static_cast<int>(min(int64_t(seg.nb - seg.blk), units));
    const int rows = min(R, qu.n * p.group - seg.rt * R);  // of them in use
    const int plain = min(qu.first, seg.len);  // all rows see the tokens before this one
    // Q: a row scaled by a power of two, in the order of the operands (see the codes' order below)
    {
      constexpr int LN = D / 8;  // lanes of a row
      uint16_t *q_s = reinterpret_cast<uint16_t *>(smem + L::kOffQ);
      for (int row = tid / LN; row < R; row += L::kThreads / LN) {
        const int c = tid % LN;
        float x[8];
        load_query<8>(p, seg, qu, row, rows, R, c * 8, x);
        if (c == 0) mask_s[row] = row < rows ? mask_word(p, qu, (seg.rt * R + row) / p.group) : ~0ull;
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
        const uint32_t lanes = LN == 32 ? 0xFFFFFFFFu : ((1u << (LN & 31)) - 1u) << (lane / LN * LN);
#pragma unroll
        for (int s = LN / 2; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, s));
        float up, unit;
        query_unit(p, top, up, unit);
        if (c == 0) qs_s[row] = unit;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int d = c * 8 + j;
          int kk, reg, pos, rr;
          float f = up;
          if constexpr (BITS == 8) {
            rr = (d >> 4) & 3;
            kk = 4 * (d >> 6) + ((d >> 2) & 3);
            reg = (d >> 1) & 1;
            pos = d & 1;
          } else {
            constexpr int PL = D >= 128 ? 32 : 16;  // codes of a lane's load
            rr = (d / PL) & 3;
            kk = (d / (4 * PL)) * (PL / 4) + 2 * ((d % PL) >> 3) + ((d >> 1) & 1);
            reg = d & 1;
            pos = (d >> 2) & 1;
            if (reg) f *= 0.0625f;
          }
          q_s[(((kk * NT + (row >> 3)) * 32 + (row & 7) * 4 + rr) * 2 + reg) * 2 + pos] = __half_as_ushort(__float2half_rn(x[j] * f));
        }
      }
    }
    __syncthreads();
    if constexpr (!L::kQSmem) {
#pragma unroll
      for (int i = 0; i < KS * NT; ++i) lds64(base + L::kOffQ + (i * 32 + lane) * 8, qreg[2 * i], qreg[2 * i + 1]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[nt][x] = -INFINITY;
        l[nt][x] = 0.f;
        qs[nt][x] = qs_s[8 * nt + 2 * r + x];
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    }
    sref = isref = 0.f;

    for (int u = 0; u < count; ++u) {
      const uint32_t v = (valid >> (TPS * stage)) & ((1u << TPS) - 1u);
      if (v != 0 && ok) {
        ok = __all_sync(0xFFFFFFFFu, wait_phase(bars + 8u * stage, (phases >> stage) & 1u, abort_flag, limit_ns, error));
        if (ok) {
          phases ^= 1u << stage;
          valid ^= v << (TPS * stage);
        }
      }
      if (v != 0 && ok) {
        const uint32_t st = ring + static_cast<uint32_t>(stage * L::kStage);
        const int t0 = ((seg.blk + u) * W + warp) * (TPS * 16);
        const bool whole = v == (1u << TPS) - 1u && t0 + TPS * 16 <= plain;  // all rows see all tokens
        // ---- scores of the step's tokens: lane: tokens g, g + 8 of each tile, rows 2 r, 2 r + 1
        float y[TPS][NT][4];
        float sv[TPS][2];
#pragma unroll
        for (int j = 0; j < TPS; ++j) {
          const uint32_t tile = st + j * L::kTile;
          const uint32_t par = tile + 32 * RB;
          const uint32_t pk0 = lds32(par + 4 * g), pk1 = lds32(par + 4 * g + 32);
          const uint32_t pv0 = lds32(par + 64 + 4 * g), pv1 = lds32(par + 64 + 4 * g + 32);
          const bool there = (v >> j) & 1u;
          const bool in0 = whole || (there && t0 + 16 * j + g < seg.len), in1 = whole || (there && t0 + 16 * j + g + 8 < seg.len);
          const float sk0 = in0 ? bits_to_float(pk0 & 0xFFFFu, L::BF) : 0.f;
          const float sk1 = in1 ? bits_to_float(pk1 & 0xFFFFu, L::BF) : 0.f;
          sv[j][0] = in0 ? bits_to_float(pv0 & 0xFFFFu, L::BF) : 0.f;
          sv[j][1] = in1 ? bits_to_float(pv1 & 0xFFFFu, L::BF) : 0.f;
          const uint32_t z0 = pk0 >> 16, z1 = pk1 >> 16;
          const uint32_t lo0 = (0x6400u + z0) * 0x10001u, lo1 = (0x6400u + z1) * 0x10001u;
          constexpr int NA = NT == 1 ? 2 : 1;  // chains of products (one row group alone would wait for each product)
          float acc[NA][NT][4];
#pragma unroll
          for (int x = 0; x < NA * NT * 4; ++x) acc[x / (4 * NT)][x / 4 % NT][x % 4] = 0.f;
          auto step = [&](int kk, const uint32_t (&a)[4]) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t b0, b1;
              if constexpr (L::kQSmem) lds64(base + L::kOffQ + ((kk * NT + nt) * 32 + lane) * 8, b0, b1);
              else b0 = qreg[2 * (kk * NT + nt)], b1 = qreg[2 * (kk * NT + nt) + 1];
              mma_16816<false>(acc[kk % NA][nt], a, b0, b1);
            }
          };
          if constexpr (BITS == 8) {
            // word w of chunk i: elements 64 i + 16 r + 4 w ..: one k step
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
              uint32_t wa[4], wb[4];
              lds_words<4>(tile + g * RB + 64 * i + 16 * r, wa);
              lds_words<4>(tile + (g + 8) * RB + 64 * i + 16 * r, wb);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t a[4] = {hsub2(prmt(wa[w], 0x64646464u, 0x4140), lo0), hsub2(prmt(wb[w], 0x64646464u, 0x4140), lo1),
                                       hsub2(prmt(wa[w], 0x64646464u, 0x4342), lo0), hsub2(prmt(wb[w], 0x64646464u, 0x4342), lo1)};
                step(4 * i + w, a);
              }
            }
          } else {
            // word w: elements n0 .. n7 as (n0, n4), 16 (n1, n5), (n2, n6), 16 (n3, n7): two k steps
            const uint32_t hi0 = (0x6400u + 16u * z0) * 0x10001u, hi1 = (0x6400u + 16u * z1) * 0x10001u;
            constexpr int PB = D >= 128 ? 16 : 8;  // bytes of a lane's load
#pragma unroll
            for (int i = 0; i < RB / (4 * PB); ++i) {
              uint32_t wa[PB / 4], wb[PB / 4];
              lds_words<PB / 4>(tile + g * RB + 4 * PB * i + PB * r, wa);
              lds_words<PB / 4>(tile + (g + 8) * RB + 4 * PB * i + PB * r, wb);
#pragma unroll
              for (int w = 0; w < PB / 4; ++w) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const uint32_t xa = x ? wa[w] >> 8 : wa[w], xb = x ? wb[w] >> 8 : wb[w];
                  const uint32_t a[4] = {hsub2(and_or(xa, 0x000F000Fu, 0x64006400u), lo0), hsub2(and_or(xb, 0x000F000Fu, 0x64006400u), lo1),
                                         hsub2(and_or(xa, 0x00F000F0u, 0x64006400u), hi0), hsub2(and_or(xb, 0x00F000F0u, 0x64006400u), hi1)};
                  step((PB / 2) * i + 2 * w + x, a);
                }
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 4; ++c) y[j][nt][c] = (NA == 2 ? acc[0][nt][c] + acc[NA - 1][nt][c] : acc[0][nt][c]) * (c < 2 ? sk0 : sk1);
          }
        }
        // ---- what the rows do not see
        uint32_t hidden = 0;  // bit (j * NT + nt) * 4 + c
        if (!whole) {
#pragma unroll
          for (int j = 0; j < TPS; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int t = t0 + 16 * j + g + 8 * (c >> 1);
              const bool there = ((v >> j) & 1u) && t < seg.len;
              const int at = t - qu.first;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const bool see = there && (at < 0 || (at < 64 && ((mask_s[8 * nt + 2 * r + (c & 1)] >> at) & 1ull)));
                if (!see) {
                  y[j][nt][c] = -INFINITY;
                  hidden |= 1u << ((j * NT + nt) * 4 + c);
                }
              }
            }
        }
        // ---- running maximum and scale
        bool raise = false;
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float t = -INFINITY;
#pragma unroll
            for (int j = 0; j < TPS; ++j) t = fmaxf(t, fmaxf(y[j][nt][x], y[j][nt][2 + x]));
            top[nt][x] = t == -INFINITY ? t : t * qs[nt][x];
            raise |= top[nt][x] > m[nt][x] + kSlack || (m[nt][x] == -INFINITY && top[nt][x] > -INFINITY);
          }
#pragma unroll
        for (int j = 0; j < TPS; ++j) raise |= !(sv[j][0] <= sref) || !(sv[j][1] <= sref);
        if (__any_sync(0xFFFFFFFFu, raise)) {
          float big = 0.f;
#pragma unroll
          for (int j = 0; j < TPS; ++j) big = fmaxf(big, fmaxf(sv[j][0], sv[j][1]));
          big = max_over_tokens(big);
          float ratio = 1.f;
          if (big > sref) {
            // the power of two above it (at least 2^-100: times its reciprocal stays finite)
            const uint32_t e = max((__float_as_uint(big) >> 23) + 1u, 27u);
            const float next = __uint_as_float(e << 23);
            ratio = sref / next;
            sref = next;
            isref = 1.f / next;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float mn = fmaxf(m[nt][x], max_over_tokens(top[nt][x]));
              const float f = mn == -INFINITY ? 1.f : exp2_approx(m[nt][x] - mn);
              m[nt][x] = mn;
              l[nt][x] *= f;
#pragma unroll
              for (int i = 0; i < KS; ++i) {
                o[i][nt][x] *= f * ratio;
                o[i][nt][2 + x] *= f * ratio;
              }
            }
        }
        // ---- probabilities, times the values' scales, as operands (rows, tokens)
        float least = INFINITY;  // the smallest of them that is not hidden
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float ms0 = kProbExp - (m[nt][0] == -INFINITY ? 0.f : m[nt][0]), ms1 = kProbExp - (m[nt][1] == -INFINITY ? 0.f : m[nt][1]);
#pragma unroll
          for (int j = 0; j < TPS; ++j) {
            float e[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              e[c] = exp2_approx(fmaf(y[j][nt][c], qs[nt][c & 1], (c & 1) ? ms1 : ms0));
              y[j][nt][c] = e[c] * (sv[j][c >> 1] * isref);
            }
            if (whole) {
              least = fminf(fminf(least, fminf(y[j][nt][0], y[j][nt][1])), fminf(y[j][nt][2], y[j][nt][3]));
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                if (hidden & (1u << ((j * NT + nt) * 4 + c))) e[c] = y[j][nt][c] = 0.f;
                else least = fminf(least, y[j][nt][c]);
              }
            }
            l[nt][0] += e[0] + e[2];
            l[nt][1] += e[1] + e[3];
          }
        }
        // ---- sums over the tokens: lane: elements g D / 8 .. of the values, tokens 2 r, 2 r + 1, 2 r + 8, 2 r + 9
        // (unit: what the sums of this product are multiplied with; one: they go straight into o)
        auto product = [&](const uint32_t (&pb)[TPS][NT][2], const bool straight, const float unit) {
#pragma unroll
          for (int j = 0; j < TPS; ++j) {
            const uint32_t tile = st + j * L::kTile + 16 * RB;
            const uint32_t par = tile + 16 * RB + 64;
            uint32_t z[4];
            lds64(par + 8 * r, z[0], z[1]);
            lds64(par + 8 * r + 32, z[2], z[3]);
            // (a slot that nothing was written to may hold any bits: kept finite, its probability is zero)
            const uint32_t zl0 = 0x64006400u + (prmt(z[0], z[1], 0x7632) & 0x00FF00FFu);
            const uint32_t zl1 = 0x64006400u + (prmt(z[2], z[3], 0x7632) & 0x00FF00FFu);
            constexpr int LB = RB / 8;                    // bytes of a lane's piece of a row
            constexpr int WL = LB / 4 > 4 ? 4 : LB / 4;   // words loaded at a time
#pragma unroll
            for (int i = 0; i < LB / 4; i += WL) {
              uint32_t a0[WL], a1[WL], a2[WL], a3[WL];
              const uint32_t at = tile + g * LB + 4 * i;
              lds_words<WL>(at + (2 * r) * RB, a0);
              lds_words<WL>(at + (2 * r + 1) * RB, a1);
              lds_words<WL>(at + (2 * r + 8) * RB, a2);
              lds_words<WL>(at + (2 * r + 9) * RB, a3);
#pragma unroll
              for (int w = 0; w < WL; ++w) {
                if constexpr (BITS == 8) {
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const uint32_t s0 = prmt(a0[w], a1[w], x ? 0x7362 : 0x5140), s1 = prmt(a2[w], a3[w], x ? 0x7362 : 0x5140);
                    const uint32_t a[4] = {hsub2(prmt(s0, 0x64646464u, 0x4140), zl0), hsub2(prmt(s0, 0x64646464u, 0x4342), zl0),
                                           hsub2(prmt(s1, 0x64646464u, 0x4140), zl1), hsub2(prmt(s1, 0x64646464u, 0x4342), zl1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) add_product(o[2 * (i + w) + x][nt], a, pb[j][nt], straight, unit);
                  }
                } else {
                  const uint32_t zh0 = 0x64006400u + 16u * (zl0 - 0x64006400u), zh1 = 0x64006400u + 16u * (zl1 - 0x64006400u);
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const uint32_t s0 = prmt(a0[w], a1[w], x ? 0x7632 : 0x5410), s1 = prmt(a2[w], a3[w], x ? 0x7632 : 0x5410);
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                      const uint32_t t0w = k2 ? s0 >> 8 : s0, t1w = k2 ? s1 >> 8 : s1;
                      // even elements as they are, odd ones times 16 (taken out at the end)
                      const uint32_t a[4] = {hsub2(and_or(t0w, 0x000F000Fu, 0x64006400u), zl0), hsub2(and_or(t0w, 0x00F000F0u, 0x64006400u), zh0),
                                             hsub2(and_or(t1w, 0x000F000Fu, 0x64006400u), zl1), hsub2(and_or(t1w, 0x00F000F0u, 0x64006400u), zh1)};
#pragma unroll
                      for (int nt = 0; nt < NT; ++nt) add_product(o[4 * (i + w) + 2 * x + k2][nt], a, pb[j][nt], straight, unit);
                    }
                  }
                }
              }
            }
          }
        };
        uint32_t pb[TPS][NT][2];
        if (!__any_sync(0xFFFFFFFFu, least < kSmall)) {
#pragma unroll
          for (int j = 0; j < TPS; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              pb[j][nt][0] = transpose8(pack_half2(y[j][nt][0], y[j][nt][1]));
              pb[j][nt][1] = transpose8(pack_half2(y[j][nt][2], y[j][nt][3]));
            }
          product(pb, true, 1.f);
        } else {
          float up = 1.f, down = 1.f;
#pragma unroll 1
          for (int plane = 0; plane < kPlanes; ++plane, up *= kPlane, down *= 1.f / kPlane) {
            bool some = false;
#pragma unroll
            for (int j = 0; j < TPS; ++j)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float x[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  // taken in this plane: what is at least 2^-14 in its unit, in the last one what is left (and NaN in the first)
                  const bool now = !(y[j][nt][c] * up < kSmall) || plane == kPlanes - 1;
                  x[c] = now ? y[j][nt][c] * up : 0.f;
                  if (now) y[j][nt][c] = 0.f;
                  some |= !(x[c] == 0.f);
                }
                pb[j][nt][0] = transpose8(pack_half2(x[0], x[1]));
                pb[j][nt][1] = transpose8(pack_half2(x[2], x[3]));
              }
            if (__any_sync(0xFFFFFFFFu, some)) product(pb, false, down);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (ok) issue(stage);
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    units -= count;
    if (units > 0) next_segment<L>(p, cur);

    // ---------------------------------------------------------------- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float sum = sum_over_tokens(l[nt][x]) * (1.f / kProbUnit);
        if (g == 0) {
          m_s[warp * R + 8 * nt + 2 * r + x] = m[nt][x];
          l_s[warp * R + 8 * nt + 2 * r + x] = sum;
        }
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, m_s[w * R + 8 * nt + 2 * r + x]);
        const float f = (m[nt][x] == -INFINITY ? (l[nt][x] == 0.f ? 0.f : 1.f) : exp2_approx(m[nt][x] - top)) * (sref * (1.f / kProbUnit));
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          o[i][nt][x] *= f;
          o[i][nt][2 + x] *= BITS == 4 ? f * 0.0625f : f;
        }
      }
    // the upper half of the warps' sums through shared memory, then those of the lower half
    auto put = [&](int slot, bool add) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float *dst = o_s + (slot * R + 8 * nt + 2 * r + x) * L::kPad + g * (D / 8);
#pragma unroll
          for (int i = 0; i < KS; i += 2) {
            float4 *d4 = reinterpret_cast<float4 *>(dst + 2 * i);
            float4 val = make_float4(o[i][nt][x], o[i][nt][2 + x], o[i + 1][nt][x], o[i + 1][nt][2 + x]);
            if (add) {
              const float4 old = *d4;
              val = make_float4(val.x + old.x, val.y + old.y, val.z + old.z, val.w + old.w);
            }
            *d4 = val;
          }
        }
    };
    if (warp >= L::MB) put(warp - L::MB, false);
    __syncthreads();
    if (warp < L::MB) put(warp, true);
    __syncthreads();
    const bool given_up = ld_flag(abort_flag) != 0;
    if (given_up) ok = false;
    const bool is_first = seg.blk == 0, is_whole = is_first && count == seg.nb;
    if (!given_up) {
      // where the segment starts and ends in the list of units: the CTAs that hold parts of it
      const int64_t seg_u = u1 - units - count - seg.blk;  // only used when nothing is extended (flags given)
      float *slot = is_whole ? nullptr : p.partials + (2 * cta + (is_first ? 1 : 0)) * int64_t(R) * (D + 2);
      for (int i = tid; i < R * D / 4; i += L::kThreads) {
        const int row = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int b = 0; b < L::MB; ++b) {
          const float4 x = *reinterpret_cast<const float4 *>(o_s + (b * R + row) * L::kPad + d);
          v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
        }
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, m_s[w * R + row]);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float mw = m_s[w * R + row], lw = l_s[w * R + row];
          sum += mw == -INFINITY ? lw : lw * exp2_approx(mw - top);  // without a maximum: zero, or a NaN
        }
        if (is_whole) {
          if (row < rows) {
            const int gr = seg.rt * R + row, qi = gr / p.group;
            const int64_t at = (qu.q0 + qi) * p.q_heads + seg.h * p.group + (gr - qi * p.group);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            store_out4(p.out, L::BF, at * D + d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            if (p.lse && d == 0) p.lse[at] = sum == 0.f ? -INFINITY : (top == -INFINITY ? sum : (top + log2f(sum)) * kLn2);
          }
        } else {
          *reinterpret_cast<float4 *>(slot + row * D + d) = v;
          if (d == 0) {
            slot[R * D + row] = top;
            slot[R * (D + 1) + row] = sum;
          }
        }
      }
      if (!is_whole) count_in<0, L::kThreads>(p, sh, seg, qu, rows, R, seg_u, int64_t(R) * (D + 2), o_s, pending, tid);
    }
    __syncthreads();  // o_s, m_s, Q and the masks are free again
  }
  for (int i = 0; i < pending->count; ++i) join_parts<R, D, L::kThreads, 64, 0>(pending->parts[i], tid);
  if (ld_flag(abort_flag) != 0) {
    // let this warp's own copies land before the shared memory is released
    for (int s = 0; s < S; ++s)
      if ((valid >> (TPS * s)) & ((1u << TPS) - 1u)) drain_phase(bars + 8u * s, (phases >> s) & 1u, error);
  }
}

template <class L>
cudaError_t start_stream(const Params &p, int num_sms, cudaStream_t stream) {
  return start_kernel<L>(stream_kernel<L>, num_sms * L::kCtas, p, stream);
}

template <int D, int BITS>
cudaError_t launch_stream(const Params &p, int rows, int num_sms, cudaStream_t stream) {
  if (rows == 8)
    return p.bf16 ? start_stream<StreamLayout<D, BITS, 1, true>>(p, num_sms, stream) : start_stream<StreamLayout<D, BITS, 1, false>>(p, num_sms, stream);
  if constexpr (D != 256) {
    if (rows == 32)
      return p.bf16 ? start_stream<StreamLayout<D, BITS, 4, true>>(p, num_sms, stream) : start_stream<StreamLayout<D, BITS, 4, false>>(p, num_sms, stream);
  }
  return p.bf16 ? start_stream<StreamLayout<D, BITS, 2, true>>(p, num_sms, stream) : start_stream<StreamLayout<D, BITS, 2, false>>(p, num_sms, stream);
}

}  // namespace attention
}  // namespace w4a16
