// Attention of many query rows (more than 32 of one cache head) over the quantised paged cache: the kernel
// whose products run on the fifth-generation tensor cores.
//
// Bound by the two products (4 D flops a row and token), the exponentials (one a row and token, 16 a clock
// and SM) and the instructions that prepare operands. A CTA (one on an SM) holds 128 rows of a cache head and
// walks over tiles of 128 tokens:
//
//  * warps 0-7: two groups of four, softmax. Tiles alternate between the groups, each with its own running
//    maximum, denominator and sums, so that the tensor cores work on one group's tile while the other's is in
//    the softmax; the groups are joined at the end of a segment. A thread has one row: no reduction
//    across threads.
//  * warps 8-15: the codes, four warps for the keys and four for the values (on four warps for both 393 us
//    where this takes 356). Loaded straight into registers one tile ahead (16 contiguous bytes a thread and
//    load; the cache tiles are brought into L2 three tiles ahead), turned into exact integers u - z by a
//    byte permutation or LOP3 and a subtraction, and stored as the operands' 128-byte-swizzled tiles: K-major
//    keys (fp16), MN-major values (bf16); a token's elements stay together in both, so nothing is transposed.
//    Inside a group of 8, 4-bit elements are stored in the order 0 4 1 5 2 6 3 7; Q uses the same order and
//    the epilogue undoes it. They also leave the tokens' scales as floats.
//  * warp 16 (it allocates tensor memory too) and warp 17: one thread each issues the MMAs, S = Q K^T (M 128,
//    N 128) and O += P V, P read from tensor memory, where it overwrites S. (One thread for both spent as long
//    on its waits and commits between them as on the MMAs.)
//
// Keys' scales multiply the fp32 scores, values' scales the probabilities. A probability times its scale is the
// sum of two bf16 numbers (upper half of the fp32 number, then the rest rounded), two products for each tile:
// 16 significant bits over the range of fp32. One fp16 number has 11 bits, but over 29 powers of two only, and
// among the 16384 probabilities of a tile some nearly always lie further apart than that. The range also leaves
// room to raise the running maximum only when a score exceeds it by 8 powers of two: with 32 rows a warp a smaller
// slack has some row raise in nearly every tile (measured: 2600 of 5960 cycles a tile with fp16 and half a power).
// The work split over CTAs, the workspace and the bounded waits are those of the streaming kernel
// (attention_stream.cuh).
//
// Measured: 6 sequences of 20000 tokens, 64 drafted tokens, 8 heads of 128 elements at 4 bits, 320 rows a head (157
// GFLOP): 352 us = 446 TFLOP/s, 0.23 of the library's dense bf16 rate; about 4600 cycles for a tile of 128 rows x
// 128 tokens. A group's tile goes through QK (700 cycles), largest score (1000), exponentials (3500 to 4000) and PV
// (1390, two products). The softmax sets the pace: with the groups made to take turns in it, so that one tile's
// products lie under the other's softmax, a call takes 381 us, so one tile's maxima and exponentials alone take about
// as long as a tile in all, and not less on more warps: two threads a row (sixteen warps of 72 registers) took 356
// us, 370 in turns. P handed to its product in two or four pieces: 356. Parts left out for timing, with two
// threads a row: codes 337, exponentials 279, both 224, the maxima too 180. No counter is near its limit
// (schedulers 54 %, shared memory's pipe 39 % without the tensor cores' reads, tensor pipe 34 %).
// 24 more registers a softmax thread (setmaxnreg): 377 -> 356. At its 96 registers the kernel spills (bytes stored and
// loaded a thread) 356 and 384 for heads of 128 at 4 bits, 456 and 440 at 8; where it spills, and what that costs, was not measured.
#pragma once

#include "attention.h"
#include "attention_common.cuh"
#include "common.cuh"

namespace w4a16 {
namespace attention {

template <int D_, int BITS_>
struct TileLayout {
  static constexpr int D = D_, BITS = BITS_;
  static constexpr int R = 128;
  static constexpr int RB = D * BITS / 8;
  static constexpr int kTile = 16 * (2 * RB + 8);  // bytes of a cache tile
  static constexpr int kUnit = 128;                // tokens of a unit
  static constexpr int kSoftmaxWarps = 8, kCodeWarps = 4;  // (four for the keys, four for the values)
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 2 * kCodeWarps + 2);
  // Registers: the kernel is compiled to kRegs a thread; the codes' warp groups give some to the softmax's.
  static constexpr int kRegs = 96, kSoftmaxRegs = 120, kCodeRegs = 72;
  static_assert(2 * kSoftmaxRegs + 2 * kCodeRegs <= 4 * kRegs, "the shares must fit into what the launch holds");
  static constexpr int kLoads = RB / 16;           // 16-byte loads of a thread for a tile's keys
  static constexpr int kOperand = 128 * D * 2;     // bytes of Q, of a tile's keys, of its values
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOperand;
  static constexpr int kOffV = kOffK + 2 * kOperand;
  static constexpr int kParam = (2 * 128 + 4) * 4;  // key scales, value scales, tiles that are there
  static constexpr int kOffParam = kOffV + 2 * kOperand;
  static constexpr int kOffRow = kOffParam + 4 * kParam;  // [2][2][128] maxima and denominators of the groups
  static constexpr int kOffQs = kOffRow + 4 * 128 * 4;
  static constexpr int kOffBar = kOffQs + 128 * 4;
  static constexpr int kBars = 2 + 2 + 2 + 2 + 4 + 2 + 2 + 2 + 4;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kSmem = kOffMisc + 64 + kThreads / 4 + sizeof(Pending) + 1024;  // + slack to align the base to 1024 bytes
  static constexpr uint32_t kTmemCols = 512;  // S of the groups at 0 and 128, O at 256 and 384
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Two 32-bit words (fp32 numbers, say) in one 64-bit register pair
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
// D (tensor memory) += A (shared memory) B (shared memory); _first: D = A B
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a),
               "l"(b), "r"(idesc)
               : "memory");
}
__device__ __forceinline__ void umma_ss_first(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, 0, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a),
               "l"(b), "r"(idesc)
               : "memory");
}
// D (tensor memory) += A (tensor memory) B (shared memory); _first: D = A B
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a),
               "l"(b), "r"(idesc)
               : "memory");
}
__device__ __forceinline__ void umma_ts_first(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, 0, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a),
               "l"(b), "r"(idesc)
               : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&x)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
}
// Shared-memory matrix descriptor: start >> 4 in bits 0-13, leading byte offset >> 4 in 16-29, stride byte
// offset >> 4 in 32-45, the fixed 0b001 in 46-48, swizzle mode in 61-63 (2: 128 bytes).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Registers of a warp group's threads from here on (all its warps execute it).
template <int N>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// Barriers of some warps (all threads of each)
template <int ID, int THREADS>
__device__ __forceinline__ void bar_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}
// The same barrier with a vote: whether any of its threads says so, one answer for all of them.
template <int ID, int THREADS>
__device__ __forceinline__ bool bar_any(bool vote) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(vote)), "n"(ID), "n"(THREADS)
      : "memory");
  return any != 0;
}

// Eight 4-bit codes as fp16 integers u - z in the order 0 4, 1 5, 2 6, 3 7 (lo = 1024 + z, hi = 64 + z, twice).
__device__ __forceinline__ void decode4(uint32_t w, uint32_t lo, uint32_t hi, uint32_t (&x)[4]) {
  const uint32_t w8 = w >> 8;
  x[0] = hsub2(and_or(w, 0x000F000Fu, 0x64006400u), lo);
  x[1] = hsub2(and_or(w, 0x00F000F0u, 0x54005400u), hi);
  x[2] = hsub2(and_or(w8, 0x000F000Fu, 0x64006400u), lo);
  x[3] = hsub2(and_or(w8, 0x00F000F0u, 0x54005400u), hi);
}
// The same as bf16 integers (base = 128 + z, twice).
__device__ __forceinline__ void decode4_bf16(uint32_t w, uint32_t base, uint32_t (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = sub2_rn<true>(and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u), base);
}
// Eight 8-bit codes, in order.
__device__ __forceinline__ void decode8(uint32_t a, uint32_t b, uint32_t lo, uint32_t (&x)[4]) {
  x[0] = hsub2(prmt(a, 0x64646464u, 0x4140), lo);
  x[1] = hsub2(prmt(a, 0x64646464u, 0x4342), lo);
  x[2] = hsub2(prmt(b, 0x64646464u, 0x4140), lo);
  x[3] = hsub2(prmt(b, 0x64646464u, 0x4342), lo);
}
// The same as bf16 integers: with v = u - 128, v = (128 + low 7 bits) - (128 or, below zero, 256); zc = z - 128, twice.
__device__ __forceinline__ uint32_t decode8_bf16_pair(uint32_t bytes, uint32_t zc) {
  const uint32_t up = and_or(bytes, 0x007F007Fu, 0x43004300u);
  const uint32_t down = and_or(~bytes, 0x00800080u, 0x43004300u);
  return sub2_rn<true>(sub2_rn<true>(up, down), zc);
}
__device__ __forceinline__ void decode8_bf16(uint32_t a, uint32_t b, uint32_t zc, uint32_t (&x)[4]) {
  x[0] = decode8_bf16_pair(prmt(a, 0u, 0x4140), zc);
  x[1] = decode8_bf16_pair(prmt(a, 0u, 0x4342), zc);
  x[2] = decode8_bf16_pair(prmt(b, 0u, 0x4140), zc);
  x[3] = decode8_bf16_pair(prmt(b, 0u, 0x4342), zc);
}
constexpr float kTileSlack = 8.f;          // how far (powers of two) scores may exceed the running maximum
constexpr float kValueUnit = 1.f / 65536;  // values' scales times this: room for the slack and the sums

__device__ __forceinline__ void unpair(uint64_t x, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) {
  float a, b;
  unpair(x, a, b);
  return pair(__float_as_uint(exp2_approx(a)), __float_as_uint(exp2_approx(b)));
}

// Two fp32 numbers as the sums of two bf16 numbers each: their upper halves, and the rest rounded.
__device__ __forceinline__ void split_pair(uint64_t x, uint32_t &upper, uint32_t &rest) {
  float a, b;
  unpair(x, a, b);
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  upper = prmt(ua, ub, 0x7632);
  float ra, rb;
  unpair(add2(x, pair((ua & 0xFFFF0000u) ^ 0x80000000u, (ub & 0xFFFF0000u) ^ 0x80000000u)), ra, rb);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(rb), "f"(ra));
}
__device__ __forceinline__ uint32_t bf16_twice(float x) { return (__float_as_uint(x) >> 16) * 0x10001u; }  // x exact in bf16
// Brings bytes (a multiple of 16, from a 16-byte boundary on) into L2.
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Multiplies 32 columns of sums in tensor memory (one row a lane).
__device__ __forceinline__ void scale_sums(uint32_t taddr, float f) {
  uint32_t x[32];
  tmem_ld32(taddr, x);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
  tmem_st32(taddr, x);
  tmem_wait_st();
}

template <class L>
__global__ void __launch_bounds__(L::kThreads, 1) tiles_kernel(const Params p) {
  constexpr int D = L::D, BITS = L::BITS, R = L::R, RB = L::RB, W = L::kThreads / 32;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const uint32_t bar0 = base + L::kOffBar;
  auto k_full = [&](int s) { return bar0 + 8u * s; };
  auto k_empty = [&](int s) { return bar0 + 8u * (2 + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (6 + s); };
  auto par_full = [&](int s) { return bar0 + 8u * (8 + s); };  // four deep
  auto s_full = [&](int g) { return bar0 + 8u * (12 + g); };
  auto p_full = [&](int g) { return bar0 + 8u * (14 + g); };
  auto pv_done = [&](int g) { return bar0 + 8u * (16 + g); };
  const uint32_t q_full = bar0 + 8u * 18, all_done = bar0 + 8u * 19, stall_bar = bar0 + 8u * 20, pv_all_done = bar0 + 8u * 21;
  const uint32_t abort_flag = base + L::kOffMisc, tmem_slot = abort_flag + 4;
  Pending *pending = reinterpret_cast<Pending *>(smem + L::kOffMisc + 64 + L::kThreads / 4);
  volatile int64_t *share_s = reinterpret_cast<volatile int64_t *>(smem + L::kOffMisc + 32);
  int64_t *scan_s = reinterpret_cast<int64_t *>(smem + L::kOffMisc + 64);

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full(s), L::kCodeWarps);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), L::kCodeWarps);
      mbar_init(v_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 4);
      mbar_init(pv_done(s), 1);
    }
    for (int s = 0; s < 4; ++s) mbar_init(par_full(s), L::kCodeWarps);
    mbar_init(q_full, L::kSoftmaxWarps);
    mbar_init(all_done, 1);
    mbar_init(pv_all_done, 1);
    mbar_init(stall_bar, 1);
    st_flag(abort_flag, 0u);
    pending->count = 0;
    mbar_init_fence();
  }
  __syncthreads();
  griddep_wait();
  const uint64_t lim = p.control->limit_ns;
  const uint64_t limit_ns = lim ? lim : kDefaultWaitNs;
  unsigned int *error = &p.control->error;

  Cursor cur;
  Shares sh;
  int64_t u1, units;
  if (!share_of<L, W>(p, scan_s, share_s, cur, sh, u1, units)) {  // nothing for this CTA
    fill_unowned<D, L::kThreads>(p, tid);
    return;
  }
  const int64_t cta = blockIdx.x;
  if (warp == 16) tmem_alloc(tmem_slot, L::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kOffMisc + 4);
  // The next kernel may start from here on (CTAs without a share are gone): one that allocates tensor memory before it waits
  // for this one, as the layer's does, must not find it free while a CTA here has yet to take it, and then wait for that CTA.
  griddep_launch_dependents();

  if (warp >= 8 && warp < 16) {
    // ---------------------------------------------------------------------------------- the codes
    registers_down<L::kCodeRegs>();
    const bool keys = warp < 12;  // warps 8-11: keys and the tokens' scales, 12-15: values
    const int cw = (warp - 8) & 3;
    const int half = lane >> 4, l16 = lane & 15;
    const int ct = cw * 2 + half;  // cache tile of the 128 tokens, 16 threads each
    // The walk over the tiles runs kAhead tiles in front (and the look into the page table one more): addresses of
    // this thread's cache tile (null when it is not there). The values' warps bring the cache tiles into L2.
    constexpr int kAhead = 2;
    const int64_t page_bytes = int64_t(p.kv_heads) * p.page_tiles * L::kTile;
    Cursor ahead = cur;
    int64_t left = units;
    int page = -1;
    uint32_t offset = 0;
    auto look = [&]() {
      page = -1;
      if (left == 0) return;
      const int tile = ahead.blk * 8 + ct;
      if (tile * 16 < ahead.len) {
        const int page_i = p.page_shift >= 0 ? tile >> p.page_shift : tile / p.page_tiles;
        page = __ldg(p.page_table + ahead.b * p.max_pages + page_i);
        offset = static_cast<uint32_t>(ahead.h * p.page_tiles + (tile - page_i * p.page_tiles));
      }
      if (--left > 0 && ++ahead.blk == ahead.nb) next_segment<L>(p, ahead);
    };
    auto found = [&]() -> const uint8_t * {
      if (page < 0 || page >= p.num_pages) return nullptr;
      const uint8_t *a = p.cache + page * page_bytes + int64_t(offset) * L::kTile;
      if (!keys && l16 == 0) prefetch_l2(a, L::kTile);
      return a;
    };
    const uint8_t *next[kAhead];  // of the tiles t + 1 ..
    uint4 codes[L::kLoads];
    uint32_t pk = 0, pv = 0;  // the parameters of token l16 of the cache tile
    auto load = [&](const uint8_t *a) {
      if (a) {
        const uint4 *src = reinterpret_cast<const uint4 *>(a + (keys ? 0 : 16 * RB)) + l16;
#pragma unroll
        for (int i = 0; i < L::kLoads; ++i) codes[i] = __ldg(src + i * 16);
        const uint32_t *par = reinterpret_cast<const uint32_t *>(a + 32 * RB) + l16;
        if (keys) pk = __ldg(par);
        pv = __ldg(par + 16);
      } else {
#pragma unroll
        for (int i = 0; i < L::kLoads; ++i) codes[i] = make_uint4(0, 0, 0, 0);
        pk = pv = 0;
      }
    };
    // Stores the operand of one kind: 16-byte piece i * 16 + l16 of the cache tile's 16 rows.
    auto store = [&](uint32_t par, uint32_t dst, const bool values) {
#pragma unroll
      for (int i = 0; i < L::kLoads; ++i) {
        constexpr int kPer = RB / 16;  // pieces of a row
        const int q = i * 16 + l16, row = q / kPer, cc = q % kPer;
        const uint32_t z = (__shfl_sync(0xFFFFFFFFu, par, (lane & 16) | row) >> 16) & 0xFFu;
        const int tok = ct * 16 + row;
        const uint32_t zero = !values ? (0x6400u + z) * 0x10001u
                                      : (BITS == 8 ? bf16_twice(static_cast<float>(static_cast<int>(z) - 128)) : (0x4300u + (z & 0x7Fu)) * 0x10001u);
        const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
        constexpr int kOut = BITS == 8 ? 2 : 4;     // 16-byte pieces of the operand
        constexpr int kHalf = D == 128 ? kPer / 2 : kPer;  // pieces of a row in one 64-element block
        const int blk = cc / kHalf;
        const int turn = blk ? kOut / 2 : 0;  // the two blocks' stores of one instruction fall into different banks
        const uint32_t at = values ? static_cast<uint32_t>(tok >> 3) * (D / 64 * 1024u) + blk * 1024u + (tok & 7) * 128u
                                   : blk * 16384u + tok * 128u;
        const uint32_t chunk0 = static_cast<uint32_t>((cc % kHalf) * kOut + turn) ^ static_cast<uint32_t>(tok & 7);
#pragma unroll
        for (int jj = 0; jj < kOut; ++jj) {  // piece jj ^ turn
          uint32_t x[4];
          if constexpr (BITS == 8) {
            const uint32_t w0 = (jj ^ turn) ? w[2] : w[0], w1 = (jj ^ turn) ? w[3] : w[1];
            if (values) decode8_bf16(w0, w1, zero, x);
            else decode8(w0, w1, zero, x);
          } else {
            const uint32_t word = turn ? w[jj ^ 2] : w[jj];
            if (values) decode4_bf16(word, zero, x);
            else decode4(word, zero, (0x5400u + 16u * z) * 0x10001u, x);
          }
          sts128(dst + at + ((chunk0 ^ jj) << 4), x);
        }
      }
    };
    bool ok = true;
    look();
    const uint8_t *a0 = found();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      look();
      next[i] = found();
    }
    look();
    load(a0);
    bool there = a0 != nullptr;
    Cursor now = cur;
    for (int64_t t = 0; t < units; ++t) {
      const int s = static_cast<int>(t & 1), ps = static_cast<int>(t & 3);
      const uint32_t par = static_cast<uint32_t>((t >> 1) & 1);
      if (keys) {
        if (ok) ok = __all_sync(0xFFFFFFFFu, wait_phase(k_empty(s), par ^ 1u, abort_flag, limit_ns, error));
        // the tokens' scales
        const bool in = there && now.blk * 128 + ct * 16 + l16 < now.len;
        float *par_s = reinterpret_cast<float *>(smem + L::kOffParam + ps * L::kParam);
        par_s[ct * 16 + l16] = in ? bits_to_float(pk & 0xFFFFu, p.bf16 != 0) : 0.f;
        par_s[128 + ct * 16 + l16] = in ? bits_to_float(pv & 0xFFFFu, p.bf16 != 0) * kValueUnit : 0.f;
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, there);
        if (lane == 0) reinterpret_cast<volatile uint8_t *>(par_s + 256)[cw] = static_cast<uint8_t>((here & 1u) | ((here >> 16 & 1u) << 1));
        __syncwarp();
        if (lane == 0) mbar_arrive(par_full(ps));
        if (ok) store(pk, base + L::kOffK + s * L::kOperand, false);
      } else {
        if (ok) ok = __all_sync(0xFFFFFFFFu, wait_phase(v_empty(s), par ^ 1u, abort_flag, limit_ns, error));
        if (ok) store(pv, base + L::kOffV + s * L::kOperand, true);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(keys ? k_full(s) : v_full(s));
      const uint8_t *a1 = next[0];
      if (t + 1 < units) {
        load(a1);
        if (keys && ++now.blk == now.nb) next_segment<L>(p, now);
      }
      there = a1 != nullptr;
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) next[i] = next[i + 1];
      next[kAhead - 1] = found();
      look();
    }
  } else if (warp == 16) {
    // ---------------------------------------------------------------------------------- S = Q K^T
    if (lane == 0) {
      constexpr uint32_t idesc = (1u << 4) | (uint32_t(128 >> 3) << 17) | (uint32_t(128 >> 4) << 24);  // fp16, both K-major
      // descriptors: the lower words move with the stage and the step, the upper ones stay
      const uint64_t km = smem_desc(base + L::kOffQ, 16u, 1024u);
      const uint32_t q_lo = static_cast<uint32_t>(km), km_hi = static_cast<uint32_t>(km >> 32);
      const uint32_t k_lo = q_lo + ((L::kOffK - L::kOffQ) >> 4);
      bool ok = true;
      uint32_t seg_i = 0, t = 0;
      int64_t left = units;
      while (left > 0 && ok) {
        const int count = static_cast<int>(min(int64_t(cur.nb - cur.blk), left));
        ok = wait_phase(q_full, seg_i & 1u, abort_flag, limit_ns, error);
        for (int i = 0; i < count && ok; ++i, ++t) {
          const uint32_t s = t & 1u;
          // the group's last P (over the same columns) has been used
          ok = wait_phase(k_full(s), (t >> 1) & 1u, abort_flag, limit_ns, error) &&
               (t < 2 || wait_phase(pv_done(s), ((t >> 1) - 1u) & 1u, abort_flag, limit_ns, error));
          if (!ok) break;
          tc_fence_after();
          const uint32_t ka = k_lo + s * (L::kOperand >> 4), da = tmem + 128u * s;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
            if (kk == 0) umma_ss_first(da, pair(q_lo, km_hi), pair(ka, km_hi), idesc);
            else umma_ss(da, pair(q_lo + off, km_hi), pair(ka + off, km_hi), idesc);
          }
          umma_commit(s_full(s));
          umma_commit(k_empty(s));
        }
        left -= count;
        ++seg_i;
        if (left > 0) next_segment<L>(p, cur);
      }
      umma_commit(all_done);
      drain_phase(all_done, 0, error);
    }
    __syncwarp();
  } else if (warp == 17) {
    // ---------------------------------------------------------------------------------- O += P V
    if (lane == 0) {
      constexpr uint32_t idesc =
          (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (uint32_t(D >> 3) << 17) | (uint32_t(128 >> 4) << 24);  // bf16, V MN-major
      const uint64_t mn = smem_desc(base + L::kOffV, 1024u, D / 64 * 1024u);
      const uint32_t v_lo = static_cast<uint32_t>(mn), mn_hi = static_cast<uint32_t>(mn >> 32);
      bool ok = true;
      uint32_t t = 0;
      int64_t left = units;
      while (left > 0 && ok) {
        const int count = static_cast<int>(min(int64_t(cur.nb - cur.blk), left));
        for (int i = 0; i < count && ok; ++i, ++t) {
          const uint32_t s = t & 1u;
          ok = wait_phase(v_full(s), (t >> 1) & 1u, abort_flag, limit_ns, error) &&
               wait_phase(p_full(s), (t >> 1) & 1u, abort_flag, limit_ns, error);
          if (!ok) break;
          tc_fence_after();
          const uint32_t va = v_lo + s * (L::kOperand >> 4), pa = tmem + 128u * s, da = tmem + 256u + 128u * s;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {  // the upper parts of 16 tokens, then the rest
            const uint64_t bd = pair(va + kk * (D / 64 * 2048u >> 4), mn_hi);
            if (kk == 0 && i < 2) umma_ts_first(da, pa, bd, idesc);  // the group's first tile of the segment
            else umma_ts(da, pa + 16u * kk, bd, idesc);
            umma_ts(da, pa + 16u * kk + 8u, bd, idesc);
          }
          umma_commit(pv_done(s));
          umma_commit(v_empty(s));
        }
        left -= count;
        if (left > 0) next_segment<L>(p, cur);
      }
      umma_commit(pv_all_done);
      drain_phase(pv_all_done, 0, error);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------------------------- softmax
    registers_up<L::kSoftmaxRegs>();
    const int grp = warp >> 2;  // group
    const int row = tid & 127;  // of the tile; the warp reads the tensor memory lanes 32 (warp % 4) ..
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + lanes + 128u * grp, o_t = tmem + lanes + 256u + 128u * grp;
    float *row_s = reinterpret_cast<float *>(smem + L::kOffRow);
    float *qs_s = reinterpret_cast<float *>(smem + L::kOffQs);
    uint32_t pv_count = 0;  // products of this group that have been asked for
    int64_t t0 = 0;
    bool ok = true;
    if (p.control->stall) ok = __all_sync(0xFFFFFFFFu, wait_phase(stall_bar, 0, abort_flag, limit_ns, error));
    while (t0 < units) {
      const Cursor seg = cur;
      const Queries qu = queries_of(p, seg.b, seg.len);
      const int count = static_cast<int>(min(int64_t(seg.nb - seg.blk), units - t0));
      const int rows = min(R, qu.n * p.group - seg.rt * R);
      const int plain = min(qu.first, seg.len);
      // ---- Q: scaled by a power of two, K-major with the 128-byte swizzle
      {
        constexpr int LN = D / 8;
        for (int rr = tid / LN; rr < R; rr += 256 / LN) {
          const int c = tid % LN;
          float x[8];
          load_query<8>(p, seg, qu, rr, rows, R, c * 8, x);
          float top = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
          const uint32_t ln = ((1u << LN) - 1u) << (lane / LN * LN);
#pragma unroll
          for (int o = LN / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(ln, top, o));
          float up, unit;
          query_unit(p, top, up, unit);
          if (c == 0) qs_s[rr] = unit;
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // halves 2 j and 2 j + 1 of the operand's order
            const int e0 = BITS == 8 ? 2 * j : j, e1 = BITS == 8 ? 2 * j + 1 : j + 4;
            h[j] = pack_half2(x[e0] * up, x[e1] * up);
          }
          sts128(base + L::kOffQ + (c >> 3) * 16384u + rr * 128u + (((c & 7) ^ (rr & 7)) << 4), h);
        }
        fence_proxy_async_smem();
        bar_sync<1, 256>();
        if (lane == 0) mbar_arrive(q_full);
      }
      const float qs = qs_s[row];
      uint64_t word = ~0ull;
      if (row < rows) word = mask_word(p, qu, (seg.rt * R + row) / p.group);
      float m = -INFINITY, l = 0.f;
      bool begun = false;

      for (int i = static_cast<int>((grp - t0) & 1); i < count; i += 2) {
        const int64_t t = t0 + i;
        const float *par_s = reinterpret_cast<const float *>(smem + L::kOffParam + (t & 3) * L::kParam);
        if (ok)
          ok = __all_sync(0xFFFFFFFFu, wait_phase(par_full(static_cast<int>(t & 3)), static_cast<uint32_t>((t >> 2) & 1), abort_flag, limit_ns, error) &&
                                           wait_phase(s_full(grp), static_cast<uint32_t>((t >> 1) & 1), abort_flag, limit_ns, error));
        tc_fence_after();
        const int at0 = (seg.blk + i) * 128;
        const uint32_t here = __float_as_uint(par_s[256]);  // two cache tiles in each byte
        const bool whole = here == 0x03030303u && at0 + 128 <= plain;
        uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
        if (!whole) {
          // what this row sees of the tile's 128 tokens
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int x0 = at0 + 32 * c;
            uint32_t v = 0;
            const int d = qu.first - x0;  // tokens of the piece before the drafted ones
            if (d >= 32) v = ~0u;
            else {
              if (d > 0) v = (1u << d) - 1u;
              v |= d >= 0 ? static_cast<uint32_t>(word << d) : (-d < 64 ? static_cast<uint32_t>(word >> -d) : 0u);
            }
            const int n = seg.len - x0;
            if (n < 32) v &= n > 0 ? (1u << n) - 1u : 0u;
            const uint32_t two = here >> (8 * c);
            v &= ((two & 1u) ? 0x0000FFFFu : 0u) | ((two & 2u) ? 0xFFFF0000u : 0u);
            vis[c] = v;
          }
        }
        auto seen = [&](int c) { return c < 2 ? (c == 0 ? vis[0] : vis[1]) : (c == 2 ? vis[2] : vis[3]); };
        // ---- largest score
        float hi = -INFINITY;
        if (whole) {
          uint32_t s0[16], s1[16];
          float hj = -INFINITY;
          auto top16 = [&](const uint32_t (&s)[16], int c) {
            const ulonglong2 *sk2 = reinterpret_cast<const ulonglong2 *>(par_s + 16 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const ulonglong2 k2 = sk2[e];
              float y0, y1, y2, y3;
              unpair(mul2(pair(s[4 * e], s[4 * e + 1]), k2.x), y0, y1);
              unpair(mul2(pair(s[4 * e + 2], s[4 * e + 3]), k2.y), y2, y3);
              hi = fmaxf(fmaxf(hi, y0), y1);
              hj = fmaxf(fmaxf(hj, y2), y3);
            }
          };
          tmem_ld16(s_t, s0);
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            tmem_wait_ld();
            tmem_ld16(s_t + 16 * c + 16, s1);
            top16(s0, c);
            tmem_wait_ld();
            if (c < 6) tmem_ld16(s_t + 16 * c + 32, s0);
            top16(s1, c + 1);
          }
          hi = fmaxf(hi, hj);
        } else {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t s[16];
            tmem_ld16(s_t + 16 * c, s);
            tmem_wait_ld();
            const uint32_t v = seen(c >> 1) >> (16 * (c & 1));
#pragma unroll
            for (int e = 0; e < 16; ++e) hi = fmaxf(hi, v >> e & 1u ? __uint_as_float(s[e]) * par_s[16 * c + e] : -INFINITY);
          }
        }
        // ---- running maximum
        const float top = hi == -INFINITY ? hi : hi * qs;
        const bool raise = top > m + kTileSlack;
        if (__any_sync(0xFFFFFFFFu, raise)) {
          const float mn = fmaxf(m, top);
          const float f = mn == -INFINITY ? 1.f : exp2_approx(m - mn);
          m = mn;
          l *= f;
          if (begun) {
            if (ok) ok = __all_sync(0xFFFFFFFFu, wait_phase(pv_done(grp), (pv_count - 1) & 1u, abort_flag, limit_ns, error));
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) scale_sums(o_t + 32 * c, f);
          }
        }
        const float ms = m == -INFINITY ? 0.f : -m;
        // ---- probabilities times the values' scales: 16 tokens at a time over their own scores, the upper halves of the
        // fp32 numbers in 8 columns, the rest in the next 8
        if (whole) {
          const uint64_t qs2 = pair(__float_as_uint(qs), __float_as_uint(qs)), ms2 = pair(__float_as_uint(ms), __float_as_uint(ms));
          uint64_t l2 = 0, l3 = 0;
          auto prob16 = [&](const uint32_t (&s)[16], int c) {
            const ulonglong2 *sk2 = reinterpret_cast<const ulonglong2 *>(par_s + 16 * c);
            const ulonglong2 *wv2 = reinterpret_cast<const ulonglong2 *>(par_s + 128 + 16 * c);
            uint32_t h[8], r[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const ulonglong2 k2 = sk2[e], w2 = wv2[e];
              const uint64_t x01 = exp2_pair(fma2(mul2(pair(s[4 * e], s[4 * e + 1]), k2.x), qs2, ms2));
              const uint64_t x23 = exp2_pair(fma2(mul2(pair(s[4 * e + 2], s[4 * e + 3]), k2.y), qs2, ms2));
              l2 = add2(l2, x01);
              l3 = add2(l3, x23);
              split_pair(mul2(x01, w2.x), h[2 * e], r[2 * e]);
              split_pair(mul2(x23, w2.y), h[2 * e + 1], r[2 * e + 1]);
            }
            tmem_st8(s_t + 16 * c, h);
            tmem_st8(s_t + 16 * c + 8, r);
          };
          uint32_t s0[16], s1[16];
          tmem_ld16(s_t, s0);
#pragma unroll 1
          for (int c = 0; c < 8; c += 2) {
            tmem_wait_ld();
            tmem_ld16(s_t + 16 * c + 16, s1);
            prob16(s0, c);
            tmem_wait_ld();
            if (c < 6) tmem_ld16(s_t + 16 * c + 32, s0);
            prob16(s1, c + 1);
          }
          float a, b;
          unpair(add2(l2, l3), a, b);
          l += a + b;
        } else {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t s[16], h[8], r[8];
            tmem_ld16(s_t + 16 * c, s);
            tmem_wait_ld();
            const uint32_t v = seen(c >> 1) >> (16 * (c & 1));
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float x[2], pr[2];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const bool see = v >> (e + z) & 1u;
                x[z] = exp2_approx(fmaf(__uint_as_float(s[e + z]) * par_s[16 * c + e + z], qs, ms));
                pr[z] = see ? x[z] * par_s[128 + 16 * c + e + z] : 0.f;
                l += see ? x[z] : 0.f;
              }
              split_pair(pair(__float_as_uint(pr[0]), __float_as_uint(pr[1])), h[e / 2], r[e / 2]);
            }
            tmem_st8(s_t + 16 * c, h);
            tmem_st8(s_t + 16 * c + 8, r);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(grp));
        ++pv_count;
        begun = true;
      }
      // ---- join the groups
      if (begun && ok) ok = __all_sync(0xFFFFFFFFu, wait_phase(pv_done(grp), (pv_count - 1) & 1u, abort_flag, limit_ns, error));
      tc_fence_after();
      row_s[grp * 128 + row] = m;
      row_s[256 + grp * 128 + row] = begun ? l : -1.f;  // (no tile: no sums either)
      // One answer for all threads of the softmax: the warps of the codes and of the MMAs, already at the next segment, may
      // set the flag at any moment, and the barriers and tensor memory loads below are for all of these threads or for none.
      // (A wait of these threads that ran out has set it too.)
      const bool given_up = bar_any<1, 256>(ld_flag(abort_flag) != 0);
      tc_fence_after();
      if (given_up) ok = false;
      const float m0 = row_s[row], m1 = row_s[128 + row];
      const bool has0 = row_s[256 + row] != -1.f, has1 = row_s[384 + row] != -1.f;
      const float l0 = has0 ? row_s[256 + row] : 0.f, l1 = has1 ? row_s[384 + row] : 0.f;
      const float top = fmaxf(m0, m1);
      const float f0 = m0 == -INFINITY ? (l0 == 0.f ? 0.f : 1.f) : exp2_approx(m0 - top);
      const float f1 = m1 == -INFINITY ? (l1 == 0.f ? 0.f : 1.f) : exp2_approx(m1 - top);
      const float sum = l0 * f0 + l1 * f1;
      const bool is_first = seg.blk == 0, is_whole = is_first && count == seg.nb;
      const int64_t seg_u = u1 - (units - t0 - count) - count - seg.blk;
      if (!given_up) {
        float *slot = is_whole ? nullptr : p.partials + (2 * cta + (is_first ? 1 : 0)) * int64_t(R) * (D + 2);
        const int gr = seg.rt * R + row, qi = gr / p.group;
        const int64_t at = (qu.q0 + qi) * p.q_heads + seg.h * p.group + (gr - qi * p.group);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        // this group takes one half of the elements, from both groups' sums
#pragma unroll 1
        for (int c = grp * (D / 2); c < (grp + 1) * (D / 2); c += 16) {
          uint32_t a[16], b[16];
          float v[16];
          tmem_ld16(tmem + lanes + 256u + c, a);
          tmem_ld16(tmem + lanes + 384u + c, b);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            // element of the operand's place e
            const int d = BITS == 8 ? e : (e & ~7) + ((e & 7) >> 1) + 4 * (e & 1);
            const float x = (has0 ? __uint_as_float(a[e]) * f0 : 0.f) + (has1 ? __uint_as_float(b[e]) * f1 : 0.f);
            v[d] = (is_whole ? x * inv : x) * (1.f / kValueUnit);
          }
          if (is_whole) {
            if (row < rows) {
              store_out8(p, at * D + c, v);
              store_out8(p, at * D + c + 8, v + 8);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4 *>(slot + row * D + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
        if (grp == 0) {
          if (is_whole) {
            if (p.lse && row < rows) p.lse[at] = sum == 0.f ? -INFINITY : (top == -INFINITY ? sum : (top + log2f(sum)) * kLn2);
          } else {
            slot[R * D + row] = top;
            slot[R * (D + 1) + row] = sum;
          }
        }
        if (!is_whole)
          count_in<1, 256>(p, sh, seg, qu, rows, R, seg_u, int64_t(R) * (D + 2), reinterpret_cast<float *>(smem + L::kOffQ), pending, tid);
      }
      tc_fence_before();
      bar_sync<1, 256>();  // the sums and row_s have been read, Q may be written
      t0 += count;
      if (t0 < units) next_segment<L>(p, cur);
    }
    for (int i = 0; i < pending->count; ++i) join_parts<R, D, 256, 8, 1>(pending->parts[i], tid);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, L::kTmemCols);
  fill_unowned<D, L::kThreads>(p, tid);
}

template <int D>
cudaError_t launch_tiles(const Params &p, int bits, int num_sms, cudaStream_t stream) {
  return bits == 8 ? start_kernel<TileLayout<D, 8>>(tiles_kernel<TileLayout<D, 8>>, num_sms, p, stream)
                   : start_kernel<TileLayout<D, 4>>(tiles_kernel<TileLayout<D, 4>>, num_sms, p, stream);
}

}  // namespace attention
}  // namespace w4a16
