// Attention of many rows per sequence over a paged KV cache on the tensor
// cores (sm_103a): the prompt form of tf_op_attention_cache for bfloat16 rows,
// over bf16 and 4-bit pages.
//
// out = sum_j p_j v_j, p = softmax_j(scale q.k_j) over what a row sees.  With
// hundreds of rows per K / V read the two products are the bound, so they run as
// tcgen05.mma (M = 128, bf16, fp32 in TMEM):
//   * A CTA takes 256 (row, query head) pairs of one KV head, so that the heads
//     of a group and 256 / G rows share every K and V tile, as two tiles A and B
//     of 128 (a pair is a TMEM lane).  While a warpgroup turns the scores of A
//     into probabilities the tensor core multiplies B's, and the other way round.
//   * TMEM (512 columns): scores of A and B (128 columns each), outputs of A and
//     B.  The probabilities go back into the first 64 columns of their scores
//     as bf16 and are the second product's A operand straight from there: no
//     shared-memory trip, and shared memory holds Q, 2 K and 2 V tiles.
//   * A key tile is four pages of the list (sink pages, then the window's), each
//     with its own base position, so that neither the sinks nor a window that
//     starts inside a tile costs a tile of its own.
//   * bf16 pages come by TMA (128-byte swizzle).  4-bit pages are converted by
//     four warps: e2m1 x e4m3 has at most 6 significant bits and is exact in bf16;
//     K's row scale multiplies the scores and V's the probabilities, in float32.
//   * The maximum is replaced, and O rescaled in TMEM, only when the probabilities
//     relative to it grow past 2^13.  Probabilities enter as bf16 (half a step: 2^-8 of
//     each, as much as the output's own rounding); their sum is of the unrounded
//     ones, in float32.
//   * Tiles that some row does not see whole are masked, and V rows that no row
//     sees are zeroed in shared memory (0 x NaN is NaN); a V row with an infinity
//     or a NaN that only some rows see is zeroed too and made a NaN probability
//     of the rows that see it.
// Measured (GB300, 32 query and 8 KV heads of 128): a tile of 128 keys takes a CTA
// about 3000 cycles with bf16 pages (the four products; 2600 at the measured dense
// rate) and 4000 with 4-bit pages (the softmax behind the products: its scales and
// the converters' instructions).  Four ragged chunks of up to 1024 rows, window 1024:
// 67 us (53 GFLOP); 2 x 1024 rows over 5120 4-bit positions: 170 us (155 GFLOP).
// Every wait is bounded; the TMEM columns are always released.
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "cache.cuh"
#include "common.cuh"
#include "device_once.h"
#include "kernels.h"
#include "tensor_map.h"

namespace tf {

namespace {

// The maximum that the exponentials are relative to is replaced when a lane's sum of a row's probabilities of a
// tile or part of it exceeds this (2^13; so no probability does).
constexpr float kMaxSum = 8192.0f;
constexpr int kInfo = 4;         // tiles of which the position / scale records are kept
constexpr int kNowhere = 0x3FFFFFFF;  // base position of a quarter that holds nothing

template <int D, int FMT>
struct PromptCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTile = 128 * D * 2;              // 128 rows of Q, K or V
  static constexpr int kSlots = 2;                       // K tiles, and V tiles, in flight
  static constexpr size_t kOffK = 2 * (size_t)kTile;
  static constexpr size_t kOffV = kOffK + (size_t)kSlots * kTile;
  static constexpr size_t kOffInfo = kOffV + (size_t)kSlots * kTile;
  // per kept tile: 4 base positions, poison words and whole flags, and for 4-bit pages 128 K and V row scales
  static constexpr int kInfoBytes = 48 + (FMT ? 2 * 128 * 4 : 0);
  static constexpr size_t kOffBar = kOffInfo + (size_t)kInfo * kInfoBytes;
  static constexpr size_t kSmem = 1024 + kOffBar + 24 * 8 + 16;
  // Warps: 8 softmax, then FMT 0: 1 MMA, 1 TMA, 2 that clean V; FMT 1: 4 converting, 1 MMA (and 3 idle ones, so
  // that whole warpgroups can trade registers: the softmax takes what the others do not need).
  static constexpr int kThreads = FMT ? 32 * 16 : 32 * 12;
  static constexpr int kMmaWarp = FMT ? 12 : 8;
  // Quarters of a tile whose p a lane keeps before it stores them: what its registers hold (FMT 1, 2 x 1024 rows
  // over 5120 positions: 170 us with 2, 184 with 1; 4 spills).
  static constexpr int kGroup = FMT ? 2 : 4;
  static constexpr uint32_t kCols = 512;
  // kind::f16, fp32 accumulate, bf16 operands, M = 128.  S: B = K tile, K-major, N = 128.
  // O: B = V tile, MN-major (bit 16), N = D.
  static constexpr uint32_t kIdescS =
      (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                      ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kWaitBudgetNs) return false;
  return true;
}
// the same, one answer for the warp (what follows is warp-collective)
__device__ __forceinline__ bool bar_wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity) ? 1 : 0) != 0;
}

__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store3(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// K-major operand tile: 8-row groups of 128-byte rows, 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | static_cast<uint64_t>(1) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
// MN-major operand tile: 64-element column blocks 16 KB apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | static_cast<uint64_t>(16384 >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{.reg .pred q; elect.sync _|q, 0xFFFFFFFF; selp.u32 %0, 1, 0, q;}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tm_ld32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// The scores' and outputs' fragment: 16 lanes x 32 columns.  Register 4 i + 2 h + e of lane (g, t) is lane
// g + 8 h of TMEM, column 8 i + 2 t + e (the shape of a warp-level product's accumulator), so a lane holds two
// columns of several rows, and what belongs to a column is loaded once for all of them.
__device__ __forceinline__ void tm_frag_ld(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tm_frag_st(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 lanes x 16 columns: register 2 i + h is lane g + 8 h, column 4 i + t.
__device__ __forceinline__ void tm_pair_st(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tm_pair_ld(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
// Waits for the loads; the registers go through it, so that nothing uses them before.
__device__ __forceinline__ void tm_wait_ld(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tm_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tm_wait_ld(uint32_t (&s)[2][16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(s[0][0]), "+r"(s[0][1]), "+r"(s[0][2]), "+r"(s[0][3]), "+r"(s[0][4]), "+r"(s[0][5]),
                 "+r"(s[0][6]), "+r"(s[0][7]), "+r"(s[0][8]), "+r"(s[0][9]), "+r"(s[0][10]), "+r"(s[0][11]),
                 "+r"(s[0][12]), "+r"(s[0][13]), "+r"(s[0][14]), "+r"(s[0][15]), "+r"(s[1][0]), "+r"(s[1][1]),
                 "+r"(s[1][2]), "+r"(s[1][3]), "+r"(s[1][4]), "+r"(s[1][5]), "+r"(s[1][6]), "+r"(s[1][7]),
                 "+r"(s[1][8]), "+r"(s[1][9]), "+r"(s[1][10]), "+r"(s[1][11]), "+r"(s[1][12]), "+r"(s[1][13]),
                 "+r"(s[1][14]), "+r"(s[1][15])
               :
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void e2m1x8(uint32_t v, uint32_t (&h)[4]) {
  asm("{.reg .b8 b0, b1, b2, b3; mov.b32 {b0, b1, b2, b3}, %4;"
      " cvt.rn.f16x2.e2m1x2 %0, b0; cvt.rn.f16x2.e2m1x2 %1, b1;"
      " cvt.rn.f16x2.e2m1x2 %2, b2; cvt.rn.f16x2.e2m1x2 %3, b3;}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(v));
}
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return h;
}
// The products of two f16 pairs as floats (mixed-precision FMA: conversion and product in one).
__device__ __forceinline__ float2 scaled(uint32_t v, uint32_t s) {
  float2 d;
  asm("{.reg .b16 vl, vh, sl, sh; mov.b32 {vl, vh}, %2; mov.b32 {sl, sh}, %3;"
      " fma.rn.f32.f16 %0, vl, sl, %4; fma.rn.f32.f16 %1, vh, sh, %4;}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(v), "r"(s), "f"(0.f));
  return d;
}
// Two floats in one 64-bit operand of the packed float32 instructions.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 16-byte chunk of row r, chunk ch of the row, in the swizzled tile layout.
__device__ __forceinline__ uint4* chunk_at(uint8_t* tile, int r, int ch) {
  return reinterpret_cast<uint4*>(tile + (ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void st_shared16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Bits of the 32 positions from base that a row at `pos` sees.
__device__ __forceinline__ uint32_t ones(int n) {  // the n lowest bits; none below 0, all from 32 on
  uint32_t d;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(d) : "r"(0), "r"(max(n, 0)));
  return d;
}
__device__ __forceinline__ uint32_t sees(int base, int pos, int low, int sinks) {
  return ones(pos - base + 1) & (~ones(low - base) | ones(sinks - base));
}

template <int D, int FMT, int NX>
__global__ void __launch_bounds__(PromptCfg<D, FMT>::kThreads, 1)
    k_cache_prompt(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_o,
                   const CacheAttnParams p, const int boxed) {
  constexpr int span = 128 * NX;  // pairs of the CTA: NX tiles
  using C = PromptCfg<D, FMT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sk = smem + C::kOffK;
  uint8_t* sv = smem + C::kOffV;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t *k_full = bar, *k_empty = bar + 2, *v_full = bar + 4, *v_empty = bar + 6;  // [2] each
  uint64_t *s_full = bar + 8, *p_full = bar + 10, *o_done = bar + 12, *drained = bar + 14, *q_full = bar + 15;
  uint64_t* v_clean = bar + 18;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 16);
  volatile uint32_t* failed = tmem_slot + 1;

  const CacheBatch& c = p.c;
  // (the shuffle, and the reduction below: values that the compiler knows to be the warp's, as the tensor core takes
  // its addresses; 184 us of the 4-bit case above without them, 174 with them)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int hkv = blockIdx.y, b = blockIdx.z;
  const int G = p.Hq / c.Hkv;
  const SeqRows sq = cache_seq(c, b);
  const int tile = static_cast<int>(gridDim.x - 1 - blockIdx.x);  // the last rows, which see most, first
  const int c0 = tile * span, ncol = min(span, sq.n * G - c0);
  if (ncol <= 0) return;
  const int first = sq.len - sq.n;
  const int posmin = first + c0 / G, posmax = first + (c0 + ncol - 1) / G;
  const bool win = p.window > 0;
  const int lowmin = win ? max(0, posmin - p.window + 1) : 0;
  const int lowmax = win ? max(0, posmax - p.window + 1) : 0;
  const int sinks = win ? p.sinks : 0;
  // The list of pages: the sinks' that the windows do not reach, then lowmin .. posmax.
  const int plow = lowmin / kKvPage;
  const int psink = min(plow, (min(sinks, lowmin) + kKvPage - 1) / kKvPage);
  const int pages = posmax < 0 ? 0 : psink + posmax / kKvPage - plow + 1;
  const int nt = (pages + 3) / 4;
  auto base_at = [&](int u) { return (u < psink ? u : plow + u - psink) * kKvPage; };
  // Tiles are taken from the second on and the first last: with a window the first is masked, and the pipeline
  // starts faster on one that is not.
  const int turn = win && nt >= 3 ? 1 : 0;
  auto tile_at = [&](int j) { return j + turn < nt ? j + turn : j + turn - nt; };
  auto quarter_whole = [&](int bq) {
    return bq + kKvPage - 1 <= posmin && (bq >= lowmax || bq + kKvPage <= sinks) ? 1 : 0;
  };
  struct Info {
    int base[4];          // position of the quarter's first key, kNowhere: nothing there
    uint32_t poison[4];   // keys whose V row is not finite (mixed quarters)
    int whole[4];         // every pair of the CTA sees every key of the quarter
    float ks[FMT ? 128 : 1], vs[FMT ? 128 : 1];
  };
  auto info = [&](int j) { return reinterpret_cast<Info*>(smem + C::kOffInfo + (j % kInfo) * C::kInfoBytes); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], FMT ? 128 : 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], FMT ? 128 : 1);
      mbar_init(&v_clean[i], 2);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(drained, 1);
    mbar_init(q_full, boxed ? 1 : 256);
    *failed = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = __reduce_or_sync(0xFFFFFFFFu, *tmem_slot);

  // FMT 1: the softmax's warpgroups take registers from the other two: 256 x 160 + 256 x 96 = the launch's
  // 512 x 128
  if (warp >= 8) {
    if constexpr (FMT == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer: the warp stays together, one
      // lane issues (a loop that only one lane runs computes every operand in its own registers and moves it to the
      // warp's: the tensor core waits for it)
      bool ok = true;
      // pairs are consecutive (row, head) rows of Q: one box per tile and 64 columns (none where no row sees a key:
      // nothing would wait for them)
      if (boxed && nt > 0 && elect_one()) {
        mbar_arrive_expect_tx(q_full, NX * C::kTile);
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_box3(smem_u32(smem) + x * C::kTile + h * 16384, &map_q, h * 64, hkv * G,
                     sq.r0 + (c0 + x * 128) / G, q_full);
      }
      auto score = [&](int x, int j) {  // S_x = Q_x K(j)^T
        const uint64_t qd = desc_k(smem_u32(smem) + x * C::kTile), kd = desc_k(smem_u32(sk) + (j & 1) * C::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          mma_ss(tmem + x * 128, qd + off, kd + off, C::kIdescS, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[x]);
      };
      if (nt > 0) {
        ok = bar_wait_warp(q_full, 0) && bar_wait_warp(&k_full[0], 0);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (ok && elect_one()) {
          score(0, 0);
          if constexpr (NX > 1) score(1, 0);
          mma_commit(&k_empty[0]);
        }
      }
      for (int j = 0; ok && j < nt; ++j) {
        const uint64_t vd = desc_mn(smem_u32(sv) + (j & 1) * C::kTile);
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          // (P last: the others are there as a rule, and nothing then lies between P and its product)
          ok = ok && (x || bar_wait_warp(FMT ? &v_full[j & 1] : &v_clean[j & 1], (j >> 1) & 1)) &&
               bar_wait_warp(&p_full[x], j & 1);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, vd + (kk * 2048 >> 4), C::kIdescO,
                     (j > 0 || kk > 0) ? 1u : 0u);
            if (x == NX - 1) mma_commit(&v_empty[j & 1]);
            if (j + 1 == nt) mma_commit(&o_done[x]);
          }
          __syncwarp();
          if (j + 1 < nt) {
            if (!x) {
              ok = bar_wait_warp(&k_full[(j + 1) & 1], ((j + 1) >> 1) & 1);
              if (!ok) break;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            }
            if (elect_one()) {
              score(x, j + 1);  // after the product that reads P_x, in issue order; its commit covers both
              if (x == NX - 1) mma_commit(&k_empty[(j + 1) & 1]);
            }
            __syncwarp();
          }
        }
      }
      if (!ok && lane == 0) *failed = 1;
      if (elect_one()) mma_commit(drained);  // nothing may be in flight when the columns are released
      if (!bar_wait_warp(drained, 0) && lane == 0) *failed = 1;
    } else {
      if constexpr (FMT == 0) {
        // -------------------------------------------------------------- TMA producer
        if (warp == 9 && lane == 0) {
          int done = 0;
          for (; done < nt; ++done) {
            const int j = done, s = j & 1;
            int pg[4];
            uint32_t boxes = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int u = 4 * tile_at(j) + q;
              pg[q] = u < pages ? cache_page(c, b, base_at(u) / kKvPage) : -1;
              boxes += pg[q] >= 0 ? 1u : 0u;
            }
            if (j >= 2 && !bar_wait(&k_empty[s], ((j >> 1) - 1) & 1)) break;
            Info* in = info(j);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int bq = pg[q] >= 0 ? base_at(4 * tile_at(j) + q) : kNowhere;
              in->base[q] = bq;
              in->poison[q] = 0;
              in->whole[q] = quarter_whole(bq);
            }
            auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* full) {
              mbar_arrive_expect_tx(full, boxes * (kKvPage * D * 2));
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (pg[q] >= 0)
                  for (int x = 0; x < C::kBoxes; ++x)
                    tma_box(smem_u32(dst) + x * 16384 + q * (kKvPage * 128), map, x * 64,
                            (pg[q] * c.Hkv + hkv) * kKvPage, full);
            };
            load(&map_k, sk + s * C::kTile, &k_full[s]);
            if (j >= 2 && !bar_wait(&v_empty[s], ((j >> 1) - 1) & 1)) {
              bar_wait(&k_full[s], (j >> 1) & 1);
              break;
            }
            load(&map_v, sv + s * C::kTile, &v_full[s]);
          }
          if (done < nt) *failed = 1;
          // every copy has landed before the CTA leaves
          for (int j = max(0, done - 2); j < done; ++j)
            if (!bar_wait(&k_full[j & 1], (j >> 1) & 1) || !bar_wait(&v_full[j & 1], (j >> 1) & 1)) break;
        } else if (warp >= 10) {
          // ------------------------------------------------------------ V cleaners: in mixed tiles, rows that
          // nobody sees or that are not finite become zeros before the product reads them
          const int t = threadIdx.x - 320;
          for (int j = 0; j < nt; ++j) {
            if (!bar_wait_warp(&v_full[j & 1], (j >> 1) & 1)) break;
            Info* in = info(j);
            uint8_t* vt = sv + (j & 1) * C::kTile;
            for (int r = t; r < 128; r += 64) {
              const int q = r >> 5, bq = in->base[q], kp = bq + (r & 31);
              if (in->whole[q]) continue;
              const bool dead = bq == kNowhere || !(kp <= posmax && (kp >= lowmin || kp < sinks));
              bool bad = false;
              if (!dead) {
#pragma unroll
                for (int ch = 0; ch < D / 8; ++ch) {
                  const uint4 v = *chunk_at(vt, r, ch);
                  const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    bad |= (w4[i] & 0x7F80u) == 0x7F80u || (w4[i] & 0x7F800000u) == 0x7F800000u;
                }
                if (bad) atomicOr(&in->poison[q], 1u << (r & 31));
              }
              if (dead || bad)
#pragma unroll
                for (int ch = 0; ch < D / 8; ++ch) *chunk_at(vt, r, ch) = make_uint4(0u, 0u, 0u, 0u);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_clean[j & 1]);
          }
        }
      } else if (warp < 12) {
        // -------------------------------------------------------------- converting warps, one page of a tile each
        using L = Kv4<D>;
        constexpr int NI = D / 32;     // 16-byte pieces of K (and of V) a lane takes
        constexpr int PR = D / 32;     // pieces of a K row
        const int w = warp - 8;
        // V piece i of this lane: unit of (position pair column j, block, t); the order differs by t so that the
        // lanes' rows fall into different banks
        auto v_unit = [&](int i) {
          if constexpr (D == 128) return ((i + lane) & 3) * 32 + lane;
          return i * 32 + lane;
        };
        auto v_row = [&](int v) { return 8 * (v & 3) + 2 * (v / (D / 4)); };
        // a piece's loads go out before the wait for its slot
        uint4 raw[NI];
        uint32_t ksb[NI], vsb[NI];
        bool ok = true;
        auto page_of = [&](int j) {  // of this warp's quarter of the j-th tile taken
          const int u = 4 * tile_at(j) + w;
          return j < nt && u < pages ? cache_page(c, b, base_at(u) / kKvPage) : -1;
        };
        int page = page_of(0);
        for (int j = 0; j < nt; ++j) {
          // (opaque to the compiler: kept across the loop, a lane's addresses would not fit its registers)
          int ln = lane;
          asm volatile("" : "+r"(ln));
          const int s = j & 1;
          const int base = page >= 0 ? base_at(4 * tile_at(j) + w) : kNowhere;
          const uint8_t* kp = c.K + ((size_t)max(page, 0) * c.Hkv + hkv) * L::kBytes;
          const uint8_t* vp = c.V + ((size_t)max(page, 0) * c.Hkv + hkv) * L::kBytes;
          float krow = 0.f, vrow = 0.f;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int e = i * 32 + lane, v = v_unit(i);  // K piece: row e / PR, elements 32 (e % PR) ..
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            ksb[i] = vsb[i] = 0;
            if (page >= 0) {
              raw[i] = __ldg(reinterpret_cast<const uint4*>(kp + e * 16));
              ksb[i] = __ldg(reinterpret_cast<const uint16_t*>(kp + L::kCodes + e * 2));
              vsb[i] = __ldg(reinterpret_cast<const uint16_t*>(vp + L::kCodes + (v % (D / 4)) / 4 * kKvPage + v_row(v)));
            }
          }
          if (page >= 0) {
            krow = __ldg(reinterpret_cast<const float*>(kp + L::kRows) + lane);
            vrow = __ldg(reinterpret_cast<const float*>(vp + L::kRows) + lane);
          }
          // the next page's id, two loads ahead of its use
          const int next = page_of(j + 1);
          const int whole = quarter_whole(base);
          uint32_t dead = 0, poison = 0;
          if (!whole) {
            const int pos = base + lane;
            dead = __ballot_sync(0xFFFFFFFFu, !(pos <= posmax && (pos >= lowmin || pos < sinks)));
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < NI; ++i)
              bad |= (((vsb[i] & 0x7Fu) == 0x7Fu ? 1u : 0u) | ((vsb[i] & 0x7F00u) == 0x7F00u ? 2u : 0u))
                     << v_row(v_unit(i));
            poison = __reduce_or_sync(0xFFFFFFFFu, bad) & ~dead;
          }
          Info* in = info(j);
          if (j >= 2 && !(ok = bar_wait_warp(&k_empty[s], ((j >> 1) - 1) & 1))) break;
          if (lane == 0) {
            in->base[w] = base;
            in->poison[w] = poison;
            in->whole[w] = whole;
          }
          in->ks[w * 32 + lane] = krow * p.scale_log2;
          in->vs[w * 32 + lane] = (dead >> lane) & 1u ? 0.f : vrow;
          // Row r = w * 32 + (32 i + lane) / PR, blocks 2 q and 2 q + 1 of it: chunk x of the four lies at the first one's
          // address ^ x * 16 (r & 7 is the same for every i).  The lanes of a row's upper half store their blocks the
          // other way round: no bank conflicts.
          const int q = ln % PR, r0 = ln / PR;
          const bool swap = (q >> 1) & 1;
          const uint32_t kt = smem_u32(sk) + s * C::kTile + (q >> 1) * 16384 + (w * 32 + r0) * 128 +
                              ((((4 * q) & 7) ^ (r0 & 7)) << 4);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const uint32_t words[4] = {swap ? raw[i].z : raw[i].x, swap ? raw[i].w : raw[i].y,
                                       swap ? raw[i].x : raw[i].z, swap ? raw[i].y : raw[i].w};
            const uint32_t s2 = e4m3x2_f16(swap ? __byte_perm(ksb[i], 0, 0x4401) : ksb[i]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t h[4], o[4];
              e2m1x8(words[x], h);
              const uint32_t sd = __byte_perm(s2, 0, x < 2 ? 0x1010 : 0x3232);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float2 f = scaled(h[y], sd);
                o[y] = pack_bf16(f.x, f.y);
              }
              st_shared16((kt ^ ((x ^ (swap ? 2 : 0)) << 4)) + i * (32 / PR) * 128, o[0], o[1], o[2], o[3]);
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_arrive(&k_full[s]);
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (page >= 0) raw[i] = __ldg(reinterpret_cast<const uint4*>(vp + v_unit(i) * 16));
          if (j >= 2 && !(ok = bar_wait_warp(&v_empty[s], ((j >> 1) - 1) & 1))) break;
          dead |= poison;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            // rows r and r + 1 (r even) of block blk: chunk h of row r at vt ^ h * 16, of row r + 1 at (vt + 128) ^ 16 ^ h * 16
            const int v = D == 128 ? ((i + ln) & 3) * 32 + ln : i * 32 + ln;
            const int r = v_row(v), blk = (v % (D / 4)) / 4;
            const uint32_t vt = smem_u32(sv) + s * C::kTile + (blk >> 2) * 16384 + (w * 32 + r) * 128 +
                                ((((2 * blk) & 7) ^ (r & 7)) << 4);
            const uint32_t words[4] = {blk & 1 ? raw[i].z : raw[i].x, blk & 1 ? raw[i].w : raw[i].y,
                                       blk & 1 ? raw[i].x : raw[i].z, blk & 1 ? raw[i].y : raw[i].w};
            uint32_t sb = vsb[i];
            if ((dead >> r) & 1u) sb &= 0xFF00u;
            if ((dead >> r) & 2u) sb &= 0x00FFu;
            const uint32_t s2 = e4m3x2_f16(sb);
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
              uint32_t h[4], g[4], o0[4], o1[4];
              e2m1x8(words[x], h);
              e2m1x8(words[x + 1], g);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float2 f0 = scaled(h[2 * y], s2), f1 = scaled(h[2 * y + 1], s2);
                const float2 g0 = scaled(g[2 * y], s2), g1 = scaled(g[2 * y + 1], s2);
                o0[y] = pack_bf16(f0.x, f1.x);
                o1[y] = pack_bf16(f0.y, f1.y);
                o0[2 + y] = pack_bf16(g0.x, g1.x);
                o1[2 + y] = pack_bf16(g0.y, g1.y);
              }
              const uint32_t h16 = (x / 2 ^ (blk & 1)) << 4;
              st_shared16(vt ^ h16, o0[0], o0[1], o0[2], o0[3]);
              st_shared16((vt + 128) ^ 16 ^ h16, o1[0], o1[1], o1[2], o1[3]);
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_arrive(&v_full[s]);
          page = next;
        }
        if (!ok && lane == 0) *failed = 1;
      }
    }
  } else {
    if constexpr (FMT == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    // ---------------------------------------------------------------- softmax: a warp has 32 pairs (its TMEM
    // lanes); lane (g, t) holds pairs g, g + 8, g + 16, g + 24 and columns 2 t, 2 t + 1 of every 8
    const int x = warp >> 2, lg = lane >> 2, lt = lane & 3;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + x * 128 + lanes, t_o = tmem + 256 + x * 128 + lanes;
    const int col0 = x * 128 + (warp & 3) * 32;   // the warp's first pair
    // Q (by these 256 threads): pair m of the CTA is row (c0 + m) / G, head (c0 + m) % G; rows past the last pair
    // are zero.  A warp copies kLines pairs at a time; lane i works out where the i-th of its 32 pairs lies.
    constexpr int kChunks = D / 8, kLines = 32 / kChunks;
    auto pair_at = [&](int m, int64_t stride) {  // element offset of a pair's row
      const int cc = c0 + m;
      return (int64_t)(sq.r0 + cc / G) * stride + (int64_t)(hkv * G + cc % G) * D;
    };
    auto from_lane = [&](int64_t v, int src) {
      return static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, static_cast<long long>(v), src));
    };
    if (!boxed && nt > 0) {
      const int64_t at = pair_at(lane / kLines * (8 * kLines) + warp * kLines + lane % kLines, p.q_stride);
#pragma unroll 4
      for (int it = 0; it < kChunks; ++it) {
        const int m = it * (8 * kLines) + warp * kLines + lane / kChunks, ch = lane % kChunks;
        uint4* dst = chunk_at(smem + (m >> 7) * C::kTile, m & 127, ch);
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + from_lane(at, it * kLines + lane / kChunks) + ch * 8;
        if (m >= ncol) {
          *dst = make_uint4(0u, 0u, 0u, 0u);
        } else if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
        } else {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = src[2 * i] | static_cast<uint32_t>(src[2 * i + 1]) << 16;
          *dst = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (!boxed && nt > 0) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full);
    }
    int pos[4], low[4];
    float ref[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int col = col0 + 8 * k + lg;
      pos[k] = col < ncol ? first + (c0 + col) / G : posmin;
      low[k] = win ? max(0, pos[k] - p.window + 1) : 0;
      ref[k] = -INFINITY;
      l[k] = 0.f;
    }
    bool ok = true;
    const int mine = x < NX ? nt : 0;
    for (int j = 0; j < mine; ++j) {
      if (!(ok = bar_wait_warp(&s_full[x], j & 1))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const Info* in = info(j);
      const int4 wq = *reinterpret_cast<const int4*>(in->whole);
      int kind = 0;  // 0: every pair sees every key; 1: a mask; 2: a mask, and V rows that are not finite
      if (!(wq.x && wq.y && wq.z && wq.w)) {
        if (FMT == 0 && !(ok = bar_wait_warp(&v_clean[j & 1], (j >> 1) & 1))) break;
        kind = (in->poison[0] | in->poison[1] | in->poison[2] | in->poison[3]) ? 2 : 1;
      }
      auto masks = [&](int q, uint32_t (&see)[4]) {  // bits 8 i + e: columns 8 i + 2 t + e of the quarter
#pragma unroll
        for (int k = 0; k < 4; ++k) see[k] = sees(in->base[q], pos[k], low[k], sinks) >> (2 * lt);
      };
      auto load = [&](int q, uint32_t (&s)[2][16]) {
        tm_frag_ld(t_s + q * 32, s[0]);
        tm_frag_ld(t_s + (16u << 16) + q * 32, s[1]);
      };
      // The largest log2 weight (relative to `ref`, or absolute) that each of the lane's rows sees in a quarter.
      auto top_of = [&](int q, bool relative, float (&mx)[4]) {
        uint32_t s[2][16], see[4];
        load(q, s);
        masks(q, see);
        tm_wait_ld(s);
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 ks = make_float2(p.scale_log2, p.scale_log2);
          if constexpr (FMT == 1) ks = *reinterpret_cast<const float2*>(in->ks + q * 32 + 8 * i + 2 * lt);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t* sr = &s[k >> 1][4 * i + 2 * (k & 1)];
            if ((see[k] >> (8 * i)) & 1u) mx[k] = fmaxf(mx[k], __uint_as_float(sr[0]) * ks.x);
            if ((see[k] >> (8 * i)) & 2u) mx[k] = fmaxf(mx[k], __uint_as_float(sr[1]) * ks.y);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xFFFFFFFFu, mx[k], 1));
          mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xFFFFFFFFu, mx[k], 2));
          if (relative) mx[k] -= ref[k];
        }
      };
      // C::kGroup quarters of the tile from q0 on: p relative to ref, their sums, and p (times V's row scale) packed for
      // the store.
      auto group = [&](auto w_, int q0, float (&sum)[4], uint32_t (&pk)[C::kGroup][2][8]) {
        constexpr int kKind = decltype(w_)::value;
        uint64_t nm2[4], sum2[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float nm = ref[k] == -INFINITY ? 0.f : -ref[k];
          nm2[k] = pair2(nm, nm);
          sum2[k] = 0;
        }
#pragma unroll
        for (int h = 0; h < C::kGroup; ++h) {
          const int q = q0 + h;
          uint32_t s[2][16], see[4], poison = 0;
          load(q, s);
          if constexpr (kKind > 0) masks(q, see);
          if constexpr (kKind == 2) poison = in->poison[q] >> (2 * lt);
          tm_wait_ld(s);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 ks = make_float2(p.scale_log2, p.scale_log2), vs = ks;
            if constexpr (FMT == 1) {  // (read where they are used: 3% of the case above against ahead of the wait)
              ks = *reinterpret_cast<const float2*>(in->ks + q * 32 + 8 * i + 2 * lt);
              vs = *reinterpret_cast<const float2*>(in->vs + q * 32 + 8 * i + 2 * lt);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t* sr = &s[k >> 1][4 * i + 2 * (k & 1)];
              float t0, t1;
              unpair2(fma2(pair2(__uint_as_float(sr[0]), __uint_as_float(sr[1])), pair2(ks.x, ks.y), nm2[k]), t0, t1);
              t0 = ex2f(t0);
              t1 = ex2f(t1);
              if constexpr (kKind > 0) {
                t0 = (see[k] >> (8 * i)) & 1u ? t0 : 0.f;
                t1 = (see[k] >> (8 * i)) & 2u ? t1 : 0.f;
              }
              if constexpr (kKind == 2) {
                if (((see[k] & poison) >> (8 * i)) & 1u) t0 = __int_as_float(0x7FFFFFFF);
                if (((see[k] & poison) >> (8 * i)) & 2u) t1 = __int_as_float(0x7FFFFFFF);
              }
              const uint64_t t2 = pair2(t0, t1);
              sum2[k] = add2(sum2[k], t2);
              if constexpr (FMT == 1) {
                unpair2(mul2(t2, pair2(vs.x, vs.y)), t0, t1);
                if constexpr (kKind > 0) {  // an unseen row's scale may be anything
                  t0 = (see[k] >> (8 * i)) & 1u ? t0 : 0.f;
                  t1 = (see[k] >> (8 * i)) & 2u ? t1 : 0.f;
                }
              }
              pk[h][k >> 1][2 * i + (k & 1)] = pack_bf16(t0, t1);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float a, b2;
          unpair2(sum2[k], a, b2);
          sum[k] = a + b2;
        }
      };
      // To begin with, any reference near the maximum does: that of the first quarters in which every row of the
      // warp sees a key.
      bool none = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) none |= ref[k] == -INFINITY;
      if (__any_sync(0xFFFFFFFFu, none)) {
#pragma unroll 1
        for (int q = 3; q >= 0; --q) {
          float mx[4];
          top_of(q, false, mx);
          none = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // (a row that has a reference keeps it; one without has only zeros so far)
            if (ref[k] == -INFINITY) ref[k] = mx[k];
            none |= ref[k] == -INFINITY;
          }
          if (!__any_sync(0xFFFFFFFFu, none)) break;
        }
      }
      // The p of a group go over the scores of the tile's first half as 16 columns a quarter: over scores that are
      // done, so that the group can be taken again.
#pragma unroll
      for (int q = 0; q < 4; q += C::kGroup) {
        uint32_t pk[C::kGroup][2][8];  // [32 keys][16 pairs][register of the store]
        float sum[4];
        auto compute = [&]() {
          if (kind == 0)
            group(std::integral_constant<int, 0>{}, q, sum, pk);
          else if (kind == 1)
            group(std::integral_constant<int, 1>{}, q, sum, pk);
          else
            group(std::integral_constant<int, 2>{}, q, sum, pk);
        };
        compute();
        const bool much = sum[0] > kMaxSum || sum[1] > kMaxSum || sum[2] > kMaxSum || sum[3] > kMaxSum;
        if (__any_sync(0xFFFFFFFFu, much)) {
          // Replace the references by a power of two, so that everything so far (sums, outputs, p of the quarters
          // before, which are in TMEM) is rescaled exactly, and take the group again.
          float mx[4], alpha[4];
          top_of(q, true, mx);
#pragma unroll 1
          for (int h = 1; h < C::kGroup; ++h) {
            float m2[4];
            top_of(q + h, true, m2);
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], m2[k]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float up = fmaxf(ceilf(mx[k]), 0.f);
            alpha[k] = ex2f(-up);
            ref[k] += up;
            l[k] *= alpha[k];
          }
          if (j > 0) {  // the product with the previous tile is done (s_full)
#pragma unroll 1
            for (int d = 0; d < 2 * D; d += 32) {
              const uint32_t at = t_o + (d >= D ? (16u << 16) + d - D : d);
              const float a0 = d >= D ? alpha[2] : alpha[0], a1 = d >= D ? alpha[3] : alpha[1];
              uint32_t r[16];
              tm_frag_ld(at, r);
              tm_wait_ld(r);
#pragma unroll
              for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * (i & 2 ? a1 : a0));
              tm_frag_st(at, r);
            }
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
#pragma unroll 1
          for (int e = 0; e < 2 * q; ++e) {
            const uint32_t at = t_s + (e & 1 ? 16u << 16 : 0u) + (e >> 1) * 16;
            uint32_t r[8];
            tm_pair_ld(at, r);
            tm_wait_ld(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a = e & 1 ? (i & 1 ? alpha[3] : alpha[2]) : (i & 1 ? alpha[1] : alpha[0]);
              r[i] = pack_bf16(bf16_lo(r[i]) * a, bf16_hi(r[i]) * a);
            }
            tm_pair_st(at, r);
          }
          compute();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) l[k] += sum[k];
#pragma unroll
        for (int h = 0; h < C::kGroup; ++h) {
          tm_pair_st(t_s + (q + h) * 16, pk[h][0]);
          tm_pair_st(t_s + (16u << 16) + (q + h) * 16, pk[h][1]);
        }
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      mbar_arrive(&p_full[x]);
    }
    if (ok && mine > 0) ok = bar_wait_warp(&o_done[x], 0);
    if (ok && x < NX) {
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      // the sums of this lane's own row (pair `lane` of the warp), whose outputs it stores
      float total = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v = l[k];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
        v = __shfl_sync(0xFFFFFFFFu, v, (lane & 7) * 4);
        if ((lane >> 3) == k) total = v;
      }
      const float inv = total == 0.f ? 0.f : 1.f / total;
      // Rows go out through the warp's 32 rows of the Q tile (every product that read it is done), so that a
      // store covers whole rows.
      uint8_t* rows = smem + x * C::kTile;
      const int r0 = (warp & 3) * 32;
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        float t[32];
        if (nt > 0) {
          tm_ld32(t_o + d, t);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) t[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t w[4];
#pragma unroll
          for (int h = 0; h < 4; ++h)
            w[h] = total == 0.f ? 0u : pack_bf16(t[i + 2 * h] * inv, t[i + 2 * h + 1] * inv);
          *chunk_at(rows, r0 + lane, (d + i) / 8) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (boxed && col0 + 32 <= ncol) {  // whole rows of the output, all of them this warp's
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_store3(&map_o, smem_u32(rows) + h * 16384 + r0 * 128, h * 64, hkv * G, sq.r0 + (c0 + col0) / G);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // (shared memory is read, then the CTA may end)
        }
      } else {
        __syncwarp();
        const int64_t at = pair_at(col0 + lane, p.out_stride);
#pragma unroll 4
        for (int it = 0; it < kChunks; ++it) {
          const int r = it * kLines + lane / kChunks, ch = lane % kChunks;
          const uint4 v = *chunk_at(rows, r0 + r, ch);
          uint16_t* dst = static_cast<uint16_t*>(p.out) + from_lane(at, r) + ch * 8;
          if (col0 + r < ncol) {
            if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
              *reinterpret_cast<uint4*>(dst) = v;
            } else {
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                dst[2 * i] = static_cast<uint16_t>(w[i]);
                dst[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
              }
            }
          }
        }
      }
    } else if (!ok && lane == 0) {
      *failed = 1;
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0 && *failed) cache_flag(c, TF_CACHE_TIMEOUT);
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
}

// CTAs of a launch with `span` pairs each (an upper bound: rows are n_rows at most in all).
int64_t prompt_ctas(const CacheAttnParams& p, int span) {
  const int64_t G = p.Hq / p.c.Hkv;
  const int64_t each = ((int64_t)p.c.max_rows * G + span - 1) / span * p.c.n_seq;
  return std::min(each, p.c.n_rows * G / span + p.c.n_seq) * p.c.Hkv;
}
// Pairs of a CTA: 128 while that still is one wave of CTAs (a tile of keys takes 1.40 us with one 128-pair tile and
// 1.54 with two, bf16, D = 128, so two pay once the CTAs queue).
int prompt_span(const CacheAttnParams& p) { return prompt_ctas(p, 128) <= 152 ? 128 : 256; }

// Rows of queries or outputs as boxes of 64 columns x G heads x `rows` rows.
bool rows_map(CUtensorMap* map, const void* base, const CacheAttnParams& p, int64_t stride, int pairs) {
  const int G = p.Hq / p.c.Hkv;
  EncodeTiled fn = encode_fn();
  if (!fn || 32 % G || reinterpret_cast<uintptr_t>(base) % 16 || stride % 8 || stride >= (1ll << 38)) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)p.c.D, (cuuint64_t)p.Hq, (cuuint64_t)p.c.n_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)p.c.D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(pairs / G)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int FMT, int NX>
cudaError_t launch_prompt_x(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p,
                            cudaStream_t s) {
  using C = PromptCfg<D, FMT>;
  static DeviceOnce once;
  cudaError_t e = device_once(once, [] {
    return cudaFuncSetAttribute(k_cache_prompt<D, FMT, NX>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  });
  if (e) return e;
  constexpr int span = 128 * NX;
  const int64_t tiles = ((int64_t)p.c.max_rows * (p.Hq / p.c.Hkv) + span - 1) / span;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
  // queries and outputs by TMA where heads divide a tile's rows and everything is 16-byte aligned
  CUtensorMap mq = {}, mo = {};
  const int boxed = rows_map(&mq, p.q, p, p.q_stride, 128) && rows_map(&mo, p.out, p, p.out_stride, 32) ? 1 : 0;
  k_cache_prompt<D, FMT, NX><<<dim3(static_cast<unsigned>(tiles), p.c.Hkv, p.c.n_seq), C::kThreads, C::kSmem, s>>>(
      mk, mv, mq, mo, p, boxed);
  return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t launch_prompt_t(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p,
                            cudaStream_t s) {
  return prompt_span(p) == 128 ? launch_prompt_x<D, FMT, 1>(mk, mv, p, s) : launch_prompt_x<D, FMT, 2>(mk, mv, p, s);
}

}  // namespace

// Measured with rows that see everything (4-bit and bf16 pages, D = 64 and 128, 512 and 1024 rows, 512 and 4608
// positions before them): start and end of a CTA, and a tile of 128 keys.
float cache_prompt_us(const CacheAttnParams& p) {
  const int span = prompt_span(p);
  const int64_t waves = (prompt_ctas(p, span) + 151) / 152;
  const int64_t rows = std::max<int64_t>(1, span / (p.Hq / p.c.Hkv));
  const int64_t keys = p.window > 0 ? std::min<int64_t>(p.c.max_len, (int64_t)p.window + p.sinks + rows + 64) : p.c.max_len;
  const float start = p.c.fmt ? (p.c.D == 128 ? 7.5f : 6.0f) : (p.c.D == 128 ? 7.0f : 6.4f);
  const float tile = (p.c.fmt ? (p.c.D == 128 ? 2.07f : 1.92f) : (p.c.D == 128 ? 1.54f : 1.23f)) * (span == 128 ? 0.91f : 1.f);
  return static_cast<float>(waves) * (start + tile * static_cast<float>((keys + 127) / 128));
}

cudaError_t launch_cache_prompt(const CacheAttnParams& p, cudaStream_t s) {
  if (p.f32) return cudaErrorInvalidValue;
  CUtensorMap mk = {}, mv = {};
  if (p.c.fmt == 0) {
    const uint64_t rows = (uint64_t)p.c.n_pages * p.c.Hkv * kKvPage;
    if (!make_map(&mk, p.c.K, rows, p.c.D, kKvPage) || !make_map(&mv, p.c.V, rows, p.c.D, kKvPage))
      return cudaErrorInvalidValue;
    return p.c.D == 128 ? launch_prompt_t<128, 0>(mk, mv, p, s) : launch_prompt_t<64, 0>(mk, mv, p, s);
  }
  return p.c.D == 128 ? launch_prompt_t<128, 1>(mk, mv, p, s) : launch_prompt_t<64, 1>(mk, mv, p, s);
}

}  // namespace tf
