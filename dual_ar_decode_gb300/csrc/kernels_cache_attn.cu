// Attention of few rows per sequence over a paged KV cache (sm_103a): the
// decode form of tf_op_attention_cache, for bf16 and 4-bit pages.
//
// out = sum_j p_j v_j with p = softmax_j(scale q.k_j) over the positions a row
// sees (window and sinks).  One row reads every visible K and V row of its KV
// head once and does 4 D flops per (head, position): memory is the bound, so
// the work is laid out to keep HBM busy and to spend few instructions per
// cached element.
//
//   * A group is (sequence, KV head, tile of 8 NT columns); a column is one
//     (row, query head) pair, so all heads of a KV head (and up to 4 rows more)
//     share each K and V read.  A cluster of up to 16 CTAs takes one group and
//     splits its list of pages; the CTAs' partial softmax results meet in
//     distributed shared memory in rank order.  So there is no workspace, no
//     second launch and no atomic, and calls on several streams cannot meet.
//   * Every warp streams its own pages through its own ring of shared-memory
//     stages (bulk copies of a head's contiguous 4-bit page, TMA boxes with the
//     128-byte swizzle for bf16): no CTA barrier inside the loop.
//   * Scores and outputs are computed as S^T = K q^T and O^T = V^T P^T with
//     mma.sync m16n8k16: keys (or head dims) on the 16-row side, columns on the
//     8-wide side.  With 8 columns a tcgen05 tile (M = 128 keys, N = 8) would
//     need its operands in shared memory in its own layout, i.e. one more trip
//     of the dequantised elements; here they go from the conversion's registers
//     into the product.  The tensor pipe is at half load at most.
//   * 4-bit elements: e2m1 x e4m3 has at most 6 significant bits and is exact in
//     f16 (values 2^-10 .. 2688), so a page costs one conversion and one multiply
//     per two elements, and row scales are applied to scores and probabilities
//     in float32.  Queries are scaled by a power of two into f16's range and
//     split in f16 hi + lo (22 bits); the probability times V's row scale is
//     split the same way against a running reference (see below).  bf16 pages:
//     three bf16 parts (24 bits) for float32 rows.
//   * The reference that a column's weights are relative to is replaced only when
//     they grow past a bound, which one vote per page finds: in the steady state a
//     page needs no shuffles.
// Measured (GB300, 32 query and 8 KV heads of 128): 32 ragged 4-bit streams of up to
// 32768 positions, bf16 rows, 100 us (6.3 TB/s; 530 warp instructions per head
// page, issue slots and HBM are both near their end); 32 bf16 streams with a
// window of 2048, float32 rows, 40 us (5.7 TB/s); 32 x 8192 bf16 positions 163 us
// (6.6 TB/s, memory); one 4-bit sequence of 4096 positions 8.2 us (latency).
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

constexpr int kSortMax = 256;  // sequences that a CTA puts in order of length
// The weights of a column are 2^(score - ref).  bf16 pages: ref is a maximum, replaced when a score exceeds it by
// more than kGrow (log2).  4-bit pages: the weights times V's row scales are multiplied in f16 parts, so ref puts the
// largest such product at 2^kRefBits when it is set and is replaced when one exceeds 2^kRefTop; it is no further than
// kRefMost below the largest score, so that the weights themselves stay far from overflow (V rows below 1e-24 lose
// bits to that).
constexpr float kGrow = 8.0f, kRefBits = 7.0f, kRefTop = 15.0f, kRefMost = 100.0f;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pair2(float a, float b) {  // two floats, one operand of the packed instructions
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
__device__ __forceinline__ float lg2f(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bounded wait that only reports (the caller decides what to do).
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kWaitBudgetNs) return false;
  return true;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

template <int FMT>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (FMT == 0)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Four bytes of e2m1 pairs -> four f16x2 (low nibble in the low half).
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
__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// (x, y) -> NP parts of 16 bits each whose sum is the pair: part 0 is the
// rounded value, the next the rounded remainder, ...; f16 (FMT 1) or bf16.
template <int FMT, int NP>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&part)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    uint32_t h;
    if constexpr (FMT == 0)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
    else
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
    part[i] = h;
    if (i + 1 < NP) {
      if constexpr (FMT == 0) {
        x -= bf16_lo(h);
        y -= bf16_hi(h);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x -= f.x;
        y -= f.y;
      }
    }
  }
}

// Shared memory and shape of one instantiation.
template <int D, int FMT, int NT, int F32, int W>
struct DecCfg {
  static constexpr int kWarps = W;
  static constexpr int kThreads = 32 * W;
  static constexpr int kPerSm = FMT ? 16 / W : 8 / W;      // CTAs an SM (registers and shared memory allow them)
  static constexpr int kKeys = FMT ? 32 : 16;               // positions of a stage (a page, or half a page)
  static constexpr int kHalf = FMT ? Kv4<D>::kBytes : 16 * D * 2;  // K (or V) bytes of a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = FMT ? 2 : (D == 64 ? 4 : NT == 3 ? 2 : 3);
  static constexpr int kQp = FMT ? (F32 ? 2 : 1) : (F32 ? 3 : 1);  // parts of a query
  static constexpr int kPp = FMT ? (F32 ? 2 : 1) : (F32 ? 3 : 2);  // parts of a probability
  static constexpr int kSteps = D / 16;
  static constexpr int kCols = 8 * NT;
  // A warp's partial outputs.  FMT 0: [col][kLd]; FMT 1: float2 (two dims of a lane) [n-tile][16-row tile]
  // [kPair: col * 10 + lane group]; both strides keep the stores and the reads free of bank conflicts.
  static constexpr int kLd = D + 4, kPair = 82;
  static constexpr int kPartFloats = FMT ? NT * kSteps * kPair * 2 : kCols * kLd;
  static constexpr int kMaxRanks = 16;
  static constexpr size_t kRing = (size_t)kWarps * kStages * kStage;
  static constexpr size_t kParts = (size_t)kWarps * kPartFloats * 4;  // overlays the ring at the end
  static constexpr size_t kOffQ = ((kRing > kParts ? kRing : kParts) + 127) / 128 * 128;
  // what the cluster's ranks send to this CTA: [rank][its share of the outputs], [rank][col] maxima and sums
  static constexpr size_t kOffC = kOffQ + (size_t)NT * kQp * kSteps * 32 * 8;
  static constexpr size_t kOffStat = kOffC + (size_t)(kCols * D / 4 + kMaxRanks) * 16 + 2 * kMaxRanks * kCols * 4;
  // per warp and column: reference, sum; per column: the queries' scale
  static constexpr size_t kOffBar = kOffStat + (size_t)(2 * kWarps + 1) * kCols * 4;
  static constexpr size_t kSmem = 1024 + kOffBar + kWarps * kStages * 8 + 16;
};

struct TileRows {
  int r0, n, len;     // the sequence's rows and length
  int c0, nc;         // the tile's first column and how many it has
};

template <int D, int FMT, int NT, int F32, int W>
__global__ void __launch_bounds__(32 * W, DecCfg<D, FMT, NT, F32, W>::kPerSm)
    k_cache_decode(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const CacheAttnParams p, const int csize, const int sorted) {
  using C = DecCfg<D, FMT, NT, F32, W>;
  constexpr int KB = C::kKeys / 8;   // blocks of 8 keys in a stage
  constexpr int MT = D / 16;         // 16-row tiles of the head dimension
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const CacheBatch& c = p.c;
  // (the shuffle: a value that the compiler knows to be the warp's, so what follows from it takes no registers of the
  // lanes'; 32 ragged 4-bit streams 106 us without it, 100 with it)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int lg = lane >> 2, lt = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % csize, tile = static_cast<int>(blockIdx.x) / csize;
  const int hkv = blockIdx.y;
  const int G = p.Hq / c.Hkv;
  // Ragged batches of more CTAs than fit at once: the longest sequences first, so that the last CTAs to
  // start are short ones.
  int b = blockIdx.z;
  SeqRows sq;
  if (sorted) {
    __shared__ int lens[kSortMax], starts[kSortMax + 1], chosen;
    const int n = c.n_seq;
    for (int t = threadIdx.x; t < n; t += C::kThreads) {
      lens[t] = __ldg(c.len + t);
      starts[t] = c.row_start ? __ldg(c.row_start + t) : t;
    }
    if (threadIdx.x == 0) starts[n] = c.row_start ? __ldg(c.row_start + n) : n;
    __syncthreads();
    for (int t = threadIdx.x; t < n; t += C::kThreads) {
      int r = 0;
      const int mine = lens[t];
      for (int i = 0; i < n; ++i) r += (lens[i] > mine || (lens[i] == mine && i < t)) ? 1 : 0;
      if (r == b) chosen = t;
    }
    __syncthreads();
    b = chosen;
    sq = cache_rows(c, starts[b], starts[b + 1], lens[b]);
  } else {
    sq = cache_seq(c, b);
  }
  const int c0 = tile * C::kCols;
  const int ncol = min(C::kCols, sq.n * G - c0);
  if (ncol <= 0) return;  // the whole cluster
  // (waited for before the first store to a peer's shared memory: it must have started)
  if (csize > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int first = sq.len - sq.n;                       // position of the sequence's row 0
  const int posmin = first + c0 / G, posmax = first + (c0 + ncol - 1) / G;
  const bool win = p.window > 0;
  const int lowmin = win ? max(0, posmin - p.window + 1) : 0;
  const int lowmax = win ? max(0, posmax - p.window + 1) : 0;
  const int sinks = win ? p.sinks : 0;

  // The list of stages: those of the sinks that the windows do not reach, then lowmin .. posmax.
  const int ulow = lowmin / C::kKeys;
  const int usink = min(ulow, (min(sinks, lowmin) + C::kKeys - 1) / C::kKeys);
  const int units = posmax < 0 ? 0 : usink + posmax / C::kKeys - ulow + 1;

  float* gpart = reinterpret_cast<float*>(smem + C::kOffC);      // from the ranks
  float* gmax = gpart + C::kCols * D + 4 * C::kMaxRanks;        // [rank][col]
  float* gsum = gmax + C::kMaxRanks * C::kCols;
  float* wmax = reinterpret_cast<float*>(smem + C::kOffStat);   // [warp][col]: references
  float* wsum = wmax + C::kWarps * C::kCols;
  float* qscale = wsum + C::kWarps * C::kCols;                  // [col]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * C::kStages;
  uint8_t* ring = smem + (size_t)warp * C::kStages * C::kStage;

  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  __syncwarp();

  // ---- this warp's stages: gw, gw + nw, ...
  const int gw = rank * C::kWarps + warp, nw = csize * C::kWarps;
  const int mine = gw < units ? (units - gw + nw - 1) / nw : 0;
  auto unit_at = [&](int i) {
    const int u = gw + i * nw;
    return u < usink ? u : ulow + u - usink;
  };
  // page ids of up to 32 stages ahead, one per lane
  int ids = -1;
  auto look_up = [&](int from) {
    const int i = from + lane;
    ids = i < mine ? cache_page(c, b, unit_at(i) / (kKvPage / C::kKeys)) : -1;
  };
  look_up(0);
  // the queries' loads go out behind the table's; they are used after the stages have been asked for
  constexpr int QC = C::kCols / C::kWarps;  // columns a warp prepares: warp, warp + kWarps, ...
  float xq[QC][D / 32];                     // dims lane, lane + 32, ...
#pragma unroll
  for (int n = 0; n < QC; ++n) {
    const int col = n * C::kWarps + warp, cc = c0 + col, row = cc / G, h = hkv * G + cc % G;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      xq[n][e] = 0.f;
      if (col < ncol) {
        const size_t o = (size_t)(sq.r0 + row) * p.q_stride + (size_t)h * D + lane + 32 * e;
        xq[n][e] = F32 ? static_cast<const float*>(p.q)[o] : bf16_to_f32(static_cast<const uint16_t*>(p.q)[o]);
      }
    }
  }
  auto issue = [&](int i) {  // all lanes; stage i of this warp into ring slot i % kStages
    if (i && (i & 31) == 0) look_up(i);
    const int page = __shfl_sync(0xFFFFFFFFu, ids, i & 31);
    if (lane == 0) {
      const int s = i % C::kStages;
      const uint32_t dst = smem_u32(ring + (size_t)s * C::kStage);
      if (page < 0) {
        mbar_arrive(&bars[s]);  // nothing to wait for; the stage is skipped
      } else if constexpr (FMT == 1) {
        const size_t off = ((size_t)page * c.Hkv + hkv) * C::kHalf;
        mbar_arrive_expect_tx(&bars[s], C::kStage);
        bulk_load(dst, c.K + off, C::kHalf, &bars[s]);
        bulk_load(dst + C::kHalf, c.V + off, C::kHalf, &bars[s]);
      } else {
        const int y = (page * c.Hkv + hkv) * kKvPage + (unit_at(i) % (kKvPage / C::kKeys)) * C::kKeys;
        mbar_arrive_expect_tx(&bars[s], C::kStage);
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          tma_box(dst + x * (16 * 128), &map_k, x * 64, y, &bars[s]);
          tma_box(dst + C::kHalf + x * (16 * 128), &map_v, x * 64, y, &bars[s]);
        }
      }
    }
    return page;
  };
  uint32_t good = 0;  // bit s: slot s holds a page of the pool
  for (int i = 0; i < min(mine, C::kStages); ++i) good |= (issue(i) >= 0 ? 1u : 0u) << (i % C::kStages);

  // ---- queries: the parts of every column in the order the products read them.  A column's queries are
  // scaled by a power of two so that the largest is in [2^14, 2^15) (FMT 1: f16 holds them).
#pragma unroll
  for (int n = 0; n < QC; ++n) {
    const int col = n * C::kWarps + warp;
    const float(&x)[D / 32] = xq[n];
    float up = 1.f;
    if constexpr (FMT == 1) {
      float am = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) am = fmaxf(am, fabsf(x[e]));
      am = warp_max(am);
      const int ex = static_cast<int>(__float_as_uint(am) >> 23) - 127;  // floor(log2 am); -127: zero or tiny
      const int sh = min(126, max(-126, 14 - ex));
      up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
      if (lane == 0) qscale[col] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
    } else if (lane == 0) {
      qscale[col] = p.scale_log2;
    }
    uint16_t* qf = reinterpret_cast<uint16_t*>(smem + C::kOffQ);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const int d = lane + 32 * e;
      // place of element d in the products: step s, lane quarter t, half (b0 / b1), low or high
      int s, t, hf, lo;
      if constexpr (FMT == 1) {
        constexpr int per = D / 4;  // a lane's elements of a row are consecutive
        t = d / per;
        s = d % per / 4;
        hf = d % 4 / 2;
        lo = d % 2;
      } else {
        s = d / 16;
        hf = d % 16 / 8;
        t = d % 8 / 2;
        lo = d % 2;
      }
      uint32_t part[C::kQp];
      split_pair<FMT, C::kQp>(x[e] * up, 0.f, part);
#pragma unroll
      for (int q = 0; q < C::kQp; ++q)
        qf[((((size_t)(col / 8) * C::kQp + q) * C::kSteps + s) * 32 + (col % 8) * 4 + t) * 4 + hf * 2 + lo] =
            static_cast<uint16_t>(part[q]);
    }
  }
  __syncthreads();
  const uint2* qf = reinterpret_cast<const uint2*>(smem + C::kOffQ) + lane;

  // ---- this lane's columns 2 lt, 2 lt + 1 of every n-tile
  int pos[NT][2], low[NT][2];
  float cs[NT][2], ref[NT][2], l[NT][2];
  float o[NT][MT][4];
  bool unset = true;  // some column of this lane has no reference yet
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = n * 8 + 2 * lt + e;
      pos[n][e] = col < ncol ? first + (c0 + col) / G : posmax;  // (a column that is not there sees what the last does)
      low[n][e] = win ? max(0, pos[n][e] - p.window + 1) : 0;
      cs[n][e] = qscale[col];
      ref[n][e] = -INFINITY;
      l[n][e] = 0.f;
    }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;

  bool ok = true;
  for (int it = 0; it < mine; ++it) {
    const int slot = it % C::kStages;
    if (!__all_sync(0xFFFFFFFFu, bar_wait(&bars[slot], (it / C::kStages) & 1) ? 1 : 0)) {
      ok = false;
      // let the copies still in flight land before the ring is reused
      for (int j = it; j < min(mine, it + C::kStages); ++j)
        if (!bar_wait(&bars[j % C::kStages], (j / C::kStages) & 1)) break;
      break;
    }
    const bool have = (good >> slot) & 1u;
    const int j0 = unit_at(it) * C::kKeys;
    const uint8_t* Ks = ring + (size_t)slot * C::kStage;
    const uint8_t* Vs = Ks + C::kHalf;
    if (have) {
      // ---- scores: S[key][col]; block bt: keys key_of(bt)
      // float32 rows: the tensor core truncates when it adds to its accumulator, so long chains drift.  The
      // leading parts of even and odd steps and the small parts have accumulators of their own, added once.
      constexpr int kAcc = F32 ? 3 : 1;
      float sc[NT][KB / 2][4], sx[NT][KB / 2][kAcc][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < KB / 2; ++i)
#pragma unroll
          for (int a = 0; a < kAcc; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) sx[n][i][a][e] = 0.f;
      auto acc_of = [](int q, int step) { return F32 ? (q > 0 ? 2 : step & 1) : 0; };
      // position in the page of this lane's key of block bt
      auto key_of = [&](int bt) { return FMT ? 8 * (lg >> 1) + 2 * bt + (lg & 1) : 8 * bt + lg; };
      if constexpr (FMT == 1) {
        uint32_t kw[KB][D / 32], ks[KB];
#pragma unroll
        for (int bt = 0; bt < KB; ++bt) {
          const int r = key_of(bt);
          if constexpr (D == 128) {
            *reinterpret_cast<uint4*>(kw[bt]) = *reinterpret_cast<const uint4*>(Ks + r * 64 + lt * 16);
            ks[bt] = e4m3x2_f16(*reinterpret_cast<const uint16_t*>(Ks + Kv4<D>::kCodes + r * 8 + 2 * lt));
          } else {
            *reinterpret_cast<uint2*>(kw[bt]) = *reinterpret_cast<const uint2*>(Ks + r * 32 + lt * 8);
            ks[bt] = e4m3x2_f16(Ks[Kv4<D>::kCodes + r * 4 + lt]);
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t a[KB][4];
#pragma unroll
          for (int bt = 0; bt < KB; ++bt) {
            const uint32_t s2 = __byte_perm(ks[bt], 0, w < 2 ? 0x1010 : 0x3232);
            e2m1x8(kw[bt][w], a[bt]);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[bt][i] = hmul2u(a[bt][i], s2);
          }
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int q = 0; q < C::kQp; ++q) {
                const uint2 bq = qf[((n * C::kQp + q) * C::kSteps + 2 * w + st) * 32];
#pragma unroll
                for (int i = 0; i < KB / 2; ++i)
                  mma16816<1>(sx[n][i][acc_of(q, st)], a[2 * i][2 * st], a[2 * i + 1][2 * st], a[2 * i][2 * st + 1],
                              a[2 * i + 1][2 * st + 1], bq.x, bq.y);
              }
        }
      } else {
        const uint32_t kb = smem_u32(Ks);
        const int r = (lane & 7) + ((lane >> 3) & 1) * 8, ch = lane >> 4;
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
          uint32_t a[4];
          const int cc = 2 * s + ch;
          ldsm4(a, kb + (cc >> 3) * (16 * 128) + r * 128 + (((cc & 7) ^ (r & 7)) << 4));
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int q = 0; q < C::kQp; ++q) {
              const uint2 bq = qf[((n * C::kQp + q) * C::kSteps + s) * 32];
              mma16816<0>(sx[n][0][acc_of(q, s)], a[0], a[1], a[2], a[3], bq.x, bq.y);
            }
        }
      }

#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < KB / 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[n][i][e] = F32 ? (sx[n][i][0][e] + sx[n][i][kAcc > 1 ? 1 : 0][e]) + sx[n][i][kAcc - 1][e]
                              : sx[n][i][0][e];

      // Does every column see every key of the stage?  Else: mask, and keep what no column sees (and
      // infinities and NaN that only some see) out of the second product.
      const int j1 = j0 + C::kKeys - 1;
      const bool whole = j1 <= posmin && (j0 >= lowmax || j1 < sinks);
      uint32_t dead = 0, poison = 0;  // bits: positions of the stage
      if (!whole) {
        const int j = j0 + (lane & (C::kKeys - 1));
        const bool any = j <= posmax && (j >= lowmin || j < sinks);
        dead = __ballot_sync(0xFFFFFFFFu, !any);
        if constexpr (FMT == 1) {
          const int blk = D == 128 ? lg : lg >> 1;
          const uint2 w = *reinterpret_cast<const uint2*>(Vs + Kv4<D>::kCodes + blk * kKvPage + 8 * lt);
          uint32_t bad = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) bad |= ((((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0x7Fu) == 0x7Fu ? 1u : 0u) << i;
          poison = __reduce_or_sync(0xFFFFFFFFu, bad << (8 * lt)) & ~dead;
        } else {
          uint32_t bad = 0;
          const uint32_t vb = smem_u32(Vs);
          const int r = (lane & 7) + ((lane >> 4) & 1) * 8, ch = (lane >> 3) & 1;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            uint32_t a[4];
            const int cc = 2 * i + ch;
            ldsm4t(a, vb + (cc >> 3) * (16 * 128) + r * 128 + (((cc & 7) ^ (r & 7)) << 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = (e >> 1) * 8 + 2 * lt;
              bad |= ((a[e] & 0x7F80u) == 0x7F80u ? 1u : 0u) << k;
              bad |= ((a[e] & 0x7F800000u) == 0x7F800000u ? 2u : 0u) << k;
            }
          }
          poison = __reduce_or_sync(0xFFFFFFFFu, bad) & ~dead;
        }
        dead |= poison;
      }

      // ---- softmax: weights 2^(score - ref), times V's row scale (4-bit pages)
      float z[NT][KB][2];
      // false, and nothing changed: a reference has to be replaced first (asked only where `checked`)
      auto weights = [&](auto mask_, bool checked) -> bool {
        constexpr bool kMask = decltype(mask_)::value;
        bool again = false;
        uint64_t sum2[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint64_t cs2 = pair2(cs[n][0], cs[n][1]);
          const uint64_t nref2 = pair2(ref[n][0] == -INFINITY ? 0.f : -ref[n][0], ref[n][1] == -INFINITY ? 0.f : -ref[n][1]);
          sum2[n] = pair2(l[n][0], l[n][1]);
          float top[2] = {0.f, 0.f};
#pragma unroll
          for (int bt = 0; bt < KB; ++bt) {
            const uint64_t s2 = pair2(sc[n][bt >> 1][(bt & 1) * 2], sc[n][bt >> 1][(bt & 1) * 2 + 1]);
            float vs = 1.f, t[2], w[2];
            if constexpr (FMT == 1) {  // the queries' scale first: it undoes what scaled them up
              const float ks = reinterpret_cast<const float*>(Ks + Kv4<D>::kRows)[key_of(bt)];
              vs = reinterpret_cast<const float*>(Vs + Kv4<D>::kRows)[key_of(bt)];
              unpair2(fma2(mul2(s2, cs2), pair2(ks, ks), nref2), t[0], t[1]);
            } else {
              unpair2(fma2(s2, cs2, nref2), t[0], t[1]);
            }
            bool on[2] = {true, true};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if constexpr (kMask) {
                const int j = j0 + key_of(bt);
                on[e] = j <= pos[n][e] && (j >= low[n][e] || j < sinks);
                t[e] = on[e] ? t[e] : -INFINITY;
              }
              if constexpr (FMT == 0) again |= t[e] > kGrow;
              w[e] = ex2f(t[e]);
              if constexpr (kMask) {
                if (((poison >> key_of(bt)) & 1u) && on[e]) w[e] = __int_as_float(0x7FFFFFFF);
              }
            }
            const uint64_t w2 = pair2(w[0], w[1]);
            sum2[n] = add2(sum2[n], w2);
            unpair2(FMT ? mul2(w2, pair2(vs, vs)) : w2, z[n][bt][0], z[n][bt][1]);
            if constexpr (FMT == 1) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if constexpr (kMask) z[n][bt][e] = on[e] ? z[n][bt][e] : 0.f;  // an unseen row's scale may be anything
                top[e] = fmaxf(top[e], z[n][bt][e]);
              }
            }
          }
          if constexpr (FMT == 1) {
            float a, b2;
            unpair2(sum2[n], a, b2);
            again |= fmaxf(top[0], top[1]) > 32768.f || fmaxf(a, b2) > 1.32922800e36f;  // 2^kRefTop, 2^120
          }
        }
        if (checked && __any_sync(0xFFFFFFFFu, again)) return false;
#pragma unroll
        for (int n = 0; n < NT; ++n) unpair2(sum2[n], l[n][0], l[n][1]);
        return true;
      };
      auto replace_refs = [&]() {
        unset = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = -INFINITY, mw = -INFINITY;  // largest score, largest score times V's row scale (log2)
#pragma unroll
            for (int bt = 0; bt < KB; ++bt) {
              const int j = j0 + key_of(bt);
              float t = sc[n][bt >> 1][(bt & 1) * 2 + e] * cs[n][e];
              if constexpr (FMT == 1) t *= reinterpret_cast<const float*>(Ks + Kv4<D>::kRows)[key_of(bt)];
              if (whole || (j <= pos[n][e] && (j >= low[n][e] || j < sinks))) {
                mx = fmaxf(mx, t);
                if constexpr (FMT == 1)
                  mw = fmaxf(mw, t + lg2f(reinterpret_cast<const float*>(Vs + Kv4<D>::kRows)[key_of(bt)]));
              }
            }
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
              mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, s));
              if constexpr (FMT == 1) mw = fmaxf(mw, __shfl_xor_sync(0xFFFFFFFFu, mw, s));
            }
            const float r = FMT ? fmaxf(mw - kRefBits, mx - kRefMost) : mx;
            if (r > (ref[n][e] == -INFINITY ? ref[n][e] : ref[n][e] + (FMT ? kRefTop - kRefBits : kGrow))) {
              const float f = ref[n][e] == -INFINITY ? 0.f : ex2f(ref[n][e] - r);
              ref[n][e] = r;
              l[n][e] *= f;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[n][i][e] *= f;
                o[n][i][2 + e] *= f;
              }
            }
            unset |= ref[n][e] == -INFINITY;
          }
      };
      // FMT 1: each weight's f16 parts are off by 2^-23 of it (two parts) or by 2^-25, half of f16's smallest step,
      // i.e. 2^-32 of the largest weight.
      auto soft = [&](auto mask_) {
        const bool start = __any_sync(0xFFFFFFFFu, unset);  // no reference yet: nothing to try first
        if (start || !weights(mask_, true)) {
          replace_refs();
          weights(mask_, false);
        }
      };
      if (whole)
        soft(std::integral_constant<bool, false>{});
      else
        soft(std::integral_constant<bool, true>{});
      // ---- probabilities as the second product's column operand: block bt holds (key, column) pairs as the
      // first product left them; the transpose gives (column, key pair)
      uint32_t pb[NT][C::kPp][KB];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int bt = 0; bt < KB; ++bt) {
          uint32_t part[C::kPp];
          if constexpr (FMT == 1)
            split_pair<1, C::kPp>(z[n][bt][0], z[n][bt][1], part);
          else
            split_pair<0, C::kPp>(z[n][bt][0], z[n][bt][1], part);
#pragma unroll
          for (int q = 0; q < C::kPp; ++q) pb[n][q][bt] = movmatrix(part[q]);
        }
      // ---- O^T += V^T P^T (float32 rows: a stage's products from zero, small parts first, then one rounded
      // addition)
      if constexpr (FMT == 1) {
        uint32_t vw[KB][D / 32], vs[KB];
        const int blk = D == 128 ? lg : lg >> 1;
        uint2 w8 = *reinterpret_cast<const uint2*>(Vs + Kv4<D>::kCodes + blk * kKvPage + 8 * lt);
        if (dead) {  // zero the scales of positions that must not enter
          const uint32_t d8 = dead >> (8 * lt);
          uint32_t keep[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i) keep[i >> 2] |= ((d8 >> i) & 1u ? 0u : 0xFFu) << (8 * (i & 3));
          w8.x &= keep[0];
          w8.y &= keep[1];
        }
        vs[0] = e4m3x2_f16(w8.x & 0xFFFFu);
        vs[1] = e4m3x2_f16(w8.x >> 16);
        vs[2] = e4m3x2_f16(w8.y & 0xFFFFu);
        vs[3] = e4m3x2_f16(w8.y >> 16);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if constexpr (D == 128)
            *reinterpret_cast<uint4*>(vw[j]) = *reinterpret_cast<const uint4*>(Vs + j * 512 + lane * 16);
          else
            *reinterpret_cast<uint2*>(vw[j]) =
                *reinterpret_cast<const uint2*>(Vs + j * 256 + (lg >> 1) * 64 + lt * 16 + (lg & 1) * 8);
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t a[KB][4];
#pragma unroll
          for (int j = 0; j < KB; ++j) {
            e2m1x8(vw[j][w], a[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[j][i] = hmul2u(a[j][i], vs[j]);
          }
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int n = 0; n < NT; ++n)
            {
              float t[4] = {0.f, 0.f, 0.f, 0.f};
              float(&to)[4] = F32 ? t : o[n][2 * w + st];
#pragma unroll
              for (int q = C::kPp - 1; q >= 0; --q)
#pragma unroll
                for (int i = 0; i < KB / 2; ++i)
                  mma16816<1>(to, a[2 * i][2 * st], a[2 * i][2 * st + 1], a[2 * i + 1][2 * st],
                              a[2 * i + 1][2 * st + 1], pb[n][q][2 * i], pb[n][q][2 * i + 1]);
              if constexpr (F32) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][2 * w + st][e] += t[e];
              }
            }
        }
      } else {
        const uint32_t vb = smem_u32(Vs);
        const int r = (lane & 7) + ((lane >> 4) & 1) * 8, ch = (lane >> 3) & 1;
        const uint32_t dl = dead >> (2 * lt);
        const uint32_t keep0 = ((dl & 1u) ? 0u : 0xFFFFu) | ((dl & 2u) ? 0u : 0xFFFF0000u);
        const uint32_t keep1 = ((dl & 0x100u) ? 0u : 0xFFFFu) | ((dl & 0x200u) ? 0u : 0xFFFF0000u);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          uint32_t a[4];
          const int cc = 2 * i + ch;
          ldsm4t(a, vb + (cc >> 3) * (16 * 128) + r * 128 + (((cc & 7) ^ (r & 7)) << 4));
          if (dead) {
            a[0] &= keep0;
            a[1] &= keep0;
            a[2] &= keep1;
            a[3] &= keep1;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            float(&to)[4] = F32 ? t : o[n][i];
#pragma unroll
            for (int q = C::kPp - 1; q >= 0; --q)
              mma16816<0>(to, a[0], a[1], a[2], a[3], pb[n][q][0], pb[n][q][1]);
            if constexpr (F32) {
#pragma unroll
              for (int e = 0; e < 4; ++e) o[n][i][e] += t[e];
            }
          }
        }
      }
    }
    __syncwarp();
    if (it + C::kStages < mine) {
      const int pg = issue(it + C::kStages);
      good = (good & ~(1u << slot)) | ((pg >= 0 ? 1u : 0u) << slot);
    }
  }
  if (!ok && lane == 0) cache_flag(c, TF_CACHE_TIMEOUT);

  // ---- the warps' partials meet in shared memory (over the ring: every copy has landed and been read)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int s = 4; s < 32; s <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], s);
  __syncthreads();
  float* wpart = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = n * 8 + 2 * lt + e;
      float* wp = wpart + (size_t)warp * C::kPartFloats;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if constexpr (FMT == 1) {
          reinterpret_cast<float2*>(wp)[(n * MT + i) * C::kPair + (2 * lt + e) * 10 + lg] =
              make_float2(o[n][i][e], o[n][i][2 + e]);
        } else {
          wp[col * C::kLd + 16 * i + lg] = o[n][i][e];
          wp[col * C::kLd + 16 * i + 8 + lg] = o[n][i][2 + e];
        }
      }
      if (lg == 0) {
        wmax[warp * C::kCols + col] = ref[n][e];
        wsum[warp * C::kCols + col] = l[n][e];
      }
    }
  __syncthreads();
  auto peer = [&](const void* a, int r) {
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(a)), "r"(r));
    return ra;
  };
  if (csize > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  // The CTA's maximum and sum of every column, to every rank.
  for (int e = threadIdx.x; e < csize * C::kCols; e += C::kThreads) {
    const int col = e % C::kCols, r = e / C::kCols;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, wmax[w * C::kCols + col]);
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      const float mw = wmax[w * C::kCols + col], lw = wsum[w * C::kCols + col];
      L += mw == -INFINITY ? lw : lw * ex2f(mw - M);  // lw: 0, or NaN
    }
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer(gmax + rank * C::kCols + col, r)), "f"(M) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer(gsum + rank * C::kCols + col, r)), "f"(L) : "memory");
  }
  // The CTA's outputs, 4 dims of a column each, to the rank that finishes them.
  const int quads = ncol * (D / 4), share = (quads + csize - 1) / csize;
  for (int e = threadIdx.x; e < quads; e += C::kThreads) {
    const int col = e / (D / 4), d = e % (D / 4) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, wmax[w * C::kCols + col]);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      const float rw = wmax[w * C::kCols + col];
      const float f = rw == -INFINITY ? 0.f : ex2f(rw - M);
      const float* wp = wpart + (size_t)w * C::kPartFloats;
      float4 v;
      if constexpr (FMT == 1) {
        const float2* w2 = reinterpret_cast<const float2*>(wp) +
                           ((col / 8) * MT + d % (D / 8) / 2) * C::kPair + (col % 8) * 10 + d / (D / 8);
        const float2 v0 = w2[0], v1 = w2[C::kPair];
        v = make_float4(v0.x, v0.y, v1.x, v1.y);
      } else {
        v = *reinterpret_cast<const float4*>(wp + col * C::kLd + d);
      }
      if (f != 0.f) {  // else what is there may be anything
        s.x = fmaf(v.x, f, s.x);
        s.y = fmaf(v.y, f, s.y);
        s.z = fmaf(v.z, f, s.z);
        s.w = fmaf(v.w, f, s.w);
      }
    }
    const int r = e / share;
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                     peer(gpart + (size_t)(rank * share + e - r * share) * 4, r)),
                 "f"(s.x), "f"(s.y), "f"(s.z), "f"(s.w)
                 : "memory");
  }
  if (csize > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
  // ---- this rank's share of the outputs, the ranks added in order
  for (int e = rank * share + threadIdx.x; e < min(quads, (rank + 1) * share); e += C::kThreads) {
    const int col = e / (D / 4), d = e % (D / 4) * 4;
    float M = -INFINITY, L = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = 0; r < csize; ++r) M = fmaxf(M, gmax[r * C::kCols + col]);
    for (int r = 0; r < csize; ++r) {
      const float mr = gmax[r * C::kCols + col], lr = gsum[r * C::kCols + col];
      const float4 v = *reinterpret_cast<const float4*>(gpart + (size_t)(r * share + e - rank * share) * 4);
      const float f = mr == -INFINITY ? 0.f : ex2f(mr - M);
      L += mr == -INFINITY ? lr : lr * f;  // lr: 0, or NaN
      y[0] = fmaf(v.x, f, y[0]);
      y[1] = fmaf(v.y, f, y[1]);
      y[2] = fmaf(v.z, f, y[2]);
      y[3] = fmaf(v.w, f, y[3]);
    }
    const float inv = 1.f / L;
    const int cc = c0 + col;
    const size_t oo = (size_t)(sq.r0 + cc / G) * p.out_stride + (size_t)(hkv * G + cc % G) * D + d;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = L == 0.f ? 0.f : y[i] * inv;
    if constexpr (F32) {
      float* o4 = static_cast<float*>(p.out) + oo;
      if ((reinterpret_cast<uintptr_t>(o4) & 15) == 0)
        *reinterpret_cast<float4*>(o4) = make_float4(y[0], y[1], y[2], y[3]);
      else
        for (int i = 0; i < 4; ++i) o4[i] = y[i];
    } else {
      uint16_t* o4 = static_cast<uint16_t*>(p.out) + oo;
      uint16_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16(y[i]);
      if ((reinterpret_cast<uintptr_t>(o4) & 7) == 0)
        *reinterpret_cast<uint2*>(o4) = make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
      else
        for (int i = 0; i < 4; ++i) o4[i] = w[i];
    }
  }
}

// How a launch is cut.
struct DecPlan {
  int64_t groups;  // (sequence, KV head, tile of columns): an upper bound, rows are n_rows at most in all
  int64_t units;   // stages of the longest group
  int cs;          // CTAs per group
};
// Columns of a tile, in eights.  bf16 pages: as many as fit the registers share a read (16 sequences x 5 rows x 4
// heads: 27 us with 24 columns, 32 with 8).  4-bit pages: 8; more would leave one CTA an SM, and the products'
// latency shows (22 us with 8, 28 with 24).
int decode_nt(const CacheAttnParams& p) {
  const int64_t cols = (int64_t)p.c.max_rows * (p.Hq / p.c.Hkv);
  return p.c.fmt || cols <= 8 ? 1 : cols <= 16 ? 2 : 3;
}
// Warps of a CTA.  bf16 pages, 8 columns: 4, two CTAs an SM, which fills the SMs more evenly (32 windowed streams
// 51 -> 44 us); wider tiles: 8 (16 x 5 rows: 27 us, 37 with 4).  4-bit pages: 8, two CTAs an SM (four CTAs of 4
// warps: 132 -> 134 us for 32 ragged streams, 9.6 -> 11.5 us for one).
constexpr int decode_warps(int fmt, int nt) { return fmt == 0 && nt == 1 ? 4 : 8; }
DecPlan decode_plan(const CacheAttnParams& p, int nt, int keys_per_stage, int warps) {
  const int64_t G = p.Hq / p.c.Hkv, cols = 8 * nt;
  const int64_t keys = p.window > 0 ? std::min<int64_t>(p.c.max_len, (int64_t)p.window + p.sinks + 8) : p.c.max_len;
  DecPlan d;
  d.groups = std::min(((int64_t)p.c.max_rows * G + cols - 1) / cols * p.c.n_seq, p.c.n_rows * G / cols + p.c.n_seq) *
             p.c.Hkv;
  d.units = (keys + keys_per_stage - 1) / keys_per_stage;
  // Enough CTAs to fill the SMs (4-bit: two each), as long as a warp still gets a stage (measured: one more doubling
  // costs 5-30%, one less leaves SMs idle).  16, beyond the portable cluster size, starts slowly and pays only for
  // one long sequence (131072 positions, 8 KV heads: 101 -> 79 us; 4096 positions: 8.9 -> 11 us).
  const int slots = (p.c.fmt ? 16 : 8) / warps * 152;
  d.cs = 1;
  // (bf16: one CTA an SM, so a doubling that starts a second wave gains nothing)
  auto more = [&](int64_t ctas) { return p.c.fmt ? ctas < slots : ctas * 2 < slots || ctas * 20 < slots * 11; };
  while (d.cs < 8 && more(d.groups * d.cs) && (int64_t)d.cs * warps < d.units) d.cs *= 2;
  if (d.cs == 8 && d.groups * 8 < 152 && d.units >= 1024) d.cs = 16;
  return d;
}

template <int D, int FMT, int NT, int F32, int W>
cudaError_t launch_decode_t(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p,
                            cudaStream_t s) {
  using C = DecCfg<D, FMT, NT, F32, W>;
  static DeviceOnce once;
  cudaError_t e = device_once(once, [] {
    cudaError_t r = cudaFuncSetAttribute(k_cache_decode<D, FMT, NT, F32, W>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (r) return r;
    return cudaFuncSetAttribute(k_cache_decode<D, FMT, NT, F32, W>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e) return e;
  const DecPlan d = decode_plan(p, NT, C::kKeys, W);
  const int64_t tiles = ((int64_t)p.c.max_rows * (p.Hq / p.c.Hkv) + C::kCols - 1) / C::kCols;
  const int cs = d.cs;
  if (tiles * cs > 0x7FFFFFFF) return cudaErrorInvalidValue;
  // (CTAs that all fit at once need no order)
  const int sorted = p.c.n_seq > 1 && p.c.n_seq <= kSortMax && d.groups * cs > C::kPerSm * 152 ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * cs), p.c.Hkv, p.c.n_seq);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_cache_decode<D, FMT, NT, F32, W>, mk, mv, p, cs, sorted);
}

template <int D, int FMT, int F32>
cudaError_t launch_decode_n(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p,
                            cudaStream_t s) {
  const int nt = decode_nt(p);
  if constexpr (FMT == 0) {
    if (nt == 3) return launch_decode_t<D, FMT, 3, F32, decode_warps(FMT, 3)>(mk, mv, p, s);
    if (nt == 2) return launch_decode_t<D, FMT, 2, F32, decode_warps(FMT, 2)>(mk, mv, p, s);
  }
  return launch_decode_t<D, FMT, 1, F32, decode_warps(FMT, 1)>(mk, mv, p, s);
}

}  // namespace

// Measured as cache_prompt_us: start and end of a CTA, and a stage of a warp (the SM full).
float cache_decode_us(const CacheAttnParams& p) {
  const int nt = decode_nt(p), warps = decode_warps(p.c.fmt, nt);
  const DecPlan d = decode_plan(p, nt, p.c.fmt ? kKvPage : kKvPage / 2, warps);
  const int slots = (p.c.fmt ? 16 : 8) / warps * 152;
  const int64_t waves = (d.groups * d.cs + slots - 1) / slots;
  const float stage = p.c.fmt ? (p.c.D == 128 ? 1.92f : 1.08f) : (p.c.D == 128 ? 1.3f : 1.05f);
  return static_cast<float>(waves) * ((p.c.fmt ? 6.f : 5.f) + stage * static_cast<float>((d.units + warps * d.cs - 1) / (warps * d.cs)));
}

cudaError_t launch_cache_decode(const CacheAttnParams& p, cudaStream_t s) {
  CUtensorMap mk = {}, mv = {};
  if (p.c.fmt == 0) {
    const uint64_t rows = (uint64_t)p.c.n_pages * p.c.Hkv * kKvPage;
    if (!make_map(&mk, p.c.K, rows, p.c.D, 16) || !make_map(&mv, p.c.V, rows, p.c.D, 16))
      return cudaErrorInvalidValue;
  }
#define TF_DEC(DV)                                                                                  \
  (p.c.fmt ? (p.f32 ? launch_decode_n<DV, 1, 1>(mk, mv, p, s) : launch_decode_n<DV, 1, 0>(mk, mv, p, s)) \
           : (p.f32 ? launch_decode_n<DV, 0, 1>(mk, mv, p, s) : launch_decode_n<DV, 0, 0>(mk, mv, p, s)))
  return p.c.D == 128 ? TF_DEC(128) : TF_DEC(64);
#undef TF_DEC
}

}  // namespace tf
