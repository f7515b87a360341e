// Cache operators (sm_103a): rows appended to and read from a paged KV cache
// in bfloat16 or 4 bits, and page copies.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "cache.cuh"
#include "common.cuh"
#include "device_once.h"
#include "kernels.h"

namespace tf {

namespace {

// ---------------------------------------------------------------- rows in and out
// Append: a lane takes one block of 16 elements of a row (D / 16 lanes a row), so a block's and a row's scale are
// worked out with few idle repeats: instructions (the quantiser's divisions), not memory, bound it.  16 x 512 bf16
// rows of 8 heads: 16.5 us, 44 MB at 2.6 TB/s (27 us with 8 elements a lane); 394 instructions for 4 rows of a head.
// Even and odd position of a pair sit in one warp: a byte of V's codes holds both, and one lane writes it.
constexpr int kRowThreads = 128, kReadThreads = 256;

template <int E>
__device__ __forceinline__ void load_row(const void* base, size_t off, int f32, float (&x)[E]) {
  if (f32) {
    const float* p = static_cast<const float*>(base) + off;
    if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < E; i += 4) *reinterpret_cast<float4*>(x + i) = __ldg(reinterpret_cast<const float4*>(p + i));
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = p[i];
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + off;
    if ((reinterpret_cast<uintptr_t>(p) & (E == 4 ? 7 : 15)) == 0) {
      uint32_t w[E / 2];
      if constexpr (E == 4) {
        *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
      } else {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) *reinterpret_cast<uint4*>(w + 4 * i) = *reinterpret_cast<const uint4*>(p + 8 * i);
      }
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = bf16_to_f32(p[i]);
    }
  }
}

template <int E>
__device__ __forceinline__ void store_row(void* base, size_t off, int f32, const float (&x)[E]) {
  if (f32) {
    float* p = static_cast<float*>(base) + off;
    if (E == 8 && (reinterpret_cast<uintptr_t>(p) & 31) == 0) {  // whole sectors
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                   "f"(x[3]), "f"(x[4 % E]), "f"(x[5 % E]), "f"(x[6 % E]), "f"(x[7 % E])
                   : "memory");
    } else if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < E; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = x[i];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + off;
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      w[i] = static_cast<uint32_t>(f32_to_bf16(x[2 * i])) | static_cast<uint32_t>(f32_to_bf16(x[2 * i + 1])) << 16;
    if ((reinterpret_cast<uintptr_t>(p) & (E * 2 - 1)) == 0) {
      if constexpr (E == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      else
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    }
  }
}

// Eight floats -> eight e2m1 codes (the first in the lowest nibble): round to nearest even, +-6 at most.
__device__ __forceinline__ uint32_t e2m1x8(const float (&r)[8]) {
  uint32_t d;
  asm("{.reg .b8 b0, b1, b2, b3;"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5; cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;"
      " mov.b32 %0, {b0, b1, b2, b3};}"
      : "=r"(d)
      : "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]));
  return d;
}
__device__ __forceinline__ float max_abs_nan(float a, float x) {  // a NaN if x is one
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(x)));
  return d;
}

// x: one block of a row, LANES lanes hold the row.  Its codes (the first element in the lowest nibble), its scale
// byte, the row's scale.
template <int LANES>
__device__ __forceinline__ void quantise_row(const float (&x)[16], uint32_t (&code)[2], uint32_t& sb, float& s) {
  float blk = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) blk = max_abs_nan(blk, x[i]);
  float row = blk;
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) row = max_abs_nan(row, __shfl_xor_sync(0xFFFFFFFFu, row, o));
  s = row < INFINITY ? __fdiv_rn(row, 2688.0f) : __int_as_float(0x7FFFFFFF);
  const float s6 = __fmul_rn(s, 6.0f);
  sb = 0;
  float step = 0.f;
  if (s6 > 0.f) {  // false for NaN
    sb = __nv_cvt_float_to_fp8(fminf(__fdiv_rn(blk, s6), 448.0f), __NV_SATFINITE, __NV_E4M3);
    step = __fmul_rn(e4m3_value(sb), s);
  }
  code[0] = code[1] = 0;
  if (!(step > 0.f)) return;
  // The code is that of the rounded quotient x / step.  x * (1 / step) is within 2^-22 of it (the roundings of the
  // reciprocal, of its scaling below and of the product, 2^-24 each), so the quotient lies between x * (1 / step) *
  // (1 -+ 2^-21).  Where both have the same code, it is the quotient's (rounding is monotonic); only a block with
  // others needs the divisions.
  const float inv = __fdiv_rn(1.0f, step), down = inv * (1.0f - 4.76837158e-7f), up = inv * (1.0f + 4.76837158e-7f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // + 0: no -0
      lo[i] = fmaf(x[8 * h + i], down, 0.f);
      hi[i] = fmaf(x[8 * h + i], up, 0.f);
    }
    code[h] = e2m1x8(lo);
    if (code[h] != e2m1x8(hi) || !(step > 1e-30f && step < 1e30f)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) lo[i] = __fdiv_rn(x[8 * h + i], step) + 0.f;
      code[h] = e2m1x8(lo);
    }
  }
}

// Grid: (position pairs / 8 (D = 128) or 16, KV heads x (K, V), sequences); 4 warps a CTA.
template <int D, int FMT>
__global__ void __launch_bounds__(kRowThreads) k_cache_append(const CacheRowsParams p) {
  constexpr int LANES = D / 16, PAIRS = 16 / LANES;      // lanes a row, pairs a warp
  using L = Kv4<D>;
  const CacheBatch& c = p.c;
  const int b = blockIdx.z, isv = blockIdx.y & 1, g = blockIdx.y >> 1;
  const int lane = threadIdx.x & 31, l = lane % LANES, half = (lane / LANES) & 1;
  const SeqRows sq = cache_seq(c, b);
  const int p0 = max(sq.len - sq.n, 0);                 // first position written
  // the pair's even position; a warp whose first pair is past the end leaves, its other lanes only idle
  const int base0 = (p0 & ~1) + 2 * PAIRS * (blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5));
  if (sq.n == 0 || base0 >= sq.len) return;
  const int base = base0 + 2 * (lane / (2 * LANES)), pos = base + half;
  const int page = base < sq.len ? cache_page(c, b, base / kKvPage) : -1;
  const bool mine = page >= 0 && pos >= p0 && pos < sq.len;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
  if (mine)
    load_row<16>(isv ? p.v : p.k, (size_t)(sq.r0 + pos - (sq.len - sq.n)) * p.stride + (size_t)g * D + l * 16, p.f32, x);
  const int r = pos % kKvPage;
  uint8_t* head = const_cast<uint8_t*>(isv ? c.V : c.K) +
                  ((size_t)max(page, 0) * c.Hkv + g) * (FMT ? L::kBytes : kKvPage * D * 2);
  if constexpr (FMT == 0) {
    if (mine) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = static_cast<uint32_t>(f32_to_bf16(x[2 * i])) | static_cast<uint32_t>(f32_to_bf16(x[2 * i + 1])) << 16;
      uint4* dst = reinterpret_cast<uint4*>(head + (r * D + l * 16) * 2);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  } else {
    uint32_t code[2], sb;
    float s;
    quantise_row<LANES>(x, code, sb, s);
    if (mine) {
      if (l == 0) reinterpret_cast<float*>(head + L::kRows)[r] = s;
      head[L::kCodes + (isv ? l * kKvPage + r : r * (D / 16) + l)] = static_cast<uint8_t>(sb);
    }
    if (!isv) {
      if (mine)
        *reinterpret_cast<uint2*>(head + r * (D / 2) + l * 8) = make_uint2(code[0], code[1]);
    } else {
      // the even position's lane writes the pair's bytes; a position that this
      // call does not write keeps its nibble
      uint32_t* dst = reinterpret_cast<uint32_t*>(head + L::v_byte(base % kKvPage, l * 16));
      const bool both = __shfl_xor_sync(0xFFFFFFFFu, mine ? 1 : 0, LANES) && mine;
      uint32_t out[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t two = __byte_perm(code[w >> 1], 0, w & 1 ? 0x4342 : 0x4140);  // elements 4 w .. + 3: a nibble each
        out[w] = (two & 0x000F000Fu) | (two & 0x00F000F0u) << 4;                      // ... a byte each
        const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, out[w], LANES);
        if (both) {
          out[w] |= o << 4;
        } else if (mine) {
          out[w] = half ? (dst[w] & 0x0F0F0F0Fu) | (out[w] << 4) : (dst[w] & 0xF0F0F0F0u) | out[w];
        }
      }
      if (both ? half == 0 : mine) *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

// Four bytes of e2m1 pairs -> f16x2 each (low nibble in the low half).
__device__ __forceinline__ void e2m1x8_f16(uint32_t v, __half2 (&h)[4]) {
  uint32_t o[4];
  asm("{.reg .b8 b0, b1, b2, b3; mov.b32 {b0, b1, b2, b3}, %4;"
      " cvt.rn.f16x2.e2m1x2 %0, b0; cvt.rn.f16x2.e2m1x2 %1, b1;"
      " cvt.rn.f16x2.e2m1x2 %2, b2; cvt.rn.f16x2.e2m1x2 %3, b3;}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(v));
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __half2*>(&o[i]);
}

// Grid: (position pairs of a sequence * KV heads / 16, 2 (K, V), sequences): half a warp takes a pair of positions
// of one head, E elements of both a lane, so V's codes (two positions in a byte) are read once.  16 x 512 rows of 8
// heads to float32: 14.1 us, 77 MB at 5.5 TB/s (18.3 us with 16-byte stores; 14.2 and 14.6 us with two and four pairs a
// half warp).
template <int D, int FMT>
__global__ void __launch_bounds__(kReadThreads) k_cache_read(const CacheRowsParams p) {
  constexpr int E = D / 16;
  using L = Kv4<D>;
  const CacheBatch& c = p.c;
  const int b = blockIdx.z, isv = blockIdx.y;
  const int l = threadIdx.x & 15;
  const SeqRows sq = cache_seq(c, b);
  const int item = blockIdx.x * (kReadThreads / 16) + (threadIdx.x >> 4);
  const int g = item % c.Hkv, first = sq.len - sq.n;
  // an even position, the first one at or below `first` (which may be negative)
  const int base = (first & ~1) + 2 * (item / c.Hkv);
  if (sq.n == 0 || base >= sq.len) return;
  const int page = base < 0 ? -1 : cache_page(c, b, base / kKvPage);
  void* dst = isv ? p.v : p.k;
  auto store = [&](int y, const float (&x)[E]) {
    if (base + y >= first && base + y < sq.len)
      store_row<E>(dst, (size_t)(sq.r0 + base + y - first) * p.stride + (size_t)g * D + l * E, p.f32, x);
  };
  if (page < 0) {
    const float zero[E] = {};
    store(0, zero);
    store(1, zero);
    return;
  }
  const int r = base % kKvPage;
  const uint8_t* head = (isv ? c.V : c.K) + ((size_t)page * c.Hkv + g) * (FMT ? L::kBytes : kKvPage * D * 2);
  float x[2][E];
  if constexpr (FMT == 0) {
    load_row<E>(head, r * D + l * E, 0, x[0]);
    load_row<E>(head, (r + 1) * D + l * E, 0, x[1]);
    store(0, x[0]);
    store(1, x[1]);
    return;
  }
  const int blk = l * E / 16;
  const float2 s = *reinterpret_cast<const float2*>(head + L::kRows + r * 4);
  const uint8_t* sb = head + L::kCodes;
  // (e2m1 * b is exact, so the row scale's product is the one rounding)
  if (isv) {
    uint32_t w[E / 4];
    const uint8_t* at = head + L::v_byte(r, l * E);
    if constexpr (E == 8)
      *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(at);
    else
      w[0] = *reinterpret_cast<const uint32_t*>(at);
    const uint32_t two = *reinterpret_cast<const uint16_t*>(sb + blk * kKvPage + r);
    const float s0 = e4m3_value(two), s1 = e4m3_value(two >> 8);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      __half2 h[4];
      e2m1x8_f16(w[i], h);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float2 f = __half22float2(h[y]);
        x[0][4 * i + y] = f.x * s0 * s.x;
        x[1][4 * i + y] = f.y * s1 * s.y;
      }
    }
    store(0, x[0]);
    store(1, x[1]);
  } else {
    uint32_t w[2], sc[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if constexpr (E == 8)
        w[y] = *reinterpret_cast<const uint32_t*>(head + (r + y) * (D / 2) + l * 4);
      else
        w[y] = *reinterpret_cast<const uint16_t*>(head + (r + y) * (D / 2) + l * 2);
      sc[y] = sb[(r + y) * (D / 16) + blk];
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const float bs = e4m3_value(sc[y]), rs = y ? s.y : s.x;
      __half2 h[4];
      e2m1x8_f16(w[y], h);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 f = __half22float2(h[i]);
        x[y][2 * i] = f.x * bs * rs;
        x[y][2 * i + 1] = f.y * bs * rs;
      }
      store(y, x[y]);
    }
  }
}

// ---------------------------------------------------------------- page copies
// The lists travel as kernel parameters, so a call needs no device staging.  64 pages of 64 KB in 72 pools: 88.6 us,
// 6.8 TB/s; one page of 19 KB in 72 pools: 1.8 us.
constexpr int kCopyPools = 128, kCopyMoves = 384;
struct CopyParams {
  uint4* pool[kCopyPools];
  int2 move[kCopyMoves];
  int32_t n_moves;
  int32_t words;    // 16-byte words of a page
  int32_t chunks;   // CTAs a page
};
constexpr int kCopyThreads = 256, kCopyUnroll = 4;

__global__ void __launch_bounds__(kCopyThreads) k_cache_copy(const __grid_constant__ CopyParams p) {
  const int m = blockIdx.x / p.chunks, ch = blockIdx.x % p.chunks;
  uint4* pool = p.pool[blockIdx.y];
  const uint4* src = pool + (size_t)p.move[m].x * p.words;
  uint4* dst = pool + (size_t)p.move[m].y * p.words;
  const int w0 = ch * kCopyThreads * kCopyUnroll + threadIdx.x;
  uint4 v[kCopyUnroll];
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u)
    if (w0 + u * kCopyThreads < p.words) v[u] = src[w0 + u * kCopyThreads];
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u)
    if (w0 + u * kCopyThreads < p.words) dst[w0 + u * kCopyThreads] = v[u];
}

}  // namespace

#define TF_CACHE_DISPATCH(KERNEL, GRID, BLOCK, S, P)                   \
  do {                                                                 \
    if ((P).c.D == 128)                                                \
      (P).c.fmt ? KERNEL<128, 1><<<GRID, BLOCK, 0, S>>>(P)             \
                : KERNEL<128, 0><<<GRID, BLOCK, 0, S>>>(P);            \
    else                                                               \
      (P).c.fmt ? KERNEL<64, 1><<<GRID, BLOCK, 0, S>>>(P)              \
                : KERNEL<64, 0><<<GRID, BLOCK, 0, S>>>(P);             \
  } while (0)

cudaError_t launch_cache_append(const CacheRowsParams& p, cudaStream_t s) {
  const int64_t pairs = (int64_t)p.c.max_rows / 2 + 1;  // that max_rows rows can touch
  const int per = (kRowThreads / 32) * (256 / p.c.D);
  const dim3 grid(static_cast<unsigned>((pairs + per - 1) / per), 2 * p.c.Hkv, p.c.n_seq);
  TF_CACHE_DISPATCH(k_cache_append, grid, kRowThreads, s, p);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheRowsParams& p, cudaStream_t s) {
  const int64_t items = ((int64_t)p.c.max_rows / 2 + 1) * p.c.Hkv;  // pairs that max_rows rows can touch
  const int per = kReadThreads / 16;
  const dim3 grid(static_cast<unsigned>((items + per - 1) / per), 2, p.c.n_seq);
  TF_CACHE_DISPATCH(k_cache_read, grid, kReadThreads, s, p);
  return cudaGetLastError();
}

cudaError_t launch_cache_copy(void* const* pools, int n_pools, int64_t page_bytes, const int32_t* src,
                              const int32_t* dst, int n, cudaStream_t s) {
  CopyParams p;
  p.words = static_cast<int32_t>(page_bytes / 16);
  p.chunks = (p.words + kCopyThreads * kCopyUnroll - 1) / (kCopyThreads * kCopyUnroll);
  for (int q0 = 0; q0 < n_pools; q0 += kCopyPools) {
    const int nq = std::min(kCopyPools, n_pools - q0);
    for (int i = 0; i < nq; ++i) p.pool[i] = static_cast<uint4*>(pools[q0 + i]);
    for (int m0 = 0; m0 < n; m0 += kCopyMoves) {
      p.n_moves = std::min(kCopyMoves, n - m0);
      for (int i = 0; i < p.n_moves; ++i) p.move[i] = make_int2(src[m0 + i], dst[m0 + i]);
      k_cache_copy<<<dim3(p.n_moves * p.chunks, nq), kCopyThreads, 0, s>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace tf
