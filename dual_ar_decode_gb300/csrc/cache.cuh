// Device helpers of the cache operators: which rows a sequence has, where a
// position lies in a page, and the 4-bit row format.
#pragma once

#include "../../include/tf.h"
#include "common.cuh"
#include "kernels.h"

namespace tf {

__device__ __forceinline__ void cache_flag(const CacheBatch& c, uint32_t bits) {
  if (c.err) atomicOr(c.err, bits);
}

// Rows r0 .. r0 + n - 1 of sequence b at positions len - n .. len - 1; n = 0
// for a sequence whose description is not usable (flagged).
struct SeqRows {
  int r0, n, len;
};
__device__ __forceinline__ SeqRows cache_rows(const CacheBatch& c, int r0, int r1, int len) {
  SeqRows s;
  s.r0 = r0;
  s.len = len;
  s.n = 0;
  if (s.r0 < 0 || r1 < s.r0 || r1 > c.n_rows || r1 - s.r0 > c.max_rows) {
    cache_flag(c, TF_CACHE_BAD_ROWS);
  } else if (s.len < 0 || s.len > c.npp * kKvPage) {
    cache_flag(c, TF_CACHE_BAD_LENGTH);
  } else {
    s.n = r1 - s.r0;
  }
  return s;
}

__device__ __forceinline__ SeqRows cache_seq(const CacheBatch& c, int b) {
  return cache_rows(c, c.row_start ? __ldg(c.row_start + b) : b, c.row_start ? __ldg(c.row_start + b + 1) : b + 1,
                    __ldg(c.len + b));
}

// Page of block-table entry i of sequence b, or -1 (flagged) outside the pool.
__device__ __forceinline__ int cache_page(const CacheBatch& c, int b, int i) {
  const int pg = __ldg(c.tbl + (size_t)b * c.npp + i);
  if (pg >= 0 && pg < c.n_pages) return pg;
  cache_flag(c, TF_CACHE_BAD_PAGE);
  return -1;
}

// 4-bit page of one head: offsets of the block scales and the row scales, and
// the byte of element d of V's position r (nibble r & 1).
template <int D>
struct Kv4 {
  static constexpr int kCodes = kKvPage * D / 2;
  static constexpr int kBlocks = kKvPage * D / 16;
  static constexpr int kRows = kCodes + kBlocks;     // float32 row scales from here
  static constexpr int kBytes = kRows + kKvPage * 4;
  __host__ __device__ static constexpr int v_byte(int r, int d) {
    return (((r >> 1) & 3) * (D / 16) + d / 16) * 64 + (r >> 3) * 16 + d % 16;
  }
};

// e4m3 bits (no NaN: the quantiser writes none) -> float.
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  return __uint_as_float((b & 0x7Fu) << 20) * 1.329227995784915873e36f;  // bits placed, x 2^120
}

}  // namespace tf
