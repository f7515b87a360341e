// C ABI of the cache operators: argument checks and launches.
#include <cmath>
#include <new>
#include <vector>

#include "../../include/tf.h"
#include "kernels.h"

namespace {

using namespace tf;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool batch_of(const tf_kv_cache* c, CacheBatch* b) {
  if (!c || !c->K || !c->V || !c->block_table || !c->lengths) return false;
  if (c->format != TF_KV_BF16 && c->format != TF_KV_NVFP4) return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->n_kv_heads < 1 || c->n_kv_heads > 32767 || c->n_pages < 1 || c->table_stride < 1 || c->n_seq < 1 ||
      c->n_seq > 65535 || c->n_rows < 0 || c->max_rows < 0 || c->max_length < 0)
    return false;
  if ((int64_t)c->n_pages * c->n_kv_heads * kKvPage >= (1ll << 31)) return false;
  if (c->table_stride > (1 << 25) || c->n_rows >= (1 << 27) || (int64_t)c->max_rows * c->n_kv_heads >= (1ll << 31)) return false;
  if (!aligned(c->K, 128) || !aligned(c->V, 128) || !aligned(c->block_table, 4) || !aligned(c->lengths, 4) ||
      !aligned(c->row_start, 4) || !aligned(c->err, 4))
    return false;
  if (!c->row_start && (c->n_rows < c->n_seq || c->max_rows < 1)) return false;
  b->fmt = c->format;
  b->Hkv = c->n_kv_heads;
  b->D = c->head_dim;
  b->n_pages = c->n_pages;
  b->K = static_cast<const uint8_t*>(c->K);
  b->V = static_cast<const uint8_t*>(c->V);
  b->tbl = c->block_table;
  b->npp = c->table_stride;
  b->n_seq = c->n_seq;
  b->len = c->lengths;
  b->row_start = c->row_start;
  b->n_rows = c->n_rows;
  // one row per sequence needs no more; rows of a sequence are rows of the buffer
  b->max_rows = c->row_start ? (c->max_rows < c->n_rows ? c->max_rows : c->n_rows) : 1;
  const int64_t whole = (int64_t)c->table_stride * kKvPage;
  b->max_len = static_cast<int32_t>(c->max_length && c->max_length < whole ? c->max_length : whole);
  b->err = c->err;
  return true;
}

bool rows_ok(int32_t dtype, const void* p) {
  return p && (dtype == TF_DTYPE_F32 ? aligned(p, 4) : dtype == TF_DTYPE_BF16 && aligned(p, 2));
}

tf_status rows_call(const tf_kv_cache* cache, const void* k, const void* v, int64_t stride, int32_t dtype,
                    void* stream, cudaError_t (*launch)(const CacheRowsParams&, cudaStream_t)) {
  CacheRowsParams p = {};
  if (!batch_of(cache, &p.c) || !rows_ok(dtype, k) || !rows_ok(dtype, v)) return TF_E_INVAL;
  const int64_t row = (int64_t)p.c.Hkv * p.c.D;
  if (stride && stride < row) return TF_E_INVAL;
  if (p.c.max_rows == 0) return TF_OK;
  p.k = const_cast<void*>(k);
  p.v = const_cast<void*>(v);
  p.stride = stride ? stride : row;
  p.f32 = dtype == TF_DTYPE_F32;
  return launch(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TF_OK : TF_E_CUDA;
}

}  // namespace

extern "C" {

int64_t tf_op_cache_page_bytes(int32_t format, int32_t n_kv_heads, int32_t head_dim) {
  if ((format != TF_KV_BF16 && format != TF_KV_NVFP4) || n_kv_heads < 1 || (head_dim != 64 && head_dim != 128))
    return 0;
  return n_kv_heads * cache_head_bytes(format, head_dim);
}

tf_status tf_op_attention_cache(const tf_kv_cache* cache, const void* q, int64_t q_stride, void* out,
                                int64_t out_stride, int32_t dtype, int32_t n_heads, int32_t window,
                                int32_t sinks, float scale, void* stream) {
  CacheAttnParams p = {};
  if (!batch_of(cache, &p.c) || !rows_ok(dtype, q) || !rows_ok(dtype, out)) return TF_E_INVAL;
  if (n_heads < 1 || n_heads % p.c.Hkv || n_heads / p.c.Hkv > 8 || window < 0 || sinks < 0) return TF_E_INVAL;
  if (!(scale >= 0.f) || !std::isfinite(scale)) return TF_E_INVAL;
  const int64_t row = (int64_t)n_heads * p.c.D;
  if ((q_stride && q_stride < row) || (out_stride && out_stride < row)) return TF_E_INVAL;
  if (p.c.max_rows == 0) return TF_OK;
  p.q = q;
  p.out = out;
  p.q_stride = q_stride ? q_stride : row;
  p.out_stride = out_stride ? out_stride : row;
  p.f32 = dtype == TF_DTYPE_F32;
  p.Hq = n_heads;
  // positions are below 2^30: a wider window or more sinks change nothing
  p.window = window < (1 << 30) ? window : 1 << 30;
  p.sinks = sinks < (1 << 30) ? sinks : 1 << 30;
  const double sc = scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)p.c.D);
  p.scale_log2 = static_cast<float>(sc * 1.4426950408889634);
  // bfloat16 rows take the tensor-core kernel where it is the faster one by what both were measured at
  const bool many = !p.f32 && cache_prompt_us(p) < cache_decode_us(p);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return (many ? launch_cache_prompt(p, s) : launch_cache_decode(p, s)) == cudaSuccess ? TF_OK : TF_E_CUDA;
}

tf_status tf_op_cache_append(const tf_kv_cache* cache, const void* k, const void* v, int64_t stride,
                             int32_t dtype, void* stream) {
  return rows_call(cache, k, v, stride, dtype, stream, launch_cache_append);
}

tf_status tf_op_cache_read(const tf_kv_cache* cache, void* k, void* v, int64_t stride, int32_t dtype,
                           void* stream) {
  return rows_call(cache, k, v, stride, dtype, stream, launch_cache_read);
}

tf_status tf_op_cache_copy(void* const* pools, int32_t n_pools, int64_t page_bytes, int32_t n_pages,
                           const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  if (!pools || n_pools < 1 || n_pages < 1 || n < 0 || (n && (!src || !dst))) return TF_E_INVAL;
  if (page_bytes < 16 || page_bytes % 16 || page_bytes > (1ll << 30)) return TF_E_INVAL;
  for (int32_t i = 0; i < n_pools; ++i)
    if (!pools[i] || !aligned(pools[i], 16)) return TF_E_INVAL;
  try {
    std::vector<uint8_t> role(n_pages, 0);  // 1: a source, 2: a destination
    for (int32_t i = 0; i < n; ++i) {
      if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages) return TF_E_INVAL;
      role[src[i]] |= 1;
    }
    for (int32_t i = 0; i < n; ++i) {
      if (role[dst[i]]) return TF_E_INVAL;
      role[dst[i]] = 2;
    }
  } catch (const std::bad_alloc&) {
    return TF_E_NOMEM;
  }
  if (n == 0) return TF_OK;
  return launch_cache_copy(pools, n_pools, page_bytes, src, dst, n, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? TF_OK
             : TF_E_CUDA;
}

}  // extern "C"
