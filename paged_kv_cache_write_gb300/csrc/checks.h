// Host-side argument checks shared by the extern "C" entry points (abi.cu
// and decode_noalloc.cu), so every entry point that takes the same
// arguments refuses the same arguments with the same status.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkv.h"
#include "launch.h"

namespace pkv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline pkv_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return PKV_OK;
  cudaGetLastError();  // clear a sticky launch-configuration error
  return PKV_ERR_CUDA;
}

// A pool descriptor: known dtype, positive sizes, token rows of whole words of
// `row_align` bytes and a flat slot index that fits in int32.
inline pkv_status check_pool(const pkv_pool_desc* pool, PoolShape* out, int row_align = 16) {
  if (pool == nullptr) return PKV_ERR_NULL;
  if (pool->dtype != PKV_F32 && pool->dtype != PKV_BF16) return PKV_ERR_DTYPE;
  if (pool->num_blocks <= 0 || pool->block_size <= 0 || pool->n_kv <= 0 || pool->head_dim <= 0)
    return PKV_ERR_SHAPE;
  *out = PoolShape{pool->num_blocks, pool->block_size, pool->n_kv, pool->head_dim, pool->dtype};
  if (out->row_bytes() % row_align != 0) return PKV_ERR_ALIGN;
  if ((int64_t)pool->num_blocks * pool->block_size > INT32_MAX) return PKV_ERR_RANGE;
  return PKV_OK;
}

// The descriptor of an 8-bit pool: as check_pool, and each KV head's row a
// whole number of 16-byte vectors.
inline pkv_status check_pool_fp8(const pkv_pool_desc* pool, PoolShape* out) {
  if (pool == nullptr) return PKV_ERR_NULL;
  if (pool->dtype != PKV_FP8_E4M3) return PKV_ERR_DTYPE;
  if (pool->num_blocks <= 0 || pool->block_size <= 0 || pool->n_kv <= 0 || pool->head_dim <= 0)
    return PKV_ERR_SHAPE;
  if (pool->head_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
  // (the kernels count a token's elements, and a block's of one head, in 32 bits)
  if ((int64_t)pool->n_kv * pool->head_dim > (1 << 26) ||
      (int64_t)pool->block_size * pool->head_dim > INT32_MAX)
    return PKV_ERR_RANGE;
  *out = PoolShape{pool->num_blocks, pool->block_size, pool->n_kv, pool->head_dim, pool->dtype};
  if ((int64_t)pool->num_blocks * pool->block_size > INT32_MAX) return PKV_ERR_RANGE;
  return PKV_OK;
}

// The descriptor of a 4-bit pool: positive sizes, rows of whole groups, a KV head
// that fits a grid's y, slots that fit in int32.
inline pkv_status check_pool_fp4(const pkv_pool_desc* pool, PoolShape* out) {
  if (pool == nullptr) return PKV_ERR_NULL;
  if (pool->dtype != PKV_FP4_E2M1) return PKV_ERR_DTYPE;
  if (pool->num_blocks <= 0 || pool->block_size <= 0 || pool->n_kv <= 0 || pool->head_dim <= 0)
    return PKV_ERR_SHAPE;
  if (pool->head_dim % 16 != 0 || pool->head_dim > 256) return PKV_ERR_UNSUPPORTED;
  if (pool->n_kv > 65535 || (int64_t)pool->num_blocks * pool->block_size > INT32_MAX ||
      (int64_t)pool->num_blocks * pool->n_kv > INT32_MAX)
    return PKV_ERR_RANGE;
  *out = PoolShape{pool->num_blocks, pool->block_size, pool->n_kv, pool->head_dim, pool->dtype};
  return PKV_OK;
}

// Rows [num_tokens, heads, head_dim] with a token stride in elements.
inline pkv_status check_rows(const void* p, int64_t stride, int32_t num_tokens, int32_t heads,
                             int32_t head_dim, int32_t dtype) {
  if (p == nullptr) return PKV_ERR_NULL;
  const int es = dtype == PKV_F32 ? 4 : 2;
  if (num_tokens > 1 && stride < (int64_t)heads * head_dim) return PKV_ERR_SHAPE;
  if (stride > INT64_MAX / 4 / num_tokens) return PKV_ERR_RANGE;
  if (!aligned16(p) || (num_tokens > 1 && stride * es % 16 != 0)) return PKV_ERR_ALIGN;
  return PKV_OK;
}

// Arguments common to decode and prefill attention, the pool already
// checked.  num_seqs == 0 passes before the pointer checks (nothing will be
// read).
inline pkv_status check_attention_args(const void* q, int32_t num_seqs, int32_t n_heads,
                                       const void* k_pool, const void* v_pool,
                                       const PoolShape& shape, const int32_t* block_tables,
                                       int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                       int32_t max_seq_len, float scale, const void* out) {
  if (num_seqs < 0 || n_heads <= 0 || max_blocks_per_seq < 0 || max_seq_len < 0)
    return PKV_ERR_SHAPE;
  if (n_heads % shape.n_kv != 0) return PKV_ERR_SHAPE;
  if (!(scale > 0.f) || scale == __builtin_inff()) return PKV_ERR_RANGE;
  if (num_seqs == 0) return PKV_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !seq_lens || !out) return PKV_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return PKV_ERR_ALIGN;
  if (max_blocks_per_seq == 0 && max_seq_len > 0) return PKV_ERR_SHAPE;
  if ((int64_t)max_seq_len > (int64_t)max_blocks_per_seq * shape.block_size) return PKV_ERR_SHAPE;
  return PKV_OK;
}

inline pkv_status check_attention(const void* q, int32_t num_seqs, int32_t n_heads,
                                  const void* k_pool, const void* v_pool,
                                  const pkv_pool_desc* pool, const int32_t* block_tables,
                                  int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                  int32_t max_seq_len, float scale, const void* out,
                                  PoolShape* shape) {
  pkv_status st = check_pool(pool, shape);
  if (st != PKV_OK) return st;
  return check_attention_args(q, num_seqs, n_heads, k_pool, v_pool, *shape, block_tables,
                              max_blocks_per_seq, seq_lens, max_seq_len, scale, out);
}

// check_attention plus what every decode entry point adds: a non-negative
// grid cap and a compiled-in shape.
inline pkv_status check_decode(const void* q, int32_t num_seqs, int32_t n_heads,
                               const void* k_pool, const void* v_pool, const pkv_pool_desc* pool,
                               const int32_t* block_tables, int32_t max_blocks_per_seq,
                               const int32_t* seq_lens, int32_t max_seq_len, float scale,
                               int32_t max_ctas, const void* out, PoolShape* shape) {
  pkv_status st = check_attention(q, num_seqs, n_heads, k_pool, v_pool, pool, block_tables,
                                  max_blocks_per_seq, seq_lens, max_seq_len, scale, out, shape);
  if (st != PKV_OK) return st;
  if (max_ctas < 0) return PKV_ERR_RANGE;
  if (!decode_supported(*shape, n_heads)) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

}  // namespace pkv
