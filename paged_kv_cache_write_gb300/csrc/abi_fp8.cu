// extern "C" entry points of the 8-bit cache (include/pkv.h): host-side
// argument checks, then the kernel launches on the caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkv.h"
#include "checks.h"
#include "launch.h"
#include "nvtx.h"

namespace {

using pkv::PoolShape;
using pkv::aligned16;
using pkv::check_pool_fp8;
using pkv::from_cuda;

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

bool float_type(int32_t dtype) { return dtype == PKV_F32 || dtype == PKV_BF16; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The attention entries' common arguments.
pkv_status check_fp8(const void* q, int32_t dtype, int32_t num_seqs, int32_t n_heads,
                     const void* k_pool, const void* v_pool, const float* k_scales,
                     const float* v_scales, const pkv_pool_desc* pool,
                     const int32_t* block_tables, int32_t max_blocks_per_seq,
                     const int32_t* seq_lens, int32_t max_seq_len, float scale, const void* out,
                     PoolShape* shape) {
  pkv_status st = check_pool_fp8(pool, shape);
  if (st != PKV_OK) return st;
  // (a KV head is a grid's y in the prefill, and 16 bits of a decode's split entry)
  if (shape->n_kv > 65535) return PKV_ERR_RANGE;
  if (!float_type(dtype)) return PKV_ERR_DTYPE;
  st = pkv::check_attention_args(q, num_seqs, n_heads, k_pool, v_pool, *shape, block_tables,
                                 max_blocks_per_seq, seq_lens, max_seq_len, scale, out);
  if (st != PKV_OK) return st;
  // (positions are 32-bit)
  if (int64_t(max_blocks_per_seq) * shape->block_size > INT32_MAX) return PKV_ERR_RANGE;
  if (num_seqs > 0 && (!k_scales || !v_scales)) return PKV_ERR_NULL;
  if (!aligned4(k_scales) || !aligned4(v_scales)) return PKV_ERR_ALIGN;
  if (!pkv::fp8_attention_supported(*shape, n_heads)) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

pkv::AttnArgs attn_args(const void* q, int32_t num_seqs, int32_t n_heads, const void* k_pool,
                        const void* v_pool, const PoolShape& shape, const int32_t* block_tables,
                        int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t max_seq_len,
                        float scale, void* out, int32_t* err_word) {
  pkv::AttnArgs a{};
  a.q = q;
  a.out = out;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.num_seqs = num_seqs;
  a.n_heads = n_heads;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_seq_len = max_seq_len;
  a.pool = shape;
  a.scale = scale;
  a.err = err_word;
  return a;
}

}  // namespace

extern "C" {

pkv_status pkv_kv_write_fp8(const void* k, const void* v, int32_t dtype,
                            const int32_t* block_tables, int32_t max_blocks_per_seq,
                            const int32_t* seq_lens, const int32_t* cu_new_lens,
                            int32_t num_seqs, int32_t num_tokens, void* k_pool, void* v_pool,
                            float* k_scales, float* v_scales, const pkv_pool_desc* pool,
                            int32_t* err_word, void* stream) {
  PKV_NVTX_RANGE("pkv_kv_write_fp8");
  PoolShape shape;
  pkv_status st = check_pool_fp8(pool, &shape);
  if (st != PKV_OK) return st;
  if (!float_type(dtype)) return PKV_ERR_DTYPE;
  if (num_seqs < 0 || num_tokens < 0 || max_blocks_per_seq < 0) return PKV_ERR_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (num_seqs == 0 || max_blocks_per_seq == 0) return PKV_ERR_SHAPE;
  if (!k || !v || !block_tables || !seq_lens || !cu_new_lens || !k_pool || !v_pool || !k_scales ||
      !v_scales)
    return PKV_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pool) || !aligned16(v_pool) ||
      !aligned4(k_scales) || !aligned4(v_scales))
    return PKV_ERR_ALIGN;
  return from_cuda(pkv::launch_kv_write_fp8(k, v, dtype, block_tables, max_blocks_per_seq,
                                            seq_lens, cu_new_lens, num_seqs, num_tokens, k_pool,
                                            v_pool, k_scales, v_scales, shape, err_word,
                                            as_stream(stream)));
}

pkv_status pkv_kv_gather_fp8(const void* k_pool, const void* v_pool, const float* k_scales,
                             const float* v_scales, const pkv_pool_desc* pool,
                             const int32_t* block_tables, int32_t max_blocks_per_seq,
                             const int32_t* seq_lens, const int32_t* cu_seq_lens,
                             int32_t num_seqs, int32_t total_tokens, int32_t dtype, void* k_out,
                             void* v_out, int32_t* err_word, void* stream) {
  PKV_NVTX_RANGE("pkv_kv_gather_fp8");
  PoolShape shape;
  pkv_status st = check_pool_fp8(pool, &shape);
  if (st != PKV_OK) return st;
  if (!float_type(dtype)) return PKV_ERR_DTYPE;
  if (num_seqs < 0 || total_tokens < 0 || max_blocks_per_seq < 0) return PKV_ERR_SHAPE;
  if (total_tokens == 0) return PKV_OK;
  if (num_seqs == 0 || max_blocks_per_seq == 0) return PKV_ERR_SHAPE;
  if (!k_pool || !v_pool || !k_scales || !v_scales || !block_tables || !seq_lens || !cu_seq_lens ||
      !k_out || !v_out)
    return PKV_ERR_NULL;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_out) || !aligned16(v_out) ||
      !aligned4(k_scales) || !aligned4(v_scales))
    return PKV_ERR_ALIGN;
  return from_cuda(pkv::launch_kv_gather_fp8(
      k_pool, v_pool, k_scales, v_scales, shape, block_tables, max_blocks_per_seq, seq_lens,
      cu_seq_lens, num_seqs, total_tokens, dtype, k_out, v_out, err_word, as_stream(stream)));
}

size_t pkv_decode_fp8_workspace_bytes(int32_t num_seqs, int32_t n_heads, int32_t head_dim,
                                      int32_t max_seq_len, int32_t max_ctas, int32_t block_size) {
  (void)max_seq_len;
  (void)max_ctas;
  (void)block_size;
  return pkv::decode_fp8_workspace_bytes(num_seqs < 0 ? 0 : num_seqs, n_heads < 1 ? 1 : n_heads,
                                         head_dim < 1 ? 1 : head_dim);
}

pkv_status pkv_paged_attention_decode_fp8(const void* q, int32_t dtype, int32_t num_seqs,
                                          int32_t n_heads, const void* k_pool, const void* v_pool,
                                          const float* k_scales, const float* v_scales,
                                          const pkv_pool_desc* pool, const int32_t* block_tables,
                                          int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                          int32_t max_seq_len, float scale, int32_t max_ctas,
                                          void* out, void* workspace, size_t workspace_bytes,
                                          int32_t* err_word, void* stream) {
  PKV_NVTX_RANGE("pkv_paged_attention_decode_fp8");
  PoolShape shape;
  const pkv_status st =
      check_fp8(q, dtype, num_seqs, n_heads, k_pool, v_pool, k_scales, v_scales, pool,
                block_tables, max_blocks_per_seq, seq_lens, max_seq_len, scale, out, &shape);
  if (st != PKV_OK) return st;
  if (max_ctas < 0) return PKV_ERR_RANGE;
  if (num_seqs == 0) return PKV_OK;
  if (!workspace || workspace_bytes < pkv::decode_fp8_workspace_bytes(num_seqs, n_heads,
                                                                      shape.head_dim))
    return PKV_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PKV_ERR_ALIGN;
  pkv::AttnArgs a = attn_args(q, num_seqs, n_heads, k_pool, v_pool, shape, block_tables,
                              max_blocks_per_seq, seq_lens, max_seq_len, scale, out, err_word);
  a.max_q_len = 1;
  a.total_q = num_seqs;
  a.max_ctas = max_ctas;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  return from_cuda(pkv::launch_decode_fp8(a, dtype, k_scales, v_scales, as_stream(stream)));
}

pkv_status pkv_paged_attention_prefill_fp8(
    const void* q, int32_t dtype, const int32_t* cu_q_lens, int32_t num_seqs, int32_t total_q,
    int32_t max_q_len, int32_t n_heads, const void* k_pool, const void* v_pool,
    const float* k_scales, const float* v_scales, const pkv_pool_desc* pool,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
    int32_t max_seq_len, float scale, void* out, int32_t* err_word, void* stream) {
  PKV_NVTX_RANGE("pkv_paged_attention_prefill_fp8");
  PoolShape shape;
  const pkv_status st =
      check_fp8(q, dtype, num_seqs, n_heads, k_pool, v_pool, k_scales, v_scales, pool,
                block_tables, max_blocks_per_seq, seq_lens, max_seq_len, scale, out, &shape);
  if (st != PKV_OK) return st;
  if (total_q < 0 || max_q_len < 0) return PKV_ERR_SHAPE;
  if (num_seqs == 0 || total_q == 0) return PKV_OK;
  if (!cu_q_lens) return PKV_ERR_NULL;
  if (max_q_len == 0 || max_q_len > total_q || max_q_len > max_seq_len) return PKV_ERR_SHAPE;
  pkv::AttnArgs a = attn_args(q, num_seqs, n_heads, k_pool, v_pool, shape, block_tables,
                              max_blocks_per_seq, seq_lens, max_seq_len, scale, out, err_word);
  a.cu_q_lens = cu_q_lens;
  a.max_q_len = max_q_len;
  a.total_q = total_q;
  return from_cuda(pkv::launch_prefill_fp8(a, dtype, k_scales, v_scales, as_stream(stream)));
}

pkv_status pkv_selftest_bounded_wait_fp8(int32_t polls, int32_t* err_word, void* stream) {
  PKV_NVTX_RANGE("pkv_selftest_bounded_wait_fp8");
  if (polls < 1) return PKV_ERR_RANGE;
  if (!err_word) return PKV_ERR_NULL;
  return from_cuda(pkv::launch_fp8_bounded_wait_selftest(static_cast<uint32_t>(polls), err_word,
                                                         as_stream(stream)));
}

}  // extern "C"
