// extern "C" entry points of the norm and rotation before the cache and of the
// 4-bit cache (include/pkv.h): host-side argument checks, then the kernel launches
// on the caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkv.h"
#include "checks.h"
#include "launch.h"
#include "nvtx.h"

namespace {

using pkv::Fp4Cache;
using pkv::NormRopeArgs;
using pkv::PoolShape;
using pkv::aligned16;
using pkv::check_pool_fp4;
using pkv::check_rows;
using pkv::from_cuda;

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

bool float_type(int32_t dtype) { return dtype == PKV_F32 || dtype == PKV_BF16; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// The norm and rotation's own arguments, and the queries and keys that they are for
// (num_tokens > 0).
pkv_status check_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const pkv_norm_rope_desc* rope, void* q_out, int64_t q_out_stride,
                           int32_t* err_word, NormRopeArgs* a) {
  if (rope == nullptr) return PKV_ERR_NULL;
  if (a->n_heads <= 0 || a->n_kv <= 0 || a->head_dim <= 0) return PKV_ERR_SHAPE;
  if (a->head_dim % 16 != 0 || a->head_dim > 256) return PKV_ERR_UNSUPPORTED;
  if (rope->rot_dim <= 0 || rope->rot_dim > a->head_dim || rope->num_positions <= 0)
    return PKV_ERR_SHAPE;
  if (rope->rot_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
  if (rope->interleaved != 0 && rope->interleaved != 1) return PKV_ERR_RANGE;
  const bool norm = rope->q_weight != nullptr || rope->k_weight != nullptr;
  if (norm && !(rope->eps >= 0.f && rope->eps < __builtin_inff())) return PKV_ERR_RANGE;
  if (a->num_tokens == 0) return PKV_OK;
  if (rope->cos_sin == nullptr || rope->positions == nullptr) return PKV_ERR_NULL;
  if (!aligned16(rope->cos_sin) || !aligned4(rope->positions) || !aligned16(rope->q_weight) ||
      !aligned16(rope->k_weight))
    return PKV_ERR_ALIGN;
  pkv_status st = check_rows(q, q_stride, a->num_tokens, a->n_heads, a->head_dim, a->dtype);
  if (st == PKV_OK) st = check_rows(k, k_stride, a->num_tokens, a->n_kv, a->head_dim, a->dtype);
  if (st == PKV_OK)
    st = check_rows(q_out, q_out_stride, a->num_tokens, a->n_heads, a->head_dim, a->dtype);
  if (st != PKV_OK) return st;
  a->q = q;
  a->q_stride = q_stride;
  a->k = k;
  a->k_stride = k_stride;
  a->q_out = q_out;
  a->q_out_stride = q_out_stride;
  a->q_weight = rope->q_weight;
  a->k_weight = rope->k_weight;
  a->eps = rope->eps;
  a->rot = rope->rot_dim;
  a->interleaved = rope->interleaved != 0;
  a->num_positions = rope->num_positions;
  a->cos_sin = rope->cos_sin;
  a->positions = rope->positions;
  a->err = err_word;
  return PKV_OK;
}

// More than the kernel counts in 32 bits.
bool too_many(const NormRopeArgs& a) {
  return a.n_heads > (1 << 20) || a.n_kv > (1 << 20) || a.num_tokens > (1 << 30);
}

// The values and the slots that keys and values go to.
pkv_status check_slots(const void* v, int64_t v_stride, const int64_t* slots, void* k_pool,
                       void* v_pool, const PoolShape& pool, NormRopeArgs* a) {
  const pkv_status st = check_rows(v, v_stride, a->num_tokens, a->n_kv, a->head_dim, a->dtype);
  if (st != PKV_OK) return st;
  if (!slots || !k_pool || !v_pool) return PKV_ERR_NULL;
  if (!aligned8(slots) || !aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_ALIGN;
  a->v = v;
  a->v_stride = v_stride;
  a->slots = slots;
  a->k_pool = k_pool;
  a->v_pool = v_pool;
  a->block_size = pool.block_size;
  a->num_slots = int64_t(pool.num_blocks) * pool.block_size;
  return PKV_OK;
}

pkv_status check_groups(const void* k_groups, const void* v_groups, const float* k_scale,
                        const float* v_scale) {
  if (!k_groups || !v_groups || !k_scale || !v_scale) return PKV_ERR_NULL;
  if (!aligned16(k_groups) || !aligned16(v_groups) || !aligned4(k_scale) || !aligned4(v_scale))
    return PKV_ERR_ALIGN;
  return PKV_OK;
}

void set_groups(void* k_groups, void* v_groups, const float* k_scale, const float* v_scale,
                NormRopeArgs* a) {
  a->k_groups = static_cast<uint8_t*>(k_groups);
  a->v_groups = static_cast<uint8_t*>(v_groups);
  a->k_scale = k_scale;
  a->v_scale = v_scale;
}

// The attention entries' common arguments, into `a` and `c`.
pkv_status check_attention_fp4(const void* q, int32_t dtype, int32_t num_seqs, int32_t n_heads,
                               const Fp4Cache& c, const pkv_pool_desc* pool,
                               const int32_t* block_tables, int32_t max_blocks_per_seq,
                               const int32_t* seq_lens, int32_t max_seq_len, float scale, void* out,
                               int32_t* err_word, pkv::AttnArgs* a) {
  PoolShape shape;
  pkv_status st = check_pool_fp4(pool, &shape);
  if (st != PKV_OK) return st;
  if (!float_type(dtype)) return PKV_ERR_DTYPE;
  st = pkv::check_attention_args(q, num_seqs, n_heads, c.k_pool, c.v_pool, shape, block_tables,
                                 max_blocks_per_seq, seq_lens, max_seq_len, scale, out);
  if (st != PKV_OK) return st;
  // (positions are 32-bit)
  if (int64_t(max_blocks_per_seq) * shape.block_size > INT32_MAX) return PKV_ERR_RANGE;
  if (num_seqs > 0) {
    st = check_groups(c.k_groups, c.v_groups, c.k_scale, c.v_scale);
    if (st != PKV_OK) return st;
  }
  if (!pkv::fp8_attention_supported(shape, n_heads)) return PKV_ERR_UNSUPPORTED;
  a->q = q;
  a->out = out;
  a->block_tables = block_tables;
  a->seq_lens = seq_lens;
  a->num_seqs = num_seqs;
  a->n_heads = n_heads;
  a->max_blocks_per_seq = max_blocks_per_seq;
  a->max_seq_len = max_seq_len;
  a->pool = shape;
  a->scale = scale;
  a->err = err_word;
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            int32_t dtype, int32_t num_tokens, int32_t n_heads, int32_t n_kv,
                            int32_t head_dim, const pkv_norm_rope_desc* rope, void* q_out,
                            int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                            int32_t* err_word, void* stream) {
  PKV_NVTX_RANGE("pkv_qk_norm_rope");
  if (!float_type(dtype)) return PKV_ERR_DTYPE;
  if (num_tokens < 0) return PKV_ERR_SHAPE;
  NormRopeArgs a{};
  a.dtype = dtype;
  a.num_tokens = num_tokens;
  a.n_heads = n_heads;
  a.n_kv = n_kv;
  a.head_dim = head_dim;
  pkv_status st = check_norm_rope(q, q_stride, k, k_stride, rope, q_out, q_out_stride, err_word, &a);
  if (st != PKV_OK || num_tokens == 0) return st;
  st = check_rows(k_out, k_out_stride, num_tokens, n_kv, head_dim, dtype);
  if (st != PKV_OK) return st;
  if (too_many(a)) return PKV_ERR_RANGE;
  a.k_out = k_out;
  a.k_out_stride = k_out_stride;
  return from_cuda(pkv::launch_norm_rope(a, as_stream(stream)));
}

pkv_status pkv_qk_norm_rope_write(const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride,
                                  int32_t num_tokens, int32_t n_heads,
                                  const pkv_norm_rope_desc* rope, void* q_out,
                                  int64_t q_out_stride, const int64_t* slot_mapping, void* k_pool,
                                  void* v_pool, const pkv_pool_desc* pool, int32_t* err_word,
                                  void* stream) {
  PKV_NVTX_RANGE("pkv_qk_norm_rope_write");
  PoolShape shape;
  pkv_status st = pkv::check_pool(pool, &shape);
  if (st != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_SHAPE;
  NormRopeArgs a{};
  a.dtype = shape.dtype;
  a.num_tokens = num_tokens;
  a.n_heads = n_heads;
  a.n_kv = shape.n_kv;
  a.head_dim = shape.head_dim;
  st = check_norm_rope(q, q_stride, k, k_stride, rope, q_out, q_out_stride, err_word, &a);
  if (st != PKV_OK || num_tokens == 0) return st;
  st = check_slots(v, v_stride, slot_mapping, k_pool, v_pool, shape, &a);
  if (st != PKV_OK) return st;
  if (too_many(a)) return PKV_ERR_RANGE;
  return from_cuda(pkv::launch_norm_rope(a, as_stream(stream)));
}

pkv_status pkv_qk_norm_rope_write_fp4(const void* q, int64_t q_stride, const void* k,
                                      int64_t k_stride, const void* v, int64_t v_stride,
                                      int32_t dtype, int32_t num_tokens, int32_t n_heads,
                                      const pkv_norm_rope_desc* rope, void* q_out,
                                      int64_t q_out_stride, const int64_t* slot_mapping,
                                      void* k_pool, void* v_pool, void* k_groups, void* v_groups,
                                      const float* k_scale, const float* v_scale,
                                      const pkv_pool_desc* pool, int32_t* err_word, void* stream) {
  PKV_NVTX_RANGE("pkv_qk_norm_rope_write_fp4");
  PoolShape shape;
  pkv_status st = check_pool_fp4(pool, &shape);
  if (st != PKV_OK) return st;
  if (!float_type(dtype)) return PKV_ERR_DTYPE;
  if (num_tokens < 0) return PKV_ERR_SHAPE;
  NormRopeArgs a{};
  a.dtype = dtype;
  a.num_tokens = num_tokens;
  a.n_heads = n_heads;
  a.n_kv = shape.n_kv;
  a.head_dim = shape.head_dim;
  st = check_norm_rope(q, q_stride, k, k_stride, rope, q_out, q_out_stride, err_word, &a);
  if (st != PKV_OK || num_tokens == 0) return st;
  st = check_slots(v, v_stride, slot_mapping, k_pool, v_pool, shape, &a);
  if (st == PKV_OK) st = check_groups(k_groups, v_groups, k_scale, v_scale);
  if (st != PKV_OK) return st;
  if (too_many(a)) return PKV_ERR_RANGE;
  set_groups(k_groups, v_groups, k_scale, v_scale, &a);
  return from_cuda(pkv::launch_norm_rope(a, as_stream(stream)));
}

pkv_status pkv_kv_write_fp4(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            int32_t dtype, const int64_t* slot_mapping, int32_t num_tokens,
                            void* k_pool, void* v_pool, void* k_groups, void* v_groups,
                            const float* k_scale, const float* v_scale, const pkv_pool_desc* pool,
                            int32_t* err_word, void* stream) {
  PKV_NVTX_RANGE("pkv_kv_write_fp4");
  PoolShape shape;
  pkv_status st = check_pool_fp4(pool, &shape);
  if (st != PKV_OK) return st;
  if (!float_type(dtype)) return PKV_ERR_DTYPE;
  if (num_tokens < 0) return PKV_ERR_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  NormRopeArgs a{};
  a.dtype = dtype;
  a.num_tokens = num_tokens;
  a.n_kv = shape.n_kv;
  a.head_dim = shape.head_dim;
  a.err = err_word;
  st = check_rows(k, k_stride, num_tokens, a.n_kv, a.head_dim, dtype);
  if (st == PKV_OK) st = check_slots(v, v_stride, slot_mapping, k_pool, v_pool, shape, &a);
  if (st == PKV_OK) st = check_groups(k_groups, v_groups, k_scale, v_scale);
  if (st != PKV_OK) return st;
  if (too_many(a)) return PKV_ERR_RANGE;
  a.k = k;
  a.k_stride = k_stride;
  set_groups(k_groups, v_groups, k_scale, v_scale, &a);
  return from_cuda(pkv::launch_norm_rope(a, as_stream(stream)));
}

pkv_status pkv_kv_gather_fp4(const void* k_pool, const void* v_pool, const void* k_groups,
                             const void* v_groups, const float* k_scale, const float* v_scale,
                             const pkv_pool_desc* pool, const int32_t* block_tables,
                             int32_t max_blocks_per_seq, const int32_t* seq_lens,
                             const int32_t* cu_seq_lens, int32_t num_seqs, int32_t total_tokens,
                             int32_t dtype, void* k_out, void* v_out, int32_t* err_word,
                             void* stream) {
  PKV_NVTX_RANGE("pkv_kv_gather_fp4");
  PoolShape shape;
  pkv_status st = check_pool_fp4(pool, &shape);
  if (st != PKV_OK) return st;
  if (!float_type(dtype)) return PKV_ERR_DTYPE;
  if (num_seqs < 0 || total_tokens < 0 || max_blocks_per_seq < 0) return PKV_ERR_SHAPE;
  if (total_tokens == 0) return PKV_OK;
  if (num_seqs == 0 || max_blocks_per_seq == 0) return PKV_ERR_SHAPE;
  if (!k_pool || !v_pool || !block_tables || !seq_lens || !cu_seq_lens || !k_out || !v_out)
    return PKV_ERR_NULL;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_out) || !aligned16(v_out))
    return PKV_ERR_ALIGN;
  if ((st = check_groups(k_groups, v_groups, k_scale, v_scale)) != PKV_OK) return st;
  const Fp4Cache c{k_pool, v_pool, k_groups, v_groups, k_scale, v_scale};
  return from_cuda(pkv::launch_kv_gather_fp4(c, shape, block_tables, max_blocks_per_seq, seq_lens,
                                             cu_seq_lens, num_seqs, total_tokens, dtype, k_out,
                                             v_out, err_word, as_stream(stream)));
}

size_t pkv_decode_fp4_workspace_bytes(int32_t num_seqs, int32_t n_heads, int32_t head_dim,
                                      int32_t max_seq_len, int32_t max_ctas, int32_t block_size) {
  (void)max_seq_len;
  (void)max_ctas;
  (void)block_size;
  return pkv::decode_fp8_workspace_bytes(num_seqs < 0 ? 0 : num_seqs, n_heads < 1 ? 1 : n_heads,
                                         head_dim < 1 ? 1 : head_dim);
}

pkv_status pkv_paged_attention_decode_fp4(
    const void* q, int32_t dtype, int32_t num_seqs, int32_t n_heads, const void* k_pool,
    const void* v_pool, const void* k_groups, const void* v_groups, const float* k_scale,
    const float* v_scale, const pkv_pool_desc* pool, const int32_t* block_tables,
    int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t max_seq_len, float scale,
    int32_t max_ctas, void* out, void* workspace, size_t workspace_bytes, int32_t* err_word,
    void* stream) {
  PKV_NVTX_RANGE("pkv_paged_attention_decode_fp4");
  const Fp4Cache c{k_pool, v_pool, k_groups, v_groups, k_scale, v_scale};
  pkv::AttnArgs a{};
  const pkv_status st =
      check_attention_fp4(q, dtype, num_seqs, n_heads, c, pool, block_tables, max_blocks_per_seq,
                          seq_lens, max_seq_len, scale, out, err_word, &a);
  if (st != PKV_OK) return st;
  if (max_ctas < 0) return PKV_ERR_RANGE;
  // (units of the work split are counted in 32 bits)
  if (int64_t(num_seqs) * a.pool.n_kv > INT32_MAX ||
      int64_t(num_seqs) * a.pool.n_kv * ((int64_t(max_seq_len) + 15) / 16) > INT32_MAX)
    return PKV_ERR_RANGE;
  if (num_seqs == 0) return PKV_OK;
  if (!workspace || workspace_bytes < pkv::decode_fp8_workspace_bytes(num_seqs, n_heads,
                                                                      a.pool.head_dim))
    return PKV_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PKV_ERR_ALIGN;
  a.max_q_len = 1;
  a.total_q = num_seqs;
  a.max_ctas = max_ctas;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  return from_cuda(pkv::launch_decode_fp4(a, dtype, c, as_stream(stream)));
}

pkv_status pkv_paged_attention_prefill_fp4(
    const void* q, int32_t dtype, const int32_t* cu_q_lens, int32_t num_seqs, int32_t total_q,
    int32_t max_q_len, int32_t n_heads, const void* k_pool, const void* v_pool,
    const void* k_groups, const void* v_groups, const float* k_scale, const float* v_scale,
    const pkv_pool_desc* pool, const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens, int32_t max_seq_len, float scale, void* out, int32_t* err_word,
    void* stream) {
  PKV_NVTX_RANGE("pkv_paged_attention_prefill_fp4");
  const Fp4Cache c{k_pool, v_pool, k_groups, v_groups, k_scale, v_scale};
  pkv::AttnArgs a{};
  const pkv_status st =
      check_attention_fp4(q, dtype, num_seqs, n_heads, c, pool, block_tables, max_blocks_per_seq,
                          seq_lens, max_seq_len, scale, out, err_word, &a);
  if (st != PKV_OK) return st;
  if (total_q < 0 || max_q_len < 0) return PKV_ERR_SHAPE;
  if (num_seqs == 0 || total_q == 0) return PKV_OK;
  if (!cu_q_lens) return PKV_ERR_NULL;
  if (max_q_len == 0 || max_q_len > total_q || max_q_len > max_seq_len) return PKV_ERR_SHAPE;
  a.cu_q_lens = cu_q_lens;
  a.max_q_len = max_q_len;
  a.total_q = total_q;
  return from_cuda(pkv::launch_prefill_fp4(a, dtype, c, as_stream(stream)));
}

}  // extern "C"
