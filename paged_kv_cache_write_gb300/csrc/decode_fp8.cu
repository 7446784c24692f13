// Decode over the 8-bit cache for bf16 queries, and the dispatch by type
// (kernels in decode_fp8.cuh).
#include "decode_fp8.cuh"

namespace pkv {

namespace fp8 {
cudaError_t decode_fp8_bf16(const AttnArgs& a, const Scales& sc, cudaStream_t s) {
  return decode_as<__nv_bfloat16>(a, sc, s);
}
}  // namespace fp8

bool fp8_attention_supported(const PoolShape& pool, int32_t n_heads) {
  const int hd = pool.head_dim;
  if (pool.block_size != fp8::kBS || n_heads % pool.n_kv != 0) return false;
  if (n_heads / pool.n_kv > attn::kMaxRep) return false;
  return hd == 16 || hd == 32 || hd == 64 || hd == 128;
}

// The plan's and the partials' layout is the bf16 decode's, and so is its bound.
size_t decode_fp8_workspace_bytes(int32_t num_seqs, int32_t n_heads, int32_t head_dim) {
  return attn::DecodeWs(num_seqs, size_t(sm_count()) * 16, size_t(n_heads), head_dim).total;
}

cudaError_t launch_decode_fp8(const AttnArgs& a, int32_t dtype, const float* k_scales,
                              const float* v_scales, cudaStream_t s) {
  const fp8::Scales sc{k_scales, v_scales};
  return dtype == PKV_F32 ? fp8::decode_fp8_f32(a, sc, s) : fp8::decode_fp8_bf16(a, sc, s);
}

}  // namespace pkv
