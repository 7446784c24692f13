// Prefill over the 8-bit cache: the warp path for bf16 queries and the
// dispatch by type (kernels in prefill_fp8.cuh).
#include "prefill_fp8.cuh"

namespace pkv {

namespace fp8 {
cudaError_t prefill_fp8_f32(const AttnArgs& a, const Scales& sc, cudaStream_t s);
}

cudaError_t launch_prefill_fp8(const AttnArgs& a, int32_t dtype, const float* k_scales,
                               const float* v_scales, cudaStream_t s) {
  using namespace fp8;
  if (a.num_seqs == 0 || a.max_q_len == 0) return cudaSuccess;
  const Scales sc{k_scales, v_scales};
  if (dtype == PKV_F32) return prefill_fp8_f32(a, sc, s);
  switch (a.pool.head_dim) {
    case 16: return prefill_run<__nv_bfloat16, 16>(a, sc, s);
    case 32: return prefill_run<__nv_bfloat16, 32>(a, sc, s);
    case 64: return prefill_run<__nv_bfloat16, 64>(a, sc, s);
    default: return prefill_run<__nv_bfloat16, 128>(a, sc, s);
  }
}

}  // namespace pkv
