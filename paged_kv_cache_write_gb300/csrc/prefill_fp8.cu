// Prefill over the 8-bit cache: the warp path for bf16 queries of narrow
// heads (kernels in prefill_fp8.cuh) and the dispatch: bf16 queries of
// head_dim 64 and 128 go to the tcgen05 kernel (prefill_fp8_tc.cu).
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
    default: return launch_prefill_fp8_tc(a, k_scales, v_scales, s);
  }
}

}  // namespace pkv
