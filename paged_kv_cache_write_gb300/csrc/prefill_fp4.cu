// Prefill over the 4-bit cache: the warp path for bf16 queries of narrow heads
// (kernels in prefill_fp4.cuh) and the dispatch: bf16 queries of head_dim 64 and 128
// go to the tcgen05 kernel (prefill_fp4_tc.cu).
#include "prefill_fp4.cuh"

namespace pkv {

namespace fp4 {
cudaError_t prefill_fp4_f32(const AttnArgs& a, const Fp4Cache& c, cudaStream_t s);
}

cudaError_t launch_prefill_fp4(const AttnArgs& a, int32_t dtype, const Fp4Cache& c, cudaStream_t s) {
  using namespace fp4;
  if (a.num_seqs == 0 || a.max_q_len == 0) return cudaSuccess;
  if (dtype == PKV_F32) return prefill_fp4_f32(a, c, s);
  switch (a.pool.head_dim) {
    case 16: return prefill_run<__nv_bfloat16, 16>(a, c, s);
    case 32: return prefill_run<__nv_bfloat16, 32>(a, c, s);
    default: return launch_prefill_fp4_tc(a, c, s);
  }
}

}  // namespace pkv
