// Prefill over the 4-bit cache for fp32 queries (kernels in prefill_fp4.cuh).
#include "prefill_fp4.cuh"

namespace pkv {
namespace fp4 {
cudaError_t prefill_fp4_f32(const AttnArgs& a, const Fp4Cache& c, cudaStream_t s) {
  switch (a.pool.head_dim) {
    case 16: return prefill_run<float, 16>(a, c, s);
    case 32: return prefill_run<float, 32>(a, c, s);
    case 64: return prefill_run<float, 64>(a, c, s);
    default: return prefill_run<float, 128>(a, c, s);
  }
}
}  // namespace fp4
}  // namespace pkv
