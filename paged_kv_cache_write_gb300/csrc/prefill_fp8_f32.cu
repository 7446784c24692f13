// Prefill over the 8-bit cache for fp32 queries (kernels in prefill_fp8.cuh).
#include "prefill_fp8.cuh"

namespace pkv {
namespace fp8 {
cudaError_t prefill_fp8_f32(const AttnArgs& a, const Scales& sc, cudaStream_t s) {
  switch (a.pool.head_dim) {
    case 16: return prefill_run<float, 16>(a, sc, s);
    case 32: return prefill_run<float, 32>(a, sc, s);
    case 64: return prefill_run<float, 64>(a, sc, s);
    default: return prefill_run<float, 128>(a, sc, s);
  }
}
}  // namespace fp8
}  // namespace pkv
