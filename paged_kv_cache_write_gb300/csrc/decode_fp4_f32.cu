// Decode over the 4-bit cache for fp32 queries (kernels in decode_fp4.cuh).
#include "decode_fp4.cuh"

namespace pkv {
namespace fp4 {
cudaError_t decode_fp4_f32(const AttnArgs& a, const Fp4Cache& c, cudaStream_t s) {
  return decode_as<float>(a, c, s);
}
}  // namespace fp4
}  // namespace pkv
