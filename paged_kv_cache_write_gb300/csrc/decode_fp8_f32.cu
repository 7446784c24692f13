// Decode over the 8-bit cache for fp32 queries (kernels in decode_fp8.cuh).
#include "decode_fp8.cuh"

namespace pkv {
namespace fp8 {
cudaError_t decode_fp8_f32(const AttnArgs& a, const Scales& sc, cudaStream_t s) {
  return decode_as<float>(a, sc, s);
}
}  // namespace fp8
}  // namespace pkv
