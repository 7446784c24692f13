// Decode over the 4-bit cache for bf16 queries, and the dispatch by type (kernels in
// decode_fp4.cuh).
#include "decode_fp4.cuh"

namespace pkv {

namespace fp4 {
cudaError_t decode_fp4_bf16(const AttnArgs& a, const Fp4Cache& c, cudaStream_t s) {
  return decode_as<__nv_bfloat16>(a, c, s);
}
}  // namespace fp4

cudaError_t launch_decode_fp4(const AttnArgs& a, int32_t dtype, const Fp4Cache& c, cudaStream_t s) {
  return dtype == PKV_F32 ? fp4::decode_fp4_f32(a, c, s) : fp4::decode_fp4_bf16(a, c, s);
}

}  // namespace pkv
