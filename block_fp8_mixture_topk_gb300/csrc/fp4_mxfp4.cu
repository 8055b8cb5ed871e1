// The experts' 4-bit products in mxfp4.
#include "fp4_experts.cuh"

namespace mfp8 {
template <>
cudaError_t fp4_experts_init<MOE_FP4_MXFP4>() {
    return Fp4Launch<MOE_FP4_MXFP4>::init();
}
template <>
cudaError_t fp4_experts_launch<MOE_FP4_MXFP4>(int dtype, int mode, const Fp4Args& a, const CUtensorMap (&tm)[5],
                                              int64_t most_items, cudaStream_t stream) {
    return Fp4Launch<MOE_FP4_MXFP4>::launch(dtype, mode, a, tm, most_items, stream);
}
}  // namespace mfp8
