// The block norms (norms.cuh) on rows of type bf16.
#include "norms.cuh"

namespace mfp8 {
cudaError_t launch_norm_bf16(const NormArgs& a, int which, int gate, bool wide, int sms, cudaStream_t stream,
                             int* ctas) {
    return launch_norm_type<__nv_bfloat16>(a, which, gate, wide, sms, stream, ctas);
}
}  // namespace mfp8
