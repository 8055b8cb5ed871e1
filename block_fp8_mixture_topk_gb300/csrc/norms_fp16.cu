// The block norms (norms.cuh) on rows of type fp16.
#include "norms.cuh"

namespace mfp8 {
cudaError_t launch_norm_fp16(const NormArgs& a, int which, int gate, bool wide, int sms, cudaStream_t stream,
                             int* ctas) {
    return launch_norm_type<__half>(a, which, gate, wide, sms, stream, ctas);
}
}  // namespace mfp8
