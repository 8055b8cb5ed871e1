// The router on fp32 logits.
#define MOE_ROUTER_KERNELS
#include "router.cuh"

namespace mfp8 {
template cudaError_t router_forward<float>(const RouterArgs&, int, cudaStream_t);
template cudaError_t router_backward<float>(const RouterBackwardArgs&, cudaStream_t);
}  // namespace mfp8
