// The router on fp16 logits.
#define MOE_ROUTER_KERNELS
#include "router.cuh"

namespace mfp8 {
template cudaError_t router_forward<__half>(const RouterArgs&, int, cudaStream_t);
template cudaError_t router_backward<__half>(const RouterBackwardArgs&, cudaStream_t);
}  // namespace mfp8
