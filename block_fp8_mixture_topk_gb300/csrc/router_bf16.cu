// The router on bf16 logits.
#define MOE_ROUTER_KERNELS
#include "router.cuh"

namespace mfp8 {
template cudaError_t router_forward<__nv_bfloat16>(const RouterArgs&, int, cudaStream_t);
template cudaError_t router_backward<__nv_bfloat16>(const RouterBackwardArgs&, cudaStream_t);
}  // namespace mfp8
