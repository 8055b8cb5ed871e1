// The router's entry points, the last step of its loads and losses, and the update of the balancing bias.
#include "router.cuh"

namespace mfp8 {
namespace {

constexpr int kFinalCtas = 8, kFinalThreads = 1024;

// The blocks' sums: expert chunk by CTA of one cluster (a thread adds every (threads / chunk)-th block, those sums in order),
// whose shares of the balance loss the first CTA adds up.
__global__ void __cluster_dims__(kFinalCtas, 1, 1) __launch_bounds__(kFinalThreads)
    router_loads_kernel(const float* share, const int32_t* count, const float* z, const int32_t* live, int blocks, int E, int k,
                        int32_t* counts, int32_t* tokens, float* losses) {
    cluster_arrive();   // this CTA runs
    grid_dependency_wait();
    __shared__ float s_share[kFinalThreads], s_part[kFinalCtas];
    __shared__ int s_count[kFinalThreads];
    __shared__ float s_z[kFinalThreads / 32];
    __shared__ int s_live[kFinalThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = (E + kFinalCtas - 1) / kFinalCtas;   // <= 128
    const int rank = static_cast<int>(cluster_rank());
    // tokens and z, in every CTA
    int n = 0;
    float zs = 0.0f;
    for (int b = threadIdx.x; b < blocks; b += kFinalThreads) {
        n += live[b];
        zs += z[b];
    }
    n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) zs += __shfl_xor_sync(0xffffffffu, zs, o);
    if (lane == 0) s_live[warp] = n, s_z[warp] = zs;
    const int rows = kFinalThreads / chunk, mine = threadIdx.x % chunk, r = threadIdx.x / chunk;
    const int e = rank * chunk + mine;
    float s = 0.0f;
    int c = 0;
    if (r < rows && e < E)
#pragma unroll 4
        for (int b = r; b < blocks; b += rows) {
            s += share[static_cast<int64_t>(b) * E + e];
            c += count[static_cast<int64_t>(b) * E + e];
        }
    s_share[threadIdx.x] = s;
    s_count[threadIdx.x] = c;
    __syncthreads();
    float part = 0.0f;
    if (r == 0 && e < E) {
        for (int i = 1; i < rows; ++i) {
            s += s_share[i * chunk + mine];
            c += s_count[i * chunk + mine];
        }
        counts[e] = c;
        part = s * static_cast<float>(c);
    }
    __syncthreads();
    s_share[threadIdx.x] = part;
    __syncthreads();
    cluster_wait();     // every CTA runs: the first one's shared memory can be written
    if (threadIdx.x < 32) {   // chunk <= 128: four to a lane
        float v = 0.0f;
        for (int i = lane; i < chunk; i += 32) v += s_share[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) {
            const uint32_t to = cluster_map(smem_addr(&s_part[rank]), 0);
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
        }
    }
    __syncwarp();
    cluster_barrier();
    if (rank == 0 && threadIdx.x == 0) {
        int tokens_all = 0;
        float z_all = 0.0f, v = 0.0f;
        for (int i = 0; i < kFinalThreads / 32; ++i) tokens_all += s_live[i], z_all += s_z[i];
        for (int i = 0; i < kFinalCtas; ++i) v += s_part[i];
        const float by = tokens_all > 0 ? 1.0f / static_cast<float>(tokens_all) : 0.0f;
        *tokens = tokens_all;
        losses[0] = v * (static_cast<float>(E) / static_cast<float>(k)) * by * by;
        losses[1] = z_all * by;
    }
}

// bias[e] += rate * sign(mean(counts) - counts[e]), over the experts that a bias of -inf does not mask: counted among them, the
// masked ones' empty loads would put the mean below what the others share evenly, and each step would push all of those down.
__global__ void __launch_bounds__(1024) router_bias_kernel(float* bias, const int32_t* counts, int E, float rate) {
    grid_dependency_wait();
    __shared__ long long s_sum[32];
    __shared__ int s_able[32];
    const int e = threadIdx.x, lane = e & 31;
    const float b = e < E ? bias[e] : -INFINITY;
    const bool able = b > -INFINITY;
    const int32_t c = able ? counts[e] : 0;
    long long sum = c;
    int n = able ? 1 : 0;
    const auto add = [&] {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        n = __reduce_add_sync(0xffffffffu, n);
    };
    add();
    if (lane == 0) s_sum[e >> 5] = sum, s_able[e >> 5] = n;
    __syncthreads();
    sum = s_sum[lane], n = s_able[lane];
    add();
    const long long mine = static_cast<long long>(c) * n;
    if (able && mine != sum) bias[e] = b + (mine < sum ? rate : -rate);
}

// Blocks of a launch: one to an SM, or to a token.
int router_blocks(int T) { return T < kPlanSms ? T : kPlanSms; }

int check_router(int dtype, int64_t ld, int T, int E, int k, const moe_router_params* p) {
    if (!p || !known_dtype(dtype) || T < 0 || E < 1 || k < 1) return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS || k > E || k > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (ld < E || (p->scoring != MOE_SCORING_SOFTMAX && p->scoring != MOE_SCORING_SIGMOID)) return MOE_ERR_INVALID_ARG;
    if (p->n_group < 1 || (p->group_score != MOE_GROUP_TOP2 && p->group_score != MOE_GROUP_MAX)) return MOE_ERR_INVALID_ARG;
    if (p->n_group > MOE_MAX_GROUPS || E % p->n_group != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (p->n_group > 1) {
        if (p->topk_group < 1 || p->topk_group > p->n_group) return MOE_ERR_INVALID_ARG;
        if (k > E / p->n_group * p->topk_group) return MOE_ERR_UNSUPPORTED_SHAPE;
    }
    return MOE_OK;
}

}  // namespace
}  // namespace mfp8

using namespace mfp8;

extern "C" {

size_t moe_router_workspace_size(int T, int E) {
    if (T < 0 || E < 1 || E > MOE_MAX_EXPERTS) return 0;
    return static_cast<size_t>(router_blocks(T)) * (2 * static_cast<size_t>(E) + 2) * 4;
}

int moe_router(const void* logits, int64_t ld, int dtype, int T, int E, int topk, const moe_router_params* p,
               const uint8_t* valid, int32_t* ids, float* weights, int32_t* counts, int32_t* tokens, float* losses,
               void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_router(dtype, ld, T, E, topk, p);
    if (rc != MOE_OK) return rc;
    const bool stats = counts != nullptr;
    if ((tokens != nullptr) != stats || (losses != nullptr) != stats) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !ids || !weights)) return MOE_ERR_INVALID_ARG;
    const uintptr_t words = address(p->bias) | address(ids) | address(weights) | address(counts) | address(tokens) |
                            address(losses) | address(workspace);
    if (words % 4 || !on_element(address(logits), dtype_bytes(dtype))) return MOE_ERR_INVALID_ARG;
    if (stats && T > 0) {
        if (!workspace) return MOE_ERR_INVALID_ARG;
        if (workspace_bytes < moe_router_workspace_size(T, E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int blocks = router_blocks(T);
    RouterArgs a = {};
    a.logits = logits, a.ld = ld, a.T = T, a.E = E, a.k = topk;
    a.sigmoid = p->scoring == MOE_SCORING_SIGMOID, a.groups = p->n_group, a.kept = p->topk_group;
    if (a.kept == a.groups) a.groups = 1;   // all of them stay
    a.top2 = p->group_score == MOE_GROUP_TOP2, a.renorm = p->renormalize != 0, a.scaling = p->routed_scaling;
    a.bias = p->bias, a.valid = valid, a.ids = ids, a.weights = weights, a.status = status;
    if (stats) {
        a.part_share = static_cast<float*>(workspace);
        a.part_count = reinterpret_cast<int32_t*>(a.part_share + static_cast<size_t>(blocks) * E);
        a.part_z = reinterpret_cast<float*>(a.part_count + static_cast<size_t>(blocks) * E);
        a.part_live = reinterpret_cast<int32_t*>(a.part_z + blocks);
    }
    if (T > 0) {
        const cudaError_t e = dtype == MOE_DTYPE_BF16   ? router_forward<__nv_bfloat16>(a, blocks, s)
                              : dtype == MOE_DTYPE_FP16 ? router_forward<__half>(a, blocks, s)
                                                        : router_forward<float>(a, blocks, s);
        if (e != cudaSuccess) return cuda_status(e);
    }
    if (!stats) return MOE_OK;
    return cuda_status(launch_pdl(router_loads_kernel, dim3(kFinalCtas), dim3(kFinalThreads), 0, s,
                                  static_cast<const float*>(a.part_share), static_cast<const int32_t*>(a.part_count),
                                  static_cast<const float*>(a.part_z), static_cast<const int32_t*>(a.part_live),
                                  T > 0 ? blocks : 0, E, topk, counts, tokens, losses));
}

int moe_router_backward(const void* logits, int64_t ld, int dtype, int T, int E, int topk, const moe_router_params* p,
                        const int32_t* ids, const float* dweights, const int32_t* counts, const int32_t* tokens,
                        float balance_coef, float z_coef, void* dlogits, void* stream) {
    int rc = check_router(dtype, ld, T, E, topk, p);
    if (rc != MOE_OK) return rc;
    if ((balance_coef != 0.0f && !counts) || ((balance_coef != 0.0f || z_coef != 0.0f) && !tokens)) return MOE_ERR_INVALID_ARG;
    if (z_coef != 0.0f && p->scoring != MOE_SCORING_SOFTMAX) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!logits || !ids || !dweights || !dlogits) return MOE_ERR_INVALID_ARG;
    const uintptr_t words = address(ids) | address(dweights) | address(counts) | address(tokens);
    if (words % 4 || !on_element(address(logits) | address(dlogits), dtype_bytes(dtype))) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    RouterBackwardArgs a = {};
    a.logits = logits, a.ld = ld, a.T = T, a.E = E, a.k = topk;
    a.sigmoid = p->scoring == MOE_SCORING_SIGMOID, a.renorm = p->renormalize != 0, a.scaling = p->routed_scaling;
    a.ids = ids, a.dweights = dweights, a.counts = counts, a.live = tokens, a.balance = balance_coef, a.z = z_coef;
    a.dlogits = dlogits, a.status = status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(dtype == MOE_DTYPE_BF16   ? router_backward<__nv_bfloat16>(a, s)
                       : dtype == MOE_DTYPE_FP16 ? router_backward<__half>(a, s)
                                                 : router_backward<float>(a, s));
}

int moe_router_update_bias(float* bias, const int32_t* counts, int E, float rate, void* stream) {
    if (!bias || !counts || E < 1 || (address(bias) | address(counts)) % 4) return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED_SHAPE;
    uint32_t* status = nullptr;
    const int rc = device_status_word(&status);
    if (rc != MOE_OK) return rc;
    return cuda_status(launch_pdl(router_bias_kernel, dim3(1), dim3(1024), 0, static_cast<cudaStream_t>(stream), bias, counts,
                                  E, rate));
}

}  // extern "C"
