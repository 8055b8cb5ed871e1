// Global norm of many gradient tensors, and their clipping.
//
//   total = sqrt(sum_i |g_i|^2) or max_i |g_i|,  scale = min(1, max_norm / (total + eps)),  g *= scale
//
// Bound by memory: one pass reads the gradients for the norm, a second reads and writes them.  The
// tensors' addresses travel in the kernels' parameters (up to kMostTensors per launch), so nothing
// is copied to the device and a captured graph holds its own copy.  The tensors are cut into
// chunks; CTA c takes chunks c, c + CTAs, ... and leaves one partial result, and every CTA of the
// scaling kernel joins all partials in one order: the result does not depend on the schedule.
// Squares are summed in fp32 within a thread's share of a chunk and in fp64 beyond it; a share
// whose largest magnitude lies outside 1e-18 .. 1e18, where fp32 squares overflow or vanish, is
// summed again in fp64.
#include <math.h>

#include "train.cuh"

namespace mfp8 {
namespace {

constexpr int kClipThreads = 512;
constexpr int kVecs = 4;                  // 16-byte vectors of a thread's share
constexpr int kChunkBytes = kClipThreads * kVecs * 16;
constexpr int kMostTensors = 960;         // per launch: their table fits the 32,764 bytes of kernel parameters
constexpr int kClipCtasPerSm = 3;
constexpr int kMostCtas = kPlanSms * kClipCtasPerSm;   // partial results

template <int N>
struct ClipTable {
    const void* src[N];
    void* dst[N];
    int64_t numel[N];
    int64_t chunk0[N + 1];                // first chunk of each tensor
    uint8_t dtype[N];
    int n;
};

template <int N>
__device__ __forceinline__ int tensor_of(const ClipTable<N>& t, int64_t chunk) {
    int lo = 0, hi = t.n - 1;             // the last tensor whose first chunk is <= chunk
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.chunk0[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Partial results joined: sums, or the largest (held as doubles of fp32 values).
__device__ __forceinline__ double join(double a, double b, int inf) {
    return inf ? static_cast<double>(max_nan(static_cast<float>(a), static_cast<float>(b))) : a + b;
}
// Over the CTA's threads; the result in every thread.
__device__ __forceinline__ double join_cta(double acc, int inf, double* warp_s) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) acc = join(acc, __shfl_xor_sync(0xffffffffu, acc, s), inf);
    if ((threadIdx.x & 31) == 0) warp_s[threadIdx.x >> 5] = acc;
    __syncthreads();
    acc = warp_s[0];
    for (int w = 1; w < kClipThreads / 32; ++w) acc = join(acc, warp_s[w], inf);
    return acc;
}

// One thread's elements of a chunk: the vectors tid, tid + threads, ... of an aligned tensor, single
// elements otherwise and past the last whole vector.  f(value) is called for each.
template <class T, class F>
__device__ __forceinline__ void each_element(const T* p, int64_t n, bool wide, F f) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    int64_t tail = 0;
    if (wide) {
        const int64_t nv = n / V;
        Pack<T, V> x[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t v = threadIdx.x + i * kClipThreads;
            if (v < nv) x[i].load(p + v * V);
            else x[i].zero();
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) f(x[i].get(e));
        tail = nv * V;
    }
    for (int64_t i = tail + threadIdx.x; i < n; i += kClipThreads) f(to_f32(p[i]));
}

template <class T>
__device__ __forceinline__ double share_norm(const T* p, int64_t n, bool wide, bool inf) {
    float ss = 0.0f, top = 0.0f;
    each_element<T>(p, n, wide, [&](float v) {
        ss = fmaf(v, v, ss);
        top = max_nan(top, fabsf(v));
    });
    if (inf) return top;
    if (top > 1e18f || (top < 1e-18f && top > 0.0f)) {
        double sd = 0.0;
        each_element<T>(p, n, wide, [&](float v) { sd = fma(static_cast<double>(v), static_cast<double>(v), sd); });
        return sd;
    }
    return ss;
}

// The partial result of CTA b: sum of squares (or largest magnitude) of chunks b, b + CTAs, ...
template <int N>
__global__ void __launch_bounds__(kClipThreads)
    grad_norm_kernel(const __grid_constant__ ClipTable<N> t, int inf, double* __restrict__ partial) {
    __shared__ double warp_s[kClipThreads / 32];
    grid_dependency_wait();
    double acc = 0.0;
    const int64_t chunks = t.chunk0[t.n];
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int k = tensor_of(t, c);
        const int64_t per = t.dtype[k] == MOE_DTYPE_FP32 ? kChunkBytes / 4 : kChunkBytes / 2;
        const int64_t e0 = (c - t.chunk0[k]) * per;
        const int64_t n = t.numel[k] - e0 < per ? t.numel[k] - e0 : per;
        const bool wide = (reinterpret_cast<uintptr_t>(t.src[k]) & 15) == 0;
        double v;
        if (t.dtype[k] == MOE_DTYPE_FP32) v = share_norm(static_cast<const float*>(t.src[k]) + e0, n, wide, inf);
        else if (t.dtype[k] == MOE_DTYPE_FP16) v = share_norm(static_cast<const __half*>(t.src[k]) + e0, n, wide, inf);
        else v = share_norm(static_cast<const __nv_bfloat16*>(t.src[k]) + e0, n, wide, inf);
        acc = join(acc, v, inf);
    }
    acc = join_cta(acc, inf, warp_s);
    if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

template <class T>
__device__ __forceinline__ void scale_share(const T* p, T* q, int64_t n, bool wide, float scale) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    int64_t tail = 0;
    if (wide) {
        const int64_t nv = n / V;
        Pack<T, V> x[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t v = threadIdx.x + i * kClipThreads;
            if (v < nv) x[i].raw = *reinterpret_cast<const typename Pack<T, V>::Raw*>(p + v * V);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t v = threadIdx.x + i * kClipThreads;
            if (v >= nv) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) x[i].set(e, x[i].get(e) * scale);
            x[i].store(q + v * V);
        }
        tail = nv * V;
    }
    for (int64_t i = tail + threadIdx.x; i < n; i += kClipThreads) q[i] = from_f32<T>(to_f32(p[i]) * scale);
}

// Every CTA joins the partial results (np of them) and scales its chunks, the last first: they are
// the ones the norm read last, so they are still in L2.  A scale of one leaves gradients that stay
// in place alone.
template <int N>
__global__ void __launch_bounds__(kClipThreads)
    grad_scale_kernel(const __grid_constant__ ClipTable<N> t, int inf, const double* __restrict__ partial, int np,
                      float max_norm, float eps, int write_total, float* __restrict__ total) {
    __shared__ double warp_s[kClipThreads / 32];
    grid_dependency_wait();
    double acc = 0.0;
    for (int i = threadIdx.x; i < np; i += kClipThreads) acc = join(acc, partial[i], inf);
    acc = join_cta(acc, inf, warp_s);
    const double norm = inf ? acc : sqrt(acc);
    if (write_total && blockIdx.x == 0 && threadIdx.x == 0) *total = static_cast<float>(norm);
    const double ratio = static_cast<double>(max_norm) / (norm + static_cast<double>(eps));
    const float scale = ratio > 1.0 ? 1.0f : static_cast<float>(ratio);   // a NaN stays
    const int64_t chunks = t.chunk0[t.n];
    for (int64_t i = blockIdx.x; i < chunks; i += gridDim.x) {
        const int64_t c = chunks - 1 - i;
        const int k = tensor_of(t, c);
        if (scale == 1.0f && t.src[k] == t.dst[k]) continue;
        const int64_t per = t.dtype[k] == MOE_DTYPE_FP32 ? kChunkBytes / 4 : kChunkBytes / 2;
        const int64_t e0 = (c - t.chunk0[k]) * per;
        const int64_t n = t.numel[k] - e0 < per ? t.numel[k] - e0 : per;
        const bool wide = ((reinterpret_cast<uintptr_t>(t.src[k]) | reinterpret_cast<uintptr_t>(t.dst[k])) & 15) == 0;
        if (t.dtype[k] == MOE_DTYPE_FP32)
            scale_share(static_cast<const float*>(t.src[k]) + e0, static_cast<float*>(t.dst[k]) + e0, n, wide, scale);
        else if (t.dtype[k] == MOE_DTYPE_FP16)
            scale_share(static_cast<const __half*>(t.src[k]) + e0, static_cast<__half*>(t.dst[k]) + e0, n, wide, scale);
        else
            scale_share(static_cast<const __nv_bfloat16*>(t.src[k]) + e0, static_cast<__nv_bfloat16*>(t.dst[k]) + e0, n,
                        wide, scale);
    }
}

int64_t chunks_of(int64_t numel, int dtype) {
    const int64_t per = kChunkBytes / static_cast<int64_t>(dtype_bytes(dtype));
    return (numel + per - 1) / per;
}

struct ClipCall {
    const void* const* src;
    void* const* dst;
    const int64_t* numel;
    const int32_t* dtype;
    int n, inf;
    float max_norm, eps;
    float* total;
    double* partial;
    cudaStream_t stream;
};

template <int N>
void fill_table(ClipTable<N>* t, const ClipCall& c, int k0, int k1) {
    t->n = k1 - k0;
    t->chunk0[0] = 0;
    for (int k = k0; k < k1; ++k) {
        const int i = k - k0;
        t->src[i] = c.src[k];
        t->dst[i] = c.dst[k];
        t->numel[i] = c.numel[k];
        t->dtype[i] = static_cast<uint8_t>(c.dtype[k]);
        t->chunk0[i + 1] = t->chunk0[i] + chunks_of(c.numel[k], c.dtype[k]);
    }
}

unsigned clip_grid(int64_t chunks) {
    return static_cast<unsigned>(chunks < 1 ? 1 : chunks < kMostCtas ? chunks : kMostCtas);
}

// Launches of at most N tensors each: the norms (their partial results one after another), then
// the scaling.
template <int N>
cudaError_t clip_launches(const ClipCall& c) {
    static thread_local ClipTable<N> t;
    cudaError_t e = cudaSuccess;
    int np = 0;
    const int batches = c.n > 0 ? (c.n + N - 1) / N : 1;
    for (int b = 0; b < batches && e == cudaSuccess; ++b) {
        fill_table(&t, c, b * N, c.n < (b + 1) * N ? c.n : (b + 1) * N);
        const unsigned grid = clip_grid(t.chunk0[t.n]);
        e = launch_pdl(grad_norm_kernel<N>, dim3(grid), dim3(kClipThreads), 0, c.stream, t, c.inf, c.partial + np);
        np += static_cast<int>(grid);
    }
    for (int b = 0; b < batches && e == cudaSuccess; ++b) {
        if (batches > 1) fill_table(&t, c, b * N, c.n < (b + 1) * N ? c.n : (b + 1) * N);
        e = launch_pdl(grad_scale_kernel<N>, dim3(clip_grid(t.chunk0[t.n])), dim3(kClipThreads), 0, c.stream, t, c.inf,
                       static_cast<const double*>(c.partial), np, c.max_norm, c.eps, b == 0 ? 1 : 0, c.total);
    }
    return e;
}

}  // namespace
}  // namespace mfp8

using namespace mfp8;

extern "C" {

size_t moe_clip_grads_workspace_size(int n) {
    if (n < 0) return 0;
    const size_t batches = n > 0 ? (static_cast<size_t>(n) + kMostTensors - 1) / kMostTensors : 1;
    return batches * kMostCtas * sizeof(double);
}

int moe_clip_grads(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* dtype, int n,
                   int norm_kind, float max_norm, float eps, float* total_norm, void* workspace,
                   size_t workspace_bytes, void* stream) {
    if (n < 0 || (norm_kind != MOE_NORM_L2 && norm_kind != MOE_NORM_INF)) return MOE_ERR_INVALID_ARG;
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || !total_norm) return MOE_ERR_INVALID_ARG;
    if (n > 0 && (!grads || !out || !numel || !dtype)) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        if (numel[i] < 0 || !known_dtype(dtype[i])) return MOE_ERR_INVALID_ARG;
        if (numel[i] > 0 && (!grads[i] || !out[i])) return MOE_ERR_INVALID_ARG;
        if (!on_element(address(grads[i]) | address(out[i]), dtype_bytes(dtype[i]))) return MOE_ERR_INVALID_ARG;
        if (numel[i] > (int64_t(1) << 50)) return MOE_ERR_UNSUPPORTED_SHAPE;
    }
    if (workspace_bytes < moe_clip_grads_workspace_size(n)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace || !on_element(address(workspace), 8)) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    const int rc = device_status_word(&status);
    if (rc != MOE_OK) return rc;
    const ClipCall c = {grads, out, numel, dtype, n, norm_kind == MOE_NORM_INF ? 1 : 0, max_norm, eps, total_norm,
                        static_cast<double*>(workspace), static_cast<cudaStream_t>(stream)};
    return cuda_status(n <= 32 ? clip_launches<32>(c) : n <= 128 ? clip_launches<128>(c)
                                                                 : clip_launches<kMostTensors>(c));
}

}  // extern "C"
