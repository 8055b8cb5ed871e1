// RMS norms before and after a block, with their gradients: kernels, templated over the rows' type.
//
// Before:    h = x * r * w,  r = 1/sqrt(mean(x^2) + eps)
// After:     out = a * residual + b * g * (y * r * w), and optionally the next block's norm of the
//            stored out in the same pass
// Backward, with n = y * r (the normalised row) and t = (gradient of n * w) * w:
//            dy = r * (t - n * mean(t * n)),  dw = sum over rows of (gradient of n * w) * n
// w stands for weight + weight_offset; g is a scalar per row, a row vector or a matrix, or its
// sigmoid.
//
// All are bound by memory: every element is read once and held in registers between the row's
// reduction and its use (at most 32 elements per thread, G threads per row).  A CTA holds R
// groups of G threads, each with its own named barrier, and walks over rows with the weights in
// registers.  The weights' gradient is summed over a CTA's rows in fp32 registers, over its groups in
// shared memory, written once per CTA and summed by a second kernel in a fixed order: no atomics,
// so the result does not depend on the schedule.
#pragma once

#include <atomic>

#include "train.cuh"

namespace mfp8 {

constexpr int kNormThreads = 512;   // most threads of a CTA
enum GateShape { kGateRow = 0, kGateChannel = 1, kGateFull = 2 };   // kGateRow also stands for no gate

struct NormArgs {
    int64_t T;
    int H, G;                   // columns, threads per row
    const void *x, *res, *gate; // x: the normed rows; res: residual (forward) / gradient joining dx (before, backward)
    int64_t ldx, ldr, ldg;
    const void* dout;           // backward: gradient of the result
    int64_t ldo;
    const void *w, *w2;         // weights of this norm and of the next
    int w_dtype;
    float w_offset, eps, a, b;
    int sigmoid;
    void *out, *h2, *dres, *dgate;
    float *rstd, *rstd2;        // forward: written; backward: rstd read
    float* partial;             // backward: [CTAs][H]
};

__device__ __forceinline__ float weight_at(const void* w, int dtype, int64_t i) {
    if (dtype == MOE_DTYPE_FP32) return static_cast<const float*>(w)[i];
    if (dtype == MOE_DTYPE_FP16) return __half2float(static_cast<const __half*>(w)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}
__device__ __forceinline__ float sigmoid_f32(float v) { return 1.0f / (1.0f + expf(-v)); }

struct Group {
    float* red;       // [2][16] of this group
    int G, tid, id, parity;
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
        if (G == 32) return v;
        float* slot = red + parity * 16;
        parity ^= 1;
        if ((tid & 31) == 0) slot[tid >> 5] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(G) : "memory");
        float t = 0.0f;
        for (int i = 0; i < G / 32; ++i) t += slot[i];
        return t;
    }
};

__device__ __forceinline__ Group make_group(float* red, int G) {
    Group g;
    g.G = G;
    g.id = threadIdx.x / G;
    g.tid = threadIdx.x % G;
    g.parity = 0;
    g.red = red + g.id * 32;
    return g;
}

template <class T, int V, int NV>
__device__ __forceinline__ void load_weights(float (&w)[NV * V], const void* p, int dtype, float offset, int tid,
                                             int G, int nvec) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int v = tid + i * G;
            w[i * V + e] = v < nvec ? weight_at(p, dtype, static_cast<int64_t>(v) * V + e) + offset : 0.0f;
        }
}
template <class T, int V, int NV>
__device__ __forceinline__ void load_row(Pack<T, V> (&r)[NV], const T* p, int tid, int G, int nvec) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = tid + i * G;
        if (v < nvec) r[i].load(p + static_cast<int64_t>(v) * V);
        else r[i].zero();
    }
}

// h = x * rstd * w
template <class T, int V, int NV>
__global__ void __launch_bounds__(kNormThreads) pre_norm_kernel(const NormArgs a) {
    __shared__ float red[16 * 32];
    Group g = make_group(red, a.G);
    const int nvec = a.H / V, R = blockDim.x / a.G;
    grid_dependency_wait();
    float w[NV * V];
    load_weights<T, V, NV>(w, a.w, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * R + g.id; t < a.T; t += static_cast<int64_t>(gridDim.x) * R) {
        Pack<T, V> x[NV];
        load_row<T, V, NV>(x, static_cast<const T*>(a.x) + t * a.ldx, g.tid, a.G, nvec);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(x[i].get(e), x[i].get(e), ss);
        const float r = __frsqrt_rn(g.sum(ss) / static_cast<float>(a.H) + a.eps);
        if (g.tid == 0) a.rstd[t] = r;
        T* out = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = g.tid + i * a.G;
            if (v >= nvec) continue;
            Pack<T, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) o.set(e, x[i].get(e) * r * w[i * V + e]);
            o.store(out + static_cast<int64_t>(v) * V);
        }
    }
}

// out = a * res + b * g * (y * rstd * w); NEXT: h2 = out * rstd2 * w2 of the stored out
template <class T, int V, int NV, int GATE, bool NEXT>
__global__ void __launch_bounds__(kNormThreads) post_norm_kernel(const NormArgs a) {
    __shared__ float red[16 * 32];
    Group g = make_group(red, a.G);
    const int nvec = a.H / V, R = blockDim.x / a.G;
    grid_dependency_wait();
    float w[NV * V], w2[NEXT ? NV * V : 1];
    load_weights<T, V, NV>(w, a.w, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
    if constexpr (NEXT) load_weights<T, V, NV>(w2, a.w2, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
    if constexpr (GATE == kGateChannel) {   // the gate scales the weight, for every row alike
        Pack<T, V> gt[NV];
        load_row<T, V, NV>(gt, static_cast<const T*>(a.gate), g.tid, a.G, nvec);
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
            const float v = gt[i / V].get(i % V);
            w[i] *= a.sigmoid ? sigmoid_f32(v) : v;
        }
    }
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * R + g.id; t < a.T; t += static_cast<int64_t>(gridDim.x) * R) {
        Pack<T, V> y[NV], s[NV], gt[GATE == kGateFull ? NV : 1];
        load_row<T, V, NV>(y, static_cast<const T*>(a.x) + t * a.ldx, g.tid, a.G, nvec);
        load_row<T, V, NV>(s, static_cast<const T*>(a.res) + t * a.ldr, g.tid, a.G, nvec);
        float b = a.b;
        if constexpr (GATE == kGateFull) {
            load_row<T, V, NV>(gt, static_cast<const T*>(a.gate) + t * a.ldg, g.tid, a.G, nvec);
        } else if constexpr (GATE == kGateRow) {
            if (a.gate) {
                const float v = to_f32(static_cast<const T*>(a.gate)[t * a.ldg]);
                b *= a.sigmoid ? sigmoid_f32(v) : v;
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(y[i].get(e), y[i].get(e), ss);
        const float r = __frsqrt_rn(g.sum(ss) / static_cast<float>(a.H) + a.eps);
        if (g.tid == 0) a.rstd[t] = r;
        T* out = static_cast<T*>(a.out) + t * a.H;
        float s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = g.tid + i * a.G;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float z = y[i].get(e) * r * w[i * V + e] * b;
                if constexpr (GATE == kGateFull) {
                    const float gv = gt[i].get(e);
                    z *= a.sigmoid ? sigmoid_f32(gv) : gv;
                }
                s[i].set(e, fmaf(a.a, s[i].get(e), z));
                if constexpr (NEXT) s2 = fmaf(s[i].get(e), s[i].get(e), s2);
            }
            if (v < nvec) s[i].store(out + static_cast<int64_t>(v) * V);
        }
        if constexpr (NEXT) {
            const float r2 = __frsqrt_rn(g.sum(s2) / static_cast<float>(a.H) + a.eps);
            if (g.tid == 0) a.rstd2[t] = r2;
            T* h2 = static_cast<T*>(a.h2) + t * a.H;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = g.tid + i * a.G;
                if (v >= nvec) continue;
                Pack<T, V> o;
#pragma unroll
                for (int e = 0; e < V; ++e) o.set(e, s[i].get(e) * r2 * w2[i * V + e]);
                o.store(h2 + static_cast<int64_t>(v) * V);
            }
        }
    }
}

// The CTA's sums over rows, group after group, into its row of the partials.
template <int V, int NV>
__device__ __forceinline__ void write_partial(const float (&acc)[NV * V], float* sum_s, const Group& g, int R,
                                              int nvec, float* partial) {
    for (int k = 0; k < R; ++k) {
        if (g.id == k) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = g.tid + i * g.G;
                if (v >= nvec) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float u = acc[i * V + e] + (k > 0 ? sum_s[v * V + e] : 0.0f);
                    if (k + 1 < R) sum_s[v * V + e] = u;
                    else partial[v * V + e] = u;
                }
            }
        }
        __syncthreads();
    }
}

// dx = rstd * (t - n * mean(t * n)) + res, t = dout * w; partial sums of dout * n
template <class T, int V, int NV>
__global__ void __launch_bounds__(kNormThreads) pre_norm_backward_kernel(const NormArgs a) {
    extern __shared__ float sum_s[];
    __shared__ float red[16 * 32];
    Group g = make_group(red, a.G);
    const int nvec = a.H / V, R = blockDim.x / a.G;
    grid_dependency_wait();
    float w[NV * V], acc[NV * V];
    load_weights<T, V, NV>(w, a.w, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
#pragma unroll
    for (int i = 0; i < NV * V; ++i) acc[i] = 0.0f;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * R + g.id; t < a.T; t += static_cast<int64_t>(gridDim.x) * R) {
        Pack<T, V> x[NV], d[NV], s[NV];
        load_row<T, V, NV>(x, static_cast<const T*>(a.x) + t * a.ldx, g.tid, a.G, nvec);
        load_row<T, V, NV>(d, static_cast<const T*>(a.dout) + t * a.ldo, g.tid, a.G, nvec);
        if (a.res) load_row<T, V, NV>(s, static_cast<const T*>(a.res) + t * a.ldr, g.tid, a.G, nvec);
        const float r = a.rstd[t];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
            const float n = x[i / V].get(i % V) * r, dv = d[i / V].get(i % V);
            m = fmaf(dv * w[i], n, m);
            acc[i] = fmaf(dv, n, acc[i]);
        }
        m = g.sum(m) / static_cast<float>(a.H);
        T* out = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = g.tid + i * a.G;
            if (v >= nvec) continue;
            Pack<T, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float n = x[i].get(e) * r;
                float u = r * fmaf(-n, m, d[i].get(e) * w[i * V + e]);
                if (a.res) u += s[i].get(e);
                o.set(e, u);
            }
            o.store(out + static_cast<int64_t>(v) * V);
        }
    }
    write_partial<V, NV>(acc, sum_s, g, R, nvec, a.partial + static_cast<int64_t>(blockIdx.x) * a.H);
}

// dy, dres = a * dout, and by the gate's shape
//   row:     dg = act'(g) * b * sum(dout * n * w); partial sums of b * g * dout * n (dw)
//   channel: partial sums of dout * n (dw and dg follow from them column by column)
//   full:    dg = act'(g) * b * dout * n * w;      partial sums of b * g * dout * n (dw)
template <class T, int V, int NV, int GATE>
__global__ void __launch_bounds__(kNormThreads) post_norm_backward_kernel(const NormArgs a) {
    extern __shared__ float sum_s[];
    __shared__ float red[16 * 32];
    Group g = make_group(red, a.G);
    const int nvec = a.H / V, R = blockDim.x / a.G;
    grid_dependency_wait();
    float w[NV * V], acc[NV * V];   // w: weight (channel: times the gate)
    load_weights<T, V, NV>(w, a.w, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
    if constexpr (GATE == kGateChannel) {
        Pack<T, V> gt[NV];
        load_row<T, V, NV>(gt, static_cast<const T*>(a.gate), g.tid, a.G, nvec);
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
            const float v = gt[i / V].get(i % V);
            w[i] *= a.sigmoid ? sigmoid_f32(v) : v;
        }
    }
#pragma unroll
    for (int i = 0; i < NV * V; ++i) acc[i] = 0.0f;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * R + g.id; t < a.T; t += static_cast<int64_t>(gridDim.x) * R) {
        Pack<T, V> y[NV], d[NV], gt[GATE == kGateFull ? NV : 1];
        load_row<T, V, NV>(y, static_cast<const T*>(a.x) + t * a.ldx, g.tid, a.G, nvec);
        load_row<T, V, NV>(d, static_cast<const T*>(a.dout) + t * a.ldo, g.tid, a.G, nvec);
        if constexpr (GATE == kGateFull)
            load_row<T, V, NV>(gt, static_cast<const T*>(a.gate) + t * a.ldg, g.tid, a.G, nvec);
        const float r = a.rstd[t];
        float gr = 1.0f, slope = 1.0f;   // the row's gate and the gate's slope
        if constexpr (GATE == kGateRow) {
            if (a.gate) {
                gr = to_f32(static_cast<const T*>(a.gate)[t * a.ldg]);
                if (a.sigmoid) {
                    gr = sigmoid_f32(gr);
                    slope = gr * (1.0f - gr);
                }
            }
        }
        float m = 0.0f;   // sum of dout (* full gate) * n * w
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
            const float n = y[i / V].get(i % V) * r;
            float dv = d[i / V].get(i % V);
            if constexpr (GATE == kGateFull) {
                const float gv = gt[i / V].get(i % V);
                dv *= a.sigmoid ? sigmoid_f32(gv) : gv;
            }
            m = fmaf(dv * w[i], n, m);
            acc[i] = fmaf(GATE == kGateChannel ? dv : dv * (gr * a.b), n, acc[i]);
        }
        m = g.sum(m);
        if constexpr (GATE == kGateRow)
            if (a.dgate && g.tid == 0) static_cast<T*>(a.dgate)[t] = from_f32<T>(slope * a.b * m);
        const float scale = a.b * gr * r;      // of t / w
        m /= static_cast<float>(a.H);
        T* dy = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = g.tid + i * a.G;
            if (v >= nvec) continue;
            Pack<T, V> o, p, q;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float n = y[i].get(e) * r;
                float dv = d[i].get(e), gv = 1.0f;
                if constexpr (GATE == kGateFull) {
                    gv = gt[i].get(e);
                    float sl = 1.0f;
                    if (a.sigmoid) {
                        gv = sigmoid_f32(gv);
                        sl = gv * (1.0f - gv);
                    }
                    q.set(e, sl * a.b * dv * n * w[i * V + e]);
                }
                o.set(e, scale * fmaf(-n, m, dv * gv * w[i * V + e]));
                p.set(e, a.a * dv);
            }
            const int64_t at = static_cast<int64_t>(v) * V;
            o.store(dy + at);
            if (a.dres) p.store(static_cast<T*>(a.dres) + t * a.H + at);
            if constexpr (GATE == kGateFull)
                if (a.dgate) q.store(static_cast<T*>(a.dgate) + t * a.H + at);
        }
    }
    write_partial<V, NV>(acc, sum_s, g, R, nvec, a.partial + static_cast<int64_t>(blockIdx.x) * a.H);
}

// ---------------------------------------------------------------- launches
enum NormKernel { kPreForward = 0, kPostForward = 1, kPreBackward = 2, kPostBackward = 3 };

// Threads per row: the fewest warps that hold the row in NV vectors per thread.
inline int norm_group(int nvec, int NV) {
    const int need = (nvec + NV - 1) / NV;
    return (need + 31) / 32 * 32;
}

// One kernel instance: CTAs of R row groups (about 256 threads forward, as many as fit backward, so
// that few partial sums leave the SM), as many CTAs as are resident at once.  *ctas: partial rows.
template <class K>
cudaError_t launch_norm(K kernel, NormArgs a, bool backward, int sms, cudaStream_t stream, int* ctas,
                        std::atomic<int>* occupancy) {
    int R = (backward ? kNormThreads : 256) / a.G;
    if (R < 1) R = 1;
    if (R > 8) R = 8;
    const int threads = R * a.G;
    // (two groups or more: at most 256 threads and 8192 columns each, so at most 32 KB)
    const size_t smem = backward && R > 1 ? static_cast<size_t>(a.H) * 4 : 0;
    int occ = 1;
    if (!backward) {
        occ = occupancy[threads / 32].load(std::memory_order_relaxed);
        if (occ == 0) {
            const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, threads, 0);
            if (e != cudaSuccess) return e;
            if (occ < 1) occ = 1;
            occupancy[threads / 32].store(occ, std::memory_order_relaxed);
        }
    }
    const int64_t need = (a.T + R - 1) / R;
    const int64_t grid = need < static_cast<int64_t>(occ) * sms ? need : static_cast<int64_t>(occ) * sms;
    *ctas = static_cast<int>(grid);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, stream, a);
}

template <class T, int V, int NV>
cudaError_t launch_norm_nv(NormArgs a, int which, int gate, int sms, cudaStream_t stream, int* ctas) {
    a.G = norm_group(a.H / V, NV);
    const bool next = a.w2 != nullptr;
#define MOE_NORM(KERNEL, BACKWARD)                                             \
    do {                                                                       \
        static std::atomic<int> occupancy[kNormThreads / 32 + 1];              \
        return launch_norm(KERNEL, a, BACKWARD, sms, stream, ctas, occupancy); \
    } while (0)
    switch (which) {
        case kPreForward: MOE_NORM((pre_norm_kernel<T, V, NV>), false);
        case kPreBackward: MOE_NORM((pre_norm_backward_kernel<T, V, NV>), true);
        case kPostForward:
            if (gate == kGateChannel) {
                if (next) MOE_NORM((post_norm_kernel<T, V, NV, kGateChannel, true>), false);
                MOE_NORM((post_norm_kernel<T, V, NV, kGateChannel, false>), false);
            }
            if (gate == kGateFull) {
                if (next) MOE_NORM((post_norm_kernel<T, V, NV, kGateFull, true>), false);
                MOE_NORM((post_norm_kernel<T, V, NV, kGateFull, false>), false);
            }
            if (next) MOE_NORM((post_norm_kernel<T, V, NV, kGateRow, true>), false);
            MOE_NORM((post_norm_kernel<T, V, NV, kGateRow, false>), false);
        default:
            if (gate == kGateChannel) MOE_NORM((post_norm_backward_kernel<T, V, NV, kGateChannel>), true);
            if (gate == kGateFull) MOE_NORM((post_norm_backward_kernel<T, V, NV, kGateFull>), true);
            MOE_NORM((post_norm_backward_kernel<T, V, NV, kGateRow>), true);
    }
#undef MOE_NORM
}

// V elements per vector (16 bytes where rows and addresses allow it, else one element); 32 elements
// per thread at most, 16 (8 without vectors) when the row then still fits a CTA's threads and
// there are fewer rows than SMs (more threads on each row).
template <class T>
cudaError_t launch_norm_type(const NormArgs& a, int which, int gate, bool wide, int sms, cudaStream_t stream,
                             int* ctas) {
    constexpr int W = 16 / static_cast<int>(sizeof(T));
    if (wide) {
        if (a.H <= 16 * kNormThreads && a.T < sms)
            return launch_norm_nv<T, W, 16 / W>(a, which, gate, sms, stream, ctas);
        return launch_norm_nv<T, W, 32 / W>(a, which, gate, sms, stream, ctas);
    }
    if (a.H <= 8 * kNormThreads) return launch_norm_nv<T, 1, 8>(a, which, gate, sms, stream, ctas);
    return launch_norm_nv<T, 1, 32>(a, which, gate, sms, stream, ctas);
}

// norms_bf16.cu, norms_fp16.cu, norms_fp32.cu
cudaError_t launch_norm_bf16(const NormArgs&, int which, int gate, bool wide, int sms, cudaStream_t, int* ctas);
cudaError_t launch_norm_fp16(const NormArgs&, int which, int gate, bool wide, int sms, cudaStream_t, int* ctas);
cudaError_t launch_norm_fp32(const NormArgs&, int which, int gate, bool wide, int sms, cudaStream_t, int* ctas);

}  // namespace mfp8
