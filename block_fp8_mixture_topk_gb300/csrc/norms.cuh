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
// All are bound by memory: every element is read once from DRAM and held between the row's reduction
// and its use (at most 32 elements per thread, G threads per row).  A CTA holds R groups of G
// threads, each with its own named barrier, and walks over rows with the weights in registers.  Two
// sources of rows: registers (RowRegs: any alignment, and few rows), or a ring in shared memory
// (RowRing: 16-byte rows; one thread of a group keeps up to four rows of bulk copies in flight
// ahead of the group, so that the reduction's latency does not stop the loads).  The weights'
// gradient is summed over a CTA's rows in fp32 registers, over its groups in shared memory, written once
// per CTA and summed by a second kernel in a fixed order: no atomics, so the result does not
// depend on the schedule.
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
    int depth;                  // RowRing: rows of a group's ring
    uint32_t* status;
};

__device__ __forceinline__ float weight_at(const void* w, int dtype, int64_t i) {
    if (dtype == MOE_DTYPE_FP32) return static_cast<const float*>(w)[i];
    if (dtype == MOE_DTYPE_FP16) return __half2float(static_cast<const __half*>(w)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}
// sigmoid(v): for 16-bit results with the fast exponential and division (a few 2^-23 relative, far
// below their rounding of 2^-9 and 2^-12)
template <class T>
__device__ __forceinline__ float sigmoid_as(float v) {
    if (sizeof(T) == 2) return __fdividef(1.0f, 1.0f + __expf(-v));
    return 1.0f / (1.0f + expf(-v));
}

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

// ---------------------------------------------------------------- sources of rows
// A source hands out a group's rows of NIN matrices: start() once, then for each row fetch(t),
// get(n, i) = vector i of this thread in matrix n (any number of times) and, after the group's
// barrier in that row, next() (the row before is done with).  finish() at the end.
template <class T, int V, int NV, int NIN>
struct RowRegs {
    Pack<T, V> r[NIN][NV];
    const T* src[NIN];
    int64_t ld[NIN];
    int G, tid, nvec;
    __device__ __forceinline__ void start(const NormArgs& a, const Group& g, int64_t, int64_t, int, uint8_t*) {
        G = a.G;
        tid = g.tid;
        nvec = a.H / V;
    }
    __device__ __forceinline__ void fetch(int64_t t) {
#pragma unroll
        for (int n = 0; n < NIN; ++n) load_row<T, V, NV>(r[n], src[n] + t * ld[n], tid, G, nvec);
    }
    __device__ __forceinline__ Pack<T, V> get(int n, int i) const { return r[n][i]; }
    __device__ __forceinline__ void next() {}
    __device__ __forceinline__ void finish() {}
};

template <class T, int V, int NV, int NIN>
struct RowRing {
    const T* src[NIN];
    int64_t ld[NIN];
    uint8_t* ring;              // this group's rows: [depth][NIN][row_bytes]
    uint64_t* bar;              // [depth]
    volatile int* abort_flag;
    uint32_t* status;
    int64_t t_load, t_end, stride;
    uint32_t row_bytes;
    int depth, slot, load_slot, G, tid, nvec;
    uint32_t phase, issued;
    bool first;

    __device__ __forceinline__ void issue() {
        if (t_load < t_end) {
            if (tid == 0) {
                const uint32_t b = smem_addr(bar + load_slot);
                mbar_arrive_expect_tx(b, NIN * row_bytes);
#pragma unroll
                for (int n = 0; n < NIN; ++n)
                    bulk_load(smem_addr(ring + (load_slot * NIN + n) * row_bytes), src[n] + t_load * ld[n], row_bytes, b);
            }
            ++issued;
            t_load += stride;
            if (++load_slot == depth) load_slot = 0;
        }
    }
    // smem: [R][depth][NIN][row_bytes], then the barriers and the abort flag
    __device__ __forceinline__ void start(const NormArgs& a, const Group& g, int64_t t0, int64_t step, int R,
                                          uint8_t* smem) {
        G = a.G;
        tid = g.tid;
        nvec = a.H / V;
        depth = a.depth;
        status = a.status;
        row_bytes = static_cast<uint32_t>(a.H) * sizeof(T);
        ring = smem + static_cast<size_t>(g.id) * depth * NIN * row_bytes;
        uint64_t* bars = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(R) * depth * NIN * row_bytes);
        bar = bars + g.id * depth;
        abort_flag = reinterpret_cast<volatile int*>(bars + R * depth);
        if (threadIdx.x == 0) {
            for (int i = 0; i < R * depth; ++i) mbar_init(smem_addr(bars + i), 1);
            *abort_flag = 0;
            fence_barrier_init();
        }
        __syncthreads();
        t_load = t0;
        t_end = a.T;
        stride = step;
        slot = depth - 1;
        load_slot = 0;
        phase = 1;
        issued = 0;
        first = true;
        for (int i = 0; i < depth; ++i) issue();
    }
    // (a wait that gave up leaves its status bit and wrong values, and all later waits return at
    // once: no thread leaves its group's barriers)
    __device__ __forceinline__ void fetch(int64_t) {
        if (++slot == depth) {
            slot = 0;
            phase ^= 1u;
        }
        mbar_wait(smem_addr(bar + slot), phase, abort_flag, status);
    }
    __device__ __forceinline__ Pack<T, V> get(int n, int i) const {
        Pack<T, V> p;
        const int v = tid + i * G;
        if (v < nvec)
            p.raw = *reinterpret_cast<const typename Pack<T, V>::Raw*>(ring + (slot * NIN + n) * row_bytes + v * 16);
        else p.zero();
        return p;
    }
    // every thread of the group has finished the row before this one: its slot takes the next row
    __device__ __forceinline__ void next() {
        if (!first) issue();
        first = false;
    }
    __device__ __forceinline__ void finish() {
        if (*abort_flag && tid == 0)   // loads may be under way: let them land
            for (int i = 0; i < depth; ++i) {
                const uint32_t n = (issued + depth - 1 - i) / depth;
                if (n > 0) mbar_wait(smem_addr(bar + i), (n - 1) & 1u, nullptr, status);
            }
    }
};

#define MOE_NORM_PROLOGUE                                                             \
    extern __shared__ __align__(128) uint8_t norm_smem[];                             \
    __shared__ float red[16 * 32];                                                    \
    Group g = make_group(red, a.G);                                                   \
    const int nvec = a.H / V, R = blockDim.x / a.G;                                   \
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * R + g.id, step = static_cast<int64_t>(gridDim.x) * R; \
    grid_dependency_wait();

// h = x * rstd * w
template <class T, int V, int NV, template <class, int, int, int> class Rows>
__global__ void __launch_bounds__(kNormThreads) pre_norm_kernel(const NormArgs a) {
    MOE_NORM_PROLOGUE
    Rows<T, V, NV, 1> in;
    in.src[0] = static_cast<const T*>(a.x);
    in.ld[0] = a.ldx;
    in.start(a, g, t0, step, R, norm_smem);
    float w[NV * V];
    load_weights<T, V, NV>(w, a.w, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
    for (int64_t t = t0; t < a.T; t += step) {
        in.fetch(t);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Pack<T, V> x = in.get(0, i);
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(x.get(e), x.get(e), ss);
        }
        const float r = __frsqrt_rn(g.sum(ss) / static_cast<float>(a.H) + a.eps);
        in.next();
        if (g.tid == 0) a.rstd[t] = r;
        T* out = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = g.tid + i * a.G;
            if (v >= nvec) continue;
            const Pack<T, V> x = in.get(0, i);
            Pack<T, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) o.set(e, x.get(e) * r * w[i * V + e]);
            o.store(out + static_cast<int64_t>(v) * V);
        }
    }
    in.finish();
}

// out = a * res + b * g * (y * rstd * w); NEXT: h2 = out * rstd2 * w2 of the stored out
template <class T, int V, int NV, int GATE, bool NEXT, template <class, int, int, int> class Rows>
__global__ void __launch_bounds__(kNormThreads) post_norm_kernel(const NormArgs a) {
    MOE_NORM_PROLOGUE
    Rows<T, V, NV, GATE == kGateFull ? 3 : 2> in;
    in.src[0] = static_cast<const T*>(a.x);
    in.ld[0] = a.ldx;
    in.src[1] = static_cast<const T*>(a.res);
    in.ld[1] = a.ldr;
    if constexpr (GATE == kGateFull) {
        in.src[2] = static_cast<const T*>(a.gate);
        in.ld[2] = a.ldg;
    }
    in.start(a, g, t0, step, R, norm_smem);
    float w[NV * V], w2[NEXT ? NV * V : 1];
    load_weights<T, V, NV>(w, a.w, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
    if constexpr (NEXT) load_weights<T, V, NV>(w2, a.w2, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
    if constexpr (GATE == kGateChannel) {   // the gate scales the weight, for every row alike
        Pack<T, V> gt[NV];
        load_row<T, V, NV>(gt, static_cast<const T*>(a.gate), g.tid, a.G, nvec);
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
            const float v = gt[i / V].get(i % V);
            w[i] *= a.sigmoid ? sigmoid_as<T>(v) : v;
        }
    }
    for (int64_t t = t0; t < a.T; t += step) {
        in.fetch(t);
        float b = a.b;
        if constexpr (GATE == kGateRow) {
            if (a.gate) {
                const float v = to_f32(static_cast<const T*>(a.gate)[t * a.ldg]);
                b *= a.sigmoid ? sigmoid_as<T>(v) : v;
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Pack<T, V> y = in.get(0, i);
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(y.get(e), y.get(e), ss);
        }
        const float r = __frsqrt_rn(g.sum(ss) / static_cast<float>(a.H) + a.eps);
        in.next();
        if (g.tid == 0) a.rstd[t] = r;
        T* out = static_cast<T*>(a.out) + t * a.H;
        float s2 = 0.0f;
        Pack<T, V> s[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = g.tid + i * a.G;
            const Pack<T, V> y = in.get(0, i), res = in.get(1, i);
            Pack<T, V> gt;
            if constexpr (GATE == kGateFull) gt = in.get(2, i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float z = y.get(e) * r * w[i * V + e] * b;
                if constexpr (GATE == kGateFull) {
                    const float gv = gt.get(e);
                    z *= a.sigmoid ? sigmoid_as<T>(gv) : gv;
                }
                s[i].set(e, fmaf(a.a, res.get(e), z));
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
    in.finish();
}

// The CTA's sums over rows, group after group, into its row of the partials.
template <int V, int NV>
__device__ __forceinline__ void write_partial(const float (&acc)[NV * V], float* sum_s, const Group& g, int R,
                                              int nvec, float* partial) {
    __syncthreads();   // sum_s is the ring's memory
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

// dx = rstd * (t - n * mean(t * n)) + res (RES), t = dout * w; partial sums of dout * n
template <class T, int V, int NV, bool RES, template <class, int, int, int> class Rows>
__global__ void __launch_bounds__(kNormThreads) pre_norm_backward_kernel(const NormArgs a) {
    MOE_NORM_PROLOGUE
    Rows<T, V, NV, RES ? 3 : 2> in;
    in.src[0] = static_cast<const T*>(a.x);
    in.ld[0] = a.ldx;
    in.src[1] = static_cast<const T*>(a.dout);
    in.ld[1] = a.ldo;
    if constexpr (RES) {
        in.src[2] = static_cast<const T*>(a.res);
        in.ld[2] = a.ldr;
    }
    in.start(a, g, t0, step, R, norm_smem);
    float w[NV * V], acc[NV * V];
    load_weights<T, V, NV>(w, a.w, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
#pragma unroll
    for (int i = 0; i < NV * V; ++i) acc[i] = 0.0f;
    for (int64_t t = t0; t < a.T; t += step) {
        const float r = a.rstd[t];
        in.fetch(t);
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Pack<T, V> x = in.get(0, i), d = in.get(1, i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float p = d.get(e) * (x.get(e) * r);
                m = fmaf(p, w[i * V + e], m);
                acc[i * V + e] += p;
            }
        }
        m = g.sum(m) / static_cast<float>(a.H);
        in.next();
        T* out = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = g.tid + i * a.G;
            if (v >= nvec) continue;
            const Pack<T, V> x = in.get(0, i), d = in.get(1, i);
            Pack<T, V> o, s;
            if constexpr (RES) s = in.get(2, i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float u = r * fmaf(-(x.get(e) * r), m, d.get(e) * w[i * V + e]);
                if constexpr (RES) u += s.get(e);
                o.set(e, u);
            }
            o.store(out + static_cast<int64_t>(v) * V);
        }
    }
    in.finish();
    write_partial<V, NV>(acc, reinterpret_cast<float*>(norm_smem), g, R, nvec,
                         a.partial + static_cast<int64_t>(blockIdx.x) * a.H);
}

// dy, dres = a * dout, and by the gate's shape
//   row:     dg = act'(g) * b * sum(dout * n * w); partial sums of b * g * dout * n (dw)
//   channel: partial sums of dout * n (dw and dg follow from them column by column)
//   full:    dg = act'(g) * b * dout * n * w;      partial sums of b * g * dout * n (dw)
template <class T, int V, int NV, int GATE, template <class, int, int, int> class Rows>
__global__ void __launch_bounds__(kNormThreads) post_norm_backward_kernel(const NormArgs a) {
    MOE_NORM_PROLOGUE
    Rows<T, V, NV, GATE == kGateFull ? 3 : 2> in;
    in.src[0] = static_cast<const T*>(a.x);
    in.ld[0] = a.ldx;
    in.src[1] = static_cast<const T*>(a.dout);
    in.ld[1] = a.ldo;
    if constexpr (GATE == kGateFull) {
        in.src[2] = static_cast<const T*>(a.gate);
        in.ld[2] = a.ldg;
    }
    in.start(a, g, t0, step, R, norm_smem);
    float w[NV * V], acc[NV * V];   // w: weight (channel: times the gate)
    load_weights<T, V, NV>(w, a.w, a.w_dtype, a.w_offset, g.tid, a.G, nvec);
    if constexpr (GATE == kGateChannel) {
        Pack<T, V> gt[NV];
        load_row<T, V, NV>(gt, static_cast<const T*>(a.gate), g.tid, a.G, nvec);
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
            const float v = gt[i / V].get(i % V);
            w[i] *= a.sigmoid ? sigmoid_as<T>(v) : v;
        }
    }
#pragma unroll
    for (int i = 0; i < NV * V; ++i) acc[i] = 0.0f;
    for (int64_t t = t0; t < a.T; t += step) {
        const float r = a.rstd[t];
        float gr = 1.0f, slope = 1.0f;   // the row's gate and the gate's slope
        if constexpr (GATE == kGateRow) {
            if (a.gate) {
                gr = to_f32(static_cast<const T*>(a.gate)[t * a.ldg]);
                if (a.sigmoid) {
                    gr = sigmoid_as<T>(gr);
                    slope = gr * (1.0f - gr);
                }
            }
        }
        in.fetch(t);
        float m = 0.0f;   // sum of dout (* full gate) * n * w
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Pack<T, V> y = in.get(0, i), d = in.get(1, i);
            Pack<T, V> gt;
            if constexpr (GATE == kGateFull) gt = in.get(2, i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float p = d.get(e) * (y.get(e) * r);
                if constexpr (GATE == kGateFull) {
                    const float gv = gt.get(e);
                    p *= a.sigmoid ? sigmoid_as<T>(gv) : gv;
                }
                m = fmaf(p, w[i * V + e], m);
                if constexpr (GATE == kGateChannel) acc[i * V + e] += p;
                else acc[i * V + e] = fmaf(p, gr * a.b, acc[i * V + e]);
            }
        }
        m = g.sum(m);
        in.next();
        if constexpr (GATE == kGateRow)
            if (a.dgate && g.tid == 0) static_cast<T*>(a.dgate)[t] = from_f32<T>(slope * a.b * m);
        const float scale = a.b * gr * r;      // of t / w
        m /= static_cast<float>(a.H);
        T* dy = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = g.tid + i * a.G;
            if (v >= nvec) continue;
            const Pack<T, V> y = in.get(0, i), d = in.get(1, i);
            Pack<T, V> o, p, q, gt;
            if constexpr (GATE == kGateFull) gt = in.get(2, i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float n = y.get(e) * r, dw = d.get(e) * w[i * V + e];
                float gv = 1.0f;
                if constexpr (GATE == kGateFull) {
                    gv = gt.get(e);
                    float sl = a.b;
                    if (a.sigmoid) {
                        gv = sigmoid_as<T>(gv);
                        sl *= gv * (1.0f - gv);
                    }
                    q.set(e, sl * dw * n);
                }
                o.set(e, scale * fmaf(-n, m, dw * gv));
                p.set(e, a.a * d.get(e));
            }
            const int64_t at = static_cast<int64_t>(v) * V;
            o.store(dy + at);
            if (a.dres) p.store(static_cast<T*>(a.dres) + t * a.H + at);
            if constexpr (GATE == kGateFull)
                if (a.dgate) q.store(static_cast<T*>(a.dgate) + t * a.H + at);
        }
    }
    in.finish();
    write_partial<V, NV>(acc, reinterpret_cast<float*>(norm_smem), g, R, nvec,
                         a.partial + static_cast<int64_t>(blockIdx.x) * a.H);
}
#undef MOE_NORM_PROLOGUE

// ---------------------------------------------------------------- launches
enum NormKernel { kPreForward = 0, kPostForward = 1, kPreBackward = 2, kPostBackward = 3 };

// Threads per row: the fewest warps that hold the row in NV vectors per thread.
inline int norm_group(int nvec, int NV) {
    const int need = (nvec + NV - 1) / NV;
    return (need + 31) / 32 * 32;
}

constexpr int kRingBytes = 196 * 1024;   // of a CTA's rings (one CTA per SM)
constexpr int kRingMostDepth = 4;

// What an instance remembers per device: that its shared-memory limit is set, and the CTAs per SM by
// the warps of a CTA.
struct NormInstance {
    std::atomic<uint64_t> limit{0};
    std::atomic<int> occupancy[kNormThreads / 32 + 1] = {};
};

// One kernel instance.  Rows in registers: CTAs of R row groups (about 256 threads forward, as many
// as fit backward, so that few partial sums leave the SM), as many CTAs as are resident at
// once.  Rows in a ring: one CTA of up to kNormThreads per SM.  *ctas: partial rows.
template <class K>
cudaError_t launch_norm(K kernel, NormArgs a, bool backward, int ring_inputs, int esize, int sms, cudaStream_t stream,
                        int* ctas, NormInstance* inst) {
    int R = (backward || ring_inputs ? kNormThreads : 256) / a.G;
    if (R < 1) R = 1;
    if (R > 8) R = 8;
    // sums over groups (two or more: at most 256 threads and 8192 columns each, so at most 32 KB)
    size_t smem = backward && R > 1 ? static_cast<size_t>(a.H) * 4 : 0;
    int occ = 1;
    if (ring_inputs) {
        const int row = ring_inputs * a.H * esize;
        while (R > 1 && 2 * R * row > kRingBytes) --R;
        a.depth = kRingBytes / (R * row);
        if (a.depth > kRingMostDepth) a.depth = kRingMostDepth;
        const size_t ring = static_cast<size_t>(R) * a.depth * row + (R * a.depth + 1) * 8;
        if (ring > smem) smem = ring;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = uint64_t(1) << (dev & 63);
        if (dev >= 64 || !(inst->limit.load(std::memory_order_acquire) & bit)) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes + 1024);
            if (e != cudaSuccess) return e;
            inst->limit.fetch_or(bit, std::memory_order_release);
        }
    } else if (!backward) {
        const int warps = R * a.G / 32;
        occ = inst->occupancy[warps].load(std::memory_order_relaxed);
        if (occ == 0) {
            const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, R * a.G, 0);
            if (e != cudaSuccess) return e;
            if (occ < 1) occ = 1;
            inst->occupancy[warps].store(occ, std::memory_order_relaxed);
        }
    }
    const int64_t need = (a.T + R - 1) / R;
    const int64_t grid = need < static_cast<int64_t>(occ) * sms ? need : static_cast<int64_t>(occ) * sms;
    *ctas = static_cast<int>(grid);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(R * a.G)), smem, stream, a);
}

template <class T, int V, int NV, template <class, int, int, int> class Rows, bool RING>
cudaError_t launch_norm_nv(NormArgs a, int which, int gate, int sms, cudaStream_t stream, int* ctas) {
    a.G = norm_group(a.H / V, NV);
    const bool next = a.w2 != nullptr;
#define MOE_NORM(INPUTS, BACKWARD, ...)                                                                          \
    do {                                                                                                         \
        static NormInstance inst;                                                                                \
        return launch_norm(__VA_ARGS__, a, BACKWARD, RING ? INPUTS : 0, static_cast<int>(sizeof(T)), sms, stream, \
                           ctas, &inst);                                                                         \
    } while (0)
    switch (which) {
        case kPreForward: MOE_NORM(1, false, pre_norm_kernel<T, V, NV, Rows>);
        case kPreBackward:
            if (a.res) MOE_NORM(3, true, pre_norm_backward_kernel<T, V, NV, true, Rows>);
            MOE_NORM(2, true, pre_norm_backward_kernel<T, V, NV, false, Rows>);
        case kPostForward:
            if (gate == kGateChannel) {
                if (next) MOE_NORM(2, false, post_norm_kernel<T, V, NV, kGateChannel, true, Rows>);
                MOE_NORM(2, false, post_norm_kernel<T, V, NV, kGateChannel, false, Rows>);
            }
            if (gate == kGateFull) {
                if (next) MOE_NORM(3, false, post_norm_kernel<T, V, NV, kGateFull, true, Rows>);
                MOE_NORM(3, false, post_norm_kernel<T, V, NV, kGateFull, false, Rows>);
            }
            if (next) MOE_NORM(2, false, post_norm_kernel<T, V, NV, kGateRow, true, Rows>);
            MOE_NORM(2, false, post_norm_kernel<T, V, NV, kGateRow, false, Rows>);
        default:
            if (gate == kGateChannel) MOE_NORM(2, true, post_norm_backward_kernel<T, V, NV, kGateChannel, Rows>);
            if (gate == kGateFull) MOE_NORM(3, true, post_norm_backward_kernel<T, V, NV, kGateFull, Rows>);
            MOE_NORM(2, true, post_norm_backward_kernel<T, V, NV, kGateRow, Rows>);
    }
#undef MOE_NORM
}

// V elements per vector: 16 bytes where rows and addresses allow it, else one element.
//   16 bytes, fewer rows than twice the SMs: registers, 16 elements per thread where the row then
//     fits a CTA's threads (more threads on each row)
//   16 bytes: the ring, 32 elements per thread (registers where two rows do not fit the ring: fp32)
//   one element: registers, 8 or 32 elements per thread
template <class T>
cudaError_t launch_norm_type(const NormArgs& a, int which, int gate, bool wide, int sms, cudaStream_t stream,
                             int* ctas) {
    constexpr int W = 16 / static_cast<int>(sizeof(T));
    if (!wide) {
        if (a.H <= 8 * kNormThreads) return launch_norm_nv<T, 1, 8, RowRegs, false>(a, which, gate, sms, stream, ctas);
        return launch_norm_nv<T, 1, 32, RowRegs, false>(a, which, gate, sms, stream, ctas);
    }
    if (a.T < 2 * sms && a.H <= 16 * kNormThreads)
        return launch_norm_nv<T, W, 16 / W, RowRegs, false>(a, which, gate, sms, stream, ctas);
    if constexpr (sizeof(T) == 4) {
        const int inputs = which == kPreForward ? 1 : which == kPreBackward ? (a.res ? 3 : 2) : gate == kGateFull ? 3 : 2;
        if (2 * inputs * a.H * 4 > kRingBytes)
            return launch_norm_nv<T, W, 32 / W, RowRegs, false>(a, which, gate, sms, stream, ctas);
    }
    return launch_norm_nv<T, W, 32 / W, RowRing, true>(a, which, gate, sms, stream, ctas);
}

// norms_bf16.cu, norms_fp16.cu, norms_fp32.cu
cudaError_t launch_norm_bf16(const NormArgs&, int which, int gate, bool wide, int sms, cudaStream_t, int* ctas);
cudaError_t launch_norm_fp16(const NormArgs&, int which, int gate, bool wide, int sms, cudaStream_t, int* ctas);
cudaError_t launch_norm_fp32(const NormArgs&, int which, int gate, bool wide, int sms, cudaStream_t, int* ctas);

}  // namespace mfp8
