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
// threads, each with its own named barrier, and walks over rows with the weights at hand.  Two
// sources of rows and weights: registers (RowRegs: few rows; RowAny: rows at any address), or shared memory
// (RowShift: rows of any width whose matrices lie alike; RowRing: 16-byte rows; one thread of a group keeps up to four rows of bulk copies in flight
// ahead of the group, so that the reduction's latency does not stop the loads).  The weights'
// gradient is summed over a CTA's rows in fp32 registers, over its groups in shared memory, written once
// per CTA and summed by a second kernel in a fixed order: no atomics, so the result does not
// depend on the schedule.
//
// Measured (bf16): before and after with the next norm, 4096 x 7168: 66 us for 352 MB (0.78 of a copy; 21
// and 43 us alone).  Both gradients of 5003 x 2880 with a sigmoid gate: 69 us for 288 MB, two launches of
// 4.7 us among them that sum the weights' partials.  One row: 6.7 us on the device.  About 4 us of
// each launch are its first loads and last stores; the after-norm with a next norm holds its weights and the
// stored row in registers (111, so 448 threads per SM) and is then bound by the two reductions' latency.
// Rows of odd widths: 8000 x 4811 before and after with the next norm 102 us, 1.5 times the bytes' time; where
// the matrices do not lie alike the vectors are joined: 165 us, bound by instructions and, in the instances of 32
// elements a thread, by spilled registers (3000 x 9001 before, backward: 88 us, 3.7 times the bytes' time).  So
// are wide rows whose matrices do not fit the ring (2000 x 16384 before, backward, with a residual's gradient: 98
// us, 2.5 times).
#pragma once

#include <atomic>

#include "train.cuh"

namespace mfp8 {

// Most threads of a CTA (128 registers); forward with rows in the ring and no next norm (64 registers)
constexpr int kNormThreads = 512, kNormWideThreads = 1024;
constexpr int kNormGroups = 15;     // groups of a CTA with a named barrier each
// kGateRow also stands for no gate; kGateFullSigmoid: the sigmoid of a full gate
enum GateShape { kGateRow = 0, kGateChannel = 1, kGateFull = 2, kGateFullSigmoid = 3 };
constexpr bool full_gate(int g) { return g == kGateFull || g == kGateFullSigmoid; }

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
// exp(-v) and 1 / v: for 16-bit results by the approximate instructions, whose product with log2(e) and
// results are off by (2 |v| + 4) 2^-24 and 2^-23 of themselves, far below the results' rounding of 2^-9 and
// 2^-12 (the division form costs three times the instructions and made the gated backward pass
// instruction-bound)
template <class T>
__device__ __forceinline__ float exp_minus(float v) {
    if (sizeof(T) != 2) return expf(-v);
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
    return e;
}
template <class T>
__device__ __forceinline__ float reciprocal(float v) {
    if (sizeof(T) != 2) return 1.0f / v;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
template <class T>
__device__ __forceinline__ float sigmoid_as(float v) {
    return reciprocal<T>(1.0f + exp_minus<T>(v));
}
template <class T>
__device__ __forceinline__ float2 sigmoid_as(float2 v) {
    return make_float2(sigmoid_as<T>(v.x), sigmoid_as<T>(v.y));
}
// The sigmoid and its slope for gradients, of e = exp(-v): s = 1 / (1 + e), and s (1 - s) with 1 - s = e s
// (1 where an infinite e leaves s = 0: fminf passes over what is no number).  The slope then keeps
// its digits where the gate saturates; 1 - s of a rounded s is off by 5e-4 of itself at v = 10 and
// is 0 from 17 on.
template <class T>
__device__ __forceinline__ float sigmoid_of(float e) {
    return reciprocal<T>(1.0f + e);
}
__device__ __forceinline__ float slope_of(float e, float s) { return s * fminf(e * s, 1.0f); }

struct Group {
    float* red;       // [2][16] of this group
    int G, tid, id, parity;
    __device__ __forceinline__ void sync() const {
        if (G == 32) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(G) : "memory");
    }
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
        if (G == 32) return v;
        float* slot = red + parity * 16;
        parity ^= 1;
        if ((tid & 31) == 0) slot[tid >> 5] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(G) : "memory");
        const float4* q = reinterpret_cast<const float4*>(slot);   // (slots past the group's warps hold zero)
        const float4 a = q[0], b = q[1], c = q[2], d = q[3];
        return ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w)) + (((c.x + c.y) + (c.z + c.w)) +
                                                                           ((d.x + d.y) + (d.z + d.w)));
    }
};

__device__ __forceinline__ Group make_group(float* red, int G) {
    Group g;
    g.G = G;
    g.id = threadIdx.x / G;
    g.tid = threadIdx.x % G;
    g.parity = 0;
    g.red = red + g.id * 32;
    if (G > 32 && g.tid < 32) g.red[g.tid] = 0.0f;
    __syncthreads();
    return g;
}

// ---------------------------------------------------------------- sources of rows
// A source hands out a group's rows of NIN matrices and a row of weights (fp32): start() and weights()
// once, then for each row fetch(t), get(n, i) = vector i of this thread in matrix n (any number of
// times) and next() (the row is done with); finish() at the end.  weight(i) = the weights of vector i;
// store(row, i, o) writes it, skip(i) tells that there is nothing of it to write.  Vectors and elements
// past the row read as zero; again(n, i) is get for values that are only stored (anything past the row).
template <int V>
struct Weights {
    float2 v[V / 2];
};

template <class T, int V, int NV, int NIN, bool ANY>
struct RowInRegs {
    static constexpr bool kWide = false, kAny = ANY, kShift = false;
    Weights<V> w[NV];
    Pack<T, V> r[NIN][NV];
    const T* src[NIN];
    int64_t ld[NIN];
    int G, tid, H, nvec;
    int64_t T_;
    __device__ __forceinline__ void start(const NormArgs& a, const Group& g, int64_t, int64_t, int, uint8_t*) {
        G = a.G;
        tid = g.tid;
        H = a.H;
        T_ = a.T;
        nvec = a.H / V;
    }
    // f(column) = its weight
    template <class F>
    __device__ __forceinline__ void weights(F f) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int c = vec(i) * V + e;
                const float x = c < H ? f(c) : 0.0f;
                if (e & 1) w[i].v[e / 2].y = x;
                else w[i].v[e / 2].x = x;
            }
    }
    __device__ __forceinline__ void weights_done() {}
    __device__ __forceinline__ Weights<V> weight(int i) const { return w[i]; }
    __device__ __forceinline__ void fetch(int64_t t) {
        if constexpr (ANY) {
            const int lane = threadIdx.x & 31;
            if (!inner_row(t, T_)) {
#pragma unroll
                for (int n = 0; n < NIN; ++n)
#pragma unroll
                    for (int i = 0; i < NV; ++i) r[n][i].raw = load_elements(src[n] + t * ld[n], H, vec(i) * V);
                return;
            }
            // the warp's NV * 32 vectors and the next one, which the first lane holds: the next lane of the last is
            // the first, one vector on
            uint4 beyond[NIN];
#pragma unroll
            for (int n = 0; n < NIN; ++n) {
                const T* row = src[n] + t * ld[n];
#pragma unroll
                for (int i = 0; i < NV; ++i) r[n][i].raw = load_around(row, H, vec(i) * V);
                beyond[n] = load_around(row, H, vec(NV) * V, lane == 0);
            }
#pragma unroll
            for (int n = 0; n < NIN; ++n) {
                const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src[n] + t * ld[n])) & 15u;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const uint4 w = r[n][i].raw, on = i + 1 < NV ? r[n][i + 1 < NV ? i + 1 : 0].raw : beyond[n];
                    const uint4 hi = shuffle(lane == 0 ? on : w, (lane + 1) & 31);
                    r[n][i].raw = inside_row<T>(bytes_from(w, hi, s), H, vec(i) * V);
                }
            }
            return;
        }
#pragma unroll
        for (int n = 0; n < NIN; ++n)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = tid + i * G;
                if (v < nvec) r[n][i].load(src[n] + t * ld[n] + v * V);
                else r[n][i].zero();
            }
    }
    // this thread's i-th vector of a row; at any address the vectors of a warp are neighbours
    __device__ __forceinline__ int column(int i) const { return vec(i) * V; }
    __device__ __forceinline__ int vec(int i) const { return ANY ? ((tid >> 5) * NV + i) * 32 + (tid & 31) : tid + i * G; }
    __device__ __forceinline__ Pack<T, V> get(int n, int i) const { return r[n][i]; }
    __device__ __forceinline__ Pack<T, V> again(int n, int i) const { return r[n][i]; }
    __device__ __forceinline__ bool skip(int i) const { return !ANY && tid + i * G >= nvec; }
    __device__ __forceinline__ void store(T* row, int i, const Pack<T, V>& o) const {
        if constexpr (ANY) store_any(row, H, vec(i), o.raw);
        else o.store(row + static_cast<int64_t>(vec(i)) * V);
    }
    __device__ __forceinline__ void next(const Group&) {}
    __device__ __forceinline__ void finish() {}
};
template <class T, int V, int NV, int NIN>
struct RowRegs : RowInRegs<T, V, NV, NIN, false> {};
template <class T, int V, int NV, int NIN>
struct RowAny : RowInRegs<T, V, NV, NIN, true> {};

// Bytes of a row in the ring, and vectors that a row touches at most; SHIFT: it may start inside a vector.
template <class T, bool SHIFT>
__host__ __device__ __forceinline__ int ring_row_bytes(int H) {
    const int bytes = H * static_cast<int>(sizeof(T));
    return SHIFT ? (bytes + 15) / 16 * 16 + 16 : bytes;
}
template <bool SHIFT>
__host__ __device__ __forceinline__ int ring_vectors(int H, int V) {
    return SHIFT ? (H + 2 * V - 2) / V : H / V;
}
// SHIFT: rows of any width whose matrices all lie alike between two 16-byte boundaries.  A row starts there
// by its number modulo 8, and so does every row of a CTA, whose rows are a multiple of 8 apart: its
// vectors are the memory's, its weights and sums are kept by those, and only a row's first and last vector
// hold columns that are not the row's.
template <class T, int V, int NV, int NIN, bool SHIFT>
struct RowInRing {
    static constexpr bool kWide = true, kAny = SHIFT, kShift = SHIFT;
    static constexpr int Q = V / 4;   // the weights of a vector: Q planes of float4, so that a warp reads 512 bytes in a row
    float4* wsm;                      // [Q][nvec], the CTA's
    const T* src[NIN];
    int64_t ld[NIN];
    uint8_t* ring;              // this group's rows: [depth][NIN][row_bytes]
    uint64_t* bar;              // [depth]
    volatile int* abort_flag;
    uint32_t* status;
    int64_t t_load, t_end, stride;
    uint32_t row_bytes;
    int depth, slot, load_slot, G, tid, H, nvec;
    int lead;                   // SHIFT: elements of a row's start past a 16-byte boundary
    uint32_t phase, issued;

    __device__ __forceinline__ void issue() {
        if (t_load < t_end) {
            if (tid == 0) {
                const uint32_t b = smem_addr(bar + load_slot);
                if constexpr (SHIFT) {
                    issue_shifted(b);
                } else {
                    mbar_arrive_expect_tx(b, NIN * row_bytes);
#pragma unroll
                    for (int n = 0; n < NIN; ++n)
                        bulk_load(smem_addr(ring + (load_slot * NIN + n) * row_bytes), src[n] + t_load * ld[n], row_bytes, b);
                }
            }
            ++issued;
            t_load += stride;
            if (++load_slot == depth) load_slot = 0;
        }
    }
    // Row t_load, by one thread: whole aligned vectors, which reach into the neighbouring rows; of the
    // matrix's first and last rows only what is in them, the elements at their ends one by one.
    __device__ __forceinline__ void issue_shifted(uint32_t b) {
        const bool inner = inner_row(t_load, t_end);
        const int before = lead * static_cast<int>(sizeof(T)), after = before + H * static_cast<int>(sizeof(T));
        const int from = inner || lead == 0 ? 0 : 16, to = inner ? (after + 15) & ~15 : after & ~15;
        const int bytes = to > from ? to - from : 0;
#pragma unroll
        for (int n = 0; n < NIN; ++n) {
            uint8_t* s = ring + (load_slot * NIN + n) * row_bytes;
            const uint8_t* g = reinterpret_cast<const uint8_t*>(src[n] + t_load * ld[n]) - before;
            if (!inner)
#pragma unroll 1
                for (int a = before; a < after; a += sizeof(T)) {
                    if (bytes && a == from) a = to;
                    if (a < after) *reinterpret_cast<T*>(s + a) = *reinterpret_cast<const T*>(g + a);
                }
        }
        if (!inner) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // later copies land in the same bytes
        mbar_arrive_expect_tx(b, NIN * bytes);
        if (bytes)
#pragma unroll
            for (int n = 0; n < NIN; ++n)
                bulk_load(smem_addr(ring + (load_slot * NIN + n) * row_bytes + from),
                          reinterpret_cast<const uint8_t*>(src[n] + t_load * ld[n]) - before + from, bytes, b);
    }
    template <class F>
    __device__ __forceinline__ void weights(F f) {
        for (int q = threadIdx.x; q < nvec * Q; q += blockDim.x) {
            const int v = q / Q, p = q - v * Q, c = v * V + p * 4 - lead;
            const auto at = [&](int k) { return !SHIFT || (c + k >= 0 && c + k < H) ? f(c + k) : 0.0f; };
            wsm[p * nvec + v] = make_float4(at(0), at(1), at(2), at(3));
        }
    }
    __device__ __forceinline__ void weights_done() { __syncthreads(); }
    __device__ __forceinline__ Weights<V> weight(int i) const {
        Weights<V> r;
        const int v = tid + i * G;
#pragma unroll
        for (int p = 0; p < Q; ++p) {
            const float4 f = v < nvec ? wsm[p * nvec + v] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            r.v[p * 2] = make_float2(f.x, f.y);
            r.v[p * 2 + 1] = make_float2(f.z, f.w);
        }
        return r;
    }
    // smem: [vectors * V] weights, [R][depth][NIN][row_bytes], then the barriers and the abort flag
    __device__ __forceinline__ void start(const NormArgs& a, const Group& g, int64_t t0, int64_t step, int R,
                                          uint8_t* smem) {
        G = a.G;
        tid = g.tid;
        H = a.H;
        nvec = ring_vectors<SHIFT>(a.H, V);
        lead = SHIFT ? static_cast<int>((reinterpret_cast<uintptr_t>(src[0] + t0 * ld[0]) & 15) / sizeof(T)) : 0;
        depth = a.depth;
        status = a.status;
        row_bytes = static_cast<uint32_t>(ring_row_bytes<T, SHIFT>(a.H));
        wsm = reinterpret_cast<float4*>(smem);
        smem += static_cast<size_t>(nvec) * V * 4;
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
        Pack<T, V> p = again(n, i);
        if constexpr (SHIFT) p.raw = inside_row<T>(p.raw, H, column(i));
        return p;
    }
    __device__ __forceinline__ Pack<T, V> again(int n, int i) const {
        Pack<T, V> p;
        const int v = tid + i * G;
        if (v < nvec)
            p.raw = *reinterpret_cast<const typename Pack<T, V>::Raw*>(ring + (slot * NIN + n) * row_bytes + v * 16);
        else p.zero();
        return p;
    }
    __device__ __forceinline__ int vec(int i) const { return tid + i * G; }
    __device__ __forceinline__ int column(int i) const { return vec(i) * V - (SHIFT ? lead : 0); }
    __device__ __forceinline__ bool skip(int i) const { return vec(i) >= nvec; }
    __device__ __forceinline__ void store(T* row, int i, const Pack<T, V>& o) const {
        if constexpr (SHIFT) store_whole(row, H, column(i), o.raw);
        else o.store(row + static_cast<int64_t>(vec(i)) * V);
    }
    // the group is done with the row: its slot takes the next one
    __device__ __forceinline__ void next(const Group& g) {
        g.sync();
        issue();
    }
    __device__ __forceinline__ void finish() {
        if (*abort_flag && tid == 0)   // loads may be under way: let them land
            for (int i = 0; i < depth; ++i) {
                const uint32_t n = (issued + depth - 1 - i) / depth;
                if (n > 0) mbar_wait(smem_addr(bar + i), (n - 1) & 1u, nullptr, status);
            }
    }
};

template <class T, int V, int NV, int NIN>
struct RowRing : RowInRing<T, V, NV, NIN, false> {};
template <class T, int V, int NV, int NIN>
struct RowShift : RowInRing<T, V, NV, NIN, true> {};

// The weight of column c, times the channel gate.
template <class T, int GATE>
__device__ __forceinline__ float gated_weight(const NormArgs& a, int c) {
    const float w = weight_at(a.w, a.w_dtype, c) + a.w_offset;
    if constexpr (GATE != kGateChannel) return w;
    const float v = to_f32(static_cast<const T*>(a.gate)[c]);
    return w * (a.sigmoid ? sigmoid_as<T>(v) : v);
}

#define MOE_NORM_PROLOGUE                                                             \
    extern __shared__ __align__(128) uint8_t norm_smem[];                             \
    __shared__ __align__(16) float red[kNormGroups * 32];                                                    \
    Group g = make_group(red, a.G);                                                   \
    constexpr int NP = V / 2;                                                   \
    const int R = blockDim.x / a.G;                                   \
    const int64_t step = static_cast<int64_t>(gridDim.x) * R;                         \
    const int64_t t0 = Rows<T, V, NV, 1>::kShift ? static_cast<int64_t>(g.id) * gridDim.x + blockIdx.x \
                                                 : static_cast<int64_t>(blockIdx.x) * R + g.id; \
    grid_dependency_wait();

// h = x * rstd * w
template <class T, int V, int NV, template <class, int, int, int> class Rows>
__global__ void __launch_bounds__(Rows<T, V, NV, 1>::kWide ? kNormWideThreads : kNormThreads)
    pre_norm_kernel(const NormArgs a) {
    MOE_NORM_PROLOGUE
    Rows<T, V, NV, 1> in;
    in.src[0] = static_cast<const T*>(a.x);
    in.ld[0] = a.ldx;
    in.start(a, g, t0, step, R, norm_smem);
    in.weights([&](int c) { return weight_at(a.w, a.w_dtype, c) + a.w_offset; });
    in.weights_done();
    for (int64_t t = t0; t < a.T; t += step) {
        in.fetch(t);
        float2 ss = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Pack<T, V> x = in.get(0, i);
#pragma unroll
            for (int e = 0; e < NP; ++e) ss = fma2(x.pair(e), x.pair(e), ss);
        }
        const float r = __frsqrt_rn(g.sum(ss.x + ss.y) / static_cast<float>(a.H) + a.eps);
        if (g.tid == 0) a.rstd[t] = r;
        T* out = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (in.skip(i)) continue;
            const Pack<T, V> x = in.again(0, i);
            const Weights<V> w = in.weight(i);
            Pack<T, V> o;
#pragma unroll
            for (int e = 0; e < NP; ++e) o.set_pair(e, mul2(mul2(x.pair(e), both(r)), w.v[e]));
            in.store(out, i, o);
        }
        in.next(g);
    }
    in.finish();
}

// out = a * res + b * g * (y * rstd * w); NEXT: h2 = out * rstd2 * w2 of the stored out
template <class T, int V, int NV, int GATE, bool NEXT, template <class, int, int, int> class Rows>
__global__ void __launch_bounds__(!Rows<T, V, NV, 1>::kWide || NEXT ? kNormThreads : kNormWideThreads)
    post_norm_kernel(const NormArgs a) {
    MOE_NORM_PROLOGUE
    Rows<T, V, NV, full_gate(GATE) ? 3 : 2> in;
    in.src[0] = static_cast<const T*>(a.x);
    in.ld[0] = a.ldx;
    in.src[1] = static_cast<const T*>(a.res);
    in.ld[1] = a.ldr;
    if constexpr (full_gate(GATE)) {
        in.src[2] = static_cast<const T*>(a.gate);
        in.ld[2] = a.ldg;
    }
    in.start(a, g, t0, step, R, norm_smem);
    in.weights([&](int c) { return gated_weight<T, GATE>(a, c); });
    in.weights_done();
    float2 w2[NEXT ? NV * NP : 1];
    if constexpr (NEXT) {
#pragma unroll
        for (int i = 0; i < NV * NP; ++i) {
            const int c = in.column(i / NP) + (i % NP) * 2;
            w2[i] = both(0.0f);
            if (c < a.H) {
                if (!in.kShift || c >= 0) w2[i].x = weight_at(a.w2, a.w_dtype, c) + a.w_offset;
                if (!in.kAny || (c + 1 >= 0 && c + 1 < a.H)) w2[i].y = weight_at(a.w2, a.w_dtype, c + 1) + a.w_offset;
            }
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
        float2 ss = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Pack<T, V> y = in.get(0, i);
#pragma unroll
            for (int e = 0; e < NP; ++e) ss = fma2(y.pair(e), y.pair(e), ss);
        }
        const float r = __frsqrt_rn(g.sum(ss.x + ss.y) / static_cast<float>(a.H) + a.eps);
        if (g.tid == 0) a.rstd[t] = r;
        T* out = static_cast<T*>(a.out) + t * a.H;
        float2 s2 = both(0.0f);
        Pack<T, V> s[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Pack<T, V> y = NEXT ? in.get(0, i) : in.again(0, i), res = NEXT ? in.get(1, i) : in.again(1, i);
            const Weights<V> w = in.weight(i);
            Pack<T, V> gt;
            if constexpr (full_gate(GATE)) gt = NEXT ? in.get(2, i) : in.again(2, i);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                float2 z = mul2(mul2(mul2(y.pair(e), both(r)), w.v[e]), both(b));
                if constexpr (GATE == kGateFull) z = mul2(z, gt.pair(e));
                if constexpr (GATE == kGateFullSigmoid) z = mul2(z, sigmoid_as<T>(gt.pair(e)));
                s[i].set_pair(e, fma2(both(a.a), res.pair(e), z));
                if constexpr (NEXT) s2 = fma2(s[i].pair(e), s[i].pair(e), s2);
            }
            if (!in.skip(i)) in.store(out, i, s[i]);
        }
        in.next(g);
        if constexpr (NEXT) {
            const float r2 = __frsqrt_rn(g.sum(s2.x + s2.y) / static_cast<float>(a.H) + a.eps);
            if (g.tid == 0) a.rstd2[t] = r2;
            T* h2 = static_cast<T*>(a.h2) + t * a.H;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (in.skip(i)) continue;
                Pack<T, V> o;
#pragma unroll
                for (int e = 0; e < NP; ++e) o.set_pair(e, mul2(mul2(s[i].pair(e), both(r2)), w2[i * NP + e]));
                in.store(h2, i, o);
            }
        }
    }
    in.finish();
}

// The CTA's sums over rows (times scale), group after group, into its row of the partials.
template <int V, int NV, class Rows>
__device__ __forceinline__ void write_partial(const float2 (&acc)[NV * (V / 2)], float scale, float* sum_s,
                                              const Rows& in, const Group& g, int R, int H, float* partial) {
    constexpr int NP = V / 2;
    __syncthreads();   // sum_s is the ring's memory
    for (int k = 0; k < R; ++k) {
        if (g.id == k) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c0 = in.column(i);
                if (c0 >= H) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (in.kAny && (c0 + e < 0 || c0 + e >= H)) continue;
                    const float2 p = acc[i * NP + e / 2];
                    const float u = (e & 1 ? p.y : p.x) + (k > 0 ? sum_s[c0 + e] : 0.0f);
                    if (k + 1 < R) sum_s[c0 + e] = u;
                    else partial[c0 + e] = u * scale;
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
    in.weights([&](int c) { return weight_at(a.w, a.w_dtype, c) + a.w_offset; });
    in.weights_done();
    float2 acc[NV * NP];
#pragma unroll
    for (int i = 0; i < NV * NP; ++i) acc[i] = both(0.0f);
    for (int64_t t = t0; t < a.T; t += step) {
        const float r = a.rstd[t];
        in.fetch(t);
        float2 m2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Pack<T, V> x = in.get(0, i), d = in.get(1, i);
            const Weights<V> w = in.weight(i);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 p = mul2(d.pair(e), mul2(x.pair(e), both(r)));
                m2 = fma2(p, w.v[e], m2);
                acc[i * NP + e] = add2(acc[i * NP + e], p);
            }
        }
        const float m = g.sum(m2.x + m2.y) / static_cast<float>(a.H);
        T* out = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (in.skip(i)) continue;
            const Pack<T, V> x = in.again(0, i), d = in.again(1, i);
            const Weights<V> w = in.weight(i);
            Pack<T, V> o, s;
            if constexpr (RES) s = in.again(2, i);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 u = fma2(mul2(x.pair(e), both(r)), both(-m), mul2(d.pair(e), w.v[e]));
                if constexpr (RES) o.set_pair(e, fma2(u, both(r), s.pair(e)));
                else o.set_pair(e, mul2(u, both(r)));
            }
            in.store(out, i, o);
        }
        in.next(g);
    }
    in.finish();
    write_partial<V, NV>(acc, 1.0f, reinterpret_cast<float*>(norm_smem), in, g, R, a.H,
                         a.partial + static_cast<int64_t>(blockIdx.x) * a.H);
}

// dy, dres = a * dout, and by the gate's shape
//   row:     dg = act'(g) * b * sum(dout * n * w); partial sums of b * g * dout * n (dw)
//   channel: partial sums of dout * n (dw and dg follow from them column by column)
//   full:    dg = act'(g) * b * dout * n * w;      partial sums of b * g * dout * n (dw)
template <class T, int V, int NV, int GATE, template <class, int, int, int> class Rows>
__global__ void __launch_bounds__(kNormThreads) post_norm_backward_kernel(const NormArgs a) {
    MOE_NORM_PROLOGUE
    // the gate's sigmoids: fp32 ones stay in registers from pass to pass (their division costs more), the slope
    // needs the exponential again either way
    constexpr bool FULL = full_gate(GATE), SIGMOID = GATE == kGateFullSigmoid, KEEP = SIGMOID && sizeof(T) == 4;
    Rows<T, V, NV, FULL ? 3 : 2> in;
    in.src[0] = static_cast<const T*>(a.x);
    in.ld[0] = a.ldx;
    in.src[1] = static_cast<const T*>(a.dout);
    in.ld[1] = a.ldo;
    if constexpr (FULL) {
        in.src[2] = static_cast<const T*>(a.gate);
        in.ld[2] = a.ldg;
    }
    in.start(a, g, t0, step, R, norm_smem);
    in.weights([&](int c) { return gated_weight<T, GATE>(a, c); });
    in.weights_done();
    float2 acc[NV * NP], kept[KEEP ? NV * NP : 1];
#pragma unroll
    for (int i = 0; i < NV * NP; ++i) acc[i] = both(0.0f);
    for (int64_t t = t0; t < a.T; t += step) {
        const float r = a.rstd[t];
        float gr = 1.0f, slope = 1.0f;   // the row's gate and the gate's slope
        if constexpr (GATE == kGateRow) {
            if (a.gate) {
                gr = to_f32(static_cast<const T*>(a.gate)[t * a.ldg]);
                if (a.sigmoid) {
                    const float e = exp_minus<T>(gr);
                    gr = sigmoid_of<T>(e);
                    slope = slope_of(e, gr);
                }
            }
        }
        in.fetch(t);
        float2 m2 = both(0.0f);   // sum of dout (* full gate) * n * w
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Pack<T, V> y = in.get(0, i), d = in.get(1, i);
            const Weights<V> w = in.weight(i);
            Pack<T, V> gt;
            if constexpr (FULL) gt = in.get(2, i);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                float2 p = mul2(d.pair(e), mul2(y.pair(e), both(r)));
                if constexpr (SIGMOID) {
                    const float2 v = gt.pair(e), x = make_float2(exp_minus<T>(v.x), exp_minus<T>(v.y));
                    const float2 s = make_float2(sigmoid_of<T>(x.x), sigmoid_of<T>(x.y));
                    if constexpr (KEEP) kept[i * NP + e] = s;
                    p = mul2(p, s);
                } else if constexpr (FULL) {
                    p = mul2(p, gt.pair(e));
                }
                m2 = fma2(p, w.v[e], m2);
                if constexpr (GATE == kGateRow) acc[i * NP + e] = fma2(p, both(gr), acc[i * NP + e]);
                else acc[i * NP + e] = add2(acc[i * NP + e], p);
            }
        }
        const float sum = g.sum(m2.x + m2.y);
        if constexpr (GATE == kGateRow)
            if (a.dgate && g.tid == 0) static_cast<T*>(a.dgate)[t] = from_f32<T>(slope * a.b * sum);
        const float2 scale = both(a.b * gr * r), m = both(-(sum / static_cast<float>(a.H)));   // scale: of t / w
        const float2 mr = both(m.x * r), rb = both(r * a.b);   // sigmoid of a full gate: n without its own product
        T* dy = static_cast<T*>(a.out) + t * a.H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (in.skip(i)) continue;
            const Pack<T, V> y = in.again(0, i), d = in.again(1, i);
            const Weights<V> w = in.weight(i);
            Pack<T, V> o, p, q, gt;
            if constexpr (FULL) gt = in.again(2, i);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 n = mul2(y.pair(e), both(r));
                float2 dw = mul2(d.pair(e), w.v[e]);
                if constexpr (SIGMOID) {
                    float2 v = gt.pair(e), s;
                    if constexpr (!KEEP) asm volatile("" : "+f"(v.x), "+f"(v.y));   // again, not kept in (spilled) registers
                    const float2 x = make_float2(exp_minus<T>(v.x), exp_minus<T>(v.y));
                    if constexpr (KEEP) s = kept[i * NP + e];
                    else s = make_float2(sigmoid_of<T>(x.x), sigmoid_of<T>(x.y));
                    const float2 slope = make_float2(slope_of(x.x, s.x), slope_of(x.y, s.y));
                    q.set_pair(e, mul2(slope, mul2(dw, mul2(y.pair(e), rb))));
                    dw = mul2(dw, s);
                } else if constexpr (FULL) {
                    q.set_pair(e, mul2(mul2(dw, n), both(a.b)));
                    dw = mul2(dw, gt.pair(e));
                }
                if constexpr (SIGMOID) o.set_pair(e, mul2(scale, fma2(y.pair(e), mr, dw)));
                else o.set_pair(e, mul2(scale, fma2(n, m, dw)));
                p.set_pair(e, mul2(both(a.a), d.pair(e)));
            }
            in.store(dy, i, o);
            if (a.dres) in.store(static_cast<T*>(a.dres) + t * a.H, i, p);
            if constexpr (FULL)
                if (a.dgate) in.store(static_cast<T*>(a.dgate) + t * a.H, i, q);
        }
        in.next(g);
    }
    in.finish();
    write_partial<V, NV>(acc, GATE == kGateChannel ? 1.0f : a.b, reinterpret_cast<float*>(norm_smem), in, g, R, a.H,
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

constexpr int kRingBytes = 222 * 1024;   // of a CTA's weights and rings (one CTA per SM)
constexpr int kRingMostDepth = 4;

// At most: vectors are 8 or 4 elements.
inline int ring_weight_bytes(int H, bool shift) { return shift ? ring_vectors<true>(H, 8) * 32 : H * 4; }

// What an instance remembers: the devices on which its shared-memory limit is set, and the CTAs per SM by the
// warps of a CTA (the same on every device that the library runs on).
struct NormInstance {
    std::atomic<uint64_t> limit{0};
    std::atomic<int> occupancy[kNormThreads / 32 + 1] = {};
};

// One kernel instance, with CTAs of as many row groups as `threads` holds.  Rows in registers: as many
// CTAs as are resident at once, backward one per SM (few partial sums).  Rows in a ring (ring_row bytes of
// it for a row of every matrix): one CTA per SM; shifted, a multiple of 8 of them, so that the rows of
// each start alike.  *ctas: partial rows.
template <class K>
cudaError_t launch_norm(K kernel, NormArgs a, int threads, bool backward, int ring_row, bool shift, int sms,
                        cudaStream_t stream, int* ctas, NormInstance* inst) {
    int R = threads / a.G;
    if (R < 1) R = 1;
    if (R > kNormGroups) R = kNormGroups;
    // sums over groups (two or more: at most 256 threads and 8192 columns each, so at most 32 KB)
    size_t smem = backward && R > 1 ? static_cast<size_t>(a.H) * 4 : 0;
    int occ = 1;
    if (ring_row) {
        const int row = ring_row, weights = ring_weight_bytes(a.H, shift), rings = kRingBytes - weights;
        while (R > 1 && 2 * R * row > rings) --R;
        a.depth = rings / (R * row);
        if (a.depth > kRingMostDepth) a.depth = kRingMostDepth;
        const size_t ring = static_cast<size_t>(weights) + static_cast<size_t>(R) * a.depth * row +
                            (R * a.depth + 1) * 8;
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
    int64_t grid = need < static_cast<int64_t>(occ) * sms ? need : static_cast<int64_t>(occ) * sms;
    if (shift) grid = grid / 8 * 8;
    *ctas = static_cast<int>(grid);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(R * a.G)), smem, stream, a);
}

template <class T, int V, int NV, template <class, int, int, int> class Rows, bool RING>
cudaError_t launch_norm_nv(NormArgs a, int which, int gate, int sms, cudaStream_t stream, int* ctas) {
    constexpr bool SHIFT = Rows<T, V, NV, 1>::kShift;
    a.G = norm_group(SHIFT ? ring_vectors<true>(a.H, V) : (a.H + V - 1) / V, NV);
    const bool next = a.w2 != nullptr;
#define MOE_NORM(INPUTS, BACKWARD, ...)                                                                          \
    do {                                                                                                         \
        static NormInstance inst;                                                                                \
        return launch_norm(__VA_ARGS__, a,                                                                       \
                           BACKWARD ? kNormThreads : !RING ? 256 : next ? kNormThreads : kNormWideThreads,       \
                           BACKWARD, RING ? INPUTS * ring_row_bytes<T, SHIFT>(a.H) : 0, SHIFT, sms, stream, ctas, &inst); \
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
            if (gate == kGateFullSigmoid) {
                if (next) MOE_NORM(3, false, post_norm_kernel<T, V, NV, kGateFullSigmoid, true, Rows>);
                MOE_NORM(3, false, post_norm_kernel<T, V, NV, kGateFullSigmoid, false, Rows>);
            }
            if (next) MOE_NORM(2, false, post_norm_kernel<T, V, NV, kGateRow, true, Rows>);
            MOE_NORM(2, false, post_norm_kernel<T, V, NV, kGateRow, false, Rows>);
        default:
            if (gate == kGateChannel) MOE_NORM(2, true, post_norm_backward_kernel<T, V, NV, kGateChannel, Rows>);
            if (gate == kGateFull) MOE_NORM(3, true, post_norm_backward_kernel<T, V, NV, kGateFull, Rows>);
            if (gate == kGateFullSigmoid) MOE_NORM(3, true, post_norm_backward_kernel<T, V, NV, kGateFullSigmoid, Rows>);
            MOE_NORM(2, true, post_norm_backward_kernel<T, V, NV, kGateRow, Rows>);
    }
#undef MOE_NORM
}

// Whether all matrices of a call lie alike between 16-byte boundaries, row by row.
inline bool alike(const NormArgs& a, int gate, int es) {
    const auto one = [&](const void* p, int64_t ld) {
        return !p || (((address(p) ^ address(a.out)) & 15) == 0 && (ld - a.H) * es % 16 == 0);
    };
    return one(a.x, a.ldx) && one(a.res, a.ldr) && one(a.dout, a.ldo) && one(a.h2, a.H) && one(a.dres, a.H) &&
           (!full_gate(gate) || (one(a.gate, a.ldg) && one(a.dgate, a.H)));
}

// Where the rows come from, by their alignment (wide: 16-byte addresses and strides), number and width:
//   fewer rows than twice the SMs: registers, 16 elements per thread where the row then fits a CTA's
//     threads (more threads on each row).  (bf16 rows of 7168, after with the next norm: 303 of them 7.5 us, 7.9
//     from the ring; 608 of them 12.0 and 11.1.  Rows of 2048: 1024 of them 7.0 and 7.3, 2048 of them 10.5 either way.)
//   else wide rows, and others whose matrices lie alike (not few: 8 CTAs need rows): the ring, 32 elements per thread (8000 bf16 rows
//     of 4811 before and after with the next norm: 102 against 165 us from registers); registers where
//     the weights and two rows do not fit a CTA's shared memory
//   else registers, 16 elements per thread up to 4096 columns, else 32 (8000 rows of 4811: 212 and 165 us;
//     of 1569: 57 and 67)
// The register instances of 32 elements do not fit 128 registers with two or three matrices: the compiler spills
// 100 to 1400 bytes of them a thread (the others at most 32).
template <class T>
cudaError_t launch_norm_type(const NormArgs& a, int which, int gate, bool wide, int sms, cudaStream_t stream,
                             int* ctas) {
    constexpr int W = 16 / static_cast<int>(sizeof(T));
    const int inputs = which == kPreForward ? 1 : which == kPreBackward ? (a.res ? 3 : 2) : full_gate(gate) ? 3 : 2;
    const bool few = a.T < 2 * sms && a.H <= 16 * kNormThreads;
    const int row = wide ? ring_row_bytes<T, false>(a.H) : ring_row_bytes<T, true>(a.H);
    const bool ring = !few && ring_weight_bytes(a.H, !wide) + 2 * inputs * row <= kRingBytes;
    if (wide) {
        if (few) return launch_norm_nv<T, W, 16 / W, RowRegs, false>(a, which, gate, sms, stream, ctas);
        if (ring) return launch_norm_nv<T, W, 32 / W, RowRing, true>(a, which, gate, sms, stream, ctas);
        return launch_norm_nv<T, W, 32 / W, RowRegs, false>(a, which, gate, sms, stream, ctas);
    }
    if (ring && a.T >= 2 * sms && ring_vectors<true>(a.H, W) <= 32 / W * kNormThreads && alike(a, gate, static_cast<int>(sizeof(T))))
        return launch_norm_nv<T, W, 32 / W, RowShift, true>(a, which, gate, sms, stream, ctas);
    if (few || a.H <= 8 * kNormThreads)
        return launch_norm_nv<T, W, 16 / W, RowAny, false>(a, which, gate, sms, stream, ctas);
    return launch_norm_nv<T, W, 32 / W, RowAny, false>(a, which, gate, sms, stream, ctas);
}

// norms_bf16.cu, norms_fp16.cu, norms_fp32.cu
cudaError_t launch_norm_bf16(const NormArgs&, int which, int gate, bool wide, int sms, cudaStream_t, int* ctas);
cudaError_t launch_norm_fp16(const NormArgs&, int which, int gate, bool wide, int sms, cudaStream_t, int* ctas);
cudaError_t launch_norm_fp32(const NormArgs&, int which, int gate, bool wide, int sms, cudaStream_t, int* ctas);

}  // namespace mfp8
