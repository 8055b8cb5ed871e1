// Global norm of many gradient tensors, and their clipping.
//
//   total = sqrt(sum_i |g_i|^2) or max_i |g_i|,  scale = min(1, max_norm / (total + eps)),  g *= scale
//
// Bound by memory: one pass reads the gradients for the norm, a second reads and writes them.  The
// tensors' addresses travel in the kernels' parameters (up to kMostTensors per launch), so nothing
// is copied to the device and a captured graph holds its own copy.  The tensors are cut into
// chunks of 8 KB; warp w of all warps takes chunks w, w + warps, ... through a ring of 2 KB bulk copies
// of its own (192 KB in flight per SM, no barrier between warps).  Every CTA leaves one partial
// result, and every CTA of the scaling kernel joins all partials in one order: the result does not
// depend on the schedule.  Squares are summed in fp32 within a lane's share of a chunk and in fp64
// beyond it; a share whose largest magnitude lies outside 1e-18 .. 1e18, where fp32 squares
// overflow or vanish, is summed again in fp64.
//
// Measured: 1.21 GB of bf16 gradients into other tensors 581 us (norm 178 us = 6.8 TB/s; scaling 377 us = 6.3 TB/s;
// the second read cannot be saved beyond what L2 keeps: 537 us at copy bandwidth); one small layer's 8
// tensors 9.5 us on the device, both launches' latency.  With vectors through registers the large case took
// 662 us; more CTAs per SM or more vectors per thread did not change that.
#include <math.h>
#include <stdlib.h>

#include <algorithm>

#include "train.cuh"

namespace mfp8 {
namespace {

constexpr int kClipThreads = 512;
constexpr int kClipWarps = kClipThreads / 32;
constexpr int kChunkBytes = 8192, kPiece = 2048;
constexpr int kSlots = 6;                 // pieces of a warp's ring
constexpr int kRingBytes = kClipWarps * kSlots * kPiece;
constexpr int kMostTensors = 960;         // per launch: their table fits the 32,764 bytes of kernel parameters
constexpr int kMostCtas = kPlanSms;       // partial results of a launch

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
// Over the lanes of a warp.
__device__ __forceinline__ double join_warp(double acc, int inf) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) acc = join(acc, __shfl_xor_sync(0xffffffffu, acc, s), inf);
    return acc;
}

// A chunk: n elements of tensor k from element e0, between two 8 KB boundaries from the 16-byte one at
// or before the tensor's start.  `bulk` bytes from element `head` come by bulk copies, what is before and
// after them (a tensor that starts or ends inside 16 bytes) element by element.
struct Chunk {
    int k;
    int64_t e0;
    int n, head, bulk;
};
// (sh: elements of 1 << sh bytes; divisions by the size made the chunks' arithmetic 40 us of 620 at 1.2 GB)
__host__ __device__ __forceinline__ int lead_elements(const void* p, int sh) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) >> sh;
}
template <int N>
__device__ __forceinline__ Chunk chunk_at(const ClipTable<N>& t, int64_t c) {
    Chunk u;
    u.k = tensor_of(t, c);
    const int sh = t.dtype[u.k] == MOE_DTYPE_FP32 ? 2 : 1, per = kChunkBytes >> sh, V = 16 >> sh;
    const int lead = lead_elements(t.src[u.k], sh);
    const bool first = c == t.chunk0[u.k];
    u.e0 = first ? 0 : (c - t.chunk0[u.k]) * per - lead;
    const int room = first ? per - lead : per;
    const int64_t left = t.numel[u.k] - u.e0;
    u.n = left < room ? static_cast<int>(left) : room;
    u.head = first && lead ? (V - lead < u.n ? V - lead : u.n) : 0;
    u.bulk = ((u.n - u.head) << sh) & ~15;
    return u;
}

// A warp's ring of pieces.  The chunks are index(0), index(1), ... of this warp; issue() brings the
// next piece of the next chunk that has one.
template <int N, bool REVERSE>
struct ClipRing {
    const ClipTable<N>& t;
    uint8_t* ring;
    uint64_t* bars;
    volatile int* abort_flag;
    uint32_t* status;
    int64_t chunks, next;      // next: chunk after the one being loaded (in this warp's order)
    int stride, slot, load_slot, left;
    uint32_t phase, issued;
    const char* src;

    __device__ __forceinline__ ClipRing(const ClipTable<N>& table, uint8_t* smem, uint64_t* barriers, volatile int* flag,
                                        uint32_t* st)
        : t(table), abort_flag(flag), status(st) {
        const int warp = threadIdx.x >> 5;
        ring = smem + warp * kSlots * kPiece;
        bars = barriers + warp * kSlots;
        chunks = t.chunk0[t.n];
        next = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
        stride = gridDim.x * kClipWarps;
        slot = load_slot = left = 0;
        phase = issued = 0;
        for (int i = 0; i < kSlots; ++i) issue();
    }
    __device__ __forceinline__ int64_t index(int64_t c) const { return REVERSE ? chunks - 1 - c : c; }
    __device__ __forceinline__ void issue() {
        while (left == 0 && next < chunks) {
            const Chunk u = chunk_at(t, index(next));
            src = static_cast<const char*>(t.src[u.k]) + (u.e0 + u.head) * (t.dtype[u.k] == MOE_DTYPE_FP32 ? 4 : 2);
            left = u.bulk;
            next += stride;
        }
        if (left == 0) return;
        const int bytes = left < kPiece ? left : kPiece;
        if ((threadIdx.x & 31) == 0) {
            const uint32_t b = smem_addr(bars + load_slot);
            mbar_arrive_expect_tx(b, bytes);
            bulk_load(smem_addr(ring + load_slot * kPiece), src, bytes, b);
        }
        ++issued;
        src += bytes;
        left -= bytes;
        if (++load_slot == kSlots) load_slot = 0;
    }
    // After a wait that gave up (its status bit is set, values are wrong): let the loads under way land.
    __device__ __forceinline__ void finish() const {
        if (*abort_flag) drain();
    }
    __device__ __forceinline__ void drain() const {
        if ((threadIdx.x & 31) == 0)
            for (int i = 0; i < kSlots; ++i) {
                const uint32_t n = (issued + kSlots - 1 - i) / kSlots;
                if (n > 0) mbar_wait(smem_addr(bars + i), (n - 1) & 1u, nullptr, status);
            }
    }
    // This lane's vectors of a piece of nv, f(vector index, vector) each; then the slot takes the next
    // piece.  ALL: f is called by whole warps, on the lanes past nv too (with no data).
    template <class T, bool ALL, class F>
    __device__ __forceinline__ void piece(int nv, F f) {
        constexpr int V = 16 / static_cast<int>(sizeof(T));
        mbar_wait(smem_addr(bars + slot), phase, abort_flag, status);
        Pack<T, V> x[kPiece / 512];
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kPiece / 512; ++i)
            if (lane + i * 32 < nv) x[i].raw = *reinterpret_cast<const uint4*>(ring + slot * kPiece + (lane + i * 32) * 16);
        __syncwarp();
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1u;
        }
        issue();
#pragma unroll
        for (int i = 0; i < kPiece / 512; ++i)
            if (ALL ? i * 32 < nv : lane + i * 32 < nv) f(lane + i * 32, x[i]);
    }
};

// This lane's share of a chunk: sum of squares, or the largest magnitude.
template <class T, class R>
__device__ __forceinline__ double share_norm(R& ring, const T* p, const Chunk& u, int inf) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const int lane = threadIdx.x & 31, nv = u.bulk / 16;
    float ss = 0.0f, top = 0.0f;
    for (int v0 = 0; v0 < nv; v0 += kPiece / 16)
        ring.template piece<T, false>(nv - v0 < kPiece / 16 ? nv - v0 : kPiece / 16, [&](int, const Pack<T, V>& x) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float v = x.get(e);
                ss = fmaf(v, v, ss);
                top = max_nan(top, fabsf(v));
            }
        });
    const auto loose = [&](auto f) {   // (less than a vector on either side)
        if (lane < u.head) f(to_f32(p[lane]));
        if (u.head + nv * V + lane < u.n) f(to_f32(p[u.head + nv * V + lane]));
    };
    loose([&](float v) {
        ss = fmaf(v, v, ss);
        top = max_nan(top, fabsf(v));
    });
    if (inf) return top;
    if (top > 1e18f || (top < 1e-18f && top > 0.0f)) {
        double sd = 0.0;
        for (int v = lane; v < nv; v += 32)
            for (int e = 0; e < V; ++e) {
                const double x = to_f32(p[u.head + v * V + e]);
                sd = fma(x, x, sd);
            }
        loose([&](float v) { sd = fma(static_cast<double>(v), static_cast<double>(v), sd); });
        return sd;
    }
    return ss;
}

#define MOE_CLIP_PROLOGUE                                                       \
    extern __shared__ __align__(128) uint8_t clip_smem[];                       \
    __shared__ uint64_t bars[kClipWarps * kSlots];                              \
    __shared__ int abort_s;                                                     \
    if (threadIdx.x < kClipWarps * kSlots) {                                    \
        mbar_init(smem_addr(bars + threadIdx.x), 1);                            \
        fence_barrier_init();                                                   \
    }                                                                           \
    if (threadIdx.x == 0) abort_s = 0;                                          \
    __syncthreads();                                                            \
    grid_dependency_wait();

// The partial result of a CTA: sum of squares (or largest magnitude) of its warps' chunks.
template <int N>
__global__ void __launch_bounds__(kClipThreads, 1)
    grad_norm_kernel(const __grid_constant__ ClipTable<N> t, int inf, double* __restrict__ partial, uint32_t* status) {
    MOE_CLIP_PROLOGUE
    ClipRing<N, false> ring(t, clip_smem, bars, &abort_s, status);
    double acc = 0.0;
    for (int64_t c = static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x; c < ring.chunks; c += ring.stride) {
        const Chunk u = chunk_at(t, c);
        double v;
        if (t.dtype[u.k] == MOE_DTYPE_FP32) v = share_norm(ring, static_cast<const float*>(t.src[u.k]) + u.e0, u, inf);
        else if (t.dtype[u.k] == MOE_DTYPE_FP16) v = share_norm(ring, static_cast<const __half*>(t.src[u.k]) + u.e0, u, inf);
        else v = share_norm(ring, static_cast<const __nv_bfloat16*>(t.src[u.k]) + u.e0, u, inf);
        acc = join(acc, v, inf);
    }
    ring.finish();
    // the threads' results through shared memory to one warp (fp64 runs at a 64th of the fp32 rate: joined
    // by all warps they took as long as the loads of a small call)
    __syncthreads();
    double* all = reinterpret_cast<double*>(clip_smem);
    all[threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    for (int i = 1; i < kClipWarps; ++i) acc = join(acc, all[threadIdx.x + i * 32], inf);
    acc = join_warp(acc, inf);
    if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// ANY: the result's 16-byte boundaries lie elsewhere than the gradient's.
template <class T, bool ANY, class R>
__device__ __forceinline__ void scale_share(R& ring, const T* p, T* q, const Chunk& u, float scale) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const int nv = u.bulk / 16, lane = threadIdx.x & 31;
    T* qb = q + u.head;
    const auto scaled = [&](const Pack<T, V>& x) {
        Pack<T, V> o;
#pragma unroll
        for (int e = 0; e < V; ++e) o.set(e, x.get(e) * scale);
        return o;
    };
    for (int v0 = 0; v0 < nv; v0 += kPiece / 16)
        ring.template piece<T, ANY>(nv - v0 < kPiece / 16 ? nv - v0 : kPiece / 16, [&](int v, const Pack<T, V>& x) {
            if constexpr (ANY) store_any(qb, nv * V, v0 + v, scaled(x).raw);
            else scaled(x).store(qb + (v0 + v) * V);
        });
    if (lane < u.head) q[lane] = from_f32<T>(to_f32(p[lane]) * scale);
    const int tail = u.head + nv * V + lane;
    if (tail < u.n) q[tail] = from_f32<T>(to_f32(p[tail]) * scale);
}

// Every CTA joins the partial results (np of them) and scales its chunks, the last first: they are
// the ones the norm read last, so they are still in L2.  A scale of one where every gradient stays in
// place leaves them alone.
template <int N, bool ANY>
__global__ void __launch_bounds__(kClipThreads, 1)
    grad_scale_kernel(const __grid_constant__ ClipTable<N> t, int inf, const double* __restrict__ partial, int np,
                      float max_norm, float eps, int write_total, int all_in_place, float* __restrict__ total,
                      uint32_t* status) {
    MOE_CLIP_PROLOGUE
    __shared__ float scale_s;
    ClipRing<N, true> ring(t, clip_smem, bars, &abort_s, status);   // the first loads run while the norm is joined
    if (threadIdx.x < 32) {
        double acc = 0.0;
        for (int i = threadIdx.x; i < np; i += 32) acc = join(acc, partial[i], inf);
        acc = join_warp(acc, inf);
        if (threadIdx.x == 0) {
            const double norm = inf ? acc : sqrt(acc);
            if (write_total && blockIdx.x == 0) *total = static_cast<float>(norm);
            const double ratio = static_cast<double>(max_norm) / (norm + static_cast<double>(eps));
            scale_s = ratio > 1.0 ? 1.0f : static_cast<float>(ratio);   // a NaN stays
        }
    }
    __syncthreads();
    const float scale = scale_s;
    if (scale == 1.0f && all_in_place) {
        ring.drain();
        return;
    }
    for (int64_t c = static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x; c < ring.chunks; c += ring.stride) {
        const Chunk u = chunk_at(t, ring.index(c));
        if (t.dtype[u.k] == MOE_DTYPE_FP32)
            scale_share<float, ANY>(ring, static_cast<const float*>(t.src[u.k]) + u.e0, static_cast<float*>(t.dst[u.k]) + u.e0, u, scale);
        else if (t.dtype[u.k] == MOE_DTYPE_FP16)
            scale_share<__half, ANY>(ring, static_cast<const __half*>(t.src[u.k]) + u.e0, static_cast<__half*>(t.dst[u.k]) + u.e0, u, scale);
        else
            scale_share<__nv_bfloat16, ANY>(ring, static_cast<const __nv_bfloat16*>(t.src[u.k]) + u.e0,
                        static_cast<__nv_bfloat16*>(t.dst[u.k]) + u.e0, u, scale);
    }
    ring.finish();
}
#undef MOE_CLIP_PROLOGUE

int64_t chunks_of(const void* src, int64_t numel, int dtype) {
    const int sh = dtype == MOE_DTYPE_FP32 ? 2 : 1;
    const int64_t per = kChunkBytes >> sh;
    return numel == 0 ? 0 : (lead_elements(src, sh) + numel + per - 1) / per;
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
    int all_in_place;
    bool apart;      // some result's 16-byte boundaries lie elsewhere than its gradient's
    uint32_t* status;
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
        t->chunk0[i + 1] = t->chunk0[i] + chunks_of(c.src[k], c.numel[k], c.dtype[k]);
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
        e = launch_pdl(grad_norm_kernel<N>, dim3(grid), dim3(kClipThreads), kRingBytes, c.stream, t, c.inf, c.partial + np,
                       c.status);
        np += static_cast<int>(grid);
    }
    for (int b = 0; b < batches && e == cudaSuccess; ++b) {
        if (batches > 1) fill_table(&t, c, b * N, c.n < (b + 1) * N ? c.n : (b + 1) * N);
        e = launch_pdl(c.apart ? grad_scale_kernel<N, true> : grad_scale_kernel<N, false>, dim3(clip_grid(t.chunk0[t.n])), dim3(kClipThreads), kRingBytes, c.stream, t,
                       c.inf, static_cast<const double*>(c.partial), np, c.max_norm, c.eps, b == 0 ? 1 : 0, c.all_in_place,
                       c.total, c.status);
    }
    return e;
}

// Whether no result shares memory with another result or with another tensor's gradient (their chunks run side by
// side, in no order).  MOE_OK, MOE_ERR_INVALID_ARG, or MOE_ERR_CUDA where the host has no memory for the check.
int check_apart(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* dtype, int n) {
    struct Span {
        uintptr_t begin, end;
        bool written;
    };
    constexpr int kOnStack = 256;
    Span few[kOnStack];
    Span* all = n <= kOnStack / 2 ? few : static_cast<Span*>(malloc(sizeof(Span) * 2 * static_cast<size_t>(n)));
    if (!all) return MOE_ERR_CUDA;
    int m = 0;
    for (int i = 0; i < n; ++i) {
        const uintptr_t bytes = static_cast<uintptr_t>(numel[i]) * dtype_bytes(dtype[i]);
        if (bytes == 0) continue;
        all[m++] = {address(out[i]), address(out[i]) + bytes, true};
        if (grads[i] != out[i]) all[m++] = {address(grads[i]), address(grads[i]) + bytes, false};
    }
    const auto before = [](const Span& a, const Span& b) { return a.begin < b.begin; };
    if (!std::is_sorted(all, all + m, before)) std::sort(all, all + m, before);
    uintptr_t any = 0, written = 0;   // where the spans so far, and those of results, end
    bool apart = true;
    for (int i = 0; i < m && apart; ++i) {
        apart = all[i].begin >= (all[i].written ? any : written);
        any = std::max(any, all[i].end);
        if (all[i].written) written = std::max(written, all[i].end);
    }
    if (all != few) free(all);
    return apart ? MOE_OK : MOE_ERR_INVALID_ARG;
}

template <int N>
cudaError_t clip_init() {
    cudaError_t e = cudaFuncSetAttribute(grad_norm_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grad_scale_kernel<N, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(grad_scale_kernel<N, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    return e;
}

}  // namespace

cudaError_t clip_init_device() {
    cudaError_t e = clip_init<32>();
    if (e == cudaSuccess) e = clip_init<128>();
    if (e == cudaSuccess) e = clip_init<kMostTensors>();
    return e;
}

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
    int all_in_place = 1;
    bool apart = false;
    for (int i = 0; i < n; ++i) {
        if (numel[i] < 0 || !known_dtype(dtype[i])) return MOE_ERR_INVALID_ARG;
        if (numel[i] > 0 && (!grads[i] || !out[i])) return MOE_ERR_INVALID_ARG;
        if (!on_element(address(grads[i]) | address(out[i]), dtype_bytes(dtype[i]))) return MOE_ERR_INVALID_ARG;
        if (numel[i] > (int64_t(1) << 50)) return MOE_ERR_UNSUPPORTED_SHAPE;
        if (numel[i] > 0 && grads[i] != out[i]) all_in_place = 0;
        if (numel[i] > 0 && ((address(grads[i]) ^ address(out[i])) & 15)) apart = true;
    }
    int rc = check_apart(grads, out, numel, dtype, n);
    if (rc != MOE_OK) return rc;
    if (workspace_bytes < moe_clip_grads_workspace_size(n)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace || !on_element(address(workspace), 8)) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    const ClipCall c = {grads, out, numel, dtype, n, norm_kind == MOE_NORM_INF ? 1 : 0, max_norm, eps, total_norm,
                        static_cast<double*>(workspace), all_in_place, apart, status, static_cast<cudaStream_t>(stream)};
    return cuda_status(n <= 32 ? clip_launches<32>(c) : n <= 128 ? clip_launches<128>(c)
                                                                 : clip_launches<kMostTensors>(c));
}

}  // extern "C"
