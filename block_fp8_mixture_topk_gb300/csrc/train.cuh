// Device helpers of the training operators (token movement, block norms, gradient clipping,
// 16-bit expert products): element types, vector loads and stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.cuh"

namespace mfp8 {

// api.cu: SMs of the current device (valid after device_status_word succeeded)
int device_sms();

// ---------------------------------------------------------------- types
template <int BYTES>
struct RawOf;
template <>
struct RawOf<16> {
    using type = uint4;
};
template <>
struct RawOf<4> {
    using type = uint32_t;
};
template <>
struct RawOf<2> {
    using type = uint16_t;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}

// V elements of type T in one register vector of 16 bytes (addresses aligned to it).
template <class T, int V>
struct Pack {
    using Raw = typename RawOf<static_cast<int>(sizeof(T)) * V>::type;
    union {
        Raw raw;
        T e[V];
    };
    __device__ __forceinline__ Pack() {}
    __device__ __forceinline__ void load(const T* p) { raw = __ldg(reinterpret_cast<const Raw*>(p)); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = raw; }
    __device__ __forceinline__ void zero() { raw = Raw{}; }
    __device__ __forceinline__ float get(int i) const { return to_f32(e[i]); }
    __device__ __forceinline__ void set(int i, float v) { e[i] = from_f32<T>(v); }
    // elements 2i and 2i + 1, for the packed fp32 arithmetic
    __device__ __forceinline__ float2 pair(int i) const { return make_float2(to_f32(e[2 * i]), to_f32(e[2 * i + 1])); }
    __device__ __forceinline__ void set_pair(int i, float2 v) {
        e[2 * i] = from_f32<T>(v.x);
        e[2 * i + 1] = from_f32<T>(v.y);
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// ---------------------------------------------------------------- rows at any address
// Rows of an odd number of elements start anywhere between two 16-byte boundaries, each row elsewhere.
// They are still read and written 16 bytes at a time: a lane loads the aligned vector that its own starts
// in and takes the rest from the next lane's; only a row's first and last results are written element by
// element.  (Element by element throughout, the same kernels took two to six times as long.)

// Bytes s .. s + 15 of the 32 bytes lo, hi (s <= 16).
__device__ __forceinline__ uint4 bytes_from(uint4 lo, uint4 hi, uint32_t s) {
    if (s & 8) lo = make_uint4(lo.z, lo.w, hi.x, hi.y), hi.x = hi.z, hi.y = hi.w;
    if (s & 4) lo = make_uint4(lo.y, lo.z, lo.w, hi.x), hi.x = hi.y;
    const uint32_t b = (s & 3) * 8;
    return make_uint4(__funnelshift_r(lo.x, lo.y, b), __funnelshift_r(lo.y, lo.z, b), __funnelshift_r(lo.z, lo.w, b),
                      __funnelshift_r(lo.w, hi.x, b));
}
// 16 bytes where `on`, else zero; without a branch, so that many of them are under way at once.
__device__ __forceinline__ uint4 load_if(bool on, uintptr_t p) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred on;\n\tsetp.ne.u32 on, %4, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@on ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%5];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "r"(static_cast<uint32_t>(on)), "l"(p));
    return v;
}
// The aligned vector in which element e of a row of n lies, where it holds any of the row (else zero).  It may
// reach up to 14 bytes to either side of the row, so only rows with kMarginRows rows of the matrix on
// either side are read by it (inner_row).
template <class T>
__device__ __forceinline__ uint4 load_around(const T* row, int n, int e, bool on = true) {
    const uintptr_t q = reinterpret_cast<uintptr_t>(row + e) & ~uintptr_t(15);
    const uint32_t past = static_cast<uint32_t>(q - reinterpret_cast<uintptr_t>(row)) + 15u;   // 1: its last byte is the row's first
    return load_if(on && past >= 1u && past < n * sizeof(T) + 15u, q);
}
constexpr int kMarginRows = 8;   // of one 2-byte element
__device__ __forceinline__ bool inner_row(int64_t r, int64_t rows) { return r >= kMarginRows && r + kMarginRows < rows; }
// Elements e .. e + V - 1 of a row of n, one by one; zero outside the row.
template <class T>
__device__ __noinline__ uint4 load_elements(const T* row, int n, int e) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    using Bits = typename RawOf<static_cast<int>(sizeof(T))>::type;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (e + i >= 0 && e + i < n)
            w[i * sizeof(T) / 4] |= static_cast<uint32_t>(reinterpret_cast<const Bits*>(row)[e + i]) << (i * sizeof(T) % 4 * 8);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 shuffle(uint4 w, int lane) {
    constexpr uint32_t kAll = 0xffffffffu;
    return make_uint4(__shfl_sync(kAll, w.x, lane), __shfl_sync(kAll, w.y, lane), __shfl_sync(kAll, w.z, lane),
                      __shfl_sync(kAll, w.w, lane));
}
// By a whole warp: V elements from p on, p one vector more from lane to lane, w this lane's aligned vector
// that p lies in.  Lanes 0 .. 30 (the last one's rest is in no lane).
constexpr int kAnyLanes = 31;
template <class T>
__device__ __forceinline__ uint4 join_lanes(uint4 w, const T* p) {
    return bytes_from(w, shuffle(w, (threadIdx.x + 1) & 31), static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u);
}
// `w` with zero for elements past n of a row, w holding elements e0 .. e0 + V - 1 (and before its first).
template <class T>
__device__ __forceinline__ uint4 inside_row(uint4 w, int n, int e0) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    if (e0 >= 0 && e0 + V <= n) return w;
    uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (e0 + e < 0 || e0 + e >= n)
            r[e * sizeof(T) / 4] &= sizeof(T) == 4 ? 0u : e & 1 ? 0xffffu : 0xffff0000u;
    return make_uint4(r[0], r[1], r[2], r[3]);
}
// `w` to elements e0 .. e0 + V - 1 of a row of n, as far as they are in it; row + e0 is a 16-byte address.
template <class T>
__device__ __forceinline__ void store_whole(T* row, int n, int e0, uint4 w) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    using Bits = typename RawOf<static_cast<int>(sizeof(T))>::type;
    if (e0 >= 0 && e0 + V <= n) {
        *reinterpret_cast<uint4*>(row + e0) = w;
    } else if (e0 + V > 0 && e0 < n) {
        const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e0 + e >= 0 && e0 + e < n)
                reinterpret_cast<Bits*>(row)[e0 + e] = static_cast<Bits>(r[e * sizeof(T) / 4] >> (e * sizeof(T) % 4 * 8));
    }
}
// By a whole warp: `w` of each lane to vector v of a row of n at any address, v one more from lane to
// lane.  The lanes write the aligned vectors between them: the end of the lane before's and the start
// of their own.  What is left, the start of the first lane's and the end of the last one's, is V
// elements together and goes one element to a lane.
template <class T>
__device__ __forceinline__ void store_any(T* row, int n, int v, uint4 w) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    using Bits = typename RawOf<static_cast<int>(sizeof(T))>::type;
    const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u;   // a vector is 16 bytes
    if (s == 0) {
        store_whole(row, n, v * V, w);
        return;
    }
    const int lane = threadIdx.x & 31, over = static_cast<int>(s / sizeof(T));   // elements past an aligned address
    const uint4 before = shuffle(w, (lane + 31) & 31);
    if (lane > 0) store_whole(row, n, v * V - over, bytes_from(before, w, 16 - s));
    const int from = lane < V - over ? 0 : 31;
    const uint4 f = shuffle(w, from);
    const int e = (v - lane + from) * V + lane;   // lane < V
    const int at = lane * static_cast<int>(sizeof(T));
    const uint32_t word = at & 8 ? (at & 4 ? f.w : f.z) : (at & 4 ? f.y : f.x);
    if (lane < V && e < n) reinterpret_cast<Bits*>(row)[e] = static_cast<Bits>(word >> (at & 3) * 8);
}

// ---------------------------------------------------------------- host helpers
inline size_t dtype_bytes(int dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 2; }
inline bool known_dtype(int dtype) {
    return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_FP16 || dtype == MOE_DTYPE_FP32;
}
inline uintptr_t address(const void* p) { return reinterpret_cast<uintptr_t>(p); }
inline bool on_element(uintptr_t bits, size_t bytes) { return bits % bytes == 0; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
// SMs of a GB300, by which chunks, partial results and so workspaces are sized
constexpr int kPlanSms = 152;

}  // namespace mfp8
