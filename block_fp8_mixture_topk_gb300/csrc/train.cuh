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
struct RawOf<8> {
    using type = uint2;
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

// V elements of type T in one register vector (V * sizeof(T) is 2, 4, 8 or 16 bytes; addresses
// aligned to it).
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
    // elements 2i and 2i + 1 (V == 1: the element and zero), for the packed fp32 arithmetic
    static constexpr int kPairs = (V + 1) / 2;
    __device__ __forceinline__ float2 pair(int i) const {
        return make_float2(to_f32(e[2 * i]), V > 1 ? to_f32(e[V > 1 ? 2 * i + 1 : 0]) : 0.0f);
    }
    __device__ __forceinline__ void set_pair(int i, float2 v) {
        e[2 * i] = from_f32<T>(v.x);
        if (V > 1) e[V > 1 ? 2 * i + 1 : 0] = from_f32<T>(v.y);
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

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
