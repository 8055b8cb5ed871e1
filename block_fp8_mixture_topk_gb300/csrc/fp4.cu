// Microscaled 4-bit quantisation of rows and weights, and the values back (formats and layouts: fp4.cuh).
//
// A group's scale and codes are the real numbers' nearest (ties to even), whatever the order of operations:
//   mxfp4  scale = the smallest power of two s with max|x| <= 6 s, code = e2m1(x / s): x / s is exact
//   nvfp4  r = fp32(max|x of the row| / 2688), b = e4m3(max|x of the group| / (6 r)), code = e2m1(x / (b r)): the
//          quotients are taken in fp32 a little too large and a little too small; where the two round differently,
//          a comparison with the border itself, exact in fp64, decides
// An infinity or NaN makes its group (mxfp4: scale NaN) or row (nvfp4: row scale NaN) NaN.
//
// Memory is the bound: a row's vectors of eight elements are loaded once, all of them before the first is used,
// and stay in registers (32 to 1024 threads to a row, up to four vectors each); the codes go out as whole words, the
// scales as words of four groups put together across lanes.
#include "fp4.cuh"

namespace mfp8 {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kVecs = 4;   // vectors of 8 elements a thread

// 8 elements from p (16-byte addresses unless !ALIGNED).
template <class T, bool ALIGNED>
struct Vec8 {
    static constexpr int kRaw = sizeof(T) == 4 ? 2 : 1;
    uint4 raw[kRaw];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int i = 0; i < kRaw; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
        } else {
            T* e = reinterpret_cast<T*>(raw);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = p[i];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kRaw; ++i) raw[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ float get(int i) const { return to_f32(reinterpret_cast<const T*>(raw)[i]); }
    // bits of the largest magnitude: they order as the magnitudes do, infinity and NaN above
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(get(i)) & 0x7fffffffu);
        return m;
    }
};

__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
// codes of x[i] * f, one word
template <class V>
__device__ __forceinline__ uint32_t e2m1_word(const V& x, float f) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= e2m1_pair(x.get(2 * i) * f, x.get(2 * i + 1) * f) << (8 * i);
    return w;
}

// e2m1(x / d) by the borders between the codes: d has at most 28 bits and a border 3, so the products are exact.
__device__ __forceinline__ uint32_t e2m1_exact(float x, double d) {
    const double a = fabs(static_cast<double>(x));
    const float border[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f};
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        const double t = border[i] * d;
        c += a > t || (a == t && (i & 1)) ? 1u : 0u;
    }
    return c | (__float_as_uint(x) >> 31 << 3);
}
template <class V>
__device__ __noinline__ uint32_t e2m1_word_exact(V x, double d) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= e2m1_exact(x.get(i), d) << (4 * i);
    return w;
}
// e4m3(x / (6 r)) for x >= 0, r > 0, likewise: the border to the next number has 5 bits.
__device__ __noinline__ uint32_t e4m3_exact(float x, float r) {
    const double d = 6.0 * static_cast<double>(r);
    const uint32_t near = e4m3x2(static_cast<float>(fmin(static_cast<double>(x) / d, 448.0)), 0.0f) & 0x7fu;
    uint32_t c = near > 0 ? near - 1 : 0;
    while (c < 126) {
        const double t = 0.5 * (e4m3_number(c) + e4m3_number(c + 1)) * d;
        if (x < t || (x == t && (c & 1) == 0)) break;
        ++c;
    }
    return c;
}

// Where a row's scales go: rows' tiles (tiles not null) or [rows, K / group].
struct QuantArgs {
    const void* x;
    int64_t ld, rows;
    int K, E;
    const int32_t* offsets;
    uint8_t* codes;
    uint8_t* tiles;
    uint8_t* plain;
    float* row_scale;
};

constexpr float kSlack = 0x1p-21f;       // over the error of a quotient or product of a few fp32 operations
constexpr float kLeastRow = 0x1p-100f;   // row scales below: fp64 throughout

template <class T, int FMT, bool ALIGNED>
__global__ void __launch_bounds__(1024) fp4_quant_kernel(const QuantArgs a, int tpr) {
    grid_dependency_wait();
    constexpr int G = fp4_group(FMT), LANES = G / 8, W = fp4_words(FMT);   // lanes of a group
    __shared__ uint32_t s_top[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int at = threadIdx.x % tpr;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = r < a.rows;
    const int KB = fp4_blocks(a.K), vecs = a.K / 8;
    const T* row = static_cast<const T*>(a.x) + r * a.ld;
    Vec8<T, ALIGNED> x[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int v = at + i * tpr;
        if (live && v < vecs) x[i].load(row + v * 8);
        else x[i].zero();
    }
    uint32_t top[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        top[i] = x[i].top();
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) top[i] = max(top[i], __shfl_xor_sync(kAll, top[i], o));
    }
    float rs = 1.0f;
    if constexpr (FMT == MOE_FP4_NVFP4) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) m = max(m, top[i]);
        m = __reduce_max_sync(kAll, m);
        if (tpr > 32) {
            if (lane == 0) s_top[warp] = m;
            __syncthreads();
            const int first = warp / (tpr / 32) * (tpr / 32);
            m = __reduce_max_sync(kAll, lane < tpr / 32 ? s_top[first + lane] : 0u);
        }
        rs = m < 0x7f800000u ? __fdiv_rn(__uint_as_float(m), 2688.0f) : __int_as_float(0x7fffffff);
        if (live && at == 0) a.row_scale[r] = rs;
    }
    if (!live) return;   // (whole warps: tpr is a multiple of 32)
    Fp4Place place = {0, 0};
    if (a.tiles) place = fp4_place(a.offsets, a.E, r);
    uint8_t* tile = a.tiles + (place.tile * KB * 2 + (place.in >> 7)) * (W * 512);
    uint32_t* codes = reinterpret_cast<uint32_t*>(a.codes + r * (a.K / 2));
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int v = at + i * tpr;
        if (v >= KB * 32) break;   // (whole warps)
        uint32_t s, w;
        if constexpr (FMT == MOE_FP4_MXFP4) {
            const uint32_t e = top[i] >> 23;
            const int byte = static_cast<int>(e) - ((top[i] & 0x7fffffu) > 0x400000u ? 1 : 2);
            s = e == 255 ? 255u : static_cast<uint32_t>(max(byte, 0));
            w = e == 255 ? 0u : e2m1_word(x[i], __uint_as_float((254u - s) << 23));   // 2^-(s - 127)
        } else {
            s = 0;
            w = 0;
            if (rs > 0.0f) {   // not zero and not NaN
                const float g = __uint_as_float(top[i]);
                bool exact = rs < kLeastRow;
                if (!exact) {
                    const float t = __fdividef(g, 6.0f * rs);
                    s = e4m3x2(t * (1.0f - kSlack), t * (1.0f + kSlack));
                    exact = (s & 0x7fu) != (s >> 8);
                    s &= 0x7fu;
                }
                if (exact) s = e4m3_exact(g, rs);
                if (s > 0) {
                    const float b = e4m3_number(s), f = __fdividef(1.0f, b * rs);
                    w = e2m1_word(x[i], f * (1.0f + kSlack));
                    if (rs < kLeastRow || w != e2m1_word(x[i], f * (1.0f - kSlack)))
                        w = e2m1_word_exact(x[i], static_cast<double>(b) * static_cast<double>(rs));
                }
            }
        }
        if (v < vecs) codes[v] = w;
        else s = 0;   // columns past K: a scale that is a number
        const int c = v / LANES;   // the group
        if (a.tiles) {
            uint32_t word = s << (8 * (c & 3));
#pragma unroll
            for (int o = LANES; o < 4 * LANES; o <<= 1) word |= __shfl_xor_sync(kAll, word, o);
            const int kb = v >> 5;
            if (lane % (4 * LANES) == 0)
                *reinterpret_cast<uint32_t*>(tile + static_cast<int64_t>(kb) * (2 * W * 512) +
                                             fp4_word(place.in & 127, (c >> 2) % W)) = word;
        } else if (lane % LANES == 0 && v < vecs) {
            a.plain[r * (a.K / G) + c] = static_cast<uint8_t>(s);
        }
    }
}

struct DequantArgs {
    const uint8_t* codes;
    const uint8_t* tiles;
    const float* row_scale;
    const int32_t* offsets;
    int64_t rows;
    int K, E;
    void* out;
};

// Values of the codes: code times group scale is exact in fp32, the row's scale and the result's type round.
template <class T, int FMT>
__global__ void __launch_bounds__(1024) fp4_dequant_kernel(const DequantArgs a, int tpr) {
    grid_dependency_wait();
    constexpr int LANES = fp4_group(FMT) / 8, W = fp4_words(FMT);
    const int at = threadIdx.x % tpr;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    if (r >= a.rows) return;   // (whole warps)
    const int KB = fp4_blocks(a.K), vecs = a.K / 8;
    const Fp4Place place = fp4_place(a.offsets, a.E, r);
    const uint8_t* tile = a.tiles + (place.tile * KB * 2 + (place.in >> 7)) * (W * 512);
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes + r * (a.K / 2));
    const float rs = FMT == MOE_FP4_NVFP4 ? a.row_scale[r] : 1.0f;
    uint32_t w[kVecs], s[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int v = at + i * tpr, c = v / LANES;
        w[i] = s[i] = 0;
        if (v >= vecs) continue;
        w[i] = __ldg(codes + v);
        s[i] = __ldg(reinterpret_cast<const uint32_t*>(tile + static_cast<int64_t>(v >> 5) * (2 * W * 512) +
                                                       fp4_word(place.in & 127, (c >> 2) % W)));
    }
    T* out = static_cast<T*>(a.out) + r * a.K;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int v = at + i * tpr, c = v / LANES;
        if (v >= vecs) continue;
        const uint32_t byte = (s[i] >> (8 * (c & 3))) & 0xffu;
        const float scale = FMT == MOE_FP4_MXFP4 ? ue8m0_number(byte) : e4m3_number(byte);
        alignas(16) T e[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h;
            asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(w[i] >> (8 * j)));
            const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
            e[2 * j] = from_f32<T>(FMT == MOE_FP4_NVFP4 ? f.x * scale * rs : f.x * scale);
            e[2 * j + 1] = from_f32<T>(FMT == MOE_FP4_NVFP4 ? f.y * scale * rs : f.y * scale);
        }
#pragma unroll
        for (int j = 0; j < static_cast<int>(sizeof(e)) / 16; ++j)
            reinterpret_cast<uint4*>(out + v * 8)[j] = reinterpret_cast<const uint4*>(e)[j];
    }
}

// Scale bytes [E, N, C] into the weights' tiles, a word to a thread; rows and columns past the end get 0.
__global__ void __launch_bounds__(256) fp4_pack_kernel(const uint8_t* s, int64_t words, int N, int C, int KB, int W,
                                                       int tiles, int gate_up, uint32_t* out) {
    grid_dependency_wait();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < words;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        // the word's place: [e][tile][kb][j][line][row / 32]
        const int in = static_cast<int>(i & 3) * 32 + static_cast<int>((i >> 2) & 31);
        int64_t rest = i >> 7;
        const int j = static_cast<int>(rest % W);
        rest /= W;
        const int kb = static_cast<int>(rest % KB);
        rest /= KB;
        const int tile = static_cast<int>(rest % tiles);
        const int64_t e = rest / tiles;
        int n = tile * 128 + in;
        bool real = n < N;
        if (gate_up) {   // 32 rows: 16 of gate, 16 of up
            const int col = (n >> 5) * 16 + (n & 15);
            real = col < N / 2;
            n = col + ((n & 16) ? N / 2 : 0);
        }
        uint32_t word = 0;
        const int c0 = (kb * W + j) * 4;
        if (real)
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (c0 + b < C) word |= static_cast<uint32_t>(s[(e * N + n) * C + c0 + b]) << (8 * b);
        out[i] = word;
    }
}

// Threads of a row: as few warps as hold it in kVecs vectors each, and rows to a block of 256 threads or more.
struct RowPlan {
    int tpr, threads;
    unsigned blocks;
};
RowPlan row_plan(int64_t rows, int K) {
    const int vecs = fp4_blocks(K) * 32;
    int tpr = 32;
    while (tpr * kVecs < vecs) tpr <<= 1;
    const int threads = tpr > 256 ? tpr : 256, per = threads / tpr;
    return {tpr, threads, static_cast<unsigned>((rows + per - 1) / per)};
}

template <class T, int FMT>
cudaError_t quant_type(const QuantArgs& a, bool on16, cudaStream_t stream) {
    const RowPlan p = row_plan(a.rows, a.K);
    return on16 ? launch_pdl(fp4_quant_kernel<T, FMT, true>, dim3(p.blocks), dim3(p.threads), 0, stream, a, p.tpr)
                : launch_pdl(fp4_quant_kernel<T, FMT, false>, dim3(p.blocks), dim3(p.threads), 0, stream, a, p.tpr);
}
template <int FMT>
cudaError_t quant_format(int dtype, const QuantArgs& a, bool on16, cudaStream_t stream) {
    return dtype == MOE_DTYPE_BF16   ? quant_type<__nv_bfloat16, FMT>(a, on16, stream)
           : dtype == MOE_DTYPE_FP16 ? quant_type<__half, FMT>(a, on16, stream)
                                     : quant_type<float, FMT>(a, on16, stream);
}
template <int FMT>
cudaError_t dequant_format(int dtype, const DequantArgs& a, cudaStream_t stream) {
    const RowPlan p = row_plan(a.rows, a.K);
    const dim3 grid(p.blocks), block(p.threads);
    return dtype == MOE_DTYPE_BF16   ? launch_pdl(fp4_dequant_kernel<__nv_bfloat16, FMT>, grid, block, 0, stream, a, p.tpr)
           : dtype == MOE_DTYPE_FP16 ? launch_pdl(fp4_dequant_kernel<__half, FMT>, grid, block, 0, stream, a, p.tpr)
                                     : launch_pdl(fp4_dequant_kernel<float, FMT>, grid, block, 0, stream, a, p.tpr);
}

bool known_format(int fmt) { return fmt == MOE_FP4_MXFP4 || fmt == MOE_FP4_NVFP4; }
int check_rows(int fmt, int dtype, const int32_t* offsets, int E, int64_t rows, int K) {
    if (!known_format(fmt) || !known_dtype(dtype) || rows < 0 || K < 1 || E < 0 || (offsets != nullptr) != (E > 0))
        return MOE_ERR_INVALID_ARG;
    if (K % 32 != 0 || K > kFp4MaxCols || E > MOE_MAX_EXPERTS || rows >= (int64_t(1) << 31) - kFp4Rows)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// The tensor maps of a product (order: fp4_experts_launch); codes and scales as bytes.
cudaError_t fp4_maps(CUtensorMap (&tm)[5], const uint8_t* codes, const uint8_t* scales, size_t scale_bytes, int fmt,
                     const uint8_t* w_codes, const uint8_t* w_scales, size_t w_scale_bytes, int64_t rows, int E, int N,
                     int K, bool silu) {
    const uint64_t row = static_cast<uint64_t>(K) / 2, n = N;
    cudaError_t e;
    if (silu) {   // [E][I / 16][gate, up][16][K / 2]: a box brings 128 rows, 16 gate and 16 up columns in turn
        const uint64_t dims[5] = {row, 16, 2, n / 32, static_cast<uint64_t>(E)};
        const uint64_t strides[4] = {row, n / 2 * row, 16 * row, n * row};
        const uint32_t box[5] = {128, 16, 2, 4, 1};
        e = encode_u8_map_nd(&tm[0], w_codes, 5, dims, strides, box, true);
    } else {
        const uint64_t dims[3] = {row, n, static_cast<uint64_t>(E)};
        const uint64_t strides[2] = {row, n * row};
        const uint32_t box[3] = {128, 128, 1};
        e = encode_u8_map_nd(&tm[0], w_codes, 3, dims, strides, box, true);
    }
    const uint64_t dims[2] = {row, static_cast<uint64_t>(rows)}, strides[1] = {row};
    const uint32_t boxes[2][2] = {{128, kFp4Rows / 2}, {128, 16}};
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) e = encode_u8_map_nd(&tm[1 + i], codes, 2, dims, strides, boxes[i], true);
    // scales as rows of 512-byte tiles
    const uint64_t s_strides[2] = {256, 512};
    const uint32_t s_box[3] = {256, 2, static_cast<uint32_t>(fp4_words(fmt))};
    const uint64_t a_dims[3] = {256, 2, w_scale_bytes / 512}, b_dims[3] = {256, 2, scale_bytes / 512};
    if (e == cudaSuccess) e = encode_u8_map_nd(&tm[3], w_scales, 3, a_dims, s_strides, s_box, false);
    if (e == cudaSuccess) e = encode_u8_map_nd(&tm[4], scales, 3, b_dims, s_strides, s_box, false);
    return e;
}

}  // namespace

cudaError_t fp4_init_device() {
    const cudaError_t e = fp4_experts_init<MOE_FP4_MXFP4>();
    return e == cudaSuccess ? fp4_experts_init<MOE_FP4_NVFP4>() : e;
}

}  // namespace mfp8

using namespace mfp8;

extern "C" {

size_t moe_fp4_row_scale_bytes(int fmt, int64_t num_rows, int E, int K) {
    if (!known_format(fmt) || num_rows < 0 || num_rows >= (int64_t(1) << 31) - kFp4Rows || E < 0 || E > MOE_MAX_EXPERTS ||
        K < 1 || K % 32 != 0 || K > kFp4MaxCols)
        return 0;
    return static_cast<size_t>(num_rows / kFp4Rows + E + 1) * fp4_blocks(K) * 2 * fp4_words(fmt) * 512;
}

size_t moe_fp4_weight_scale_bytes(int fmt, int E, int N, int K) {
    if (!known_format(fmt) || E < 1 || N < 1 || K < 1 || K % 32 != 0) return 0;
    return static_cast<size_t>(E) * ((static_cast<size_t>(N) + 127) / 128) * fp4_blocks(K) * fp4_words(fmt) * 512;
}

int moe_fp4_quant(const void* x, int64_t ldx, int dtype, int fmt, const int32_t* expert_offsets, int E, int64_t num_rows,
                  int K, uint8_t* codes, uint8_t* scales, float* row_scale, void* stream) {
    int rc = check_rows(fmt, dtype, expert_offsets, E, num_rows, K);
    if (rc != MOE_OK) return rc;
    if (ldx < K || (row_scale != nullptr) != (fmt == MOE_FP4_NVFP4 && num_rows > 0)) return MOE_ERR_INVALID_ARG;
    if (num_rows == 0) return MOE_OK;
    if (!x || !codes || !scales || address(codes) % 16 || address(scales) % 16 || address(row_scale) % 4 ||
        !on_element(address(x), dtype_bytes(dtype)))
        return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    const QuantArgs a = {x, ldx, num_rows, K, E, expert_offsets, codes, scales, nullptr, row_scale};
    const bool on16 = address(x) % 16 == 0 && (num_rows == 1 || ldx * dtype_bytes(dtype) % 16 == 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(fmt == MOE_FP4_MXFP4 ? quant_format<MOE_FP4_MXFP4>(dtype, a, on16, s)
                                            : quant_format<MOE_FP4_NVFP4>(dtype, a, on16, s));
}

int moe_fp4_dequant(const uint8_t* codes, const uint8_t* scales, const float* row_scale, int fmt,
                    const int32_t* expert_offsets, int E, int64_t num_rows, int K, int dtype, void* out, void* stream) {
    int rc = check_rows(fmt, dtype, expert_offsets, E, num_rows, K);
    if (rc != MOE_OK) return rc;
    if ((row_scale != nullptr) != (fmt == MOE_FP4_NVFP4 && num_rows > 0)) return MOE_ERR_INVALID_ARG;
    if (num_rows == 0) return MOE_OK;
    if (!codes || !scales || !out || address(codes) % 16 || address(scales) % 16 || address(row_scale) % 4 ||
        address(out) % 16)
        return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    const DequantArgs a = {codes, scales, row_scale, expert_offsets, num_rows, K, E, out};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(fmt == MOE_FP4_MXFP4 ? dequant_format<MOE_FP4_MXFP4>(dtype, a, s)
                                            : dequant_format<MOE_FP4_NVFP4>(dtype, a, s));
}

int moe_mxfp4_quant_weight(const void* w, int dtype, int E, int N, int K, uint8_t* codes, uint8_t* scales, void* stream) {
    if (E < 0 || N < 0 || static_cast<int64_t>(E) * N >= (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(E) * N;
    int rc = check_rows(MOE_FP4_MXFP4, dtype, nullptr, 0, rows, K);
    if (rc != MOE_OK || rows == 0) return rc;
    if (!w || !codes || !scales || address(w) % 16 || address(codes) % 16) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    const QuantArgs a = {w, K, rows, K, 0, nullptr, codes, nullptr, scales, nullptr};
    return cuda_status(quant_format<MOE_FP4_MXFP4>(dtype, a, true, static_cast<cudaStream_t>(stream)));
}

int moe_fp4_pack_scales(const uint8_t* s, int fmt, int E, int N, int K, int gate_up, uint8_t* out, void* stream) {
    if (!known_format(fmt) || E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
    if (K % 32 != 0 || (gate_up && N % 32 != 0)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!s || !out || address(out) % 16) return MOE_ERR_INVALID_ARG;
    int rc;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    const int64_t words = static_cast<int64_t>(moe_fp4_weight_scale_bytes(fmt, E, N, K) / 4);
    const int64_t blocks = (words + 255) / 256, most = static_cast<int64_t>(kPlanSms) * 16;
    return cuda_status(launch_pdl(fp4_pack_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0,
                                  static_cast<cudaStream_t>(stream), s, words, N, K / fp4_group(fmt), fp4_blocks(K),
                                  fp4_words(fmt), (N + 127) / 128, gate_up, reinterpret_cast<uint32_t*>(out)));
}

int moe_fp4_expert_gemm(const uint8_t* codes, const uint8_t* scales, const float* row_scale, int fmt, const uint8_t* w_codes,
                        const uint8_t* w_scales, const float* w_global, const int32_t* expert_offsets, int64_t num_rows,
                        int E, int N, int K, int epilogue, int dtype, void* out, void* stream) {
    const bool silu = epilogue == MOE_EXPERT_SILU_MUL;
    if (!silu && epilogue != MOE_EXPERT_STORE) return MOE_ERR_INVALID_ARG;
    int rc = check_rows(fmt, dtype, expert_offsets, expert_offsets ? E : 0, num_rows, K);
    if (rc != MOE_OK) return rc;
    if (E < 1 || N < 1 || (!expert_offsets && E != 1) || (silu && dtype == MOE_DTYPE_FP32)) return MOE_ERR_INVALID_ARG;
    if (N % (silu ? 32 : 8) != 0 || N >= (1 << 24)) return MOE_ERR_UNSUPPORTED_SHAPE;
    const bool nv = fmt == MOE_FP4_NVFP4;
    if (!w_codes || !w_scales || (w_global != nullptr) != nv || (row_scale != nullptr) != (nv && num_rows > 0))
        return MOE_ERR_INVALID_ARG;
    if (address(w_codes) % 16 || address(w_scales) % 16 || address(w_global) % 4 || address(row_scale) % 4)
        return MOE_ERR_INVALID_ARG;
    if (num_rows == 0) return MOE_OK;
    if (!codes || !scales || !out || address(codes) % 16 || address(scales) % 16 || address(out) % 16)
        return MOE_ERR_INVALID_ARG;
    const size_t scale_bytes = moe_fp4_row_scale_bytes(fmt, num_rows, expert_offsets ? E : 0, K);
    const size_t w_scale_bytes = moe_fp4_weight_scale_bytes(fmt, E, N, K);
    if (scale_bytes / 512 >= (size_t(1) << 31) || w_scale_bytes / 512 >= (size_t(1) << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    CUtensorMap tm[5];
    if (fp4_maps(tm, codes, scales, scale_bytes, fmt, w_codes, w_scales, w_scale_bytes, num_rows, E, N, K, silu) != cudaSuccess)
        return MOE_ERR_CUDA;
    const Fp4Args a = {expert_offsets, E, num_rows, N, K, row_scale, w_global, out, status};
    const int64_t row_tiles = num_rows / kFp4Rows + (num_rows < E ? num_rows : E) + 1;
    const int64_t items = row_tiles * (silu ? (N / 2 + 127) / 128 : (N + 255) / 256);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(nv ? fp4_experts_launch<MOE_FP4_NVFP4>(dtype, silu, a, tm, items, s)
                          : fp4_experts_launch<MOE_FP4_MXFP4>(dtype, silu, a, tm, items, s));
}

}  // extern "C"
