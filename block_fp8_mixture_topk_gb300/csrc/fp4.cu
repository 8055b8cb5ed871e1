// Microscaled 4-bit quantisation of rows and weights, and the values back (formats and layouts: fp4.cuh).
//
// A group's scale and codes are the real numbers' nearest (ties to even), whatever the order of operations:
//   mxfp4  scale = the smallest power of two s with max|x| <= 6 s, code = e2m1(x / s): x / s is exact
//   nvfp4  r = fp32(max|x of the row| / 2688), b = e4m3(max|x of the group| / (6 r)), code = e2m1(x / (b r)): the
//          quotients are taken in fp32 a little too large and a little too small; where the two round differently,
//          a comparison with the border itself, its product exact in two fp32 parts, decides; 16-bit rows, whose quotients
//          are often nearly a border, need neither (border_side)
// An infinity or NaN makes its group (mxfp4: scale NaN) or row (nvfp4: row scale NaN) NaN.
//
// Memory is the bound: a thread loads its vectors of 16 elements whole (32 bytes at a time) before it uses the first,
// so a group is one lane's or two lanes'; they stay in registers for the row's maximum (32 to 1024 threads to a row).
// The codes go out as eight bytes a vector, the scales as words of four groups put together across lanes.
//
// Measured (GB300; rows read, codes and scales written): mxfp4 131072 x 2048 bf16 98 us, 6.9 TB/s; 4096 x 32768 53 us, 6.4 TB/s;
// 5003 x 2880 fp32 8.7 us.  nvfp4 116 us, 5.9 TB/s; 65 us, 5.3 TB/s; 10.2 us: its row's maximum is a barrier, and its quotients make
// 200 instructions of 16 elements, 2.7 of 4 issue slots.  So a row takes small blocks (64 threads in place of 256: 121 ->
// 116 us), and a long row four vectors a thread in place of two (32768 columns: 84 -> 65 us, mxfp4 68 -> 53; 7168: 31 and 32).
// Values back: 131072 x 2048 100 us, 6.8 TB/s.
#include "fp4.cuh"

namespace mfp8 {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

// Whether a >= 0 is rounded up from code c past the border m r to the next: m has few bits, the product's two parts are
// exact (r not below kLeastRow), ties go to the even code.
__device__ __forceinline__ bool past_border(float a, float m, float r, uint32_t c) {
    const float p = m * r, rest = fmaf(m, r, -p);
    return a > p || (a == p && (rest < 0.0f || (rest == 0.0f && (c & 1u))));
}
// Border between e2m1 codes c and c + 1.
__device__ __forceinline__ float e2m1_border(uint32_t c) {
    return 0.25f * static_cast<float>(static_cast<uint32_t>(0x00140e0a07050301ull >> (8 * c)) & 0xffu);
}

// Row scales below kLeastRow, in fp64: e2m1(x / d), e4m3(x / (6 r)) by the borders between codes.
__device__ __noinline__ uint32_t e2m1_tiny(float x, double d) {
    const double a = fabs(static_cast<double>(x));
    uint32_t c = 0;
    for (uint32_t i = 0; i < 7; ++i) {
        const double t = e2m1_border(i) * d;
        c += a > t || (a == t && (i & 1)) ? 1u : 0u;
    }
    return c | (__float_as_uint(x) >> 31 << 3);
}
__device__ __noinline__ uint32_t e4m3_tiny(float x, float r) {
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
    int align;                 // bytes of which every row's address is a multiple: 32, 16 or less
    int warps;                 // of a row
};

constexpr float kSlack = 0x1p-21f;       // over the error of a quotient or product of a few fp32 operations
constexpr float kLeastRow = 0x1p-100f;

// Rows of 16 bits need no borders.  With the largest magnitude m, r is m / 2688 rounded, and a quotient by the exact m / 2688 is
// g * 448 / m or x * 2688 / (b m).  Against a border h that is 21 x (16 bits of an fp16 row) against h b m (3, 4 and 11 bits; scales: 7 g
// against 5 and 11 bits), whole numbers up to a power of two: equal, or apart by 1 or more in at most 65 * 2047 of the smaller
// unit (x = 1584, m = 2047, b = 13, h = 5), 2^-17.02 of the quotient (of a bf16 row 2^-13.9).  The rounding of r (2^-24) only decides on
// which side of a border that it would meet a quotient lies: below where r is too large.  A factor of 1 -+ 2^-20 takes it there in
// spite of the arithmetic's 2^-21.  0 where r is exact: those rows meet borders, and are decided as 32-bit ones.
template <class T>
__device__ __forceinline__ float border_side(float m, float rs) {
    if (sizeof(T) == 4) return 0.0f;
    const float over = fmaf(rs, 2688.0f, -m);
    return over > 0.0f ? 1.0f - 0x1p-20f : over < 0.0f ? 1.0f + 0x1p-20f : 0.0f;
}

// A group's scale byte and its part's codes, nvfp4 (rs > 0; side: border_side; by: 1 / (6 rs)).
template <class T>
__device__ __forceinline__ uint32_t nvfp4_group(const Vec16<T>& x, uint32_t top, float rs, float side, float by, uint2* codes) {
    const float g = __uint_as_float(top);
    *codes = make_uint2(0, 0);
    if (sizeof(T) == 2 && side != 0.0f && rs >= kLeastRow) {
        const uint32_t s = e4m3x2(g * (by * side), 0.0f) & 0xffu;
        if (s > 0) *codes = e2m1_words(x, __fdividef(1.0f, e4m3_number(s) * rs) * side);
        return s;
    }
    if (rs < kLeastRow) {
        const uint32_t s = e4m3_tiny(g, rs);
        if (s > 0) {
            const double d = static_cast<double>(e4m3_number(s)) * static_cast<double>(rs);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                codes->x |= e2m1_tiny(x.get(i), d) << (4 * i);
                codes->y |= e2m1_tiny(x.get(8 + i), d) << (4 * i);
            }
        }
        return s;
    }
    const float t = g * by;
    const uint32_t two = e4m3x2(t * (1.0f - kSlack), t * (1.0f + kSlack));
    uint32_t s = two & 0xffu;
    if (s != two >> 8) s += past_border(g, 3.0f * (e4m3_number(s) + e4m3_number(s + 1)), rs, s) ? 1u : 0u;
    if (s == 0) return 0;
    const float b = e4m3_number(s), f = __fdividef(1.0f, b * rs);
    uint2 lo = e2m1_words(x, f * (1.0f - kSlack));
    const uint2 hi = e2m1_words(x, f * (1.0f + kSlack));
    if (lo.x != hi.x || lo.y != hi.y) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            uint32_t& w = i < 8 ? lo.x : lo.y;
            const uint32_t c = w >> (4 * (i & 7)) & 7u;
            if (((w ^ (i < 8 ? hi.x : hi.y)) >> (4 * (i & 7)) & 0xfu) && past_border(fabsf(x.get(i)), e2m1_border(c) * b, rs, c))
                w += 1u << (4 * (i & 7));
        }
    }
    *codes = lo;
    return s;
}

// Blocks to an SM: with two vectors of 16-bit elements a thread 1536 threads (40 registers), 98 KB of rows under way, else 1024.
template <class T, int VECS>
constexpr int quant_blocks(int threads) {
    return (sizeof(T) == 2 && VECS == 2 ? 1536 : 1024) / threads;
}

template <class T, int FMT, int THREADS, int VECS>
__global__ void __launch_bounds__(THREADS, quant_blocks<T, VECS>(THREADS)) fp4_quant_kernel(const QuantArgs a) {
    grid_dependency_wait();
    constexpr int G = fp4_group(FMT), LANES = G / 16, W = fp4_words(FMT);   // lanes of a group
    __shared__ uint32_t s_top[32];
    const int at = threadIdx.x, own = threadIdx.y, tpr = blockDim.x;   // the thread of a row, the block's row
    const int lane = at & 31;
    const uint32_t row_of = blockIdx.x * blockDim.y + own;
    const bool live = row_of < static_cast<uint32_t>(a.rows);
    const int r = static_cast<int>(row_of), KB = fp4_blocks(a.K), vecs = a.K / 16;
    const T* row = static_cast<const T*>(a.x) + r * a.ld;
    Vec16<T> x[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int v = at + i * tpr;
        if (live && v < vecs) x[i].load(row + v * 16, a.align);
        else x[i].zero();
    }
    Fp4Place place = {0, 0};
    if (a.tiles && live) place = fp4_place(a.offsets, a.E, r);
    uint32_t top[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        top[i] = x[i].top();
        if (LANES == 2) top[i] = max(top[i], __shfl_xor_sync(kAll, top[i], 1));
    }
    uint32_t most = top[0];
#pragma unroll
    for (int i = 1; i < VECS; ++i) most = max(most, top[i]);
    float rs = 1.0f, side = 0.0f, by = 0.0f;
    if constexpr (FMT == MOE_FP4_NVFP4) {
        uint32_t m = __reduce_max_sync(kAll, most);
        if (a.warps > 1) {
            if (lane == 0) s_top[own * a.warps + (at >> 5)] = m;
            __syncthreads();
            m = __reduce_max_sync(kAll, lane < a.warps ? s_top[own * a.warps + lane] : 0u);
        }
        rs = m < 0x7f800000u ? __fdiv_rn(__uint_as_float(m), 2688.0f) : __int_as_float(0x7fffffff);
        side = border_side<T>(__uint_as_float(m), rs);
        by = __fdividef(1.0f, 6.0f * rs);
        if (live && at == 0) a.row_scale[r] = rs;
    }
    if (!live) return;   // (whole warps)
    uint8_t* tile = fp4_scale_row(a.tiles, place.tile, place.in, KB, W);
    uint2* codes = reinterpret_cast<uint2*>(a.codes + static_cast<int64_t>(r) * (a.K / 2));
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int v = at + i * tpr;
        if ((v & ~31) >= KB * 16) break;   // (whole warps)
        uint32_t s = 0;
        uint2 w = make_uint2(0, 0);
        if constexpr (FMT == MOE_FP4_MXFP4) {
            s = mxfp4_group(x[i], top[i], &w);
        } else if (rs > 0.0f) {   // not zero and not NaN
            s = nvfp4_group(x[i], top[i], rs, side, by, &w);
        }
        if (v < vecs) codes[v] = w;
        else s = 0;   // columns past K: a scale that is a number
        const int c = v / LANES;   // the group
        if (a.tiles) {
            uint32_t word = s << (8 * (c & 3));
#pragma unroll
            for (int o = LANES; o < 4 * LANES; o <<= 1) word |= __shfl_xor_sync(kAll, word, o);
            const int kb = v >> 4;
            if (lane % (4 * LANES) == 0 && kb < KB)
                *reinterpret_cast<uint32_t*>(tile + static_cast<int64_t>(kb) * (2 * W * 512) + (c >> 2) % W * 512) = word;
        } else if (lane % LANES == 0 && v < vecs) {
            a.plain[static_cast<int64_t>(r) * (a.K / G) + c] = static_cast<uint8_t>(s);
        }
    }
}

constexpr int kVecs = 4;   // vectors of 8 elements a thread, of the values' kernel

struct DequantArgs {
    const uint8_t* codes;
    const uint8_t* tiles;
    const float* row_scale;
    const int32_t* offsets;
    int64_t rows;
    int K, E;
    void* out;
    bool align32;              // out is at a 32-byte address
};

// Values of the codes: code times group scale is exact in fp32, the row's scale and the result's type round.
template <class T, int FMT>
__global__ void __launch_bounds__(1024) fp4_dequant_kernel(const DequantArgs a) {
    grid_dependency_wait();
    constexpr int LANES = fp4_group(FMT) / 8, W = fp4_words(FMT);
    const int at = threadIdx.x, tpr = blockDim.x;
    const uint32_t row_of = blockIdx.x * blockDim.y + threadIdx.y;
    if (row_of >= static_cast<uint32_t>(a.rows)) return;   // (whole warps)
    const int64_t r = row_of;
    const int KB = fp4_blocks(a.K), vecs = a.K / 8;
    const Fp4Place place = fp4_place(a.offsets, a.E, static_cast<int>(r));
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
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(out + v * 8) = *reinterpret_cast<const uint4*>(e);
        } else {   // 32 bytes at once (rows at 16-byte addresses: K is a multiple of 32, out of 16 bytes)
            const uint32_t* u = reinterpret_cast<const uint32_t*>(e);
            if (a.align32)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + v * 8), "r"(u[0]), "r"(u[1]),
                             "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                             : "memory");
            else
#pragma unroll
                for (int j = 0; j < 2; ++j) reinterpret_cast<uint4*>(out + v * 8)[j] = reinterpret_cast<const uint4*>(e)[j];
        }
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

template <class T, int FMT>
cudaError_t quant_type(QuantArgs a, cudaStream_t stream) {
    const uintptr_t bits = address(a.x) | (a.rows > 1 ? static_cast<uintptr_t>(a.ld) * sizeof(T) : 0);
    a.align = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 1;
    const int all = fp4_blocks(a.K) * 16;                                       // vectors of a row
    const auto launch = [&](auto kernel, int vecs) {
        a.warps = (all + 32 * vecs - 1) / (32 * vecs);
        const int most = FMT == MOE_FP4_NVFP4 ? 2 : 8, per = a.warps < most ? most / a.warps : 1;   // rows of a block
        return launch_pdl(kernel, dim3(static_cast<unsigned>((a.rows + per - 1) / per)), dim3(32 * a.warps, per), 0, stream, a);
    };
    if (all <= 8 * 64) return launch(fp4_quant_kernel<T, FMT, 256, 2>, 2);
    if constexpr (sizeof(T) == 2) return launch(fp4_quant_kernel<T, FMT, 512, 4>, 4);
    else return all <= 16 * 64 ? launch(fp4_quant_kernel<T, FMT, 512, 2>, 2) : launch(fp4_quant_kernel<T, FMT, 1024, 2>, 2);
}
template <int FMT>
cudaError_t quant_format(int dtype, const QuantArgs& a, cudaStream_t stream) {
    return dtype == MOE_DTYPE_BF16   ? quant_type<__nv_bfloat16, FMT>(a, stream)
           : dtype == MOE_DTYPE_FP16 ? quant_type<__half, FMT>(a, stream)
                                     : quant_type<float, FMT>(a, stream);
}
template <int FMT>
cudaError_t dequant_format(int dtype, const DequantArgs& a, cudaStream_t stream) {
    // as few warps as hold a row, kVecs vectors a thread; blocks of up to 256 threads or one row
    const int warps = (a.K / 8 + 32 * kVecs - 1) / (32 * kVecs), per = warps < 8 ? 8 / warps : 1;
    const dim3 grid(static_cast<unsigned>((a.rows + per - 1) / per)), block(32 * warps, per);
    return dtype == MOE_DTYPE_BF16   ? launch_pdl(fp4_dequant_kernel<__nv_bfloat16, FMT>, grid, block, 0, stream, a)
           : dtype == MOE_DTYPE_FP16 ? launch_pdl(fp4_dequant_kernel<__half, FMT>, grid, block, 0, stream, a)
                                     : launch_pdl(fp4_dequant_kernel<float, FMT>, grid, block, 0, stream, a);
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
    const uint32_t a_box[3] = {256, 2, static_cast<uint32_t>(fp4_words(fmt))};
    const uint32_t b_box[3] = {256, 2, 2 * static_cast<uint32_t>(fp4_words(fmt))};
    const uint64_t a_dims[3] = {256, 2, w_scale_bytes / 512}, b_dims[3] = {256, 2, scale_bytes / 512};
    if (e == cudaSuccess) e = encode_u8_map_nd(&tm[3], w_scales, 3, a_dims, s_strides, a_box, false);
    if (e == cudaSuccess) e = encode_u8_map_nd(&tm[4], scales, 3, b_dims, s_strides, b_box, false);
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
    if (!known_format(fmt) || E < 1 || E > MOE_MAX_EXPERTS || N < 1 || N % 8 != 0 || N >= kFp4MaxOut || K < 1 || K % 32 != 0 ||
        K > kFp4MaxCols)
        return 0;
    const size_t tiles = static_cast<size_t>(E) * ((static_cast<size_t>(N) + 127) / 128) * fp4_blocks(K) * fp4_words(fmt);
    return tiles < (size_t(1) << 31) ? tiles * 512 : 0;
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
    const QuantArgs a = {x, ldx, num_rows, K, E, expert_offsets, codes, scales, nullptr, row_scale, 0, 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(fmt == MOE_FP4_MXFP4 ? quant_format<MOE_FP4_MXFP4>(dtype, a, s)
                                            : quant_format<MOE_FP4_NVFP4>(dtype, a, s));
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
    const DequantArgs a = {codes, scales, row_scale, expert_offsets, num_rows, K, E, out, address(out) % 32 == 0};
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
    const QuantArgs a = {w, K, rows, K, 0, nullptr, codes, nullptr, scales, nullptr, 0, 0};
    return cuda_status(quant_format<MOE_FP4_MXFP4>(dtype, a, static_cast<cudaStream_t>(stream)));
}

int moe_fp4_pack_scales(const uint8_t* s, int fmt, int E, int N, int K, int gate_up, uint8_t* out, void* stream) {
    if (!known_format(fmt) || E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
    if (moe_fp4_weight_scale_bytes(fmt, E, N, K) == 0 || (gate_up && N % 32 != 0)) return MOE_ERR_UNSUPPORTED_SHAPE;
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
                        int E, int N, int K, int epilogue, int dtype, void* out, uint8_t* out_scales, void* stream) {
    const bool quant = epilogue == MOE_EXPERT_SILU_MUL_QUANT, silu = epilogue == MOE_EXPERT_SILU_MUL || quant;
    if (!silu && epilogue != MOE_EXPERT_STORE) return MOE_ERR_INVALID_ARG;
    if (quant && (fmt != MOE_FP4_MXFP4 || dtype != MOE_DTYPE_BF16)) return MOE_ERR_INVALID_ARG;
    int rc = check_rows(fmt, dtype, expert_offsets, expert_offsets ? E : 0, num_rows, K);
    if (rc != MOE_OK) return rc;
    if (E < 1 || N < 1 || (!expert_offsets && E != 1) || (silu && dtype == MOE_DTYPE_FP32)) return MOE_ERR_INVALID_ARG;
    if (N % (quant ? 64 : silu ? 32 : 8) != 0 || N >= kFp4MaxOut) return MOE_ERR_UNSUPPORTED_SHAPE;
    const bool nv = fmt == MOE_FP4_NVFP4;
    if (!w_codes || !w_scales || (w_global != nullptr) != nv || (row_scale != nullptr) != (nv && num_rows > 0))
        return MOE_ERR_INVALID_ARG;
    if (address(w_codes) % 16 || address(w_scales) % 16 || address(w_global) % 4 || address(row_scale) % 4)
        return MOE_ERR_INVALID_ARG;
    if (num_rows == 0) return MOE_OK;
    if (!codes || !scales || !out || address(codes) % 16 || address(scales) % 16 || address(out) % 16 ||
        (out_scales != nullptr) != quant || address(out_scales) % 16)
        return MOE_ERR_INVALID_ARG;
    const size_t scale_bytes = moe_fp4_row_scale_bytes(fmt, num_rows, expert_offsets ? E : 0, K);
    const size_t w_scale_bytes = moe_fp4_weight_scale_bytes(fmt, E, N, K);
    if (scale_bytes / 512 >= (size_t(1) << 31) || w_scale_bytes == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t row_tiles = num_rows / kFp4Rows + (num_rows < E ? num_rows : E) + 1;
    const int64_t items = row_tiles * (silu ? (N / 2 + 127) / 128 : (N + 255) / 256);
    if (items >= int64_t(1) << 31) return MOE_ERR_UNSUPPORTED_SHAPE;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    CUtensorMap tm[5];
    if (fp4_maps(tm, codes, scales, scale_bytes, fmt, w_codes, w_scales, w_scale_bytes, num_rows, E, N, K, silu) != cudaSuccess)
        return MOE_ERR_CUDA;
    const Fp4Args a = {expert_offsets, E, num_rows, N, K, row_scale, w_global, out, out_scales, status};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(nv ? fp4_experts_launch<MOE_FP4_NVFP4>(dtype, epilogue, a, tm, items, s)
                          : fp4_experts_launch<MOE_FP4_MXFP4>(dtype, epilogue, a, tm, items, s));
}

}  // extern "C"
