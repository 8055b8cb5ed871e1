// Microscaled 4-bit rows and weights: formats, the tiles of scales that the products read, and the rows' places.
//
//   MOE_FP4_MXFP4  e2m1 codes, 32 along K to a UE8M0 scale (a power of two)
//   MOE_FP4_NVFP4  e2m1 codes, 16 along K to an e4m3 scale, and an fp32 scale per row (rows) or expert (weights)
//
// The products take K in blocks of 256 (128 bytes of codes, a swizzled row).  The scales of 128 rows over a block
// are W = 2 (mxfp4) or 4 (nvfp4) tiles of 512 bytes, each as tensor memory holds it: 32 lines of 16 bytes, line l the
// words of rows l, l + 32, l + 64, l + 96, a word the scales of four consecutive groups.
//   weights [E][tiles of 128][K blocks][W][512]: of w's rows; with gate_up (rows gate, then up), 16 gate rows and
//           the 16 up rows of the same columns in turn, as the SiLU product's tile has them
//   rows    [tiles of 224][K blocks][2][W][512]: a product takes up to 224 rows of one expert at a time, so the
//           tiles start with the expert: row r of expert e, whose rows begin at o_e, is row (r - o_e) % 224 of tile
//           o_e / 224 + e + (r - o_e) / 224.  (Tiles of different experts never meet: floor(o/224 + n/224) + 1 is more
//           than floor(o/224) + n/224.)  Rows of no expert follow as an expert E.
#pragma once

#include <type_traits>

#include "train.cuh"

namespace mfp8 {

constexpr int kFp4Rows = 224;      // rows of an item of the products, and of a tile of their scales
constexpr int kFp4Block = 256;     // columns of a K block
constexpr int kFp4MaxCols = 32768;
constexpr int kFp4MaxOut = 1 << 24;   // output columns of a product are fewer

__host__ __device__ constexpr int fp4_group(int fmt) { return fmt == MOE_FP4_MXFP4 ? 32 : 16; }
__host__ __device__ constexpr int fp4_words(int fmt) { return fmt == MOE_FP4_MXFP4 ? 2 : 4; }
__host__ __device__ __forceinline__ int fp4_blocks(int K) { return (K + kFp4Block - 1) / kFp4Block; }

// Byte of the first scale of word j of row `in` (0 .. 127) in 128 rows' tiles of one K block.
__host__ __device__ __forceinline__ int fp4_word(int in, int j) { return j * 512 + (in & 31) * 16 + (in >> 5) * 4; }

// Tile of an expert's first rows, which begin at row o; the scales' bytes of row `in` of a tile (word 0 of K block 0).
__host__ __device__ __forceinline__ int64_t fp4_tile(int64_t o, int e) { return o / kFp4Rows + e; }
__device__ __forceinline__ uint8_t* fp4_scale_row(uint8_t* tiles, int64_t tile, int in, int blocks, int words) {
    return tiles + (tile * blocks * 2 + (in >> 7)) * (words * 512) + fp4_word(in & 127, 0);
}

// The tile and the place in it of row r, found by a whole warp: e is the last expert whose rows begin at or before
// r, o where they begin.  Offsets out of order or range count as the running maximum of the clamped ones, from 0,
// as the products take them.
struct Fp4Place {
    int64_t tile;
    int in;
};
__device__ __forceinline__ Fp4Place fp4_place(const int32_t* offsets, int E, int r) {
    int e = 0, o = 0;
    if (offsets) {
        const int lane = threadIdx.x & 31;
        int most = 0;   // of the lane's offsets up to r
        e = E;
        for (int i0 = 1; i0 <= E; i0 += 32) {
            const int i = i0 + lane;
            const int32_t v = i <= E ? __ldg(offsets + i) : 0;
            const uint32_t past = __ballot_sync(0xffffffffu, v > r);
            if (past) {
                const int first = __ffs(static_cast<int>(past)) - 1;
                if (lane < first) most = max(most, v);
                e = i0 + first - 1;
                break;
            }
            most = max(most, v);
        }
        o = __reduce_max_sync(0xffffffffu, most);
    }
    const uint32_t past = static_cast<uint32_t>(r - o), m = past / kFp4Rows;
    return {static_cast<int64_t>(static_cast<uint32_t>(o) / kFp4Rows + e + m), static_cast<int>(past - m * kFp4Rows)};
}

// e4m3 number of a byte without its sign.
__device__ __forceinline__ float e4m3_number(uint32_t code) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(code));
    return __low2float(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ float ue8m0_number(uint32_t byte) {   // 255 is NaN
    return byte == 255 ? __int_as_float(0x7fffffff) : byte ? __uint_as_float(byte << 23) : __uint_as_float(1u << 22);
}

// The larger magnitudes of two pairs of elements, NaN above all.
template <class T>
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                             __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    const __half2 m = __hmax2_nan(__habs2(*reinterpret_cast<const __half2*>(&a)), __habs2(*reinterpret_cast<const __half2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// 16 elements.
template <class T>
struct Vec16 {
    static constexpr int kWords = 4 * static_cast<int>(sizeof(T));
    uint32_t w[kWords];
    // from a row at 32-byte addresses, 16-byte ones or any
    __device__ __forceinline__ void load(const T* p, int align) {
        if (align == 32) {
#pragma unroll
            for (int i = 0; i < kWords; i += 8)
                asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                               "=r"(w[i + 6]), "=r"(w[i + 7])
                             : "l"(reinterpret_cast<const uint32_t*>(p) + i));
        } else if (align == 16) {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
                w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
            }
        } else if constexpr (sizeof(T) == 2) {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = e[2 * i] | static_cast<uint32_t>(e[2 * i + 1]) << 16;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    // elements 2 i and 2 i + 1
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else return __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    }
    __device__ __forceinline__ float get(int i) const { return (i & 1) ? pair(i / 2).y : pair(i / 2).x; }
    // fp32 bits of the largest magnitude: they order as the magnitudes do, infinity and NaN above
    __device__ __forceinline__ uint32_t top() const {
        if constexpr (sizeof(T) == 4) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        } else {
            uint32_t m = abs_max2<T>(w[0], w[1]);
#pragma unroll
            for (int i = 2; i < kWords; ++i) m = abs_max2<T>(m, w[i]);
            m = max(m & 0x7fffu, m >> 16 & 0x7fffu);
            if constexpr (std::is_same<T, __nv_bfloat16>::value) return m << 16;
            return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
        }
    }
};

// Codes of x * f, two words.
template <class V>
__device__ __forceinline__ uint2 e2m1_words(const V& x, float f) {
    uint32_t r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(x.pair(4 * h + i), both(f));
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(r[h])
            : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
    }
    return make_uint2(r[0], r[1]);
}

// A group's UE8M0 byte and its part's codes, for the fp32 bits of its largest magnitude: the smallest power of two
// that takes it to 6 or below; 255 (NaN) where it is not finite.
template <class T>
__device__ __forceinline__ uint32_t mxfp4_group(const Vec16<T>& x, uint32_t top, uint2* codes) {
    const uint32_t e = top >> 23;
    *codes = make_uint2(0, 0);
    if (e == 255) return 255u;
    const int byte = static_cast<int>(e) - ((top & 0x7fffffu) > 0x400000u ? 1 : 2);
    const uint32_t s = static_cast<uint32_t>(max(byte, 0));
    *codes = e2m1_words(x, __uint_as_float((254u - s) << 23));   // times 2^-(s - 127), exact
    return s;
}

// fp4_mxfp4.cu, fp4_nvfp4.cu: the products, a format to a translation unit.  tm: weights' codes, rows' codes in boxes
// of kFp4Rows / 2 and of 16 rows, weights' scales, rows' scales.
struct Fp4Args {
    const int32_t* offsets;    // null: one expert owns all rows
    int E;
    int64_t rows;
    int N, K;
    const float* row_scale;    // nvfp4
    const float* w_global;     // nvfp4, [E]
    void* out;
    uint8_t* out_scales;       // kFp4SiluQuant
    uint32_t* status;
};
enum Fp4Mode { kFp4Store = MOE_EXPERT_STORE, kFp4Silu = MOE_EXPERT_SILU_MUL, kFp4SiluQuant = MOE_EXPERT_SILU_MUL_QUANT };
template <int FMT>
cudaError_t fp4_experts_init();
template <int FMT>
cudaError_t fp4_experts_launch(int dtype, int mode, const Fp4Args& a, const CUtensorMap (&tm)[5], int64_t most_items,
                               cudaStream_t stream);

}  // namespace mfp8
