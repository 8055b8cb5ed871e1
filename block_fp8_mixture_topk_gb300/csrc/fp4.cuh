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

#include "train.cuh"

namespace mfp8 {

constexpr int kFp4Rows = 224;      // rows of an item of the products, and of a tile of their scales
constexpr int kFp4Block = 256;     // columns of a K block
constexpr int kFp4MaxCols = 32768;

__host__ __device__ constexpr int fp4_group(int fmt) { return fmt == MOE_FP4_MXFP4 ? 32 : 16; }
__host__ __device__ constexpr int fp4_words(int fmt) { return fmt == MOE_FP4_MXFP4 ? 2 : 4; }
__host__ __device__ __forceinline__ int fp4_blocks(int K) { return (K + kFp4Block - 1) / kFp4Block; }

// Byte of the first scale of word j of row `in` (0 .. 127) in 128 rows' tiles of one K block.
__host__ __device__ __forceinline__ int fp4_word(int in, int j) { return j * 512 + (in & 31) * 16 + (in >> 5) * 4; }

// The tile and the place in it of row r, found by a whole warp: e is the last expert whose rows begin at or before
// r, o where they begin.  Offsets out of order or range count as the running maximum of the clamped ones, from 0,
// as the products take them.
struct Fp4Place {
    int64_t tile;
    int in;
};
__device__ __forceinline__ Fp4Place fp4_place(const int32_t* offsets, int E, int64_t r) {
    int64_t e = 0, o = 0;
    if (offsets) {
        const int lane = threadIdx.x & 31;
        int most = 0;
        e = E;
        for (int i0 = 1; i0 <= E; i0 += 32) {
            const int i = i0 + lane;
            const int32_t v = i <= E ? __ldg(offsets + i) : 0;
            const uint32_t past = __ballot_sync(0xffffffffu, v > r);
            const int first = past ? __ffs(static_cast<int>(past)) - 1 : 32;
            most = max(most, __reduce_max_sync(0xffffffffu, lane < first ? max(v, 0) : 0));
            if (past) {
                e = i0 + first - 1;
                break;
            }
        }
        o = most;
    }
    const int64_t m = (r - o) / kFp4Rows;
    return {o / kFp4Rows + e + m, static_cast<int>(r - o - m * kFp4Rows)};
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
    uint32_t* status;
};
template <int FMT>
cudaError_t fp4_experts_init();
template <int FMT>
cudaError_t fp4_experts_launch(int dtype, bool silu, const Fp4Args& a, const CUtensorMap (&tm)[5], int64_t most_items,
                               cudaStream_t stream);

}  // namespace mfp8
