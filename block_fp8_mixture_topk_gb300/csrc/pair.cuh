// What the products on pairs of CTAs share: loads and the issuing lane of their control warps, and the staging of
// their epilogue, whose accumulators hold an output column per lane.
#pragma once

#include "train.cuh"

namespace mfp8 {

constexpr int X_PITCH = 256 + 16;                  // bytes of a staged row of 128 outputs
constexpr int X_STAGED = 32 * X_PITCH;             // of a block of 32 rows

// As tma_load_2d_pair, in five dimensions.
__device__ __forceinline__ void tma_load_5d_pair(uint32_t smem_dst, const CUtensorMap* map, int32_t x, int32_t y,
                                                 int32_t z, int32_t w, int32_t v, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
        "%4, %5, %6}], [%7];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
        : "memory");
}
// One lane of a converged warp, the same every time.  The TMA and MMA warps run their loops as whole
// warps on warp-uniform values and elect the issuing lane, so that the tensor instructions' operands stay
// in uniform registers (with one thread in the loop each MMA cost it about 70 cycles).
__device__ __forceinline__ bool elect_lane() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// An accumulator lane is an output column: the four warps that hold a CTA's 128 columns turn a block of 32
// rows over in shared memory, so that it is stored (and gate and up are loaded) by whole 128-byte
// lines.  (Stored by each warp from registers, 32 or 64 bytes of a row at a time, the writes were a
// quarter of the L2's requests.)
struct Block {
    uint8_t* stage;            // [32] rows of X_PITCH bytes
    int bar, et;               // named barrier of the 128 threads, this thread among them
    __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory"); }
    // this thread's 16-byte pieces of a block whose rows have `pieces` of them (16 or 8): f(row, piece, address)
    template <int PIECES, class F>
    __device__ __forceinline__ void each_piece(F f) const {
#pragma unroll
        for (int i = 0; i < PIECES / 4; ++i) {
            const int k = i * 128 + et, r = k / PIECES, q = k % PIECES;
            f(i, r, q, stage + r * X_PITCH + q * 16);
        }
    }
    template <class T>
    __device__ __forceinline__ void put(int row, int col, float v) const {
        *reinterpret_cast<T*>(stage + row * X_PITCH + col * 2) = from_f32<T>(v);
    }
    template <class T>
    __device__ __forceinline__ float get(int row, int col) const {
        return to_f32(*reinterpret_cast<const T*>(stage + row * X_PITCH + col * 2));
    }
    // column `col` of 32 staged rows from v, then the block to rows [0, nrow) of out, from column c
    template <class T>
    __device__ __forceinline__ void store(const float* v, int col, T* out, int64_t ld, int nrow, int c, int cols) const {
#pragma unroll
        for (int i = 0; i < 32; ++i) put<T>(i, col, v[i]);
        sync();
        each_piece<16>([&](int, int r, int q, uint8_t* p) {
            if (r < nrow && c + q * 8 < cols)
                *reinterpret_cast<uint4*>(out + r * ld + c + q * 8) = *reinterpret_cast<const uint4*>(p);
        });
        sync();
    }
    // the reverse, in two steps: this thread's pieces of the block; column `col` of them all
    template <class T>
    __device__ __forceinline__ void fetch(uint4 (&u)[4], const T* in, int64_t ld, int nrow, int c, int cols) const {
        each_piece<16>([&](int i, int r, int q, uint8_t*) {
            u[i] = make_uint4(0, 0, 0, 0);
            if (r < nrow && c + q * 8 < cols) u[i] = __ldg(reinterpret_cast<const uint4*>(in + r * ld + c + q * 8));
        });
    }
    template <class T>
    __device__ __forceinline__ void turn(const uint4 (&u)[4], float* v, int col) const {
        each_piece<16>([&](int i, int, int, uint8_t* p) { *reinterpret_cast<uint4*>(p) = u[i]; });
        sync();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = get<T>(i, col);
        sync();
    }
};

// Whether all four warps of an epilogue half got through their wait: the same answer in all of them (the
// second barrier keeps a later item's answer away from this one's readers).
__device__ __forceinline__ bool half_ok(bool ok, const Block& block, volatile int* bad) {
    if (!ok) *bad = 1;
    block.sync();
    const bool fine = *bad == 0;
    block.sync();
    return fine;
}

// 32 columns of the warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t a[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
          "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(a[16]),
          "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]), "=r"(a[24]),
          "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(a[i]);
}

}  // namespace mfp8
