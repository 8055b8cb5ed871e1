// The experts' products on 4-bit rows and weights, over rows sorted by expert, with fp32 accumulation:
//
//   product            c[r] = a[r] @ w[e]^T                a [rows, K], w [E, N, K], c [rows, N]
//   ... SiLU(gate)*up  h[r] = silu(c[r, :N/2]) * c[r, N/2:]
// where expert e owns rows [offsets[e], offsets[e+1]) and a and w stand for codes and scales (fp4.cuh); the scale
// of a row and of an expert (nvfp4) multiply the fp32 sum.
//
// One persistent kernel on clusters of two CTAs, one CTA per SM, built like the 16-bit products.  An item is a
// tile of 256 output columns (the weights, 128 lanes of tensor memory in each CTA) by up to 224 rows (N of the MMA,
// in steps of 32, half of them loaded by each CTA), so an expert's last tile costs its rows.  One thread of CTA 0
// issues tcgen05.mma.cta_group::2 of kind mxf4 (a scale per 32) or mxf4nvf4 (per 16), K = 64 a step; a stage is a
// block of 256 K, four steps: 30 KB of codes and 3 or 6 KB of scales into an SM for 448 cycles of its tensor pipe.
//
// Tensor memory: two accumulators of 224 columns leave 64 for scales (with 256 rows nothing would be left, and one
// accumulator alone would stop the tensor pipe while it is read).  A slot of scales is two words of the weights'
// 128 rows and of the item's rows, 24 columns; the two slots are filled in turn by tcgen05.cp, issued by the MMA
// thread ahead of the MMAs that read them: the two run in the order in which one thread issues them.
//
// The rows' scales lie in tiles of 224 rows that start with the expert (fp4.cuh), so an item reads whole tiles; both
// CTAs need the scales of all its rows.
//
// Measured (GB300; the tensor cores' 4-bit rate taken as four times a measured 16-bit 1941 TFLOP/s):
//   8192 rows of 8 experts, nvfp4, 4096 -> 2 x 14336 with SiLU 302-312 us, 6370 TFLOP/s, 0.82 (359 under the power cap, at 1380 MHz);
//   14336 -> 4096 150 us, 0.82, fp32 results 160.  A stage's 33 or 36 KB come into an SM at 63 bytes a cycle (counted: 70 of the cycles
//   with work), 520 or 560 cycles for 448 of its tensor pipe: the bound.
//   131072 rows of 128 skewed experts, mxfp4, 2048 -> 2 x 768 with requantisation 145 us, 0.73 (eight K blocks an item: the
//   start and the end of an item show); 768 -> 2048 121 us, 5.7 TB/s: the results' stores.
//   131072 even rows, 768 -> 2048, nvfp4: bf16 results 179 us, fp32 245 (4.8 TB/s).
//   One token's 8 rows, 2048 -> 2 x 768 7 us, 768 -> 2048 6 us: a launch, and one stage's way after the other.
// Weights fetched into L2 ahead of the stages were slower (5003 rows, 2048 -> 7168: 28 -> 31 us: the copies' issue is
// what is short); two row tiles of an item on the same weights, too (302 -> 355 us: the epilogue no longer hidden).
#pragma once

#include "fp4.cuh"
#include "pair.cuh"

namespace mfp8 {
namespace {

constexpr int F_N = kFp4Rows;
constexpr int F_A = 128 * 128;                      // bytes of the weights' codes of a stage in one CTA
constexpr int F_B = F_N / 2 * 128;                  // of the rows'
constexpr int F_EPI_WARPS = 8, F_FIRST_EPI = 4;     // warps 0: TMA, 1: MMA, 2: tile table
constexpr int F_THREADS = (F_FIRST_EPI + F_EPI_WARPS) * 32;
constexpr uint32_t F_TMEM = 512;
constexpr int F_GROUP = 4;                          // row tiles visited together
constexpr int F_SLOT = 24;                          // columns of a slot of scales: 2 words of 128 and of 256 rows
constexpr int F_STAGED = 2048;                      // bytes of staged results a warp
constexpr int F_ITEMS = 128;                        // a cluster's first items, in a table
__host__ __device__ constexpr int f_stages(int fmt) { return fmt == MOE_FP4_MXFP4 ? 6 : 5; }
__host__ __device__ constexpr int f_scales(int fmt) { return 3 * fp4_words(fmt) * 512; }   // bytes of a stage
__host__ __device__ constexpr int f_stage(int fmt) { return F_A + F_B + f_scales(fmt); }

// One output tile: rows [r0, r0 + nrow) of column tile n of expert e, the m-th of its row tiles.
struct FItem {
    int e, n, m, r0, nrow;
};

struct FCtl {
    uint64_t full[6];           // (CTA 0) both CTAs' operands of the stage are in place
    uint64_t empty[6];          // the stage's MMAs completed
    uint64_t tfull[2];          // the accumulators are complete
    uint64_t tempty[2];         // (CTA 0) both CTAs' epilogue warps moved them out
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int half_bad[2];
    int row0[MOE_MAX_EXPERTS + 1];    // first row of each expert, checked against the rows
    int tile0[MOE_MAX_EXPERTS + 1];   // first row tile of each expert
    FItem item[F_ITEMS];              // the cluster's first
};
__host__ __device__ constexpr size_t f_smem(int fmt) {
    return 1024 + static_cast<size_t>(f_stages(fmt)) * f_stage(fmt) + F_EPI_WARPS * F_STAGED + sizeof(FCtl);
}
static_assert(f_smem(MOE_FP4_MXFP4) <= 232448 && f_smem(MOE_FP4_NVFP4) <= 232448, "more shared memory than a CTA has");
static_assert(2 * (256 + F_SLOT) > static_cast<int>(F_TMEM) && F_N + F_SLOT <= 256, "an accumulator and a slot to each half");

// Item w of the launch: the expert whose tiles hold tile w / NT; within it F_GROUP row tiles by all column tiles, row
// tiles fastest, so that the items under way at one time share rows and weights in L2.
__device__ __forceinline__ FItem f_item_at(const Fp4Args& a, const FCtl* ctl, uint32_t w, uint32_t NT) {
    FItem t;
    const int g = static_cast<int>(w / NT);
    int lo = 0, hi = a.E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ctl->tile0[mid] <= g) lo = mid;
        else hi = mid - 1;
    }
    const int mt = ctl->tile0[lo + 1] - ctl->tile0[lo];
    uint32_t local = w - static_cast<uint32_t>(ctl->tile0[lo]) * NT;
    const uint32_t grp = local / (F_GROUP * NT);
    local -= grp * F_GROUP * NT;
    const int left = mt - static_cast<int>(grp) * F_GROUP;
    const uint32_t gm = left < F_GROUP ? left : F_GROUP;
    t.n = static_cast<int>(local / gm);
    t.m = static_cast<int>(grp * F_GROUP + local - t.n * gm);
    t.e = lo;
    t.r0 = ctl->row0[lo] + t.m * F_N;
    const int rows = ctl->row0[lo + 1] - t.r0;
    t.nrow = rows < F_N ? rows : F_N;
    return t;
}
// The k-th item of this cluster, from the table or (a long launch) worked out; the same values in every lane, which the
// compiler knows.  (Worked out by every role, an item took each of them 520 cycles, a quarter of a short one.)
__device__ __forceinline__ FItem f_item(const Fp4Args& a, const FCtl* ctl, uint32_t k, uint32_t w, uint32_t NT) {
    const FItem t = k < F_ITEMS ? ctl->item[k] : f_item_at(a, ctl, w, NT);
    FItem u;
    u.e = __shfl_sync(0xffffffffu, t.e, 0);
    u.n = __shfl_sync(0xffffffffu, t.n, 0);
    u.m = __shfl_sync(0xffffffffu, t.m, 0);
    u.r0 = __shfl_sync(0xffffffffu, t.r0, 0);
    u.nrow = __shfl_sync(0xffffffffu, t.nrow, 0);
    return u;
}
__device__ __forceinline__ int f_rows_mma(int nrow) { return (nrow + 31) / 32 * 32; }

// Instruction descriptor: e2m1 operands, both K-major, M = 256; sf: the first byte of the scales' words (2 of them
// per row and step with mxfp4, all 4 with nvfp4).
template <int FMT>
__device__ __forceinline__ uint32_t f_idesc(int n, int sf) {
    return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           ((FMT == MOE_FP4_MXFP4 ? 1u : 0u) << 23) | (2u << 27) | (static_cast<uint32_t>(sf) << 29);
}
// D (256 x N over both CTAs) (+)= (A * scales) * (B * scales)^T, K = 64; issued by one thread of CTA 0.
template <int FMT>
__device__ __forceinline__ void f_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                      uint32_t accumulate) {
    if constexpr (FMT == MOE_FP4_MXFP4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}
// Each CTA's 512-byte tile at this shared-memory address into 4 columns of its own tensor memory.
__device__ __forceinline__ void f_copy_scales(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// A block of 32 rows in the warp's 32 tensor-memory lanes (output columns), as fragments of 16 lanes by 8 rows: element
// 4 q + i of v[h] is lane 16 h + 8 (i / 2) + t / 4, row 8 q + 2 (t % 4) + i % 2 of thread t.  The values are there after
// f_wait_block, which names them so that nothing reads them earlier.
__device__ __forceinline__ void f_load_block(uint32_t taddr, float (&v)[2][16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
            "[%16];"
            : "=f"(v[h][0]), "=f"(v[h][1]), "=f"(v[h][2]), "=f"(v[h][3]), "=f"(v[h][4]), "=f"(v[h][5]), "=f"(v[h][6]),
              "=f"(v[h][7]), "=f"(v[h][8]), "=f"(v[h][9]), "=f"(v[h][10]), "=f"(v[h][11]), "=f"(v[h][12]), "=f"(v[h][13]),
              "=f"(v[h][14]), "=f"(v[h][15])
            : "r"(taddr + (static_cast<uint32_t>(16 * h) << 16))
            : "memory");
}
__device__ __forceinline__ void f_wait_block(float (&v)[2][16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0][0]), "+f"(v[0][1]), "+f"(v[0][2]), "+f"(v[0][3]), "+f"(v[0][4]), "+f"(v[0][5]), "+f"(v[0][6]),
                   "+f"(v[0][7]), "+f"(v[0][8]), "+f"(v[0][9]), "+f"(v[0][10]), "+f"(v[0][11]), "+f"(v[0][12]),
                   "+f"(v[0][13]), "+f"(v[0][14]), "+f"(v[0][15])
                 :
                 : "memory");
    asm volatile(""
                 : "+f"(v[1][0]), "+f"(v[1][1]), "+f"(v[1][2]), "+f"(v[1][3]), "+f"(v[1][4]), "+f"(v[1][5]), "+f"(v[1][6]),
                   "+f"(v[1][7]), "+f"(v[1][8]), "+f"(v[1][9]), "+f"(v[1][10]), "+f"(v[1][11]), "+f"(v[1][12]),
                   "+f"(v[1][13]), "+f"(v[1][14]), "+f"(v[1][15])
                 :
                 : "memory");
}
// Four 8 x 8 fragments of 16-bit values stored transposed, 16 bytes a row; lane t gives the address of row t % 8 of t / 8.
__device__ __forceinline__ void f_store_turned(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return bf16x2(lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// (The result is rounded to 16 bits: 9.8e-6 of the values elsewhere than the exact h's, 7.1e-6 with expf and a full division, which took
// 239 us in place of 129 at 131072 x 2048 -> 2 x 768.)
__device__ __forceinline__ float silu_mul(float gate, float up) { return __fdividef(gate, 1.0f + __expf(-gate)) * up; }

template <class T, int FMT, int MODE>
__global__ void __launch_bounds__(F_THREADS, 1)
    fp4_expert_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmB16, const __grid_constant__ CUtensorMap tmSA,
                      const __grid_constant__ CUtensorMap tmSB, const Fp4Args a) {
    constexpr int STAGES = f_stages(FMT), W = fp4_words(FMT);
    constexpr bool SILU = MODE != kFp4Store;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    uint8_t* smA = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);   // [STAGES][F_A]
    uint8_t* smB = smA + STAGES * F_A;                                      // [STAGES][F_B]
    uint8_t* smS = smB + STAGES * F_B;                                      // [STAGES][weights W, rows 2 W][512]
    uint8_t* smE = smS + STAGES * f_scales(FMT);                            // [F_EPI_WARPS][F_STAGED]
    FCtl* ctl = reinterpret_cast<FCtl*>(smE + F_EPI_WARPS * F_STAGED);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank());
    const int OC = SILU ? a.N / 2 : a.N;                        // output columns
    const int NT = SILU ? (OC + 127) / 128 : (OC + 255) / 256;
    const int KB = fp4_blocks(a.K);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_addr(&ctl->full[s]), 1);
            mbar_init(smem_addr(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&ctl->tfull[b]), 1);
            mbar_init(smem_addr(&ctl->tempty[b]), 2 * F_EPI_WARPS);
        }
        mbar_init(smem_addr(&ctl->drain), 1);
        ctl->abort_flag = 0;
        ctl->half_bad[0] = ctl->half_bad[1] = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
        tma_prefetch_map(&tmSA);
        tma_prefetch_map(&tmSB);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&ctl->tmem_base), F_TMEM);
        tmem_relinquish_pair();
    }
    grid_dependency_wait();
    // the experts' rows, offsets out of range or order repaired and reported, as in the 16-bit products
    int bad = 0;
    for (int e = threadIdx.x; e <= a.E; e += F_THREADS) {
        if (!a.offsets) {
            ctl->row0[e] = e == 0 ? 0 : static_cast<int>(a.rows);
            continue;
        }
        const int64_t o = a.offsets[e], prev = e > 0 ? a.offsets[e - 1] : 0;
        bad |= o < 0 || o > a.rows || prev > o || (e == 0 && o != 0);
        ctl->row0[e] = static_cast<int>(e == 0 || o < 0 ? 0 : o > a.rows ? a.rows : o);
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) {
            status_set(a.status, MOE_STATUS_BAD_COUNT);
            for (int e = 1; e <= a.E; ++e)
                if (ctl->row0[e] < ctl->row0[e - 1]) ctl->row0[e] = ctl->row0[e - 1];
        }
        __syncthreads();
    }
    if (warp == 2) {
        int carry = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int cnt = e < a.E ? ctl->row0[e + 1] - ctl->row0[e] : 0;
            const int own = (cnt + F_N - 1) / F_N;
            int v = own;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, s);
                if (lane >= s) v += u;
            }
            if (e < a.E) ctl->tile0[e] = carry + v - own;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) ctl->tile0[a.E] = carry;
    }
    tc_fence_before();
    __syncthreads();
    const uint32_t total = static_cast<uint32_t>(ctl->tile0[a.E]) * NT;   // (below 2^31: checked with the sizes)
    const uint32_t cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    if (threadIdx.x < F_ITEMS && cluster + threadIdx.x * clusters < total)
        ctl->item[threadIdx.x] = f_item_at(a, ctl, cluster + threadIdx.x * clusters, NT);
    __syncthreads();
    cluster_barrier();   // both CTAs' barriers are initialised before any arrival from the other
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int* abort_flag = &ctl->abort_flag;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA (both CTAs)
        int stage = 0;
        uint32_t phase = 0, issued = 0;
        bool ok = true;
        const uint32_t smA0 = smem_addr(smA), smB0 = smem_addr(smB), smS0 = smem_addr(smS);
        const uint32_t full = smem_addr(&ctl->full[0]), full0 = cluster_map(full, 0);
        const int w_tiles = SILU ? (OC + 63) / 64 : (a.N + 127) / 128;   // of the weights' scales, an expert
        uint32_t k = 0;
        for (uint32_t w = cluster; w < total && ok; w += clusters, ++k) {
            const FItem t = f_item(a, ctl, k, w, NT);
            const int c0 = t.n * (SILU ? 128 : 256) + rank * (SILU ? 64 : 128);   // this CTA's output columns
            const int nn = f_rows_mma(t.nrow);
            const int32_t r0 = t.r0 + rank * (nn / 2);
            const int small = nn <= 64 ? nn / 32 : 0;   // few rows: in boxes of 16, only as many as the MMAs read
            const uint32_t bytes = F_A + (small ? small * 2048 : F_B) + f_scales(FMT);
            // 512-byte tiles of scales; a tile of weights past the last is not multiplied into anything stored
            const int wt = 2 * t.n + rank;
            int32_t sa = static_cast<int32_t>((static_cast<int64_t>(t.e) * w_tiles + (wt < w_tiles ? wt : w_tiles - 1)) * KB * W);
            int32_t sb = static_cast<int32_t>((static_cast<int64_t>(ctl->row0[t.e] / F_N) + t.e + t.m) * KB * 2 * W);
            for (int kb = 0; kb < KB; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait<true>(smem_addr(&ctl->empty[stage]), phase ^ 1u, abort_flag, a.status));
                if (!ok) break;
                if (elect_lane()) {
                    const uint32_t bar = full0 + stage * 8;
                    if (rank == 0) mbar_arrive_expect_tx(full + stage * 8, 2 * bytes);
                    const uint32_t da = smA0 + stage * F_A, db = smB0 + stage * F_B, ds = smS0 + stage * f_scales(FMT);
                    if (SILU) tma_load_5d_pair(da, &tmA, kb * 128, 0, 0, c0 / 16, t.e, bar);   // 16 of gate, 16 of up in turn
                    else tma_load_3d_pair(da, &tmA, kb * 128, c0, t.e, bar);
                    if (small == 0) tma_load_2d_pair(db, &tmB, kb * 128, r0, bar);
                    for (int i = 0; i < small; ++i) tma_load_2d_pair(db + i * 2048, &tmB16, kb * 128, r0 + i * 16, bar);
                    tma_load_3d_pair(ds, &tmSA, 0, 0, sa, bar);
                    tma_load_3d_pair(ds + W * 512, &tmSB, 0, 0, sb, bar);
                }
                __syncwarp();
                sa += W;
                sb += 2 * W;
                ++issued;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // after an abort CTA 0 lets the loads of the stages it armed land, both CTAs' bytes; CTA 1, which
        // cannot see its loads' completion, waits for CTA 0 at the closing cluster barrier
        if (!ok && rank == 0 && lane == 0) {
            for (int s = 0; s < STAGES; ++s) {
                const uint32_t n_s = (issued + STAGES - 1 - s) / STAGES;
                if (n_s > 0) mbar_wait<true>(smem_addr(&ctl->full[s]), (n_s - 1) & 1u, nullptr, a.status);
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------------------------------------ MMA (CTA 0)
            const uint64_t ad0 = smem_desc_k128_sw128(smem_addr(smA)), bd0 = smem_desc_k128_sw128(smem_addr(smB));
            const uint64_t sd0 = smem_desc_sf_tile(smem_addr(smS));
            int stage = 0;
            uint32_t phase = 0, buf = 0, bphase = 0, slot = 0;
            bool ok = true;
            uint32_t k = 0;
            for (uint32_t w = cluster; w < total && ok; w += clusters, ++k) {
                const FItem t = f_item(a, ctl, k, w, NT);
                ok = __all_sync(0xffffffffu, mbar_wait<true>(smem_addr(&ctl->tempty[buf]), bphase ^ 1u, abort_flag, a.status));
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * 256;
                const int nn = f_rows_mma(t.nrow);
                const uint32_t idesc = f_idesc<FMT>(nn, 0);
                for (int kb = 0; kb < KB; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait<true>(smem_addr(&ctl->full[stage]), phase, abort_flag, a.status));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = ad0 + stage * (F_A >> 4), bd = bd0 + stage * (F_B >> 4);
                    const uint64_t sd = sd0 + stage * (f_scales(FMT) >> 4);
                    const int left = a.K - kb * kFp4Block;
                    const int steps = left >= kFp4Block ? 4 : (left + 63) / 64;
                    if (elect_lane()) {
                        constexpr int PER = FMT == MOE_FP4_MXFP4 ? 4 : 2;   // steps of a slot
#pragma unroll
                        for (int k0 = 0; k0 < 4; k0 += PER) {
                            if (k0 < steps) {
                                const uint32_t sfa = tmem + (((slot + k0 / PER) & 1u) ? 256 : 0) + F_N, sfb = sfa + 8;
                                const int word = k0 / PER * 2;
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    f_copy_scales(sfa + j * 4, sd + (word + j) * 32);
                                    f_copy_scales(sfb + j * 8, sd + (W + word + j) * 32);
                                    if (nn > 128) f_copy_scales(sfb + j * 8 + 4, sd + (2 * W + word + j) * 32);
                                }
#pragma unroll
                                for (int k = k0; k < k0 + PER; ++k) {
                                    const int j = FMT == MOE_FP4_MXFP4 ? k >> 1 : k - k0;
                                    const uint32_t id = idesc | (FMT == MOE_FP4_MXFP4 && (k & 1) ? (2u << 4) | (2u << 29) : 0u);
                                    if (k < steps)
                                        f_mma<FMT>(d, ad + k * 2, bd + k * 2, id, sfa + j * 4, sfb + j * 8, (kb | k) > 0 ? 1u : 0u);
                                }
                            }
                        }
                        mma_commit_pair(smem_addr(&ctl->empty[stage]), 3);
                        if (kb + 1 == KB) mma_commit_pair(smem_addr(&ctl->tfull[buf]), 3);
                    }
                    __syncwarp();
                    slot ^= FMT == MOE_FP4_MXFP4 || steps <= 2 ? 1u : 0u;   // (a stage of nvfp4 takes two)
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                buf ^= 1u;
                if (buf == 0) bphase ^= 1u;
            }
            // every MMA complete before the CTAs can leave (they read both CTAs' shared memory)
            if (elect_lane()) {
                mma_commit_pair(smem_addr(&ctl->drain), 1);
                mbar_wait(smem_addr(&ctl->drain), 0, nullptr, a.status);
            }
        }
    } else if (warp >= F_FIRST_EPI) {
        // ---------------------------------------------------------------- epilogue
        // The four warps of a half hold the CTA's 128 columns; the halves take blocks of 32 rows in turn.  Lanes are output
        // columns: 16-bit results go into shared memory transposed (8 x 8 at a time by stmatrix) and leave by rows.
        //   store         each warp by itself, 64 bytes (fp32: 128) of a row: no barrier in the loop (with one, and whole
        //                 rows of 256 bytes, warps stood at it half of the time)
        //   SiLU          the half together, 128 bytes of a row (a warp has 32), from two buffers in turn: one barrier a block
        // Rows are staged without padding, their 16-byte pieces exchanged by row so that no bank is hit twice.
        const int g = (warp - F_FIRST_EPI) >> 2;
        const int sp = warp & 3;                   // tensor-memory lane quarter
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(sp * 32) << 16);
        T* out = static_cast<T*>(a.out);
        uint8_t* const half_stage = smE + g * (4 * F_STAGED);
        uint8_t* const warp_stage = half_stage + sp * F_STAGED;
        const Block block = {half_stage, 1 + g, sp * 32 + lane};   // (for its barrier)
        uint32_t buf = 0, bphase = 0, side = 0;
        bool ok = true;
        const uint32_t tempty0 = cluster_map(smem_addr(&ctl->tempty[0]), 0), tempty1 = cluster_map(smem_addr(&ctl->tempty[1]), 0);
        uint32_t k = 0;
        for (uint32_t w = cluster; w < total; w += clusters, ++k) {
            const FItem t = f_item(a, ctl, k, w, NT);
            const int c0 = t.n * (SILU ? 128 : 256) + rank * (SILU ? 64 : 128);   // this CTA's columns
            const int blocks = (t.nrow + 31) / 32;
            float wg = 1.0f, rs = 0.0f;
            const auto row_scale = [&](int blk) {   // of the lane's row, times the expert's
                const int r = blk * 32 + lane;
                return r < t.nrow ? __ldg(a.row_scale + t.r0 + r) * wg : 0.0f;
            };
            if constexpr (FMT == MOE_FP4_NVFP4) {
                wg = __ldg(a.w_global + t.e);
                if (g < blocks) rs = row_scale(g);
            }
            ok = __all_sync(0xffffffffu, mbar_wait<true>(smem_addr(&ctl->tfull[buf]), bphase, abort_flag, a.status));
            if (SILU ? !half_ok(ok, block, &ctl->half_bad[g]) : !ok) break;
            tc_fence_after();
            const uint32_t acc = lane_base + buf * 256;
            if constexpr (sizeof(T) == 4) {
                for (int blk = g; blk < blocks; blk += 2) {
                    float v[32];
                    tmem_ld32(acc + blk * 32, v);
                    if constexpr (FMT == MOE_FP4_NVFP4) {
                        if (blk != g) rs = row_scale(blk);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= __shfl_sync(0xffffffffu, rs, i);
                    }
                    const int c = c0 + sp * 32 + (lane & 7) * 4;
#pragma unroll
                    for (int part = 0; part < 2; ++part) {   // 16 rows of 32 columns at a time
#pragma unroll
                        for (int i = 0; i < 16; ++i) *reinterpret_cast<float*>(warp_stage + i * 128 + lane * 4) = v[part * 16 + i];
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int q = i * 4 + (lane >> 3), r = blk * 32 + part * 16 + q;
                            const uint4 u = *reinterpret_cast<const uint4*>(warp_stage + q * 128 + (lane & 7) * 16);
                            if (r < t.nrow && c < OC)
                                *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(t.r0) + r) * OC + c) = u;
                        }
                        __syncwarp();
                    }
                }
            } else {
                float v[2][16];
                if (g < blocks) f_load_block(acc + g * 32, v);
                for (int blk = g; blk < blocks; blk += 2) {
                    f_wait_block(v);
                    if constexpr (FMT == MOE_FP4_NVFP4) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float s0 = __shfl_sync(0xffffffffu, rs, 8 * q + 2 * (lane & 3));
                            const float s1 = __shfl_sync(0xffffffffu, rs, 8 * q + 2 * (lane & 3) + 1);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                v[h][4 * q] *= s0, v[h][4 * q + 2] *= s0;
                                v[h][4 * q + 1] *= s1, v[h][4 * q + 3] *= s1;
                            }
                        }
                        if (blk + 2 < blocks) rs = row_scale(blk + 2);
                    }
                    // row r at r * PITCH, its piece p at p ^ swap(r)
                    constexpr int PITCH = SILU ? 128 : 64;
                    uint8_t* stage = SILU ? half_stage + side * (2 * F_STAGED) : warp_stage;
                    side ^= 1u;
                    if constexpr (SILU) {   // lanes 0 .. 15 gate, 16 .. 31 the up of the same columns
                        const int r = (lane >> 4) * 8 + (lane & 7);
                        const uint32_t to = smem_addr(stage) + r * PITCH + (((sp * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4);
#pragma unroll
                        for (int q = 0; q < 4; q += 2) {
                            uint32_t p[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                p[i] = pack2<T>(silu_mul(v[0][4 * q + 2 * i], v[1][4 * q + 2 * i]),
                                                silu_mul(v[0][4 * q + 2 * i + 1], v[1][4 * q + 2 * i + 1]));
                            f_store_turned(to + q * 8 * PITCH, p[0], p[1], p[2], p[3]);
                        }
                    } else {
                        const int r = lane & 7;
                        const uint32_t to = smem_addr(stage) + r * PITCH + (((lane >> 3) ^ (r >> 1)) << 4);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            f_store_turned(to + q * 8 * PITCH, pack2<T>(v[0][4 * q], v[0][4 * q + 1]),
                                           pack2<T>(v[0][4 * q + 2], v[0][4 * q + 3]), pack2<T>(v[1][4 * q], v[1][4 * q + 1]),
                                           pack2<T>(v[1][4 * q + 2], v[1][4 * q + 3]));
                    }
                    if (blk + 2 < blocks) f_load_block(acc + (blk + 2) * 32, v);
                    if (SILU) block.sync();
                    else __syncwarp();
                    const int64_t r0 = static_cast<int64_t>(t.r0) + blk * 32;
                    const int nrow = t.nrow - blk * 32;
                    if constexpr (MODE == kFp4SiluQuant) {
                        // a thread 16 of a row's 64 columns, two threads a group
                        const int r = block.et >> 2, part = block.et & 3, c = c0 + part * 16;
                        Vec16<T> x;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint4 u = *reinterpret_cast<const uint4*>(stage + r * PITCH + (((part * 2 + i) ^ (r & 7)) << 4));
                            x.w[4 * i] = u.x, x.w[4 * i + 1] = u.y, x.w[4 * i + 2] = u.z, x.w[4 * i + 3] = u.w;
                        }
                        uint32_t top = x.top();
                        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        uint2 codes;
                        const uint32_t s = mxfp4_group(x, top, &codes);
                        if (r < nrow) {
                            const int in = blk * 32 + r, group = c >> 5;
                            if (c < OC) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + (r0 + r) * (OC / 2) + c / 2) = codes;
                            uint8_t* tile = fp4_scale_row(a.out_scales, fp4_tile(ctl->row0[t.e], t.e) + t.m, in, fp4_blocks(OC), 2);
                            if ((part & 1) == 0)
                                tile[(group >> 3) * 2048 + ((group >> 2) & 1) * 512 + (group & 3)] =
                                    static_cast<uint8_t>(c < OC ? s : 0u);
                            // the K block's other 128 columns, where no item has them
                            if (t.n == NT - 1 && (NT & 1) && rank == 1 && part == 0)
                                *reinterpret_cast<uint32_t*>(tile + (group >> 3) * 2048 + 512) = 0u;
                        }
                    } else if constexpr (SILU) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int k = i * 128 + block.et, r = k >> 3, q = k & 7;
                            if (r < nrow && c0 + q * 8 < OC)
                                *reinterpret_cast<uint4*>(out + (r0 + r) * OC + c0 + q * 8) =
                                    *reinterpret_cast<const uint4*>(stage + r * PITCH + ((q ^ (r & 7)) << 4));
                        }
                    } else {
                        const int c = c0 + sp * 32 + (lane & 3) * 8;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = i * 8 + (lane >> 2);
                            const uint4 u = *reinterpret_cast<const uint4*>(stage + r * PITCH + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
                            if (r < nrow && c < OC) *reinterpret_cast<uint4*>(out + (r0 + r) * OC + c) = u;
                        }
                        __syncwarp();   // before the next block is staged
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(buf ? tempty1 : tempty0);
            buf ^= 1u;
            if (buf == 0) bphase ^= 1u;
        }
        if (ok) {   // rows of no expert: zero
            const int64_t first = ctl->row0[a.E], left = a.rows - first;
            const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (F_EPI_WARPS * 32) + threadIdx.x - F_FIRST_EPI * 32;
            const int64_t step = static_cast<int64_t>(gridDim.x) * (F_EPI_WARPS * 32);
            const int64_t row_bytes = MODE == kFp4SiluQuant ? OC / 2 : static_cast<int64_t>(OC) * static_cast<int64_t>(sizeof(T));
            uint4* zero = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + first * row_bytes);
            for (int64_t i = i0; i < left * row_bytes / 16; i += step) zero[i] = make_uint4(0, 0, 0, 0);
            if constexpr (MODE == kFp4SiluQuant) {   // their scales: those of an expert E
                const int words = fp4_blocks(OC) * 2;
                for (int64_t i = i0; i < left * words; i += step) {
                    const int64_t r = i / words;
                    const int j = static_cast<int>(i - r * words), m = static_cast<int>(r / F_N);
                    uint8_t* tile = fp4_scale_row(a.out_scales, fp4_tile(first, a.E) + m, static_cast<int>(r - static_cast<int64_t>(m) * F_N),
                                                  words / 2, 2);
                    *reinterpret_cast<uint32_t*>(tile + (j >> 1) * 2048 + (j & 1) * 512) = 0u;
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_barrier();   // no CTA leaves while the other's MMAs, loads or arrivals may still reach it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, F_TMEM);
}

void f_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int fmt, unsigned clusters, cudaStream_t stream) {
    *cfg = {};
    cfg->gridDim = dim3(2 * clusters);
    cfg->blockDim = dim3(F_THREADS);
    cfg->dynamicSmemBytes = f_smem(fmt);
    cfg->stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 2;
}

template <int FMT>
struct Fp4Launch {
    static int clusters;   // of two CTAs resident at once (the same for every instance: one CTA per SM)
    template <class T, int MODE>
    static cudaError_t one(const Fp4Args& a, const CUtensorMap (&tm)[5], int64_t most_items, cudaStream_t stream) {
        if (clusters < 1) return cudaErrorNotSupported;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        f_config(&cfg, attr, FMT, static_cast<unsigned>(most_items < clusters ? most_items : clusters), stream);
        return cudaLaunchKernelEx(&cfg, fp4_expert_kernel<T, FMT, MODE>, tm[0], tm[1], tm[2], tm[3], tm[4], a);
    }
    static cudaError_t launch(int dtype, int mode, const Fp4Args& a, const CUtensorMap (&tm)[5], int64_t items,
                              cudaStream_t s) {
        if constexpr (FMT == MOE_FP4_MXFP4)
            if (mode == kFp4SiluQuant) return one<__nv_bfloat16, kFp4SiluQuant>(a, tm, items, s);
        if (mode == kFp4Silu)
            return dtype == MOE_DTYPE_BF16 ? one<__nv_bfloat16, kFp4Silu>(a, tm, items, s) : one<__half, kFp4Silu>(a, tm, items, s);
        return dtype == MOE_DTYPE_BF16   ? one<__nv_bfloat16, kFp4Store>(a, tm, items, s)
               : dtype == MOE_DTYPE_FP16 ? one<__half, kFp4Store>(a, tm, items, s)
                                         : one<float, kFp4Store>(a, tm, items, s);
    }
    template <class T, int MODE>
    static cudaError_t smem() {
        return cudaFuncSetAttribute(fp4_expert_kernel<T, FMT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(f_smem(FMT)));
    }
    static cudaError_t init() {
        cudaError_t e = smem<__nv_bfloat16, kFp4Silu>();
        if constexpr (FMT == MOE_FP4_MXFP4)
            if (e == cudaSuccess) e = smem<__nv_bfloat16, kFp4SiluQuant>();
        if (e == cudaSuccess) e = smem<__half, kFp4Silu>();
        if (e == cudaSuccess) e = smem<__nv_bfloat16, kFp4Store>();
        if (e == cudaSuccess) e = smem<__half, kFp4Store>();
        if (e == cudaSuccess) e = smem<float, kFp4Store>();
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        f_config(&cfg, attr, FMT, 1, nullptr);
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, fp4_expert_kernel<__nv_bfloat16, FMT, kFp4Store>, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        clusters = n;
        return cudaSuccess;
    }
};
template <int FMT>
int Fp4Launch<FMT>::clusters = 0;

}  // namespace

}  // namespace mfp8
