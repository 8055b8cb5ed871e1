// The experts' products over rows sorted by expert, in bf16 or fp16 with fp32 accumulation, and
// their gradients ("w13 [num_experts, N, K]", page "Quantization and MoE Optimizations", section
// FusedMoE Class):
//
//   product            c[r]  = a[r] @ w[e]^T              a [rows, K], w [E, N, K], c [rows, N]
//   ... SiLU(gate)*up  h[r]  = silu(c[r, :N/2]) * c[r, N/2:]
//   rows' gradient     da[r] = dc[r] @ w[e]               dc [rows, N], da [rows, K]
//   ... through SiLU(gate)*up (gate, up [rows, 2K]):
//                      dgate = da * up * s * (1 + gate * (1 - s)),  dup = da * gate * s,  s = sigmoid(gate)
//   weights' gradient  dw[e] = dc[rows of e]^T @ a[rows of e]
// where expert e owns rows [offsets[e], offsets[e+1]).
//
// One persistent kernel on clusters of two CTAs, one CTA per SM.  An item is a tile of 256 x up to 256
// outputs: one thread of CTA 0 issues tcgen05.mma.cta_group::2 (256 x N x 16), which reads both CTAs'
// operands (128 of the 256, half of the N each) and leaves each CTA its 128 x N in its own tensor
// memory (two accumulators).  A 64-wide K block then brings 32 KB into an SM for 512 cycles of its
// tensor pipe.  A TMA warp per CTA fills a ring of six 64-wide stages, eight warps per CTA drain an
// accumulator while the next one fills.
//
// Products and rows' gradient: the 256 run along the output columns (the weights) and N along the
// rows, so that the tile in which an expert ends costs its rows rounded up to 32, not to 256 (a
// skewed router leaves most experts few rows: with rows along the 256, 19% of the multiply-adds of
// the Qwen3-shaped batch were padding).  The accumulators then hold one output column per lane,
// and the epilogue turns them over.  Weights' gradient: 256 columns of a by 256 of dc, the rows are
// the reduction.
//
// The operands keep the caller's layout; where the reduction runs along the slow axis (w of the
// rows' gradient, both operands of the weights' gradient) the 128-byte rows of a TMA box run along the
// other axis and the MMA reads the tile transposed (MN-major).  Rows need no padding: a tile that
// ends inside an expert computes rows of the next and does not store them; in the weights' gradient
// the stage in which an expert ends is finished by a warp of each CTA that zeroes the rows past the
// end, for both operands, so that nothing a neighbour holds (a NaN, say) reaches the sum.
//
// Measured: 131072 rows of bf16 over 128 skewed experts, K 2048, N 1536 with SiLU: 526 us in short loops (1568
// TFLOP/s, tensor pipe 79% busy), 600 us in a long one, where the power limit lowers the clocks (a library
// product of 8192^3 falls from 1904 to 1710 TFLOP/s the same way).  The rows' gradient of the same batch 540 us, through
// SiLU (2048 to 768 columns) 342 us, the weights' gradient 566 us (638 us in a long loop).  Decode, 64 rows over 128
// experts: 54 us for 321 MB (0.88 of a copy); rows' gradient of 1024 rows, 8 experts of 14336 x 4096: 165 us
// (0.95 of a copy).
#include <type_traits>

#include "train.cuh"

namespace mfp8 {
namespace {

enum Mode { kForward = 0, kForwardSilu = 1, kRows = 2, kRowsSilu = 3, kWeights = 4 };

constexpr int XM = 256, XN = 256, XK = 64;         // item; XK elements are one 128-byte swizzled row
constexpr int X_STAGES = 6;                        // of the ring, one K block each
constexpr int X_TILE = 128 * XK * 2;               // one operand's K block in one CTA
constexpr int X_BOX = 64 * 128;                    // bytes of a transposed operand's box: 64 rows of 64 elements
constexpr int X_EPI_WARPS = 8, X_FIRST_EPI = 4;    // warps 0: TMA, 1: MMA, 2: tile table, 3: ends of experts
constexpr int X_THREADS = (X_FIRST_EPI + X_EPI_WARPS) * 32;
constexpr uint32_t X_TMEM = 512;
constexpr int X_PITCH = 256 + 16;                  // bytes of a staged row of 128 outputs
constexpr int X_STAGED = 32 * X_PITCH;             // of a block of 32 rows
constexpr int X_GROUP = 4;                         // row tiles visited together (see item_at)

struct ExpertArgs {
    const int32_t* offsets;
    int E;
    int64_t rows;
    int N, K;                  // w is [E, N, K]
    void* out;                 // c, h, da, dgate|dup or dw
    void* gate_up;             // kForwardSilu: written [rows, N] (null: not); kRowsSilu: read [rows, 2K]
    int64_t ld_gu;
    int turn;                  // kForwardSilu: gate and up columns alternate in the tile by this many (8 or 16)
    uint32_t* status;
};

struct XCtl {
    uint64_t full[X_STAGES];     // (CTA 0) both CTAs' operands of the stage are in place
    uint64_t empty[X_STAGES];    // the stage's MMAs completed
    uint64_t tail[X_STAGES];     // this CTA's loads of an expert's last stage landed (weights' gradient)
    uint64_t tfull[2];          // the accumulators are complete
    uint64_t tempty[2];         // (CTA 0) both CTAs' epilogue warps moved them out
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int half_bad[2];            // a warp of the epilogue's half gave up
    int row0[MOE_MAX_EXPERTS + 1];    // first row of each expert, checked against the rows
    int tile0[MOE_MAX_EXPERTS + 1];   // first row tile of each expert; weights' gradient: experts by falling rows
};
constexpr size_t X_SMEM = 1024 + X_STAGES * 2 * X_TILE + 2 * X_STAGED + sizeof(XCtl);
static_assert(X_SMEM <= 232448, "more shared memory than a CTA has");

// One output tile: rows [r0, r0 + nrow) of column tile n of expert e; kblocks of the reduction
// (length red).
struct XItem {
    int e, n, kblocks, red;
    int64_t r0;
    int nrow;
};

template <int MODE>
__device__ __forceinline__ int64_t item_count(const ExpertArgs& a, const XCtl* ctl, int NT) {
    if (MODE == kWeights) return static_cast<int64_t>(a.E) * ((a.N + XM - 1) / XM) * NT;
    return static_cast<int64_t>(ctl->tile0[a.E]) * NT;
}

// The item this cluster takes in its v-th round.  Rows' products: cluster c takes items c, c + clusters,
// ... (about equal work).  Weights' gradient: an item takes as long as its expert has rows, so the
// experts come by falling rows, every other round is dealt backwards (no cluster always gets the
// longer ones), and rounds are taken from both ends in turn, the odd clusters one step behind, so that
// items bound by their stores run beside the multiply-adds of the others.
template <int MODE>
__device__ __forceinline__ int64_t item_of_round(int64_t v, int64_t rounds) {
    const int64_t c = blockIdx.x >> 1, n = gridDim.x >> 1;
    if (MODE != kWeights) return v * n + c;
    const int64_t r = ((v + c) & 1) ? rounds - 1 - (v >> 1) : v >> 1;
    return r * n + ((r & 1) ? n - 1 - c : c);
}

template <int MODE>
__device__ __forceinline__ XItem item_at(const ExpertArgs& a, const XCtl* ctl, int64_t w, int NT) {
    XItem t;
    if (MODE == kWeights) {
        const int MT = (a.N + XM - 1) / XM, per = MT * NT;
        const int k = static_cast<int>(w / per);
        t.e = ctl->tile0[k];
        const int local = static_cast<int>(w - static_cast<int64_t>(k) * per);
        const int m = local % MT;
        t.n = local / MT;
        t.r0 = m * XM;
        t.nrow = a.N - m * XM < XM ? a.N - m * XM : XM;
        t.red = ctl->row0[t.e + 1] - ctl->row0[t.e];
    } else {
        // the expert whose tiles hold tile w / NT; within it X_GROUP row tiles by all column tiles, row
        // tiles fastest, so that the items under way at one time share rows and weights in L2
        const int g = static_cast<int>(w / NT);
        int lo = 0, hi = a.E - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (ctl->tile0[mid] <= g) lo = mid;
            else hi = mid - 1;
        }
        t.e = lo;
        const int mt = ctl->tile0[lo + 1] - ctl->tile0[lo];
        int local = static_cast<int>(w - static_cast<int64_t>(ctl->tile0[lo]) * NT);
        const int grp = local / (X_GROUP * NT);
        local -= grp * X_GROUP * NT;
        const int gm = mt - grp * X_GROUP < X_GROUP ? mt - grp * X_GROUP : X_GROUP;
        const int m = grp * X_GROUP + local % gm;
        t.n = local / gm;
        const int cnt = ctl->row0[t.e + 1] - ctl->row0[t.e];
        t.r0 = ctl->row0[t.e] + m * XN;
        t.nrow = cnt - m * XN < XN ? cnt - m * XN : XN;
        t.red = MODE == kRows || MODE == kRowsSilu ? a.N : a.K;
    }
    t.kblocks = t.red > 0 ? (t.red + XK - 1) / XK : 0;
    return t;
}

// Rows that the MMAs of a tile with nrow rows take (N: a multiple of 32 for a pair of CTAs).
__device__ __forceinline__ int rows_mma(int nrow) { return (nrow + 31) / 32 * 32; }

// The same item, in values the compiler knows to be the same in every lane.
__device__ __forceinline__ XItem uniform(const XItem& t) {
    XItem u;
    u.e = __shfl_sync(0xffffffffu, t.e, 0);
    u.n = __shfl_sync(0xffffffffu, t.n, 0);
    u.kblocks = __shfl_sync(0xffffffffu, t.kblocks, 0);
    u.red = __shfl_sync(0xffffffffu, t.red, 0);
    u.r0 = __shfl_sync(0xffffffffu, t.r0, 0);
    u.nrow = __shfl_sync(0xffffffffu, t.nrow, 0);
    return u;
}

// Descriptor of a tile read transposed: 64-element rows of 128 bytes along M or N (swizzled, as
// TMA writes them), one per reduction index; 8 of them (1024 bytes) to a group, the next 64
// elements of M or N one box further.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(X_BOX >> 4) << 16;         // leading byte offset: next 64 of M or N
    d |= static_cast<uint64_t>(1024 >> 4) << 32;          // stride byte offset: next 8 of K
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

template <class T>
__host__ __device__ constexpr uint32_t idesc_16bit(int n, bool a_mn, bool b_mn) {
    const uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return (1u << 4)                                       // D format: f32
           | (fmt << 7) | (fmt << 10)                      // A, B format: bf16 or f16
           | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16)   // transposed
           | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(XM >> 4) << 24);
}

// As tma_load_2d_pair, in five dimensions.
__device__ __forceinline__ void tma_load_5d_pair(uint32_t smem_dst, const CUtensorMap* map, int32_t x, int32_t y,
                                                 int32_t z, int32_t w, int32_t v, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
        "%4, %5, %6}], [%7];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
        : "memory");
}
// D (256 x N over both CTAs) (+)= A * B^T, K = 16, 16-bit operands, fp32 accumulation; issued by one
// thread of CTA 0.
__device__ __forceinline__ void mma_16bit_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on a barrier of either CTA, releasing this thread's writes to the cluster.
__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// One lane of a converged warp, the same every time.  The TMA and MMA warps run their loops as whole
// warps on warp-uniform values and elect the issuing lane, so that the tensor instructions' operands stay
// in uniform registers (with one thread in the loop each MMA cost it about 70 cycles).
__device__ __forceinline__ bool elect_lane() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
// Acquire at cluster scope what the arrivals on a completed phase released.
__device__ __forceinline__ void mbar_acquire_cluster(uint32_t bar, uint32_t parity) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(bar),
        "r"(parity)
        : "memory");
}
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async;" ::: "memory"); }

template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if (std::is_same<T, __nv_bfloat16>::value)
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<__half2*>(&v));
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

template <class T, int MODE>
__global__ void __launch_bounds__(X_THREADS, 1)
    expert_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmB16, const ExpertArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    uint8_t* base = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    uint8_t* smA = base;                                   // [X_STAGES][X_TILE]
    uint8_t* smB = base + X_STAGES * X_TILE;        // likewise
    uint8_t* smE = smB + X_STAGES * X_TILE;         // [2][X_STAGED]
    XCtl* ctl = reinterpret_cast<XCtl*>(smE + 2 * X_STAGED);
    constexpr bool A_MN = MODE == kWeights || MODE == kRows || MODE == kRowsSilu;
    constexpr bool B_MN = MODE == kWeights;
    constexpr bool SILU = MODE == kForwardSilu;

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank());
    const int OC = MODE == kForward ? a.N : SILU ? a.N / 2 : a.K;   // output columns (of h, for kForwardSilu)
    const int NT = SILU ? (OC + 127) / 128 : (OC + XN - 1) / XN;

    if (threadIdx.x == 0) {
        for (int s = 0; s < X_STAGES; ++s) {
            mbar_init(smem_addr(&ctl->full[s]), MODE == kWeights ? 2 : 1);
            mbar_init(smem_addr(&ctl->empty[s]), 1);
            mbar_init(smem_addr(&ctl->tail[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&ctl->tfull[b]), 1);
            mbar_init(smem_addr(&ctl->tempty[b]), 2 * X_EPI_WARPS);
        }
        mbar_init(smem_addr(&ctl->drain), 1);
        ctl->abort_flag = 0;
        ctl->half_bad[0] = ctl->half_bad[1] = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&ctl->tmem_base), X_TMEM);
        tmem_relinquish_pair();
    }
    grid_dependency_wait();
    // the experts' rows: every row up to the last offset belongs to exactly one expert.  Offsets that leave
    // [0, rows], start above 0 or run backwards are reported, and replaced by 0 for the first and the running
    // maximum of the clamped ones for the others.
    int bad = 0;
    for (int e = threadIdx.x; e <= a.E; e += X_THREADS) {
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
    if (MODE == kWeights) {
        for (int e = threadIdx.x; e < a.E; e += X_THREADS) {
            const int n = ctl->row0[e + 1] - ctl->row0[e];
            int place = 0;   // experts with more rows, or as many and a lower index
#pragma unroll 8
            for (int o = 0; o < a.E; ++o) {
                const int m = ctl->row0[o + 1] - ctl->row0[o];
                place += m > n || (m == n && o < e);
            }
            ctl->tile0[place] = e;
        }
    } else if (warp == 2) {
        int carry = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int cnt = e < a.E ? ctl->row0[e + 1] - ctl->row0[e] : 0;
            const int own = cnt > 0 ? (cnt + XN - 1) / XN : 0;
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
    cluster_barrier();   // both CTAs' barriers are initialised before any arrival from the other
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int* abort_flag = &ctl->abort_flag;
    const int64_t total = item_count<MODE>(a, ctl, NT);
    const int64_t rounds = (total + (gridDim.x >> 1) - 1) / (gridDim.x >> 1);

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA (both CTAs)
        int stage = 0;
        uint32_t phase = 0, issued = 0;
        bool ok = true;
        const uint32_t smA0 = smem_addr(smA), smB0 = smem_addr(smB);
        const uint32_t full = smem_addr(&ctl->full[0]), full0 = cluster_map(full, 0);
        for (int64_t round = 0; round < rounds && ok; ++round) {
            const int64_t w = item_of_round<MODE>(round, rounds);
            if (w >= total) continue;
            const XItem t = uniform(item_at<MODE>(a, ctl, w, NT));
            const int c0 = t.n * (SILU ? 128 : 256) + rank * (SILU ? 64 : 128);   // this CTA's output columns
            const int nn = rows_mma(t.nrow);                                      // rows the MMAs take
            const int32_t r0 = static_cast<int32_t>(t.r0) + rank * (MODE == kWeights ? 128 : nn / 2);
            // few rows: in boxes of 16, only as many as the MMAs read
            const int small = MODE != kWeights && nn <= 64 ? nn / 32 : 0;
            const int n_bytes = small ? small * 2048 : X_TILE;
            const int32_t first = MODE == kWeights ? ctl->row0[t.e] : 0;
            for (int kb = 0; kb < t.kblocks; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait<true>(smem_addr(&ctl->empty[stage]), phase ^ 1u, abort_flag, a.status));
                if (!ok) break;
                const bool tail = MODE == kWeights && t.red - kb * XK < XK;
                const uint32_t bar = tail ? smem_addr(&ctl->tail[stage]) : full0 + stage * 8;
                if (elect_lane()) {
                    if (tail) mbar_arrive_expect_tx(bar, 2 * X_TILE);
                    else if (rank == 0) mbar_arrive_expect_tx(full + stage * 8, 2 * (X_TILE + n_bytes));
                    else if (MODE == kWeights) mbar_arrive_cluster(bar);
                    const uint32_t sa = smA0 + stage * X_TILE, sb = smB0 + stage * X_TILE;
                    if (MODE == kWeights) {
                        // 64 rows of the expert, 128 columns of a and of dc
                        const int32_t r = first + kb * XK;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (tail) {
                                tma_load_2d(sa + i * X_BOX, &tmA, (c0 + i * 64) * 2, r, bar);
                                tma_load_2d(sb + i * X_BOX, &tmB, (r0 + i * 64) * 2, r, bar);
                            } else {
                                tma_load_2d_pair(sa + i * X_BOX, &tmA, (c0 + i * 64) * 2, r, bar);
                                tma_load_2d_pair(sb + i * X_BOX, &tmB, (r0 + i * 64) * 2, r, bar);
                            }
                        }
                    } else {
                        if (MODE == kForwardSilu) {   // gate and up columns in turn, a.turn of each
                            tma_load_5d_pair(sa, &tmA, kb * XK * 2, 0, 0, c0 / a.turn, t.e, bar);
                        } else if (MODE == kForward) {
                            tma_load_3d_pair(sa, &tmA, kb * XK * 2, c0, t.e, bar);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                tma_load_3d_pair(sa + i * X_BOX, &tmA, (c0 + i * 64) * 2, kb * XK, t.e, bar);
                        }
                        if (small == 0) tma_load_2d_pair(sb, &tmB, kb * XK * 2, r0, bar);
                        for (int i = 0; i < small; ++i)
                            tma_load_2d_pair(sb + i * 2048, &tmB16, kb * XK * 2, r0 + i * 16, bar);
                    }
                }
                __syncwarp();
                ++issued;
                if (++stage == X_STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // after an abort CTA 0 lets the loads of the stages it armed land, both CTAs' bytes; CTA 1, which
        // cannot see its loads' completion, waits for CTA 0 at the closing cluster barrier
        if (!ok && rank == 0 && lane == 0) {
            for (int s = 0; s < X_STAGES; ++s) {
                const uint32_t n_s = (issued + X_STAGES - 1 - s) / X_STAGES;
                if (n_s > 0) mbar_wait<true>(smem_addr(&ctl->full[s]), (n_s - 1) & 1u, nullptr, a.status);
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ------------------------------------------------------------ MMA (CTA 0)
            const uint64_t ad0 = A_MN ? smem_desc_mn_sw128(smem_addr(smA)) : smem_desc_k128_sw128(smem_addr(smA));
            const uint64_t bd0 = B_MN ? smem_desc_mn_sw128(smem_addr(smB)) : smem_desc_k128_sw128(smem_addr(smB));
            constexpr uint32_t a_step = (A_MN ? 2048 : 32) >> 4, b_step = (B_MN ? 2048 : 32) >> 4;
            constexpr uint32_t stage_step = X_TILE >> 4;
            int stage = 0;
            uint32_t phase = 0, buf = 0, bphase = 0;
            bool ok = true;
            for (int64_t round = 0; round < rounds && ok; ++round) {
                const int64_t w = item_of_round<MODE>(round, rounds);
                if (w >= total) continue;
                const XItem t = uniform(item_at<MODE>(a, ctl, w, NT));
                if (t.kblocks == 0) continue;
                ok = __all_sync(0xffffffffu, mbar_wait<true>(smem_addr(&ctl->tempty[buf]), bphase ^ 1u, abort_flag, a.status));
                if (!ok) break;
                const uint32_t d = tmem + buf * XN;
                const uint32_t idesc = idesc_16bit<T>(MODE == kWeights ? XN : rows_mma(t.nrow), A_MN, B_MN);
                for (int kb = 0; kb < t.kblocks; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait<true>(smem_addr(&ctl->full[stage]), phase, abort_flag, a.status));
                    if (!ok) break;
                    const int left = t.red - kb * XK;
                    if (MODE == kWeights && left < XK) mbar_acquire_cluster(smem_addr(&ctl->full[stage]), phase);
                    tc_fence_after();
                    const uint64_t ad = ad0 + stage * stage_step, bd = bd0 + stage * stage_step;
                    if (elect_lane()) {
                        if (left >= XK) {
                            mma_16bit_pair(d, ad, bd, idesc, kb > 0 ? 1u : 0u);
#pragma unroll
                            for (int k = 1; k < XK / 16; ++k)
                                mma_16bit_pair(d, ad + k * a_step, bd + k * b_step, idesc, 1u);
                        } else {
                            const int steps = (left + 15) / 16;
                            for (int k = 0; k < steps; ++k)
                                mma_16bit_pair(d, ad + k * a_step, bd + k * b_step, idesc, (kb | k) > 0 ? 1u : 0u);
                        }
                        mma_commit_pair(smem_addr(&ctl->empty[stage]), 3);
                        if (kb + 1 == t.kblocks) mma_commit_pair(smem_addr(&ctl->tfull[buf]), 3);
                    }
                    __syncwarp();
                    if (++stage == X_STAGES) {
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
    } else if (warp == 3 && MODE == kWeights) {
        // ---------------------------------------------------------------- ends of experts (both CTAs)
        int stage = 0;
        uint32_t tails = 0;   // bit s: parity of stage s's tail barrier
        bool ok = true;
        for (int64_t round = 0; round < rounds && ok; ++round) {
            const int64_t w = item_of_round<MODE>(round, rounds);
            if (w >= total) continue;
            const XItem t = item_at<MODE>(a, ctl, w, NT);
            if (t.kblocks == 0) continue;
            const int live = t.red - (t.kblocks - 1) * XK;   // rows of the last stage, 1 .. 64
            const int last = (stage + t.kblocks - 1) % X_STAGES;
            stage = (last + 1) % X_STAGES;
            if (live == XK) continue;
            ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&ctl->tail[last]), (tails >> last) & 1u, abort_flag, a.status));
            if (!ok) break;
            tails ^= 1u << last;
            // the MMAs run in steps of 16 rows: the rest of the last step's rows, in this CTA's four boxes
            const int pieces = ((live + 15) / 16 * 16 - live) * 8;   // 16-byte pieces of a box
            uint8_t* at = smA + last * X_TILE + live * 128;
            for (int i = lane; i < pieces * 4; i += 32) {
                const int box = i / pieces, p = i - box * pieces;
                *reinterpret_cast<uint4*>(at + (box & 1) * X_BOX + (box >> 1) * (smB - smA) + p * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive_release_cluster(cluster_map(smem_addr(&ctl->full[last]), 0));
        }
    } else if (warp >= X_FIRST_EPI) {
        // ---------------------------------------------------------------- epilogue
        const int g = (warp - X_FIRST_EPI) >> 2;
        const int sp = warp & 3;                   // tensor-memory lane quarter
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(sp * 32) << 16);
        T* out = static_cast<T*>(a.out);
        const T* gu_in = static_cast<const T*>(a.gate_up);   // kRowsSilu
        const Block block = {smE + g * X_STAGED, 1 + g, sp * 32 + lane};
        uint32_t buf = 0, bphase = 0;
        bool ok = true;
        const uint32_t tempty0 = cluster_map(smem_addr(&ctl->tempty[0]), 0), tempty1 = cluster_map(smem_addr(&ctl->tempty[1]), 0);
        for (int64_t round = 0; round < rounds; ++round) {
            const int64_t w = item_of_round<MODE>(round, rounds);
            if (w >= total) continue;
            const XItem t = item_at<MODE>(a, ctl, w, NT);
            // output columns in the lanes; the tile's rows in blocks of 32, dealt to the halves g in turn
            const int c0 = t.n * (SILU ? 128 : 256) + rank * (SILU ? 64 : 128);   // this CTA's columns
            const int col = sp * 32 + lane;
            const int blocks = (t.nrow + 31) / 32;
            const int64_t row = t.r0 + (MODE == kWeights ? static_cast<int64_t>(t.e) * a.N : 0);
            if (MODE == kWeights && t.kblocks == 0) {   // an expert without rows: zero
                for (int blk = g; blk < blocks; blk += 2)
                    block.each_piece<16>([&](int, int r, int q, uint8_t*) {
                        if (r < t.nrow - blk * 32 && c0 + q * 8 < OC)
                            *reinterpret_cast<uint4*>(out + (row + blk * 32 + r) * OC + c0 + q * 8) = make_uint4(0, 0, 0, 0);
                    });
                continue;
            }
            uint4 gq[4], uq[4];
            if constexpr (MODE == kRowsSilu) {   // gate and up of the first block, ahead of the products
                block.fetch<T>(gq, gu_in + (row + g * 32) * a.ld_gu, a.ld_gu, t.nrow - g * 32, c0, OC);
                block.fetch<T>(uq, gu_in + (row + g * 32) * a.ld_gu + OC, a.ld_gu, t.nrow - g * 32, c0, OC);
            }
            ok = __all_sync(0xffffffffu, mbar_wait<true>(smem_addr(&ctl->tfull[buf]), bphase, abort_flag, a.status));
            if (!half_ok(ok, block, &ctl->half_bad[g])) break;
            tc_fence_after();
            for (int blk = g; blk < blocks; blk += 2) {
                float v[32];
                tmem_ld32(lane_base + buf * XN + blk * 32, v);
                const int64_t r0 = row + blk * 32;
                const int nrow = t.nrow - blk * 32;
                if constexpr (SILU) {
                    // lanes: a.turn gate columns, then the up columns of the same, and so on; hc: the column of h
                    const bool up = (lane & a.turn) != 0;
                    const int hc = sp * 16 + (a.turn == 16 ? lane & 15 : ((lane >> 4) * 8) + (lane & 7));
                    T* gu = static_cast<T*>(a.gate_up);
                    if (gu) {   // staged as 64 gate and 64 up columns
#pragma unroll
                        for (int i = 0; i < 32; ++i) block.put<T>(i, hc + (up ? 64 : 0), v[i]);
                        block.sync();
                        block.each_piece<16>([&](int, int r, int q, uint8_t* p) {
                            const int c = c0 + (q & 7) * 8;
                            if (r < nrow && c < OC)
                                *reinterpret_cast<uint4*>(gu + (r0 + r) * (2 * OC) + c + (q & 8 ? OC : 0)) =
                                    *reinterpret_cast<const uint4*>(p);
                        });
                        block.sync();
                    }
                    // a gate lane gives the up lane beside it its rows 16 .. 31 for that lane's up of rows
                    // 0 .. 15: each then holds 16 rows of one column of h
                    const int first = up ? 16 : 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float o = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[16 + i], a.turn);
                        const float gate = up ? o : v[i], u = up ? v[16 + i] : o;
                        block.put<T>(first + i, hc, __fdividef(gate, 1.0f + __expf(-gate)) * u);
                    }
                    block.sync();
                    block.each_piece<8>([&](int, int r, int q, uint8_t* p) {
                        if (r < nrow && c0 + q * 8 < OC)
                            *reinterpret_cast<uint4*>(out + (r0 + r) * OC + c0 + q * 8) = *reinterpret_cast<const uint4*>(p);
                    });
                    block.sync();
                } else if constexpr (MODE == kRowsSilu) {
                    float gt[32], up[32];
                    block.turn<T>(gq, gt, col);
                    block.turn<T>(uq, up, col);
                    if (blk + 2 < blocks) {
                        block.fetch<T>(gq, gu_in + (r0 + 64) * a.ld_gu, a.ld_gu, nrow - 64, c0, OC);
                        block.fetch<T>(uq, gu_in + (r0 + 64) * a.ld_gu + OC, a.ld_gu, nrow - 64, c0, OC);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float s = __fdividef(1.0f, 1.0f + __expf(-gt[i])), d = v[i];
                        v[i] = d * up[i] * s * (1.0f + gt[i] * (1.0f - s));
                        up[i] = d * gt[i] * s;
                    }
                    block.store<T>(v, col, out + r0 * (2 * OC), 2 * OC, nrow, c0, OC);
                    block.store<T>(up, col, out + r0 * (2 * OC) + OC, 2 * OC, nrow, c0, OC);
                } else {
                    block.store<T>(v, col, out + r0 * OC, OC, nrow, c0, OC);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(buf ? tempty1 : tempty0);
            buf ^= 1u;
            if (buf == 0) bphase ^= 1u;
        }
        if (MODE != kWeights && ok) {
            // rows of no expert: zero
            const int64_t cols = MODE == kRowsSilu ? 2 * OC : OC, first = ctl->row0[a.E], left = a.rows - first;
            const int64_t n = left * cols / 8, n2 = SILU && a.gate_up ? left * a.N / 8 : 0;
            const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (X_EPI_WARPS * 32) + threadIdx.x - X_FIRST_EPI * 32;
            const int64_t step = static_cast<int64_t>(gridDim.x) * (X_EPI_WARPS * 32);
            for (int64_t i = i0; i < n; i += step)
                reinterpret_cast<uint4*>(out + first * cols)[i] = make_uint4(0, 0, 0, 0);
            for (int64_t i = i0; i < n2; i += step)
                reinterpret_cast<uint4*>(static_cast<T*>(a.gate_up) + first * a.N)[i] = make_uint4(0, 0, 0, 0);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_barrier();   // no CTA leaves while the other's MMAs, loads or arrivals may still reach it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, X_TMEM);
}

// Tensor map of 16-bit rows [n1, n0] (n2 of them; 0: two dimensions), boxes of 64 elements by box1
// rows, as bytes.
cudaError_t map_16bit(CUtensorMap* map, const void* p, int64_t n0, int64_t ld, int64_t n1, int64_t n2, int box1) {
    const uint64_t dims[3] = {static_cast<uint64_t>(n0) * 2, static_cast<uint64_t>(n1), static_cast<uint64_t>(n2)};
    const uint64_t strides[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(ld) * 2 * n1};
    const uint32_t box[3] = {128, static_cast<uint32_t>(box1), 1};
    return encode_u8_map_nd(map, static_cast<const uint8_t*>(p), n2 > 0 ? 3 : 2, dims, strides, box, true);
}

// The rows of a product in boxes of 128 and of 16 (tm[1], tm[2]).
cudaError_t map_rows(CUtensorMap (&tm)[3], const void* p, int64_t cols, int64_t ld, int64_t rows) {
    const cudaError_t e = map_16bit(&tm[1], p, cols, ld, rows, 0, 128);
    return e == cudaSuccess ? map_16bit(&tm[2], p, cols, ld, rows, 0, 16) : e;
}

// w [E, 2I, K] as [E][I / turn][gate, up][turn][K]: one box brings 128 rows, turn gate columns and
// the up columns of the same in turn (I a multiple of turn).
cudaError_t map_gate_up(CUtensorMap* map, const void* w, int64_t K, int64_t I, int64_t E, int turn) {
    const uint64_t row = static_cast<uint64_t>(K) * 2, n = static_cast<uint64_t>(I);
    const uint64_t dims[5] = {row, static_cast<uint64_t>(turn), 2, n / turn, static_cast<uint64_t>(E)};
    const uint64_t strides[4] = {row, n * row, turn * row, 2 * n * row};
    const uint32_t box[5] = {128, static_cast<uint32_t>(turn), 2, static_cast<uint32_t>(64 / turn), 1};
    return encode_u8_map_nd(map, static_cast<const uint8_t*>(w), 5, dims, strides, box, true);
}

int g_clusters = 0;   // clusters of two CTAs resident at once (the same for every instance: one CTA per SM)

void pair_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned clusters, cudaStream_t stream) {
    *cfg = {};
    cfg->gridDim = dim3(2 * clusters);
    cfg->blockDim = dim3(X_THREADS);
    cfg->dynamicSmemBytes = X_SMEM;
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

template <class T, int MODE>
cudaError_t launch_experts(const ExpertArgs& a, const CUtensorMap (&tm)[3], int64_t most_items, cudaStream_t stream) {
    if (g_clusters < 1) return cudaErrorNotSupported;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    pair_config(&cfg, attr, static_cast<unsigned>(most_items < g_clusters ? most_items : g_clusters), stream);
    return cudaLaunchKernelEx(&cfg, expert_gemm_kernel<T, MODE>, tm[0], tm[1], tm[2], a);
}

template <int MODE>
cudaError_t launch_experts_type(int dtype, const ExpertArgs& a, const CUtensorMap (&tm)[3], int64_t most_items,
                                cudaStream_t stream) {
    return dtype == MOE_DTYPE_BF16 ? launch_experts<__nv_bfloat16, MODE>(a, tm, most_items, stream)
                                   : launch_experts<__half, MODE>(a, tm, most_items, stream);
}

template <class T, int MODE>
cudaError_t set_smem() {
    return cudaFuncSetAttribute(expert_gemm_kernel<T, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(X_SMEM));
}
template <class T>
cudaError_t set_smem_all() {
    cudaError_t e = set_smem<T, kForward>();
    if (e == cudaSuccess) e = set_smem<T, kForwardSilu>();
    if (e == cudaSuccess) e = set_smem<T, kRows>();
    if (e == cudaSuccess) e = set_smem<T, kRowsSilu>();
    if (e == cudaSuccess) e = set_smem<T, kWeights>();
    return e;
}

int64_t most_row_tiles(int64_t rows, int E) { return rows / XM + (rows < E ? rows : E) + 1; }

// Checks that all three products share.
int check_experts(int dtype, int64_t rows, int E, int N, int K) {
    if (rows < 0 || E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS || N % 8 != 0 || K % 8 != 0 || rows >= (int64_t(1) << 31) || N >= (1 << 29) ||
        K >= (1 << 29))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}
bool on_16(const void* p) { return (address(p) & 15) == 0; }

}  // namespace

cudaError_t experts_init_device() {
    cudaError_t e = set_smem_all<__nv_bfloat16>();
    if (e == cudaSuccess) e = set_smem_all<__half>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    pair_config(&cfg, attr, 1, nullptr);
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, expert_gemm_kernel<__nv_bfloat16, kForward>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
    }
    g_clusters = n;
    return cudaSuccess;
}

}  // namespace mfp8

using namespace mfp8;

extern "C" {

int moe_expert_gemm(const void* rows_a, int64_t lda, int dtype, const void* w, const int32_t* expert_offsets,
                    int64_t num_rows, int E, int N, int K, int epilogue, void* out, void* gate_up, void* stream) {
    int rc = check_experts(dtype, num_rows, E, N, K);
    if (rc != MOE_OK) return rc;
    if (epilogue != MOE_EXPERT_STORE && epilogue != MOE_EXPERT_SILU_MUL) return MOE_ERR_INVALID_ARG;
    if (lda < K || (gate_up && epilogue == MOE_EXPERT_STORE)) return MOE_ERR_INVALID_ARG;
    if (lda % 8 != 0 || (epilogue == MOE_EXPERT_SILU_MUL && N % 16 != 0)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!w || !expert_offsets || (num_rows > 0 && (!rows_a || !out))) return MOE_ERR_INVALID_ARG;
    if (!on_16(rows_a) || !on_16(w) || !on_16(out) || !on_16(gate_up)) return MOE_ERR_INVALID_ARG;
    if (num_rows == 0) return MOE_OK;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    const int I = N / 2, turn = I % 16 == 0 ? 16 : 8;
    const bool silu = epilogue == MOE_EXPERT_SILU_MUL;
    CUtensorMap tm[3];   // weights, rows, rows in small boxes
    if ((silu ? map_gate_up(&tm[0], w, K, I, E, turn) : map_16bit(&tm[0], w, K, K, N, E, 128)) != cudaSuccess ||
        map_rows(tm, rows_a, K, lda, num_rows) != cudaSuccess)
        return MOE_ERR_CUDA;
    const ExpertArgs a = {expert_offsets, E, num_rows, N, K, out, gate_up, 0, turn, status};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t tiles = most_row_tiles(num_rows, E);
    if (silu) return cuda_status(launch_experts_type<kForwardSilu>(dtype, a, tm, tiles * ((I + 127) / 128), s));
    return cuda_status(launch_experts_type<kForward>(dtype, a, tm, tiles * ((N + XN - 1) / XN), s));
}

int moe_expert_gemm_dgrad(const void* dc, int64_t lddc, int dtype, const void* w, const int32_t* expert_offsets,
                          int64_t num_rows, int E, int N, int K, const void* gate_up, int64_t ldgu, void* out,
                          void* stream) {
    int rc = check_experts(dtype, num_rows, E, N, K);
    if (rc != MOE_OK) return rc;
    if (lddc < N || (gate_up && ldgu < 2 * static_cast<int64_t>(K))) return MOE_ERR_INVALID_ARG;
    if (lddc % 8 != 0 || (gate_up && ldgu % 8 != 0)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!w || !expert_offsets || (num_rows > 0 && (!dc || !out))) return MOE_ERR_INVALID_ARG;
    if (!on_16(dc) || !on_16(w) || !on_16(out) || !on_16(gate_up)) return MOE_ERR_INVALID_ARG;
    if (num_rows == 0) return MOE_OK;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    CUtensorMap tm[3];
    if (map_16bit(&tm[0], w, K, K, N, E, XK) != cudaSuccess || map_rows(tm, dc, N, lddc, num_rows) != cudaSuccess)
        return MOE_ERR_CUDA;
    const ExpertArgs a = {expert_offsets, E, num_rows, N, K, out, const_cast<void*>(gate_up), ldgu, 0, status};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t items = most_row_tiles(num_rows, E) * ((K + XN - 1) / XN);
    if (gate_up) return cuda_status(launch_experts_type<kRowsSilu>(dtype, a, tm, items, s));
    return cuda_status(launch_experts_type<kRows>(dtype, a, tm, items, s));
}

int moe_expert_gemm_wgrad(const void* dc, int64_t lddc, const void* rows_a, int64_t lda, int dtype,
                          const int32_t* expert_offsets, int64_t num_rows, int E, int N, int K, void* dw,
                          void* stream) {
    int rc = check_experts(dtype, num_rows, E, N, K);
    if (rc != MOE_OK) return rc;
    if (lddc < N || lda < K) return MOE_ERR_INVALID_ARG;
    if (lddc % 8 != 0 || lda % 8 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!dw || !expert_offsets || (num_rows > 0 && (!dc || !rows_a))) return MOE_ERR_INVALID_ARG;
    if (!on_16(dc) || !on_16(rows_a) || !on_16(dw)) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (num_rows == 0) return cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(E) * N * K * 2, s));
    CUtensorMap tm[3];
    if (map_16bit(&tm[0], rows_a, K, lda, num_rows, 0, XK) != cudaSuccess ||
        map_16bit(&tm[1], dc, N, lddc, num_rows, 0, XK) != cudaSuccess)
        return MOE_ERR_CUDA;
    tm[2] = tm[1];   // not read
    const ExpertArgs a = {expert_offsets, E, num_rows, N, K, dw, nullptr, 0, 0, status};
    const int64_t items = static_cast<int64_t>(E) * ((N + XM - 1) / XM) * ((K + XN - 1) / XN);
    return cuda_status(launch_experts_type<kWeights>(dtype, a, tm, items, s));
}

}  // extern "C"
