// Token rows sorted by expert and back, with their gradients (the training form of the "sorted
// token" pattern and of the router-weighted gather, page "Quantization and MoE Optimizations",
// sections Triton Fused MoE Kernel and Modular Kernel Architecture).
//
//   dispatch            rows[pos[t, j]] = x[t]            (stable sort of the pairs by expert)
//   combine             out[t] = sum_j w[t, j] * y[pos[t, j]]
//   combine, backward   dy[pos[t, j]] = w[t, j] * dout[t],  dw[t, j] = <dout[t], y[pos[t, j]]>
//   dispatch, backward  dx[t] = sum_j drows[pos[t, j]]
//
// All four are bound by memory: every row is read or written once and the arithmetic is one fused
// multiply-add per element.  Rows of 16-byte addresses and strides move by bulk copies through
// shared memory, with more than 100 KB in flight per SM: the dispatch copies a row in once and out topk
// times without touching a register, the sums read a slab of columns of a token's topk rows at a time.
// Sums are fp32, in j order, rounded once to the rows' type; there are no atomics on values, so
// results do not depend on the schedule.
//
// Measured (bf16): dispatch and combine of 4096 tokens x 7168, top-8 of 256, 185 us for 1.06 GB (5.7 TB/s,
// 0.85 of a copy); the dispatch takes half, about 10 us of it the sort before its first store.  Both
// gradients for 16384 x 2048, top-8 of 128, skewed: 292 us for 1.75 GB (0.88 of a copy).  Eight tokens:
// 6.2 us on the device for both.  With vectors through registers the first shape took 211 us.  Rows at any
// address are bound by instructions (joining the vectors): 8000 x 4070 fp16, top-2 of 64, 108 us, 1.9 times
// the bytes' time.
#include "train.cuh"

namespace mfp8 {
namespace {

constexpr int kSortThreads = 1024;   // one thread per expert in the scan (MOE_MAX_EXPERTS)
// Up to so many pairs every CTA counts all ids itself: 16384 pairs (512 columns, 128 experts) take 7.9 us, and 10.3
// with a launch that counts them; 32768 take 12.0 and 12.7, 65536 23.3 and 18.5.
constexpr int64_t kDirectPairs = 16384;

// Counts of one chunk's pairs per expert.
__global__ void __launch_bounds__(kSortThreads) pair_count_kernel(const int32_t* __restrict__ ids, int64_t P,
                                                                  int chunk, int E, int32_t* __restrict__ counts) {
    grid_dependency_wait();
    __shared__ int hist[MOE_MAX_EXPERTS];
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * chunk;
    const int64_t p1 = p0 + chunk < P ? p0 + chunk : P;
    for (int64_t p = p0 + threadIdx.x; p < p1; p += blockDim.x) {
        const int id = ids[p];
        if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) counts[static_cast<int64_t>(blockIdx.x) * E + e] = hist[e];
}

struct DispatchArgs {
    const char* x;
    int64_t ld_bytes;
    const int32_t* ids;
    int64_t P;
    int topk, E;
    int chunk;                 // pairs per chunk (blockIdx.x), a multiple of topk
    int nch;
    const int32_t* counts;     // [nch][E], or null: every CTA counts the ids itself
    int H;
    int vecs, slab;            // most vectors of a row, vectors per column slab (blockIdx.y)
    char* rows;
    int32_t* expert_offsets;
    int32_t* pair_ids;
    int32_t* pos;
    int piece, slots, ring;    // bulk copies: bytes of a piece of a row, slots of a warp's ring, their offset in shared memory
    uint32_t* status;
};

constexpr int kCopyWarps = 8;              // warps that issue bulk copies
constexpr int kMostPiece = 8192;           // bytes of a piece of a row
constexpr int kMostSlots = 8;
constexpr int kSmemLimit = 232448, kStaticSmem = 2048;   // a CTA's shared memory; upper bound of what is declared statically

__device__ __forceinline__ void bulk_store(void* dst, uint32_t smem_src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the last N of this thread's groups of bulk stores have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// One warp's share of a round's copies: pieces warp, warp + kCopyWarps, ... of the round's tokens (token
// by token).  A ring of slots: lane 0 loads a piece, lanes j < topk store it to the pair's row; a slot
// is loaded again some pieces after its stores were issued, once every lane has seen its store's read of
// the slot finish.
__device__ __forceinline__ void copy_round(const DispatchArgs& a, const int* pos_s, int64_t t0, int tokens, uint8_t* ring,
                                           uint64_t* bars, uint32_t* phases, volatile int* abort_flag) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row_bytes = a.vecs * 16, pieces = (row_bytes + a.piece - 1) / a.piece, items = tokens * pieces;
    auto load = [&](int i, int slot) {
        const int t = i / pieces, c = (i - t * pieces) * a.piece;
        const uint32_t bytes = row_bytes - c < a.piece ? row_bytes - c : a.piece;
        const uint32_t b = smem_addr(bars + slot);
        mbar_arrive_expect_tx(b, bytes);
        bulk_load(smem_addr(ring + slot * a.piece), a.x + (t0 + t) * a.ld_bytes + c, bytes, b);
    };
    const int n = items > warp ? (items - warp + kCopyWarps - 1) / kCopyWarps : 0;   // this warp's pieces
    if (lane == 0)
        for (int k = 0; k < a.slots && k < n; ++k) load(warp + k * kCopyWarps, k);
    const int lag = a.slots >= 4 ? 2 : a.slots >= 2 ? 1 : 0;   // pieces between a store and its slot's next load
    int slot = 0;
    for (int k = 0; k < n; ++k) {
        mbar_wait(smem_addr(bars + slot), (*phases >> slot) & 1u, abort_flag, a.status);
        *phases ^= 1u << slot;
        const int i = warp + k * kCopyWarps, t = i / pieces, c = (i - t * pieces) * a.piece;
        const uint32_t bytes = row_bytes - c < a.piece ? row_bytes - c : a.piece;
        if (lane < a.topk) {
            const int r = pos_s[t * a.topk + lane];
            if (r >= 0) bulk_store(a.rows + static_cast<int64_t>(r) * row_bytes + c, smem_addr(ring + slot * a.piece), bytes);
        }
        bulk_commit();
        if (k >= lag) {
            if (lag == 2) bulk_wait_read<2>();
            else if (lag == 1) bulk_wait_read<1>();
            else bulk_wait_read<0>();
            __syncwarp();
            const int next = k - lag + a.slots;   // the slot of piece k - lag takes it
            if (lane == 0 && next < n) load(warp + next * kCopyWarps, (k - lag) % a.slots);
        }
        if (++slot == a.slots) slot = 0;
    }
    bulk_wait_read<0>();
    __syncwarp();
    if (*abort_flag && lane == 0)   // a wait gave up (its status bit is set): let the loads under way land
        for (int i = 0; i < a.slots; ++i) mbar_wait(smem_addr(bars + i), ((*phases >> i) & 1u) ^ 1u, nullptr, a.status);
}

// Vectors that a row of H elements of E touches at most: it may start and end inside one.
template <class E>
constexpr int vectors_any(int H) {
    return (H + 2 * (16 / static_cast<int>(sizeof(E))) - 2) / (16 / static_cast<int>(sizeof(E)));
}
// First element of the row's v-th aligned vector (negative for the first one of a row that starts inside it).
template <class E>
__device__ __forceinline__ int vector_any(const E* row, int v) {
    constexpr int V = 16 / static_cast<int>(sizeof(E));
    return v * V - static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(E));
}

// A round's copies for rows at any address: a warp to a pair, vectors v0 .. v0 + nv - 1 of its row in parts of
// kAnyLanes.
template <class E>
__device__ __forceinline__ void copy_round_any(const DispatchArgs& a, const int* pos_s, int64_t t0, int pairs, int v0,
                                               int nv) {
    constexpr int V = 16 / static_cast<int>(sizeof(E)), U = 4;
    const int64_t ld = a.ld_bytes / static_cast<int64_t>(sizeof(E)), T_ = a.P / a.topk;
    const int lane = threadIdx.x & 31;
    for (int p = threadIdx.x >> 5; p < pairs; p += kSortThreads / 32) {
        const int r = pos_s[p];
        if (r < 0) continue;
        const int64_t t = t0 + p / a.topk;
        const E* src = reinterpret_cast<const E*>(a.x) + t * ld;
        E* dst = reinterpret_cast<E*>(a.rows) + static_cast<int64_t>(r) * a.H;
        const int e0 = vector_any(dst, v0), e1 = min(a.H, e0 + nv * V);   // (whole vectors from e0 on)
        if (!inner_row(t, T_)) {
            for (int e = e0 + lane * V; e < e1; e += 32 * V) store_whole(dst, a.H, e, load_elements(src, a.H, e));
            continue;
        }
        for (int e = e0 + lane * V; e - lane * V < e1; e += U * kAnyLanes * V) {
            uint4 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) w[u] = load_around(src, a.H, e + u * kAnyLanes * V);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = e + u * kAnyLanes * V;
                if (at - lane * V >= e1) break;
                w[u] = join_lanes(w[u], src + at);
                if (lane < kAnyLanes && at < e1) store_whole(dst, a.H, at, w[u]);
            }
        }
    }
}

// The sort and the copies of one chunk of tokens and one slab of columns.  Every CTA derives the
// first row of its chunk for each expert from the pair counts (a scan over experts of the totals,
// plus the pairs of earlier chunks), ranks its pairs with a warp match, and copies its tokens: a
// row is read once and written topk times.  The slab-0 CTAs also write the tables.  R: the vector, or the
// element of rows at any address.
template <class R, bool BULK>
__global__ void __launch_bounds__(kSortThreads) dispatch_kernel(const DispatchArgs a) {
    extern __shared__ __align__(128) int smem[];
    int* before = smem;                    // [E] pairs of earlier chunks, then the next row of each expert
    int* after = smem + a.E;               // [E] pairs of this and later chunks
    int* pos_s = smem + 2 * a.E;           // [kSortThreads] rows of the current round's pairs
    int16_t* warp_count = reinterpret_cast<int16_t*>(pos_s + kSortThreads);   // [32][E]
    __shared__ int warp_sums[32];
    __shared__ int total_s;
    __shared__ uint64_t bars[kCopyWarps * kMostSlots];
    __shared__ int abort_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t phases = 0;
    if (BULK && tid < kCopyWarps * kMostSlots) {
        mbar_init(smem_addr(bars + tid), 1);
        fence_barrier_init();
    }
    if (tid == 0) abort_s = 0;
    for (int e = tid; e < 2 * a.E; e += kSortThreads) smem[e] = 0;
    __syncthreads();
    grid_dependency_wait();
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int64_t p1 = p0 + a.chunk < a.P ? p0 + a.chunk : a.P;
    if (a.counts) {
        const int G = kSortThreads / a.E;
        const int e = tid % a.E, g = tid / a.E;
        if (g < G) {
            int b = 0, t = 0;
#pragma unroll 8
            for (int c = g; c < a.nch; c += G) {
                const int v = a.counts[static_cast<int64_t>(c) * a.E + e];
                if (c < static_cast<int>(blockIdx.x)) b += v;
                else t += v;
            }
            atomicAdd(&before[e], b);
            atomicAdd(&after[e], t);
        }
    } else {
#pragma unroll 4
        for (int64_t p = tid; p < a.P; p += kSortThreads) {
            const int id = __ldg(a.ids + p);
            if (id >= 0 && id < a.E) atomicAdd(p < p0 ? &before[id] : &after[id], 1);
        }
    }
    __syncthreads();
    const int mine = tid < a.E ? before[tid] + after[tid] : 0;
    const int off = block_exclusive_scan(mine, warp_sums);
    if (tid < a.E) {
        before[tid] += off;
        if (blockIdx.x == 0 && blockIdx.y == 0) a.expert_offsets[tid] = off;
        if (tid == a.E - 1) {
            total_s = off + mine;
            if (blockIdx.x == 0 && blockIdx.y == 0) a.expert_offsets[a.E] = off + mine;
        }
    }
    __syncthreads();
    const int64_t total = total_s;
    const int v0 = blockIdx.y * a.slab;
    const int nv = a.vecs - v0 < a.slab ? a.vecs - v0 : a.slab;
    const bool tables = blockIdx.y == 0;
    const int round = kSortThreads / a.topk * a.topk;
    for (int64_t r0 = p0; r0 < p1; r0 += round) {
        for (int i = tid; i < 32 * a.E / 2; i += kSortThreads) reinterpret_cast<int*>(warp_count)[i] = 0;
        __syncthreads();
        const int n = static_cast<int>(p1 - r0 < round ? p1 - r0 : round);
        int id = -1;
        if (tid < n) {
            id = a.ids[r0 + tid];
            if (id >= a.E) {
                if (tables) status_set(a.status, MOE_STATUS_BAD_EXPERT_ID);
                id = -1;
            }
            if (id < 0) id = -1;
        }
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        const int rank = __popc(same & ((1u << lane) - 1));
        if (id >= 0 && rank == 0) warp_count[warp * a.E + id] = static_cast<int16_t>(__popc(same));
        __syncthreads();
        int at = -1;
        if (id >= 0) {
            int b = before[id];
            for (int w = 0; w < warp; ++w) b += warp_count[w * a.E + id];
            at = b + rank;
        }
        pos_s[tid] = at;
        if (tables && tid < n) {
            a.pos[r0 + tid] = at;
            if (at >= 0) a.pair_ids[at] = static_cast<int32_t>(r0 + tid);
        }
        __syncthreads();
        if (tid < a.E) {
            int c = 0;
#pragma unroll 8
            for (int w = 0; w < 32; ++w) c += warp_count[w * a.E + tid];
            before[tid] += c;
        }
        const int tokens = n / a.topk;
        const int64_t t0 = r0 / a.topk;
        if constexpr (BULK) {
            if (warp < kCopyWarps)
                copy_round(a, pos_s, t0, tokens, reinterpret_cast<uint8_t*>(smem) + a.ring + warp * a.slots * a.piece,
                           bars + warp * kMostSlots, &phases, &abort_s);
            __syncthreads();
            continue;
        } else if constexpr (sizeof(R) < 16) {
            copy_round_any<R>(a, pos_s, t0, n, v0, nv);
            __syncthreads();
            continue;
        }
        R* rows = reinterpret_cast<R*>(a.rows);
        const int items = tokens * nv;
        constexpr int U = 4;
        for (int i = tid; i < items; i += U * kSortThreads) {
            R val[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = i + u * kSortThreads;
                if (k < items)
                    val[u] = __ldg(reinterpret_cast<const R*>(a.x + (t0 + k / nv) * a.ld_bytes) + v0 + k % nv);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = i + u * kSortThreads;
                if (k >= items) break;
                const int t = k / nv, v = v0 + k % nv;
                for (int j = 0; j < a.topk; ++j) {
                    const int r = pos_s[t * a.topk + j];
                    if (r >= 0) rows[static_cast<int64_t>(r) * a.vecs + v] = val[u];
                }
            }
        }
        __syncthreads();
    }
    if constexpr (BULK) bulk_wait_all();
    // rows of no pair (as many as there are pairs without an expert): zero, at the end
    const int64_t left = (a.P - total) * nv;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSortThreads + tid; i < left;
         i += static_cast<int64_t>(gridDim.x) * kSortThreads) {
        const int64_t r = total + i / nv;
        const int v = v0 + static_cast<int>(i % nv);
        R* rows = reinterpret_cast<R*>(a.rows);
        if constexpr (sizeof(R) < 16) store_whole(rows + r * a.H, a.H, vector_any(rows + r * a.H, v), make_uint4(0u, 0u, 0u, 0u));
        else rows[r * a.vecs + v] = R{};
    }
    if (tables)
        for (int64_t r = total + static_cast<int64_t>(blockIdx.x) * kSortThreads + tid; r < a.P;
             r += static_cast<int64_t>(gridDim.x) * kSortThreads)
            a.pair_ids[r] = -1;
}

// out[t] = sum_j w[t, j] * y[pos[t, j]] (w null: 1), one thread per 16-byte vector of the result.
template <class T>
__global__ void __launch_bounds__(256) combine_kernel(const T* __restrict__ y, int64_t ld,
                                                      const int32_t* __restrict__ pos,
                                                      const float* __restrict__ w, int64_t n_tokens, int topk,
                                                      int vecs, int64_t num_rows, T* __restrict__ out,
                                                      uint32_t* status) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    grid_dependency_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n_tokens * vecs) return;
    const int64_t t = i / vecs;
    const int v = static_cast<int>(i - t * vecs);
    const int32_t* tp = pos + t * topk;
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    constexpr int U = 8;
    for (int j0 = 0; j0 < topk; j0 += U) {
        Pack<T, V> val[U];
        float wj[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int64_t r = j0 + u < topk ? tp[j0 + u] : -1;
            if (r >= num_rows) {
                if (v == 0) status_set(status, MOE_STATUS_BAD_EXPERT_ID);
                r = -1;
            }
            live[u] = r >= 0;
            if (live[u]) {
                val[u].load(y + r * ld + static_cast<int64_t>(v) * V);
                wj[u] = w ? w[t * topk + j0 + u] : 1.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!live[u]) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(wj[u], val[u].get(e), acc[e]);
        }
    }
    Pack<T, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) o.set(e, acc[e]);
    o.store(out + (t * vecs + v) * V);
}

// The same for rows at any address: a warp to a token and a part of kAnyLanes vectors of the result; lane j
// holds the row and the weight of pair j.
template <class T>
__global__ void __launch_bounds__(256) combine_any_kernel(const T* __restrict__ y, int64_t ld,
                                                          const int32_t* __restrict__ pos,
                                                          const float* __restrict__ w, int n_tokens, int topk, int H,
                                                          int parts, int num_rows, T* __restrict__ out,
                                                          uint32_t* status) {
    constexpr int V = 16 / static_cast<int>(sizeof(T)), U = 4;
    grid_dependency_wait();
    const uint32_t i = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, t = i / parts, part = i - t * parts;
    if (t >= n_tokens) return;
    const int lane = threadIdx.x & 31;
    int mine = -1;
    float weight = 1.0f;
    if (lane < topk) {
        mine = pos[static_cast<int64_t>(t) * topk + lane];
        if (w) weight = w[static_cast<int64_t>(t) * topk + lane];
        if (mine >= num_rows) {
            if (part == 0) status_set(status, MOE_STATUS_BAD_EXPERT_ID);
            mine = -1;
        }
    }
    T* row = out + static_cast<int64_t>(t) * H;
    const int e0 = vector_any(row, static_cast<int>(part) * kAnyLanes + lane);
    float2 acc[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) acc[e] = both(0.0f);
    for (uint32_t live = __ballot_sync(0xffffffffu, mine >= 0); live;) {
        uint4 x[U];
        const T* src[U];
        float wj[U];
        uint32_t inner = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            src[u] = nullptr;
            if (!live) continue;
            const int j = __ffs(live) - 1, r = __shfl_sync(0xffffffffu, mine, j);
            live &= live - 1;
            wj[u] = __shfl_sync(0xffffffffu, weight, j);
            src[u] = y + r * ld;
            if (!inner_row(r, num_rows)) continue;
            inner |= 1u << u;
            x[u] = load_around(src[u], H, e0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!src[u]) break;
            Pack<T, V> p;
            p.raw = inner >> u & 1 ? join_lanes(x[u], src[u] + e0) : load_elements(src[u], H, e0);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) acc[e] = fma2(both(wj[u]), p.pair(e), acc[e]);
        }
    }
    Pack<T, V> o;
#pragma unroll
    for (int e = 0; e < V / 2; ++e) o.set_pair(e, acc[e]);
    if (lane < kAnyLanes) store_whole(row, H, e0, o.raw);
}

// The same for rows of 16-byte addresses and strides and many tokens.  A CTA holds groups of G threads; a
// group walks over items (token, slab of G vectors), its first warp keeping `depth` items of bulk
// copies ahead: lane j < topk brings pair j's piece of the slab, the pairs without a row left out.
// Each thread then sums one vector over the token's rows from shared memory.
struct CombineArgs {
    const char* y;
    int64_t ld_bytes;
    const int32_t* pos;
    const float* w;
    int64_t tokens;
    int topk, vecs, slabs, G, depth;
    int64_t num_rows;
    char* out;
    uint32_t* status;
};
constexpr int kCombineThreads = 512, kCombineGroups = 15, kCombineDepth = 8;
constexpr int kCombineMeta = (MOE_MAX_TOPK + 4) * 4;   // of a slot: the weights of its pieces, then their number

// A place in the items of a group: token and slab, moved on by a fixed number of items.
struct CombineAt {
    int64_t t;
    int s;
    __device__ __forceinline__ void next(int64_t step_t, int step_s, int slabs) {
        t += step_t;
        s += step_s;
        if (s >= slabs) {
            s -= slabs;
            ++t;
        }
    }
};

template <class T>
__global__ void __launch_bounds__(kCombineThreads) combine_ring_kernel(const CombineArgs a) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    extern __shared__ __align__(128) uint8_t ring_smem[];
    __shared__ uint64_t bars[kCombineGroups * kCombineDepth];
    __shared__ int abort_s;
    const int G = a.G, R = blockDim.x / G, g = threadIdx.x / G, tid = threadIdx.x - g * G, lane = threadIdx.x & 31;
    const int slot_bytes = a.topk * G * 16 + kCombineMeta, piece = G * 16;
    uint8_t* ring = ring_smem + static_cast<size_t>(g) * a.depth * slot_bytes;
    uint64_t* bar = bars + g * kCombineDepth;
    for (int i = threadIdx.x; i < kCombineGroups * kCombineDepth; i += blockDim.x) mbar_init(smem_addr(bars + i), 1);
    fence_barrier_init();
    if (threadIdx.x == 0) abort_s = 0;
    __syncthreads();
    grid_dependency_wait();
    const int64_t step = static_cast<int64_t>(gridDim.x) * R, first = static_cast<int64_t>(blockIdx.x) * R + g;
    const int64_t step_t = step / a.slabs;
    const int step_s = static_cast<int>(step - step_t * a.slabs);
    CombineAt now = {first / a.slabs, static_cast<int>(first % a.slabs)}, load = now;
    // first warp: row and weight of this lane's pair in the item to load next, fetched one item early
    int64_t row = -1;
    float weight = 1.0f;
    uint32_t issued = 0;
    auto fetch = [&] {
        row = -1;
        if (lane < a.topk && load.t < a.tokens) {
            row = a.pos[load.t * a.topk + lane];
            if (a.w) weight = a.w[load.t * a.topk + lane];
        }
    };
    auto issue = [&](int slot) {
        if (load.t >= a.tokens) return;
        const int v0 = load.s * G, nv = a.vecs - v0 < G ? a.vecs - v0 : G;
        if (row >= a.num_rows) {
            if (v0 == 0) status_set(a.status, MOE_STATUS_BAD_EXPERT_ID);
            row = -1;
        }
        const uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
        const int at = __popc(live & ((1u << lane) - 1)), n = __popc(live);
        uint8_t* s = ring + static_cast<size_t>(slot) * slot_bytes;
        float* meta = reinterpret_cast<float*>(s + a.topk * piece);
        if (row >= 0) meta[at] = weight;
        if (lane == 0) reinterpret_cast<int*>(meta)[MOE_MAX_TOPK] = n;
        __syncwarp();
        const uint32_t b = smem_addr(bar + slot);
        if (lane == 0) mbar_arrive_expect_tx(b, n * nv * 16);
        __syncwarp();
        if (row >= 0) bulk_load(smem_addr(s + at * piece), a.y + row * a.ld_bytes + static_cast<int64_t>(v0) * 16, nv * 16, b);
        ++issued;
        load.next(step_t, step_s, a.slabs);
        fetch();
    };
    if (tid < 32) {
        fetch();
        for (int d = 0; d < a.depth; ++d) issue(d);
    }
    int slot = 0;
    uint32_t phase = 0;
    for (; now.t < a.tokens; now.next(step_t, step_s, a.slabs)) {
        mbar_wait(smem_addr(bar + slot), phase, &abort_s, a.status);
        const int v = now.s * G + tid;
        const uint8_t* s = ring + static_cast<size_t>(slot) * slot_bytes;
        const float* meta = reinterpret_cast<const float*>(s + a.topk * piece);
        const int n = reinterpret_cast<const int*>(meta)[MOE_MAX_TOPK];
        if (v < a.vecs) {
            float2 acc[V / 2];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) acc[e] = both(0.0f);
#pragma unroll 8
            for (int j = 0; j < n; ++j) {
                Pack<T, V> x;
                x.raw = *reinterpret_cast<const uint4*>(s + j * piece + tid * 16);
                const float2 w = both(meta[j]);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) acc[e] = fma2(w, x.pair(e), acc[e]);
            }
            Pack<T, V> o;
#pragma unroll
            for (int e = 0; e < V / 2; ++e) o.set_pair(e, acc[e]);
            *reinterpret_cast<uint4*>(a.out + (now.t * a.vecs + v) * 16) = o.raw;
        }
        if (G == 32) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(G) : "memory");
        if (tid < 32) issue(slot);
        if (++slot == a.depth) {
            slot = 0;
            phase ^= 1u;
        }
    }
    if (*static_cast<volatile int*>(&abort_s) && tid == 0)   // a wait gave up: let the loads under way land
        for (int d = 0; d < a.depth; ++d) {
            const uint32_t n = (issued + a.depth - 1 - d) / a.depth;
            if (n > 0) mbar_wait(smem_addr(bar + d), (n - 1) & 1u, nullptr, a.status);
        }
}

// One warp per pair: dy[pos] = w * dout[t] and dw = <dout[t], y[pos]>.  The pairs of one token are
// neighbouring warps, so that dout comes from DRAM once.  The warps past the pairs zero the rows
// that belong to no pair, 32 rows each.
template <class T, bool ANY>
__global__ void __launch_bounds__(256)
    combine_backward_kernel(const T* __restrict__ dout, int64_t ldo, const T* __restrict__ y, int64_t ldy,
                            const int32_t* __restrict__ pos, const int32_t* __restrict__ pair_ids,
                            const float* __restrict__ w, int64_t P, int topk, int H, int vecs, int64_t num_rows,
                            T* __restrict__ dy, float* __restrict__ dw, uint32_t* status) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t p = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (p >= P) {
        const int64_t r0 = (p - P) * 32;
        if (r0 >= num_rows) return;
        uint32_t empty = __ballot_sync(0xffffffffu, r0 + lane < num_rows && pair_ids[r0 + lane] < 0);
        Pack<T, V> z;
        z.zero();
        while (empty) {
            const int64_t r = r0 + __ffs(empty) - 1;
            empty &= empty - 1;
            T* dr = dy + r * H;
            for (int v = lane; v < vecs; v += 32) {
                if constexpr (ANY) store_whole(dr, H, vector_any(dr, v), z.raw);
                else z.store(dr + v * V);
            }
        }
        return;
    }
    const int64_t r = pos[p];
    if (r < 0 || r >= num_rows) {
        if (lane == 0) {
            dw[p] = 0.0f;
            if (r >= num_rows) status_set(status, MOE_STATUS_BAD_EXPERT_ID);
        }
        return;
    }
    const float wp = w ? w[p] : 1.0f;
    const T* o = dout + p / topk * ldo;
    const T* yr = y + r * ldy;
    T* dr = dy + r * H;
    float dot = 0.0f;
    if constexpr (ANY)
        if (!inner_row(p / topk, P / topk) || !inner_row(r, num_rows)) {
            for (int v = lane; v < vecs; v += 32) {
                const int e0 = vector_any(dr, v);
                Pack<T, V> a, b, d;
                a.raw = load_elements(o, H, e0);
                b.raw = load_elements(yr, H, e0);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    dot = fmaf(a.get(e), b.get(e), dot);
                    d.set(e, wp * a.get(e));
                }
                store_whole(dr, H, e0, d.raw);
            }
            vecs = 0;
        }
    constexpr int U = 4, LANES = ANY ? kAnyLanes : 32;
    for (int v0 = 0; v0 < vecs; v0 += LANES * U) {
        Pack<T, V> a[U], b[U];
        const int first = ANY ? vector_any(dr, v0 + lane) : (v0 + lane) * V;   // element
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e0 = first + u * LANES * V;
            if constexpr (ANY) {
                a[u].raw = load_around(o, H, e0);
                b[u].raw = load_around(yr, H, e0);
            } else if (e0 < H) {
                a[u].load(o + e0);
                b[u].load(yr + e0);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e0 = first + u * LANES * V;
            if constexpr (ANY) {
                if (v0 + u * LANES >= vecs) break;
                const int n = lane < kAnyLanes ? H : 0;
                a[u].raw = inside_row<T>(join_lanes(a[u].raw, o + e0), n, e0);
                b[u].raw = inside_row<T>(join_lanes(b[u].raw, yr + e0), n, e0);
            } else if (e0 >= H) {
                break;
            }
            Pack<T, V> d;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float g = a[u].get(e);
                dot = fmaf(g, b[u].get(e), dot);
                d.set(e, wp * g);
            }
            if constexpr (!ANY) d.store(dr + e0);
            else if (lane < kAnyLanes) store_whole(dr, H, e0, d.raw);
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
    if (lane == 0) dw[p] = dot;
}

// Whether rows of these addresses (bits: addresses and strides in bytes, or-ed) go in whole 16-byte vectors.
bool whole_rows(int64_t row_bytes, uintptr_t bits) { return ((bits | static_cast<uintptr_t>(row_bytes)) & 15) == 0; }

struct DispatchPlan {
    int chunk, nch;
    bool direct;
};
// Chunks of whole tokens, about one per SM, so that every SM copies; few pairs: no counting launch.
DispatchPlan dispatch_plan(int64_t P, int topk) {
    DispatchPlan d;
    const int64_t T = P / topk;
    const int64_t per = (T + kPlanSms - 1) / kPlanSms;
    d.chunk = static_cast<int>(per * topk);
    d.nch = static_cast<int>((P + d.chunk - 1) / d.chunk);
    d.direct = P <= kDirectPairs;
    return d;
}

size_t dispatch_smem(int E) { return (2 * E + kSortThreads) * 4 + 32 * static_cast<size_t>(E) * 2 + 4; }

template <class R>
cudaError_t launch_dispatch(const DispatchArgs& a, dim3 grid, cudaStream_t stream) {
    return launch_pdl(dispatch_kernel<R, false>, grid, dim3(kSortThreads), dispatch_smem(a.E), stream, a);
}
// With bulk copies: one CTA per SM, what the sort leaves of its shared memory divided among the
// copying warps.
cudaError_t launch_dispatch_bulk(DispatchArgs a, dim3 grid, cudaStream_t stream) {
    const int row_bytes = a.vecs * 16, pieces = (row_bytes + kMostPiece - 1) / kMostPiece;
    a.piece = ((row_bytes + pieces - 1) / pieces + 15) / 16 * 16;
    a.ring = static_cast<int>((dispatch_smem(a.E) + 127) / 128 * 128);
    a.slots = (kSmemLimit - kStaticSmem - a.ring) / (kCopyWarps * a.piece);
    if (a.slots > kMostSlots) a.slots = kMostSlots;
    return launch_pdl(dispatch_kernel<uint4, true>, grid, dim3(kSortThreads),
                      static_cast<size_t>(a.ring) + static_cast<size_t>(kCopyWarps) * a.slots * a.piece, stream, a);
}

template <class T, bool ANY>
cudaError_t launch_combine(const void* y, int64_t ld, const int32_t* pos, const float* w, int64_t T_, int topk, int H,
                           int64_t num_rows, void* out, uint32_t* status, cudaStream_t stream) {
    if constexpr (ANY) {
        const int parts = (vectors_any<T>(H) + kAnyLanes - 1) / kAnyLanes;
        return launch_pdl(combine_any_kernel<T>, dim3(static_cast<unsigned>((T_ * parts + 7) / 8)), dim3(256), 0, stream,
                          static_cast<const T*>(y), ld, pos, w, static_cast<int>(T_), topk, H, parts,
                          static_cast<int>(num_rows), static_cast<T*>(out), status);
    }
    const int vecs = H / (16 / static_cast<int>(sizeof(T)));
    const int64_t n = T_ * vecs;
    return launch_pdl(combine_kernel<T>, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream,
                      static_cast<const T*>(y), ld, pos, w, T_, topk, vecs, num_rows, static_cast<T*>(out), status);
}

// Whether the ring takes a combine: two items or more for every group; and its launch.  (bf16, top-8, rows that are
// not in L2: 512 tokens of 2048 columns 5.7 us, 6.1 with vectors through registers; 512 of 7168 12.8 and 14.1; 256
// of 7168 7.9 and 7.7.  Of rows in L2 the ring is the slower one up to about 1024 tokens, by at most 1.1 us.)
bool combine_ring_shape(int64_t T_, int topk, int vecs, CombineArgs* a, int* groups) {
    int G = topk <= 8 ? 128 : topk <= 16 ? 64 : 32;
    while (G > 32 && G / 2 >= vecs) G /= 2;
    const int slot = topk * G * 16 + kCombineMeta;
    int R = kCombineThreads / G < kCombineGroups ? kCombineThreads / G : kCombineGroups;
    const int room = kSmemLimit - kStaticSmem;
    while (R > 1 && 2 * R * slot > room) --R;
    a->G = G;
    a->slabs = (vecs + G - 1) / G;
    a->depth = room / (R * slot) < kCombineDepth ? room / (R * slot) : kCombineDepth;
    *groups = R;
    return T_ * a->slabs >= 2ll * R * kPlanSms;
}
template <class T>
cudaError_t launch_combine_ring(const CombineArgs& a, int groups, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(groups) * a.depth * (a.topk * a.G * 16 + kCombineMeta);
    return launch_pdl(combine_ring_kernel<T>, dim3(kPlanSms), dim3(groups * a.G), smem, stream, a);
}

template <class T, bool ANY>
cudaError_t launch_combine_backward(const void* dout, int64_t ldo, const void* y, int64_t ldy, const int32_t* pos,
                                    const int32_t* pair_ids, const float* w, int64_t P, int topk, int H,
                                    int64_t num_rows, void* dy, float* dw, uint32_t* status, cudaStream_t stream) {
    const int64_t warps = P + (num_rows + 31) / 32;
    return launch_pdl(combine_backward_kernel<T, ANY>, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0,
                      stream, static_cast<const T*>(dout), ldo, static_cast<const T*>(y), ldy, pos, pair_ids, w, P,
                      topk, H, ANY ? vectors_any<T>(H) : H / (16 / static_cast<int>(sizeof(T))), num_rows,
                      static_cast<T*>(dy), dw, status);
}

// F<T, ANY> for the type and the rows' alignment
#define MOE_BY_TYPE(F, dtype, whole, ...)                                                                 \
    ((dtype) == MOE_DTYPE_FP32   ? ((whole) ? F<float, false>(__VA_ARGS__) : F<float, true>(__VA_ARGS__)) \
     : (dtype) == MOE_DTYPE_FP16 ? ((whole) ? F<__half, false>(__VA_ARGS__) : F<__half, true>(__VA_ARGS__)) \
                                 : ((whole) ? F<__nv_bfloat16, false>(__VA_ARGS__) : F<__nv_bfloat16, true>(__VA_ARGS__)))

int check_rows(int T, int topk, int H, int64_t ld, int64_t num_rows, int dtype) {
    if (T < 0 || topk < 1 || H < 1 || ld < H || num_rows < 0 || !known_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    if (topk > MOE_MAX_TOPK || H > MOE_MAX_HIDDEN || static_cast<int64_t>(T) * topk >= (int64_t(1) << 31) ||
        num_rows >= (int64_t(1) << 31) || static_cast<int64_t>(T) * H / 256 >= (int64_t(1) << 31))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

template <class T>
cudaError_t combine_ring_init() {
    return cudaFuncSetAttribute(combine_ring_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmemLimit - kStaticSmem);
}

}  // namespace

cudaError_t tokens_init_device() {
    const int bytes = static_cast<int>(dispatch_smem(MOE_MAX_EXPERTS));
    cudaError_t e = cudaFuncSetAttribute(dispatch_kernel<uint4, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(dispatch_kernel<uint32_t, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(dispatch_kernel<uint16_t, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(dispatch_kernel<uint4, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemLimit - kStaticSmem);
    if (e == cudaSuccess) e = combine_ring_init<float>();
    if (e == cudaSuccess) e = combine_ring_init<__half>();
    if (e == cudaSuccess) e = combine_ring_init<__nv_bfloat16>();
    return e;
}

}  // namespace mfp8

using namespace mfp8;

extern "C" {

size_t moe_dispatch_workspace_size(int T, int topk, int E) {
    if (T < 0 || topk < 1 || topk > MOE_MAX_TOPK || E < 1 || E > MOE_MAX_EXPERTS) return 0;
    const int64_t P = static_cast<int64_t>(T) * topk;
    if (P == 0 || P >= (int64_t(1) << 31)) return 0;   // (the plan counts pairs in ints)
    const DispatchPlan d = dispatch_plan(P, topk);
    return d.direct ? 0 : static_cast<size_t>(d.nch) * E * 4;
}

int moe_dispatch(const void* x, int64_t ldx, int dtype, const int32_t* topk_ids, int T, int topk, int E, int H,
                 void* rows, int32_t* expert_offsets, int32_t* pair_ids, int32_t* pos, void* workspace,
                 size_t workspace_bytes, void* stream) {
    int rc = check_rows(T, topk, H, ldx, 0, dtype);
    if (rc != MOE_OK) return rc;
    if (E < 1) return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t P = static_cast<int64_t>(T) * topk;
    if (!expert_offsets || (P > 0 && (!x || !topk_ids || !rows || !pair_ids || !pos))) return MOE_ERR_INVALID_ARG;
    if (!on_element(address(x) | address(rows), dtype_bytes(dtype))) return MOE_ERR_INVALID_ARG;
    const size_t need = moe_dispatch_workspace_size(T, topk, E);
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (need > 0 && !workspace) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (P == 0) return cuda_status(cudaMemsetAsync(expert_offsets, 0, (static_cast<size_t>(E) + 1) * 4, s));
    const DispatchPlan d = dispatch_plan(P, topk);
    const int es = static_cast<int>(dtype_bytes(dtype));
    const int64_t row_bytes = static_cast<int64_t>(H) * es;
    const bool whole = whole_rows(row_bytes, address(x) | address(rows) | static_cast<uintptr_t>(ldx * es));
    DispatchArgs a;
    a.x = static_cast<const char*>(x);
    a.ld_bytes = ldx * es;
    a.ids = topk_ids;
    a.P = P;
    a.topk = topk;
    a.E = E;
    a.chunk = d.chunk;
    a.nch = d.nch;
    a.counts = d.direct ? nullptr : static_cast<const int32_t*>(workspace);
    a.H = H;
    a.vecs = whole ? static_cast<int>(row_bytes / 16) : es == 4 ? vectors_any<uint32_t>(H) : vectors_any<uint16_t>(H);
    // few tokens: several CTAs share a chunk, each with a slab of at least 128 vectors of the columns
    int slabs = kPlanSms / d.nch;
    if (slabs > (a.vecs + 127) / 128) slabs = (a.vecs + 127) / 128;
    if (slabs < 1) slabs = 1;
    a.slab = (a.vecs + slabs - 1) / slabs;
    slabs = (a.vecs + a.slab - 1) / a.slab;
    a.rows = static_cast<char*>(rows);
    a.expert_offsets = expert_offsets;
    a.pair_ids = pair_ids;
    a.pos = pos;
    a.status = status;
    cudaError_t e = cudaSuccess;
    if (!d.direct)
        e = launch_pdl(pair_count_kernel, dim3(static_cast<unsigned>(d.nch)), dim3(kSortThreads), 0, s, topk_ids, P,
                       d.chunk, E, static_cast<int32_t*>(workspace));
    const dim3 grid(static_cast<unsigned>(d.nch), static_cast<unsigned>(slabs));
    if (e == cudaSuccess) {
        e = !whole      ? es == 4 ? launch_dispatch<uint32_t>(a, grid, s) : launch_dispatch<uint16_t>(a, grid, s)
            : slabs > 1 ? launch_dispatch<uint4>(a, grid, s)
                        : launch_dispatch_bulk(a, grid, s);
    }
    return cuda_status(e);
}

int moe_combine(const void* y, int64_t ldy, int dtype, const int32_t* pos, const float* weights, int T, int topk,
                int H, int64_t num_rows, void* out, void* stream) {
    int rc = check_rows(T, topk, H, ldy, num_rows, dtype);
    if (rc != MOE_OK) return rc;
    if (T == 0) return MOE_OK;
    if (!pos || !out || (num_rows > 0 && !y)) return MOE_ERR_INVALID_ARG;
    if (!on_element(address(y) | address(out), dtype_bytes(dtype))) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    const int es = static_cast<int>(dtype_bytes(dtype));
    const bool whole = whole_rows(static_cast<int64_t>(H) * es,
                                  address(y) | address(out) | static_cast<uintptr_t>(ldy * es));
    if (whole) {
        CombineArgs a = {};
        int groups = 0;
        a.vecs = H * es / 16;
        if (combine_ring_shape(T, topk, a.vecs, &a, &groups)) {
            a.y = static_cast<const char*>(y);
            a.ld_bytes = ldy * es;
            a.pos = pos;
            a.w = weights;
            a.tokens = T;
            a.topk = topk;
            a.num_rows = num_rows;
            a.out = static_cast<char*>(out);
            a.status = status;
            cudaStream_t s = static_cast<cudaStream_t>(stream);
            return cuda_status(dtype == MOE_DTYPE_FP32   ? launch_combine_ring<float>(a, groups, s)
                               : dtype == MOE_DTYPE_FP16 ? launch_combine_ring<__half>(a, groups, s)
                                                         : launch_combine_ring<__nv_bfloat16>(a, groups, s));
        }
    }
    return cuda_status(MOE_BY_TYPE(launch_combine, dtype, whole, y, ldy, pos, weights, T, topk, H, num_rows, out, status,
                                   static_cast<cudaStream_t>(stream)));
}

int moe_dispatch_backward(const void* drows, int64_t lddrows, int dtype, const int32_t* pos, int T, int topk, int H,
                          int64_t num_rows, void* dx, void* stream) {
    return moe_combine(drows, lddrows, dtype, pos, nullptr, T, topk, H, num_rows, dx, stream);
}

int moe_combine_backward(const void* dout, int64_t lddout, const void* y, int64_t ldy, int dtype, const int32_t* pos,
                         const int32_t* pair_ids, const float* weights, int T, int topk, int H, int64_t num_rows,
                         void* dy, float* dweights, void* stream) {
    int rc = check_rows(T, topk, H, ldy, num_rows, dtype);
    if (rc != MOE_OK) return rc;
    if (lddout < H) return MOE_ERR_INVALID_ARG;
    const int64_t P = static_cast<int64_t>(T) * topk;
    if (P == 0 && num_rows == 0) return MOE_OK;
    if (P > 0 && (!dout || !pos || !dweights)) return MOE_ERR_INVALID_ARG;
    if (num_rows > 0 && (!y || !dy || !pair_ids)) return MOE_ERR_INVALID_ARG;
    if (!on_element(address(dout) | address(y) | address(dy), dtype_bytes(dtype))) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    const int es = static_cast<int>(dtype_bytes(dtype));
    const bool whole = whole_rows(static_cast<int64_t>(H) * es,
                                  address(dout) | address(y) | address(dy) | static_cast<uintptr_t>(lddout * es) |
                                      static_cast<uintptr_t>(ldy * es));
    return cuda_status(MOE_BY_TYPE(launch_combine_backward, dtype, whole, dout, lddout, y, ldy, pos, pair_ids, weights, P,
                                   topk, H, num_rows, dy, dweights, status, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
