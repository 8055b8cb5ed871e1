// The router in its training form, one warp to a token: the choice of experts with the loads and losses that it
// is trained by, and the gradient of the logits ("router — top-K router", page "Quantization and MoE Optimizations",
// section FusedMoE Class; the grouped variant of section Key Environment Variables).
//
//   score  s = softmax(l) or sigmoid(l), key = s + bias (order of the logits where there is no bias)
//   groups a group's value is its largest key or the sum of its two largest; the best groups stay
//   choice the k largest keys, ties to the lower expert; an expert of logit -inf is never chosen
//   weight w_j = c s_j / (sum over the chosen) or c s_j
//   loads  counts_e, n tokens that chose; P = s / sum(s): balance = sum_e (E counts_e / (k n)) mean_t(P_te);
//          z = mean_t(logsumexp(l_t)^2)
// Gradient, q = w / c, g = c dw, phi = 1 (softmax) or 1 - s (sigmoid):
//   renormalised  dl_j = phi_j q_j (g_j - sum q g);   else  softmax: dl_e = s_e (g_e - sum s g), sigmoid: dl_j = phi_j s_j g_j
//   balance a     dl_e += phi_e P_e (h_e - sum P h), h_e = a E counts_e / (k n^2);   z b  dl_e += 2 b lse s_e / n
//
// The choice is that of fp64 keys: they are formed in fp32, and where two of them that a decision compares are closer than their
// error (and not of the same logit and bias) the token's choice is repeated in fp64.  Keys that are equal there are ordered by
// their logits and then their biases, groups by their scores without the bias and what these leave to 1: where a score is lost in
// the bias, or is 1 to fp64's last bit (sigmoid from 37 on), that is the order of the real numbers if the biases are the same.
//
// Lanes hold V experts each in registers.  Where a token's experts fit eight lanes and there are many tokens, a warp takes four
// at a time, so that most instructions work for four tokens; else a token has a warp.  The lanes are dealt to the groups, a
// power of two of them to a group, so that a group's value is found among its lanes (a lane may then hold fewer than V
// experts); slot lane V + v is expert v of the lane.  The choice: keys from the k-th largest of the largest of 32 parts of the
// experts on hold the k largest and are hardly more; they are gathered in shared memory, and each counts the ones ahead of
// it.  Of four tokens, one whose keys are too near, or with too many that are equal, is taken by the whole warp afterwards.
// A token is one long chain of such steps, so the bound is how many of them an SM has under way and the instructions of a
// token: everything that a warp keeps across tokens but its score sums lies in shared memory, and 24 or 32 warps of 80 or 64
// registers fit.  Score sums are added across warps, then blocks (a last small launch) in a fixed order; the loads are
// integers.
//
// Measured (GB300; choice alone, with loads and losses, gradient, gradient with the losses'), us:
//   58368 x 256 fp32, sigmoid, bias, 4 of 8 groups, 8 experts    59, 66, 18, 33   (the bytes: 9, 9, 9, 18)
//   58368 x 128 bf16, softmax, 8 experts                         19, 26, 8, 14    (2.8, 2.8, 2.8, 4.5)
//   152 x 256 as the first                                       4, 9, 2.4, 3.7   (launches)
// The choice issues an instruction in 54% of the cycles with 24 warps to an SM and waits for shuffles and shared memory in
// between; DRAM is below 20%.
#pragma once

#include <type_traits>

#include "train.cuh"

namespace mfp8 {

constexpr int router_warps(int V, int L) {   // of a block, one block to an SM
    return V <= 4 || (V == 8 && L == 8) ? 32 : V == 8 || (V == 16 && L == 8) ? 24 : V == 16 ? 16 : V == 32 ? 8 : 2;
}
constexpr int kNearest = 24, kSorted = 16;   // gathered keys of a token, and sorted ones
constexpr int kBackwardWarps = 8;

struct RouterArgs {
    const void* logits;
    int64_t ld;
    int T, E, k;
    int sigmoid, groups, kept, top2, renorm;
    float scaling;
    const float* bias;
    const uint8_t* valid;
    int32_t* ids;
    float* weights;
    // loads and losses: [blocks][E] each, [blocks] each (null: not wanted)
    float* part_share;
    int32_t* part_count;
    float* part_z;
    int32_t* part_live;
    uint32_t* status;
    int vector;                // rows can be loaded V elements at a time
    int lanes;                 // of a group (of the L lanes of a token)
};

struct RouterBackwardArgs {
    const void* logits;
    int64_t ld;
    int T, E, k;
    int sigmoid, renorm;
    float scaling;
    const int32_t* ids;
    const float* dweights;
    const int32_t* counts;     // with balance
    const int32_t* live;       // number of tokens that chose; with balance or z
    float balance, z;
    void* dlogits;             // [T, E] dense
    uint32_t* status;
    int vector, vector_out;
};

// One type to a translation unit (router_*.cu).  blocks: of the grid.
template <class T>
cudaError_t router_forward(const RouterArgs& a, int blocks, cudaStream_t stream);
template <class T>
cudaError_t router_backward(const RouterBackwardArgs& a, cudaStream_t stream);

#ifdef MOE_ROUTER_KERNELS
// Rows that can be loaded V elements at a time: E a multiple of V, addresses of the vectors (32 bytes at most).
template <class T>
bool router_vectors(const void* p, int64_t ld, int E, int V) {
    const int64_t size = V * static_cast<int64_t>(sizeof(T)), bytes = size < 32 ? size : 32;
    return E % V == 0 && address(p) % bytes == 0 && ld * static_cast<int64_t>(sizeof(T)) % bytes == 0;
}
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kNone = -INFINITY;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
// Sum over the first k lanes (the others hold 0), the same in every lane.
__device__ __forceinline__ float chosen_sum(float v, int k) {
    if (k > 8) {
        v += __shfl_xor_sync(kAll, v, 16);
        v += __shfl_xor_sync(kAll, v, 8);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return __shfl_sync(kAll, v, 0);
}
// fp32 as integers of the same order, both zeros alike.
__device__ __forceinline__ uint32_t ordered(float v) {
    const int b = __float_as_int(v + 0.0f);
    return static_cast<uint32_t>(b ^ ((b >> 31) | INT32_MIN));
}
__device__ __forceinline__ float of_ordered(uint32_t u) {
    return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}

// (No NaN.)
__device__ __forceinline__ float warp_max(float v) { return of_ordered(__reduce_max_sync(kAll, ordered(v))); }

// V logits from p on, those past `count` -inf (vector: count is 0 or V).
template <class T, int V>
struct Logits {
    static constexpr int kBytes = V * static_cast<int>(sizeof(T));
    static constexpr int kWords = kBytes >= 16 ? kBytes / 16 : 1;
    using Word = typename std::conditional<kBytes >= 16, uint4,
                 typename std::conditional<kBytes == 8, uint2, typename std::conditional<kBytes == 4, uint32_t, uint16_t>::type>::type>::type;
    union {
        Word w[kWords];
        uint32_t u[kBytes >= 4 ? kBytes / 4 : 1];
        T e[V];
    };
    __device__ __forceinline__ Logits() {}
    __device__ __forceinline__ void load(const T* p, int count, bool vector) {
        if (vector && count > 0) {
            if constexpr (kBytes % 32 == 0) {   // whole sectors
#pragma unroll
                for (int i = 0; i < kBytes / 4; i += 8)
                    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                                 : "=r"(u[i]), "=r"(u[i + 1]), "=r"(u[i + 2]), "=r"(u[i + 3]), "=r"(u[i + 4]), "=r"(u[i + 5]),
                                   "=r"(u[i + 6]), "=r"(u[i + 7])
                                 : "l"(reinterpret_cast<const uint32_t*>(p) + i));
            } else {
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const Word*>(p) + i);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) e[v] = v < count ? p[v] : from_f32<T>(-INFINITY);
        }
    }
    __device__ __forceinline__ void store(T* p, int count, bool vector) const {
        if (vector) {
            if (count <= 0) return;
            if constexpr (kBytes % 32 == 0) {
#pragma unroll
                for (int i = 0; i < kBytes / 4; i += 8)
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                                     reinterpret_cast<uint32_t*>(p) + i),
                                 "r"(u[i]), "r"(u[i + 1]), "r"(u[i + 2]), "r"(u[i + 3]), "r"(u[i + 4]), "r"(u[i + 5]),
                                 "r"(u[i + 6]), "r"(u[i + 7])
                                 : "memory");
            } else {
#pragma unroll
                for (int i = 0; i < kWords; ++i) reinterpret_cast<Word*>(p)[i] = w[i];
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v < count) p[v] = e[v];
        }
    }
};

// A lane's logits; NaN and +inf count as -inf (true in *odd).
template <class T, int V>
__device__ __forceinline__ void finite_logits(const Logits<T, V>& raw, float (&l)[V], bool* odd) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float x = to_f32(raw.e[v]);
        l[v] = x < INFINITY ? x : kNone;
        *odd |= !(x < INFINITY);
    }
}
constexpr uint32_t kLeastKey = 0x00800000u;   // of a finite number; -inf is below

// Accurate where it vanishes, too.
__device__ __forceinline__ float sigmoid32(float l) {
    const float e = expf(-fabsf(l));
    return __fdividef(l < 0.0f ? e : 1.0f, 1.0f + e);
}

// The choice on fp64 keys, compared as ordered integers (fp64 instructions are a 64th of the others' rate here).  Returns on
// lane j < k the j-th expert or -1.
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return b ^ (b >> 63 ? ~uint64_t(0) : uint64_t(1) << 63);
}
__device__ __forceinline__ double of_ordered(uint64_t u) {
    return __longlong_as_double(static_cast<long long>(u >> 63 ? u ^ (uint64_t(1) << 63) : ~u));
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, static_cast<uint64_t>(__shfl_xor_sync(kAll, static_cast<unsigned long long>(v), o)));
    return v;
}
// exp(x) in fp64 for x <= 0, to a few 2^-53 of itself: x = n ln2 / 32 + r, 2^(n / 32) from a table and exp(r) by its series
// (|r| < 0.011: the sixth power's term is the last above 2^-55; a table-driven exponential after Tang, ACM TOMS 15, 1989).
// A third of the fp64 instructions of exp(), which has more to take care of.  Below 2^-1000: 0.
__device__ const double kPowers[32] = {
    0x1.0000000000000p+0, 0x1.059b0d3158574p+0, 0x1.0b5586cf9890fp+0, 0x1.11301d0125b51p+0,
    0x1.172b83c7d517bp+0, 0x1.1d4873168b9aap+0, 0x1.2387a6e756238p+0, 0x1.29e9df51fdee1p+0,
    0x1.306fe0a31b715p+0, 0x1.371a7373aa9cbp+0, 0x1.3dea64c123422p+0, 0x1.44e086061892dp+0,
    0x1.4bfdad5362a27p+0, 0x1.5342b569d4f82p+0, 0x1.5ab07dd485429p+0, 0x1.6247eb03a5585p+0,
    0x1.6a09e667f3bcdp+0, 0x1.71f75e8ec5f74p+0, 0x1.7a11473eb0187p+0, 0x1.82589994cce13p+0,
    0x1.8ace5422aa0dbp+0, 0x1.93737b0cdc5e5p+0, 0x1.9c49182a3f090p+0, 0x1.a5503b23e255dp+0,
    0x1.ae89f995ad3adp+0, 0x1.b7f76f2fb5e47p+0, 0x1.c199bdd85529cp+0, 0x1.cb720dcef9069p+0,
    0x1.d5818dcfba487p+0, 0x1.dfc97337b9b5fp+0, 0x1.ea4afa2a490dap+0, 0x1.f50765b6e4540p+0};
__device__ __forceinline__ double exp64(double x) {
    const double magic = 0x1.8p52;
    const double t = fma(x, 0x1.71547652b82fep+5, magic), n = t - magic;
    const int k = __double2loint(t);
    double r = fma(n, -0x1.62e42fee00000p-6, x);   // the first part of ln2 / 32 has 32 bits: exact
    r = fma(n, -0x1.a39ef35793c76p-38, r);
    double p = fma(r, 1.0 / 720.0, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p * r, r, r);
    const double power = kPowers[k & 31], value = fma(power, p, power);
    const int up = k >> 5;
    return x < -693.0 ? 0.0 : __hiloint2double(__double2hiint(value) + up * (1 << 20), __double2loint(value));
}

__device__ __forceinline__ double sigmoid64(double x) {
    const double e = exp64(-fabs(x));
    return (x < 0.0 ? e : 1.0) / (1.0 + e);
}

// Orders equal fp64 keys: the larger logit first, then the larger bias.
__device__ __forceinline__ uint64_t tie_key(float l, float b) { return static_cast<uint64_t>(ordered(l)) << 32 | ordered(b); }

// A key t and its tie_key p among the two largest so far.
__device__ __forceinline__ void two_best(uint64_t t, uint64_t p, uint64_t& t1, uint64_t& p1, uint64_t& t2, uint64_t& p2) {
    const bool top = t > t1 || (t == t1 && p > p1);
    if (top || t > t2 || (t == t2 && p > p2)) t2 = top ? t1 : t, p2 = top ? p1 : p;
    if (top) t1 = t, p1 = p;
}
// Whether the last group that stays and the first that does not have the same value, *meet (by a whole warp; of the lanes that
// are `real`, each place is one group's).
__device__ __forceinline__ bool border_ties(uint64_t value, int place, int kept, bool real, uint64_t* meet) {
    const uint32_t last = __ballot_sync(kAll, real && place == kept - 1);
    const uint32_t out = __ballot_sync(kAll, real && place == kept);
    if (last == 0u || out == 0u) return false;   // (the same in every lane)
    *meet = __shfl_sync(kAll, static_cast<unsigned long long>(value), __ffs(static_cast<int>(last)) - 1);
    const uint64_t next = __shfl_sync(kAll, static_cast<unsigned long long>(value), __ffs(static_cast<int>(out)) - 1);
    return *meet == next && next != 0;
}

// The places of groups of which some at the border have the same fp64 value, meet: as they are, if it is by the same logits and
// biases (16-bit logits often meet), else by the scores of their two best experts, and then by what these leave to 1 (scores that vanish
// or reach 1).
template <int V, bool SIGMOID>
__device__ __noinline__ int tied_place(const float* l, const uint64_t* key, float m, const RouterArgs& a, int first, int lanes,
                                       uint64_t mine, uint64_t meet, int place) {
    const int own = (threadIdx.x & 31) / lanes;
    uint64_t t1 = 0, t2 = 0, p1 = 0, p2 = 0;   // the two largest keys and their tie_key
    const auto join = [&](uint64_t t, uint64_t p) { two_best(t, p, t1, p1, t2, p2); };
    for (int v = 0; v < V; ++v)
        if (key[v] != 0) join(key[v], tie_key(l[v], a.bias ? a.bias[first + v] : 0.0f));
    for (int o = 1; o < lanes; o <<= 1) {
        const uint64_t u1 = __shfl_xor_sync(kAll, static_cast<unsigned long long>(t1), o), u2 = __shfl_xor_sync(kAll, static_cast<unsigned long long>(t2), o);
        const uint64_t q1 = __shfl_xor_sync(kAll, static_cast<unsigned long long>(p1), o), q2 = __shfl_xor_sync(kAll, static_cast<unsigned long long>(p2), o);
        join(u1, q1);
        join(u2, q2);
    }
    if (!a.top2) t2 = p2 = 0;
    const bool equal = own < a.groups && mine == meet;
    const int src = __ffs(static_cast<int>(__ballot_sync(kAll, equal))) - 1;
    const uint64_t r1 = __shfl_sync(kAll, static_cast<unsigned long long>(p1), src), r2 = __shfl_sync(kAll, static_cast<unsigned long long>(p2), src);
    if (!__any_sync(kAll, equal && (p1 != r1 || p2 != r2))) return place;
    const double x1 = of_ordered(static_cast<uint32_t>(p1 >> 32)), x2 = of_ordered(static_cast<uint32_t>(p2 >> 32));
    const bool one = t1 != 0, two = t2 != 0;
    const auto score = [&](double x) { return SIGMOID ? sigmoid64(x) : exp64(x - m); };
    const uint64_t sum = ordered((one ? score(x1) : 0.0) + (two ? score(x2) : 0.0));
    const uint64_t rest = SIGMOID ? ~ordered((one ? sigmoid64(-x1) : 0.0) + (two ? sigmoid64(-x2) : 0.0)) : 0;
    place = 0;
    for (int g = 0; g < a.groups; ++g) {
        const uint64_t o = __shfl_sync(kAll, static_cast<unsigned long long>(mine), g * lanes);
        const uint64_t os = __shfl_sync(kAll, static_cast<unsigned long long>(sum), g * lanes);
        const uint64_t orest = __shfl_sync(kAll, static_cast<unsigned long long>(rest), g * lanes);
        place += o != mine ? o > mine : os != sum ? os > sum : orest != rest ? orest > rest : g < own;
    }
    return place;
}

template <int V, bool SIGMOID>
__device__ __noinline__ int choose_exact(const float* l, float m, const RouterArgs& a, int first, int count, int lanes) {
    const int lane = threadIdx.x & 31;
    uint64_t key[V];   // 0: not to be chosen
    double s[V], z = 1.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const double x = l[v];
        s[v] = l[v] == kNone ? 0.0 : exp64(SIGMOID ? -fabs(x) : x - m);
    }
    if (!SIGMOID) {
        z = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) z += s[v];
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const double b = a.bias && v < count ? static_cast<double>(a.bias[first + v]) : 0.0;
        key[v] = l[v] == kNone || b == static_cast<double>(kNone)
                     ? 0u
                     : ordered((SIGMOID ? (l[v] < 0.0f ? s[v] : 1.0) / (1.0 + s[v]) : s[v] / z) + b);
    }
    if (a.groups > 1) {
        uint64_t t1 = 0, t2 = 0;
        const auto join = [&](uint64_t u1, uint64_t u2) {
            t2 = max(min(t1, u1), max(t2, u2));
            t1 = max(t1, u1);
        };
#pragma unroll
        for (int v = 0; v < V; ++v) join(key[v], 0);
        for (int o = 1; o < lanes; o <<= 1) {
            const uint64_t u1 = __shfl_xor_sync(kAll, static_cast<unsigned long long>(t1), o);
            const uint64_t u2 = __shfl_xor_sync(kAll, static_cast<unsigned long long>(t2), o);
            join(u1, u2);
        }
        const uint64_t mine = a.top2 && t2 > 0 ? ordered(of_ordered(t1) + of_ordered(t2)) : t1;
        const int own = lane / lanes;
        int place = 0;
        for (int g = 0; g < a.groups; ++g) {
            const uint64_t o = __shfl_sync(kAll, static_cast<unsigned long long>(mine), g * lanes);
            place += o > mine || (o == mine && g < own);
        }
        uint64_t meet = 0;
        if (border_ties(mine, place, a.kept, own < a.groups, &meet)) {
            uint64_t copy[V];   // (so that the keys stay in registers)
#pragma unroll
            for (int v = 0; v < V; ++v) copy[v] = key[v];
            place = tied_place<V, SIGMOID>(l, copy, m, a, first, lanes, mine, meet, place);
        }
        if (own >= a.groups || place >= a.kept) {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = 0;
        }
    }
    int id = -1;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) best = max(best, key[v]);
        const uint64_t top = warp_max(best);
        if (top == 0) break;
        int at = 0, equal = 0;
#pragma unroll
        for (int v = V - 1; v >= 0; --v) {
            if (key[v] == top) at = v;
            equal += key[v] == top ? 1 : 0;
        }
        bool has = best == top;
        if (__reduce_add_sync(kAll, equal) > 1) {
            uint64_t tie = 0;
#pragma unroll
            for (int v = V - 1; v >= 0; --v) {
                if (key[v] == top) {
                    const uint64_t p = tie_key(l[v], a.bias ? a.bias[first + v] : 0.0f);
                    if (p >= tie) at = v;
                    tie = max(tie, p);
                }
            }
            const uint64_t first_of = warp_max(tie);
            has = has && tie == first_of;
        }
        const int src = __ffs(static_cast<int>(__ballot_sync(kAll, has))) - 1;
        const int e = __shfl_sync(kAll, first + at, src);
        if (lane == src) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v == at) key[v] = 0;
        }
        if (lane == j) id = e;
    }
    return id;
}

// More than the error of a difference of keys is key_slack() and kRel of the larger.  A score is off by 2^-22.4 of itself (the
// quotient, a sum) and by its exponential: 2^-22 and 1.44 * 2^-24 of the exponent d, that is by less than 2^-23.5 (sigmoid:
// s (1 - s) <= 1/4, s (1 - s) d < 0.23) or 2^-24 of the largest score (softmax: d e^-d < 0.37) and 2^-22 of itself; a score is at most
// the key and b_most, so kRel and 2^-20 b_most cover what goes by the score.  Softmax scores share a factor, the sum's: in units of
// 2^-24 its V + 4 additions (V experts a lane, five exchanges), its exponentials' 4 and 1.44 of the entropy (10 at most), and its
// reciprocal's 4.  That counts by the difference of the scores, at most 2 b_most over the keys'.
constexpr float kRel = 0x1p-20f;
template <int V, bool SIGMOID>
__device__ __forceinline__ float key_slack(float b_most, float per) {
    constexpr float kShared = 2 * (V + 22) * 0x1p-24f;
    return (SIGMOID ? 0x1p-20f : 0x1p-20f + kShared) * b_most + (SIGMOID ? 0x1p-22f : 0x1p-22f * per);
}
// Scores from logits (softmax: times z, m the largest logit); exp(-inf) = 0: one that cannot be chosen has score 0.  __expf and
// __fdividef are off by 2 ulp each and by |x| 2^-24 of the exponent, in place of expf's and the division's 1 and 1/2.  It is within the
// slack, and what is summed of them is as near to 64 bits: shares' gradient 2.4e-7 in the 2-norm with either at 16384 x 256 sigmoid,
// 9.2e-8 and 8.9e-8 at 65536 x 128 softmax, the choice 20.3 and 23.0, 21.5 and 22.6 us.
template <bool SIGMOID>
__device__ __forceinline__ float score32(float l, float m) {
    if (!SIGMOID) return __expf(l - m);
    const float e = __expf(-fabsf(l));
    return __fdividef(l < 0.0f ? e : 1.0f, 1.0f + e);
}

// A group's value, of finite keys: held finite, so that it is not taken for that of a group without experts, nor two that overflow for
// far apart (equal or near, they are compared in fp64).
__device__ __forceinline__ float within_fp32(float v) { return fminf(fmaxf(v, -0x1.fffffep127f), 0x1.fffffep127f); }

// A sum of sigmoid scores below which they vanish (e^-69): there s is e^l to fp32's last bit, and shares are formed as e^(l - m), the
// largest logit's being 1, which no underflow reaches.
constexpr float kVanished = 1e-30f;

// The lane's place among 32 that take a token: its group, its first expert and how many it has.
struct Seat {
    int lanes, own, first, count;   // lanes: of a group
    __device__ __forceinline__ Seat(const RouterArgs& a, int V, int lanes_, int lane) : lanes(lanes_), own(lane / lanes_) {
        const int G = a.E / a.groups, inside = lane % lanes_ * V;
        first = own * G + inside;
        count = own < a.groups ? min(max(G - inside, 0), V) : 0;
    }
};

// Whether one of a lane's keys that are left (kNone: taken) is near the k-th largest, last, and of another logit or bias.
template <int V>
__device__ __noinline__ bool left_near(const float* keys, const float* l, const float* bias, float last, float l_last, float b_last,
                                       float slack) {
    bool near = false;
    for (int v = 0; v < V; ++v)
        near |= keys[v] > kNone && last - keys[v] <= slack + kRel * fmaxf(fabsf(last), fabsf(keys[v])) &&
                (l[v] != l_last || bias[v] != b_last);
    return near;
}

// The choice and the weights of token t by a whole warp, for its logits l, the largest m (some expert can be chosen).  s_bias:
// by slot; loads: null, or to be counted into; STATS: the shares are added to share, *lse is set.
template <class T, int V, bool SIGMOID, bool STATS>
__device__ __forceinline__ void route_warp(const RouterArgs& a, const T* logits, int64_t t, const Seat& seat, const float (&l)[V], float m,
                                           float b_most, const float* s_bias, int* loads, uint2* s_near, float (&share)[V],
                                           float* lse) {
    const int lane = threadIdx.x & 31, lanes = seat.lanes, own = seat.own, first = seat.first, count = seat.count;
    const uint32_t below = (1u << lane) - 1u;
    float s[V], per = 1.0f;
    const bool scored = a.bias || (a.groups > 1 && a.top2);
    if (scored || STATS || !SIGMOID) {
        float z = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = score32<SIGMOID>(l[v], m);
            z += s[v];
        }
        z = warp_sum(z);
        per = __fdividef(1.0f, fmaxf(z, 1e-37f));
        if constexpr (STATS) {
            if (SIGMOID && z < kVanished) {   // (the same in every lane)
                float u[V], sum = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) sum += u[v] = __expf(l[v] - m);
                sum = warp_sum(sum);
#pragma unroll
                for (int v = 0; v < V; ++v) share[v] += __fdividef(u[v], sum);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) share[v] = fmaf(s[v], per, share[v]);
            }
            *lse = SIGMOID ? 0.0f : m + logf(z);
        }
    }
    const float slack = key_slack<V, SIGMOID>(b_most, per);
    uint32_t key[V];
    if (scored) {   // s: keys as numbers
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = l[v] > kNone ? (SIGMOID ? s[v] : s[v] * per) + s_bias[lane * V + v] : kNone;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = l[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = ordered(a.bias ? s[v] : l[v]);
    bool close = false;
    if (a.groups > 1) {
        float t1 = kNone, t2 = kNone;
        const auto join = [&](float u1, float u2) {
            t2 = fmaxf(fminf(t1, u1), fmaxf(t2, u2));
            t1 = fmaxf(t1, u1);
        };
#pragma unroll
        for (int v = 0; v < V; ++v) join(s[v], kNone);
        for (int o = 1; o < lanes; o <<= 1) {
            const float u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
            join(u1, u2);
        }
        const float mine = a.top2 && t2 > kNone ? within_fp32(t1 + t2) : t1;
        const bool real = own < a.groups;
        int place = 0;
        for (int g = 0; g < a.groups; ++g) {
            const float o = __shfl_sync(kAll, mine, g * lanes);
            place += o > mine || (o == mine && g < own);
        }
        if (scored && a.kept < a.groups) {
            const float last = warp_max(real && place == a.kept - 1 ? mine : kNone);
            const float out = warp_max(real && place == a.kept ? mine : kNone);
            const float limit = 4.0f * slack + 2.0f * kRel * fmaxf(fabsf(last), fabsf(out));
            close = out > kNone && last - out <= limit;
            if (SIGMOID && close) {
                // the groups at the border by the fp64 keys of their two best (and what may be), a lane each
                const bool border = real && (fabsf(mine - last) <= limit || fabsf(mine - out) <= limit);
                const float best = a.top2 && t2 > kNone ? t2 : t1, low = best - (slack + kRel * fabsf(best));
                int found = 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const bool in = border && s[v] >= low;
                    const uint32_t all = __ballot_sync(kAll, in);
                    const int at = found + __popc(all & below);
                    if (in && at < 32) s_near[at] = make_uint2(first + v, own);
                    found += __popc(all);
                }
                __syncwarp();
                if (found <= 32) {
                    uint64_t wide = 0;
                    uint32_t group = 0xffffffffu;
                    if (lane < found) {
                        const uint32_t e = s_near[lane].x;
                        group = s_near[lane].y;
                        const double x64 = to_f32(logits[e]);
                        wide = ordered(sigmoid64(x64) + (a.bias ? static_cast<double>(a.bias[e]) : 0.0));
                    }
                    uint64_t u1 = 0, u2 = 0;
                    for (int i = 0; i < found; ++i) {
                        const uint64_t o = __shfl_sync(kAll, static_cast<unsigned long long>(wide), i);
                        if (__shfl_sync(kAll, group, i) == static_cast<uint32_t>(own)) {
                            u2 = max(min(u1, o), u2);
                            u1 = max(u1, o);
                        }
                    }
                    const uint64_t value = a.top2 && u2 > 0 ? ordered(of_ordered(u1) + of_ordered(u2)) : u1;
                    const uint32_t borders = __ballot_sync(kAll, border);
                    place = 0;
                    for (int g = 0; g < a.groups; ++g) {
                        const uint64_t o = __shfl_sync(kAll, static_cast<unsigned long long>(value), g * lanes);
                        const float of = __shfl_sync(kAll, mine, g * lanes);
                        const bool both = border && ((borders >> (g * lanes)) & 1u);
                        place += both ? o > value || (o == value && g < own) : of > mine || (of == mine && g < own);
                    }
                    close = false;
                    uint64_t meet = 0;
                    if (border_ties(value, place, a.kept, border, &meet)) {
                        // equal in fp64, too: alike, if it is by the same logits and biases, else decided by those
                        uint64_t tie = 0, t1 = 0, t2 = 0, p1 = 0, p2 = 0;
                        if (lane < found) {
                            const uint32_t e = s_near[lane].x;
                            tie = tie_key(to_f32(logits[e]), a.bias ? a.bias[e] : 0.0f);
                        }
                        for (int i = 0; i < found; ++i) {
                            const uint64_t o = __shfl_sync(kAll, static_cast<unsigned long long>(wide), i);
                            const uint64_t ot = __shfl_sync(kAll, static_cast<unsigned long long>(tie), i);
                            if (__shfl_sync(kAll, group, i) == static_cast<uint32_t>(own)) two_best(o, ot, t1, p1, t2, p2);
                        }
                        const bool equal = border && value == meet;
                        if (!a.top2) p2 = 0;
                        const int src = __ffs(static_cast<int>(__ballot_sync(kAll, equal))) - 1;
                        const uint64_t q1 = __shfl_sync(kAll, static_cast<unsigned long long>(p1), src);
                        const uint64_t q2 = __shfl_sync(kAll, static_cast<unsigned long long>(p2), src);
                        close = __any_sync(kAll, equal && (p1 != q1 || p2 != q2));
                    }
                }
                __syncwarp();
            }
        }
        if (!real || place >= a.kept) {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = 0u;
        }
    }
    const int need = a.bias ? a.k + 1 : a.k;
    uint32_t most = key[0], least = 1u;
#pragma unroll
    for (int v = 1; v < V; ++v) most = max(most, key[v]);
    for (int j = 0; j < need; ++j) {
        least = __reduce_max_sync(kAll, most);
        if (least < kLeastKey) break;
        if (most == least) most = 0u;
    }
    least = max(least, kLeastKey);
    if (a.bias && least > kLeastKey) {   // (keys in fp32: all that may be among them)
        const float low = of_ordered(least);
        least = max(ordered(low - (slack + kRel * fabsf(low))), kLeastKey);
    }
    int slot[V], found = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const uint32_t in = __ballot_sync(kAll, key[v] >= least);
        slot[v] = key[v] >= least ? found + __popc(in & below) : 32;
        found += __popc(in);
    }
    int id = -1;
    if (found <= 32) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (slot[v] < 32) s_near[slot[v]] = make_uint2(key[v], first + v);
        __syncwarp();
        const uint2 mine = lane < found ? s_near[lane] : make_uint2(0u, 0u);
        int place = 0;
        for (int i = 0; i < found; ++i) {
            const uint2 o = s_near[i];
            place += o.x > mine.x || (o.x == mine.x && o.y < mine.y);
        }
        __syncwarp();
        if (lane < found) s_near[place] = mine;
        __syncwarp();
        if (a.bias) {
            // each key of the first k with the one before it, and all others with the k-th: the next may be of the same logit
            // and bias as the k-th, and a nearer one behind it
            bool near = false;
            if (lane > 0 && lane < found) {
                const uint2 u = s_near[min(lane, a.k) - 1], n = s_near[lane];
                const float before = of_ordered(u.x), now = of_ordered(n.x);
                if (before - now <= slack + kRel * fmaxf(fabsf(before), fabsf(now)))
                    near = to_f32(logits[u.y]) != to_f32(logits[n.y]) || a.bias[u.y] != a.bias[n.y];
            }
            if (__any_sync(kAll, near)) {   // their order by fp64 keys, a lane each
                double all = 1.0;
                if (!SIGMOID) {
                    all = 0.0;
                    #pragma unroll
                    for (int v = 0; v < V; ++v) all += l[v] > kNone ? exp64(static_cast<double>(l[v]) - m) : 0.0;
                    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(kAll, all, o);
                }
                uint64_t wide = 0;
                float x = 0.0f, b = 0.0f;
                if (lane < found) {
                    x = to_f32(logits[mine.y]), b = a.bias[mine.y];
                    const double x64 = x;
                    const double s64 = SIGMOID ? sigmoid64(x64) : exp64(x64 - m) / all;
                    wide = ordered(s64 + static_cast<double>(b));
                }
                bool tied = false;   // (equal in fp64, too)
                place = 0;
                for (int i = 0; i < found; ++i) {
                    const uint64_t o = __shfl_sync(kAll, static_cast<unsigned long long>(wide), i);
                    const uint32_t oe = __shfl_sync(kAll, mine.y, i);
                    place += o > wide || (o == wide && oe < mine.y);
                    tied |= o == wide && i != lane;
                }
                if (__any_sync(kAll, tied)) {
                    const uint64_t tie = tie_key(x, b);
                    place = 0;
                    for (int i = 0; i < found; ++i) {
                        const uint64_t o = __shfl_sync(kAll, static_cast<unsigned long long>(wide), i);
                        const uint64_t ot = __shfl_sync(kAll, static_cast<unsigned long long>(tie), i);
                        const uint32_t oe = __shfl_sync(kAll, mine.y, i);
                        place += o != wide ? o > wide : ot != tie ? ot > tie : oe < mine.y;
                    }
                }
                __syncwarp();
                if (lane < found) s_near[place] = mine;
                __syncwarp();
            }
        }
        if (lane < a.k && lane < found) id = static_cast<int>(s_near[lane].y);
        __syncwarp();
    } else {   // many equal keys: one after the other
        float before = 0.0f;
        int before_id = -1;
        for (int j = 0; j < need; ++j) {
            most = key[0];
#pragma unroll
            for (int v = 1; v < V; ++v) most = max(most, key[v]);
            const uint32_t top = __reduce_max_sync(kAll, most);
            if (top < kLeastKey) break;
            const int src = __ffs(static_cast<int>(__ballot_sync(kAll, most == top))) - 1;
            int at = 0;
#pragma unroll
            for (int v = V - 1; v >= 0; --v)
                if (key[v] == top) at = v;
            const int e = __shfl_sync(kAll, first + at, src);
            if (a.bias && j == a.k) {
                const float now = of_ordered(top);
                if (before - now <= slack + kRel * fmaxf(fabsf(before), fabsf(now))) {   // (the same in every lane)
                    float keys[V], logit[V];   // (copies, so that the registers stay those of the loop above)
#pragma unroll
                    for (int v = 0; v < V; ++v) keys[v] = key[v] >= kLeastKey ? of_ordered(key[v]) : kNone, logit[v] = l[v];
                    const bool near = left_near<V>(keys, logit, s_bias + lane * V, before, to_f32(logits[before_id]), a.bias[before_id], slack);
                    close |= __any_sync(kAll, near);
                }
                break;
            }
            if (a.bias) {
                const float now = of_ordered(top);
                if (j > 0 && before - now <= slack + kRel * fmaxf(fabsf(before), fabsf(now)))
                    close |= to_f32(logits[e]) != to_f32(logits[before_id]) || a.bias[e] != a.bias[before_id];
                before = now;
                before_id = e;
            }
            if (lane == src) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v == at) key[v] = 0u;
            }
            if (lane == j) id = e;
        }
    }
    if (close) {   // (the same in every lane)
        float copy[V];   // (so that l itself stays in registers)
#pragma unroll
        for (int v = 0; v < V; ++v) copy[v] = l[v];
        id = choose_exact<V, SIGMOID>(copy, m, a, first, count, lanes);
    }
    // weights, on lane j
    const float x = id >= 0 ? to_f32(logits[id]) : kNone;
    float w;
    if (SIGMOID) {
        w = sigmoid32(x);
        if (a.renorm) {
            const float sum = chosen_sum(w, a.k);
            if (sum > 1e-30f) {   // (the same in every lane)
                w = __fdividef(w, sum);
            } else {              // all far below: s ~ exp(l)
                w = expf(x - warp_max(x));
                w /= chosen_sum(w, a.k);
            }
        }
    } else if (a.renorm) {
        w = expf(x - warp_max(x));
        w = __fdividef(w, chosen_sum(w, a.k));
    } else {
        w = expf(x - m) * per;
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.weights[t * a.k + lane] = id >= 0 ? w * a.scaling : 0.0f;
        if (loads && id >= 0) atomicAdd(loads + id, 1);   // (whole numbers: in any order)
    }
}

// A token that its lanes left to the whole warp (it has an expert that can be chosen, and its shares are counted).
template <class T, int V, bool SIGMOID>
__device__ __noinline__ void route_token(const RouterArgs& a, int64_t t, int lanes, float b_most, const float* s_bias, int* loads,
                                         uint2* s_near) {
    const T* logits = static_cast<const T*>(a.logits) + t * a.ld;
    const Seat seat(a, V, lanes, threadIdx.x & 31);
    Logits<T, V> raw;
    raw.load(logits + seat.first, seat.count, false);
    float l[V], none[V], lse;
    bool odd = false;
    finite_logits(raw, l, &odd);
    float m = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
    route_warp<T, V, SIGMOID, false>(a, logits, t, seat, l, warp_max(m), b_most, s_bias, loads, s_near, none, &lse);
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// Shared memory of the choice: bias and loads by slot or expert, then the warps' gathered keys (or, at the end, score sums).
template <int V, int L>
constexpr size_t router_smem(bool stats) {
    const size_t slots = 32 * V * sizeof(float);   // (L V of them are used)
    const size_t near = static_cast<size_t>(router_warps(V, L)) * (32 / L) * (kNearest + kSorted) * sizeof(uint2);
    const size_t sums = stats ? static_cast<size_t>(router_warps(V, L)) * L * V * sizeof(float) : 0;
    return 2 * slots + (near > sums ? near : sums);
}

// (A bias of -inf masks its expert.)
__device__ __forceinline__ float finite_magnitude(float b) { return fabsf(b) < INFINITY ? fabsf(b) : 0.0f; }
// Whether a token (the lanes of `lanes` from base on) has a logit above -inf whose bias is, too.
template <int V>
__device__ __forceinline__ bool some_unmasked(const float (&l)[V], const float* bias, int base, uint32_t lanes) {
    bool able = false;
#pragma unroll
    for (int v = 0; v < V; ++v) able |= l[v] > kNone && bias[v] > kNone;
    return ((__ballot_sync(kAll, able) >> base) & lanes) != 0u;
}
// Bias by slot, loads at zero.
template <int V, int WARPS, bool STATS>
__device__ __forceinline__ void router_start(const RouterArgs& a, float* s_bias, int* s_loads) {
    const int G = a.E / a.groups, per_group = a.lanes * V;
    for (int i = threadIdx.x; i < 32 * V; i += WARPS * 32) {
        const int g = i / per_group, r = i - g * per_group;
        s_bias[i] = a.bias && g < a.groups && r < G ? __ldg(a.bias + g * G + r) : 0.0f;
        if constexpr (STATS) s_loads[i] = 0;
    }
    __syncthreads();
}
// A block's sums: z_sum of a warp, live of each lane, share of each lane's experts.
template <int V, int L, int WARPS>
__device__ __forceinline__ void router_sums(const RouterArgs& a, float (&share)[V], float z_sum, int live, const int* s_loads,
                                            float* s_rest, int per_group) {
    __shared__ float s_z[WARPS];
    __shared__ int s_live[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.E / a.groups;
    live = __reduce_add_sync(kAll, live);
    if (lane == 0) s_z[warp] = z_sum, s_live[warp] = live;
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += WARPS * 32) a.part_count[static_cast<int64_t>(blockIdx.x) * a.E + e] = s_loads[e];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        for (int o = L; o < 32; o <<= 1) share[v] += __shfl_xor_sync(kAll, share[v], o);
        if (lane < L) s_rest[warp * (L * V) + lane * V + v] = share[v];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += WARPS * 32) {
        const int slot = e / G * per_group + e % G;
        float sum = 0.0f;
        for (int i = 0; i < WARPS; ++i) sum += s_rest[i * (L * V) + slot];
        a.part_share[static_cast<int64_t>(blockIdx.x) * a.E + e] = sum;
    }
    if (threadIdx.x == 0) {
        float z = 0.0f;
        int n = 0;
        for (int i = 0; i < WARPS; ++i) z += s_z[i], n += s_live[i];
        a.part_z[blockIdx.x] = z;
        a.part_live[blockIdx.x] = n;
    }
}

template <class T, int V, int L, bool STATS, bool SIGMOID>
__global__ void __launch_bounds__(router_warps(V, L) * 32, 1) router_kernel(const RouterArgs a) {
    grid_dependency_wait();
    extern __shared__ __align__(16) float s_mem[];
    constexpr int WARPS = router_warps(V, L), TOKENS = 32 / L;
    float* s_bias = s_mem;                                    // [L V]
    int* s_loads = reinterpret_cast<int*>(s_mem + 32 * V);    // [E]
    float* s_rest = s_mem + 2 * 32 * V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % L, base = lane - sub;
    const int G = a.E / a.groups, per_group = a.lanes * V;    // slots of a group
    const int own = sub / a.lanes, inside = sub % a.lanes * V;
    const int first = own * G + inside, count = own < a.groups ? min(max(G - inside, 0), V) : 0;
    uint2* const near = reinterpret_cast<uint2*>(s_rest) + (warp * TOKENS + lane / L) * (kNearest + kSorted);
    uint2* const sorted = near + kNearest;
    const T* logits = static_cast<const T*>(a.logits);
    router_start<V, WARPS, STATS>(a, s_bias, s_loads);
    float b_most = 0.0f;
    bool masks = false;   // a bias of -inf
    if (a.bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            b_most = fmaxf(b_most, finite_magnitude(s_bias[sub * V + v]));
            masks |= s_bias[sub * V + v] == kNone;
        }
        b_most = lanes_max<L>(b_most);
        masks = __any_sync(kAll, masks);
    }
    const bool scored = a.bias || (a.groups > 1 && a.top2);   // keys are needed as numbers, not only their order
    const int need = a.bias ? a.k + 1 : a.k;
    const bool all_hard = need > kSorted;
    float share[V];
    float z_sum = 0.0f;
    int live = 0;
    if constexpr (STATS) {
#pragma unroll
        for (int v = 0; v < V; ++v) share[v] = 0.0f;
    }
    bool odd = false;

    // a block's tokens are one in gridDim.x (of TOKENS together): few tokens spread over the SMs
    const int64_t step = static_cast<int64_t>(gridDim.x) * WARPS * TOKENS;
    for (int64_t t0 = (blockIdx.x + static_cast<int64_t>(warp) * gridDim.x) * TOKENS; t0 < a.T; t0 += step) {
        const int64_t t = t0 + lane / L;
        const bool real = t < a.T;
        const T* row = logits + t * a.ld;
        Logits<T, V> raw;
        const bool wanted = real && (!a.valid || a.valid[t] != 0);
        raw.load(row + first, wanted ? count : 0, a.vector);
        float l[V], s[V];
        finite_logits(raw, l, &odd);
        float m = l[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
        m = lanes_max<L>(m);
        bool alive = m > kNone;   // some expert can be chosen
        m = alive ? m : 0.0f;
        if (masks) alive = some_unmasked<V>(l, s_bias + sub * V, base, (1u << L) - 1u);
        float per = 1.0f;
        if (scored || STATS || !SIGMOID) {
            float z = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = score32<SIGMOID>(l[v], m);
                z += s[v];
            }
            z = lanes_sum<L>(z);
            per = __fdividef(1.0f, fmaxf(z, 1e-37f));
            if constexpr (STATS) {
                const bool gone = SIGMOID && alive && z < kVanished;   // (the same in a token's lanes)
#pragma unroll
                for (int v = 0; v < V; ++v) share[v] = fmaf(s[v], alive && !gone ? per : 0.0f, share[v]);
                if (SIGMOID && __any_sync(kAll, gone)) {
                    float u[V], sum = 0.0f;
#pragma unroll
                    for (int v = 0; v < V; ++v) sum += u[v] = __expf(l[v] - m);
                    sum = lanes_sum<L>(sum);
#pragma unroll
                    for (int v = 0; v < V; ++v) share[v] += gone ? __fdividef(u[v], sum) : 0.0f;
                }
                const float lse = SIGMOID || !alive ? 0.0f : m + logf(z);
                if (sub == 0) {
                    z_sum = fmaf(lse, lse, z_sum);
                    live += alive ? 1 : 0;
                }
            }
        }
        const float slack = key_slack<V, SIGMOID>(b_most, per);
        // keys as numbers (s, where they are needed) and as ordered integers
        uint32_t key[V];
        if (scored) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                s[v] = l[v] > kNone ? (SIGMOID ? s[v] : s[v] * per) + s_bias[sub * V + v] : kNone;
        }
        if (a.bias) {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = ordered(s[v]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = ordered(l[v]);
        }
        bool hard = all_hard;   // for the whole warp, afterwards (the same in a token's lanes)
        if (a.groups > 1) {
            float t1 = kNone, t2 = kNone;
            const auto join = [&](float u1, float u2) {
                t2 = fmaxf(fminf(t1, u1), fmaxf(t2, u2));
                t1 = fmaxf(t1, u1);
            };
            if (scored) {
#pragma unroll
                for (int v = 0; v < V; ++v) join(s[v], kNone);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) t1 = fmaxf(t1, l[v]);
            }
            for (int o = 1; o < a.lanes; o <<= 1) {
                const float u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
                join(u1, u2);
            }
            const float mine = a.top2 && t2 > kNone ? within_fp32(t1 + t2) : t1;
            int place = 0;
            for (int g = 0; g < a.groups; ++g) {
                const float o = __shfl_sync(kAll, mine, base + g * a.lanes);
                place += o > mine || (o == mine && g < own);
            }
            if (scored && a.kept < a.groups) {
                const float last = lanes_max<L>(own < a.groups && place == a.kept - 1 ? mine : kNone);
                const float out = lanes_max<L>(own < a.groups && place == a.kept ? mine : kNone);
                hard |= out > kNone && last - out <= 4.0f * slack + 2.0f * kRel * fmaxf(fabsf(last), fabsf(out));
            }
            if (own >= a.groups || place >= a.kept) {
#pragma unroll
                for (int v = 0; v < V; ++v) key[v] = 0u;
            }
        }
        // the k largest, and, with keys in fp32, one more to see how near it is: those from the k-th largest of the largest of
        // each PART of a lane's experts on (32 parts of a token or more, so that hardly more than k are)
        constexpr int PARTS = 4, PART = V / PARTS;
        uint32_t most[PARTS], least = kLeastKey;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            most[p] = key[p * PART];
#pragma unroll
            for (int v = 1; v < PART; ++v) most[p] = max(most[p], key[p * PART + v]);
        }
        for (int j = 0; j < need; ++j) {
            least = most[0];
#pragma unroll
            for (int p = 1; p < PARTS; ++p) least = max(least, most[p]);
            least = lanes_max<L>(least);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) most[p] = most[p] == least ? 0u : most[p];
        }
        least = max(least, kLeastKey);
        if (a.bias && least > kLeastKey) {   // (keys in fp32: all that may be among them)
            const float low = of_ordered(least);
            least = max(ordered(low - (slack + kRel * fabsf(low))), kLeastKey);
        }
        int found = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) found += key[v] >= least ? 1 : 0;
        int at = found;   // sum over the token's lanes up to this one
#pragma unroll
        for (int o = 1; o < L; o <<= 1) {
            const int u = __shfl_up_sync(kAll, at, o, L);
            if (sub >= o) at += u;
        }
        const int mine_found = found;
        found = __shfl_sync(kAll, at, base + L - 1);
        at -= mine_found;
        hard |= found > kNearest;
        const int n = hard ? 0 : found;   // (0: nothing is gathered)
        if (n > 0) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (key[v] >= least) near[at++] = make_uint2(key[v], first + v);
        }
        __syncwarp();
        const int most_found = __reduce_max_sync(kAll, n);
        for (int c = sub; c < most_found; c += L) {
            if (c < n) {
                const uint2 u = near[c];
                int place = 0;
                for (int i = 0; i < n; ++i) {
                    const uint2 o = near[i];
                    place += o.x > u.x || (o.x == u.x && o.y < u.y);
                }
                if (place < kSorted) sorted[place] = u;
            }
        }
        __syncwarp();
        // choices j = sub and sub + L (k <= kSorted <= 2 L)
        int id[2];
        float x[2];
        bool close = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = sub + i * L;
            id[i] = -1;
            x[i] = kNone;
            if (j < a.k && j < n) {
                const uint2 u = sorted[j];
                id[i] = static_cast<int>(u.y);
                x[i] = a.bias ? to_f32(row[u.y]) : of_ordered(u.x);
                if (a.bias && j + 1 < n) {
                    const uint2 o = sorted[j + 1];
                    const float before = of_ordered(u.x), now = of_ordered(o.x);
                    if (before - now <= slack + kRel * fmaxf(fabsf(before), fabsf(now))) {
                        close |= x[i] != to_f32(row[o.y]) || s_bias[u.y / G * per_group + u.y % G] != s_bias[o.y / G * per_group + o.y % G];
                        // the k-th and the next are alike: one behind them may be as near
                        if (j + 1 == a.k && j + 2 < n) {
                            const float third = j + 2 < kSorted ? of_ordered(sorted[j + 2].x) : before;
                            close |= before - third <= slack + kRel * fmaxf(fabsf(before), fabsf(third));
                        }
                    }
                }
            }
        }
        const uint32_t closes = __ballot_sync(kAll, close);
        constexpr uint32_t kToken = (1u << L) - 1u;
        hard |= ((closes >> base) & kToken) != 0u;
        // weights
        float w[2];
        if (SIGMOID) {
            w[0] = sigmoid32(x[0]), w[1] = sigmoid32(x[1]);
            if (a.renorm) {
                const float sum = lanes_sum<L>(w[0] + w[1]);
                const bool tiny = !(sum > 1e-30f);   // all far below: s ~ exp(l)
                w[0] = __fdividef(w[0], sum), w[1] = __fdividef(w[1], sum);
                if (__any_sync(kAll, tiny && n > 0)) {
                    const float top = lanes_max<L>(fmaxf(x[0], x[1]));
                    const float u0 = x[0] > kNone ? expf(x[0] - top) : 0.0f, u1 = x[1] > kNone ? expf(x[1] - top) : 0.0f;
                    const float all = lanes_sum<L>(u0 + u1);
                    if (tiny) w[0] = u0 / all, w[1] = u1 / all;
                }
            }
        } else if (a.renorm) {
            const float top = lanes_max<L>(fmaxf(x[0], x[1])), from = top > kNone ? top : 0.0f;
            w[0] = expf(x[0] - from), w[1] = expf(x[1] - from);
            const float sum = lanes_sum<L>(w[0] + w[1]);
            w[0] = __fdividef(w[0], sum), w[1] = __fdividef(w[1], sum);
        } else {
            w[0] = expf(x[0] - m) * per, w[1] = expf(x[1] - m) * per;
        }
        if (real && !(hard && alive)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = sub + i * L;
                if (j < a.k) {
                    a.ids[t * a.k + j] = id[i];
                    a.weights[t * a.k + j] = id[i] >= 0 ? w[i] * a.scaling : 0.0f;
                    if constexpr (STATS)
                        if (id[i] >= 0) atomicAdd(s_loads + id[i], 1);   // (whole numbers: in any order)
                }
            }
            if (all_hard)   // no expert can be chosen, and more slots than the lanes' two
                for (int j = sub + 2 * L; j < a.k; j += L) a.ids[t * a.k + j] = -1, a.weights[t * a.k + j] = 0.0f;
        }
        __syncwarp();
        uint32_t left = __ballot_sync(kAll, sub == 0 && real && hard && alive);
        while (left) {   // (the same in every lane)
            const int src = __ffs(static_cast<int>(left)) - 1;
            left &= left - 1;
            const int64_t hard_t = t0 + src / L;
            route_token<T, V * L / 32, SIGMOID>(a, hard_t, a.lanes * (32 / L), b_most, s_bias, STATS ? s_loads : nullptr,
                                                reinterpret_cast<uint2*>(s_rest) + warp * TOKENS * (kNearest + kSorted));
            __syncwarp();
        }
    }
    if (odd) status_set(a.status, MOE_STATUS_BAD_LOGIT);
    if constexpr (STATS) router_sums<V, L, WARPS>(a, share, warp_sum(z_sum), live, s_loads, s_rest, per_group);
}

// The same with a warp to a token: the choice of few tokens, and of more than 128 experts.
template <class T, int V, bool STATS, bool SIGMOID>
__global__ void __launch_bounds__(router_warps(V, 32) * 32, 1) router_warp_kernel(const RouterArgs a) {
    grid_dependency_wait();
    extern __shared__ __align__(16) float s_mem[];
    constexpr int WARPS = router_warps(V, 32);
    float* s_bias = s_mem;                                    // [32 V]
    int* s_loads = reinterpret_cast<int*>(s_mem + 32 * V);    // [E]
    float* s_rest = s_mem + 2 * 32 * V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Seat seat(a, V, a.lanes, lane);
    uint2* const near = reinterpret_cast<uint2*>(s_rest) + warp * 32;
    const T* logits = static_cast<const T*>(a.logits);
    router_start<V, WARPS, STATS>(a, s_bias, s_loads);
    float b_most = 0.0f;
    bool masks = false;   // a bias of -inf
    if (a.bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            b_most = fmaxf(b_most, finite_magnitude(s_bias[lane * V + v]));
            masks |= s_bias[lane * V + v] == kNone;
        }
        b_most = warp_max(b_most);
        masks = __any_sync(kAll, masks);
    }
    float share[V], z_sum = 0.0f;
    int live = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) share[v] = 0.0f;
    bool odd = false;
    const int64_t step = static_cast<int64_t>(gridDim.x) * WARPS;
    for (int64_t t = blockIdx.x + static_cast<int64_t>(warp) * gridDim.x; t < a.T; t += step) {
        const T* row = logits + t * a.ld;
        Logits<T, V> raw;
        const bool wanted = !a.valid || a.valid[t] != 0;
        raw.load(row + seat.first, wanted ? seat.count : 0, a.vector);
        float l[V];
        finite_logits(raw, l, &odd);
        float m = l[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
        m = warp_max(m);
        bool alive = m > kNone;   // some expert can be chosen
        if (masks) alive = some_unmasked<V>(l, s_bias + lane * V, 0, kAll);
        if (alive) {
            float lse = 0.0f;
            route_warp<T, V, SIGMOID, STATS>(a, row, t, seat, l, m, b_most, s_bias, STATS ? s_loads : nullptr, near, share, &lse);
            z_sum = fmaf(lse, lse, z_sum);
            live += lane == 0 ? 1 : 0;
            __syncwarp();
        } else if (lane < a.k) {
            a.ids[t * a.k + lane] = -1;
            a.weights[t * a.k + lane] = 0.0f;
        }
    }
    if (odd) status_set(a.status, MOE_STATUS_BAD_LOGIT);
    if constexpr (STATS) router_sums<V, 32, WARPS>(a, share, z_sum, live, s_loads, s_rest, a.lanes * V);
}

// The gradient: L lanes to a token, V experts to a lane (a warp has 32 / L tokens under way, its sums take log2 L steps).
template <class T, int V, int L, bool SIGMOID>
__global__ void __launch_bounds__(kBackwardWarps * 32, V <= 16 ? 4 : 2) router_backward_kernel(const RouterBackwardArgs a) {
    grid_dependency_wait();
    // the loads' factors h, rows of chosen gradients [tokens]; expert e of one at e % V * P + e / V (P odd: neighbours and a
    // lane's own fall into different banks)
    constexpr int P = L + 1;
    extern __shared__ float s_mem[];
    constexpr int TOKENS = kBackwardWarps * 32 / L;
    const int lane = threadIdx.x & 31, sub = lane % L, slot = threadIdx.x / L;
    const int first = sub * V, count = min(max(a.E - first, 0), V);
    const T* logits = static_cast<const T*>(a.logits);
    float* row = s_mem + (slot + 1) * (P * V);
    const bool shares = a.balance != 0.0f;
    const bool dense = shares || a.z != 0.0f || (!SIGMOID && !a.renorm);   // every logit has a gradient
    // the first token's logits are under way while the loads' factors are made
    const int64_t step = static_cast<int64_t>(gridDim.x) * TOKENS;
    int64_t t0 = static_cast<int64_t>(blockIdx.x) * TOKENS;
    Logits<T, V> raw;
    if (a.vector) raw.load(logits + (t0 + slot) * a.ld + first, dense && t0 + slot < a.T ? count : 0, true);
    float z_by = 0.0f;
    if (shares || a.z != 0.0f) {
        const float n = fmaxf(static_cast<float>(*a.live), 1.0f);
        z_by = 2.0f * a.z / n;
        const float by = a.balance * static_cast<float>(a.E) / (static_cast<float>(a.k) * n) / n;
        for (int e = threadIdx.x; e < L * V; e += kBackwardWarps * 32)
            s_mem[e % V * P + e / V] = shares && e < a.E ? by * static_cast<float>(a.counts[e]) : 0.0f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) row[v * P + sub] = 0.0f;
    __syncthreads();
    bool bad = false;

    for (; t0 < a.T; t0 += step) {   // (the same for a whole block)
        const int64_t t = t0 + slot;
        const bool real = t < a.T;
        const int32_t* ids = a.ids + t * a.k;
        // a chosen expert j of this lane: its id (else -1)
        const auto chosen = [&](int j) { return real && j < a.k ? __ldg(ids + j) : -1; };
        const int id0 = chosen(sub);
        bool any = id0 >= 0 && id0 < a.E;
        for (int j = sub + L; j < a.k; j += L) {
            const int id = chosen(j);
            any |= id >= 0 && id < a.E;
        }
        const bool some = lanes_max<L>(any ? 1.0f : 0.0f) > 0.0f;   // the token has an expert
        // of each expert c: softmax the score times z, sigmoid the score times 1 - score, which is e / (1 + e)^2 with e = exp(-|l|);
        // 0 of an expert that cannot be chosen
        float c[V], m = 0.0f, z = 1.0f, mean_h = 0.0f;
        if (dense) {
            bool odd = false;
            if (a.vector) {
                finite_logits(raw, c, &odd);
            } else {   // by neighbouring lanes, through the token's row
                if (real)
                    for (int e = sub; e < a.E; e += L) row[e % V * P + e / V] = to_f32(logits[t * a.ld + e]);
                __syncwarp();
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float x = real && v < count ? row[v * P + sub] : kNone;
                    c[v] = x < INFINITY ? x : kNone;
                    row[v * P + sub] = 0.0f;
                }
                __syncwarp();
            }
            if (!SIGMOID) {
                m = c[0];
#pragma unroll
                for (int v = 1; v < V; ++v) m = fmaxf(m, c[v]);
                m = lanes_max<L>(m);
                m = m > kNone ? m : 0.0f;
            }
            z = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float score;
                if (SIGMOID) {
                    const float e = __expf(-fabsf(c[v])), r = __fdividef(1.0f, 1.0f + e), er = e * r;
                    score = c[v] < 0.0f ? er : r;
                    c[v] = er * r;
                } else {
                    score = c[v] = __expf(c[v] - m);
                }
                z += score;
                if (shares) mean_h = fmaf(score, s_mem[v * P + sub], mean_h);
            }
            z = lanes_sum<L>(z);
            if (shares) mean_h = lanes_sum<L>(mean_h);
            if (SIGMOID && shares) {
                const bool gone = some && z < kVanished;   // (the same in a token's lanes)
                if (__any_sync(kAll, gone)) {   // the logits once more, twice: kept, they would cost registers in every token
                    const auto logit = [&](int v) {
                        const float x = gone && v < count ? to_f32(logits[t * a.ld + first + v]) : kNone;
                        return x < INFINITY ? x : kNone;
                    };
                    float top = kNone, all = 0.0f, h = 0.0f;
#pragma unroll
                    for (int v = 0; v < V; ++v) top = fmaxf(top, logit(v));
                    top = lanes_max<L>(top);
                    top = top > kNone ? top : 0.0f;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float u = __expf(logit(v) - top);
                        all += u;
                        h = fmaf(u, s_mem[v * P + sub], h);
                        c[v] = gone ? u : c[v];   // (1 - s is 1)
                    }
                    all = lanes_sum<L>(all);
                    h = lanes_sum<L>(h);
                    z = gone ? all : z, mean_h = gone ? h : mean_h;
                }
            }
        }
        if (a.vector && t + step < a.T) raw.load(logits + (t + step) * a.ld + first, dense ? count : 0, true);
        const float per = some ? __fdividef(1.0f, fmaxf(z, 1e-37f)) : 0.0f;
        mean_h *= per;
        // the chosen experts' part: sums over them, then each one's gradient (a lane has one, or every L-th)
        const auto part = [&](int id, float dw, float* q, float* g, float* phi) {
            const bool chose = id >= 0 && id < a.E;
            const float x = chose ? to_f32(logits[t * a.ld + id]) : kNone;
            *g = chose ? a.scaling * dw : 0.0f;
            *q = !chose ? 0.0f : SIGMOID ? sigmoid32(x) : a.renorm ? x : expf(x - m) * per;
            *phi = SIGMOID && chose ? sigmoid32(-x) : 1.0f;
            return x;
        };
        const auto dweight = [&](int j) { return real && j < a.k ? __ldg(a.dweights + t * a.k + j) : 0.0f; };
        float q0, g0, phi0;
        const float x0 = part(id0, dweight(sub), &q0, &g0, &phi0);
        bad |= id0 >= a.E;
        float most = x0, sum = 0.0f, sum_g = 0.0f;
        bool tiny = false;   // sigmoid scores that vanish: s ~ exp(l)
        if (a.renorm) {
            float all = q0;
            for (int j = sub + L; j < a.k; j += L) {
                float q, g, phi;
                most = fmaxf(most, part(chosen(j), 0.0f, &q, &g, &phi));
                all += q;
            }
            most = lanes_max<L>(most);
            if (SIGMOID) sum = lanes_sum<L>(all);
            tiny = SIGMOID && !(sum > 1e-30f);
            const bool logs = !SIGMOID || tiny;
            if (__any_sync(kAll, logs)) {   // (the warp's tokens together: the sum below is over lanes)
                all = x0 > kNone ? expf(x0 - most) : 0.0f;
                if (logs) q0 = all;
                for (int j = sub + L; j < a.k; j += L) {
                    float q, g, phi;
                    const float x = part(chosen(j), 0.0f, &q, &g, &phi);
                    all += x > kNone ? expf(x - most) : 0.0f;
                }
                const float other = lanes_sum<L>(all);
                if (logs) sum = other;
            }
        }
        const float by = a.renorm ? 1.0f / fmaxf(sum, 1e-37f) : 1.0f;
        q0 *= by;
        // (of a further choice j: q as q0, in the same way)
        const auto again = [&](int j, float* q, float* g, float* phi) {
            const int id = chosen(j);
            bad |= id >= a.E;
            const float x = part(id, dweight(j), q, g, phi);
            if (a.renorm && (!SIGMOID || tiny)) *q = x > kNone ? expf(x - most) : 0.0f;
            *q *= by;
            return id >= 0 && id < a.E ? id : -1;
        };
        sum_g = q0 * g0;
        for (int j = sub + L; j < a.k; j += L) {
            float q, g, phi;
            again(j, &q, &g, &phi);
            sum_g = fmaf(q, g, sum_g);
        }
        sum_g = lanes_sum<L>(sum_g);
        const float inner = a.renorm ? sum_g : 0.0f;
        if (any && id0 >= 0 && id0 < a.E) row[id0 % V * P + id0 / V] = phi0 * q0 * (g0 - inner);
        for (int j = sub + L; j < a.k; j += L) {
            float q, g, phi;
            const int id = again(j, &q, &g, &phi);
            if (id >= 0) row[id % V * P + id / V] = phi * q * (g - inner);
        }
        __syncwarp();
        // of every softmax logit: the z loss, and the chosen sum where it is not renormalised
        const float each = SIGMOID || !some ? 0.0f : (a.z != 0.0f ? z_by * (m + logf(z)) : 0.0f) - (a.renorm ? 0.0f : sum_g);
        T* to = static_cast<T*>(a.dlogits) + t * a.E;
        const auto gradient = [&](int v) {
            const float r = row[v * P + sub];
            return dense ? fmaf(c[v] * per, shares ? s_mem[v * P + sub] - mean_h + each : each, r) : r;
        };
        if (a.vector_out) {
            Logits<T, V> out;
#pragma unroll
            for (int v = 0; v < V; ++v) out.e[v] = from_f32<T>(gradient(v));
            __syncwarp();
            if (id0 >= 0 && id0 < a.E) row[id0 % V * P + id0 / V] = 0.0f;
            for (int j = sub + L; j < a.k; j += L) {
                const int id = chosen(j);
                if (id >= 0 && id < a.E) row[id % V * P + id / V] = 0.0f;
            }
            if (real) out.store(to + first, count, true);
        } else {   // rows of odd sizes: by neighbouring lanes (element by element from each lane's own, they took twice as long)
#pragma unroll
            for (int v = 0; v < V; ++v) row[v * P + sub] = gradient(v);
            __syncwarp();
            if (real)
                for (int e = sub; e < a.E; e += L) to[e] = from_f32<T>(row[e % V * P + e / V]);
            __syncwarp();
#pragma unroll
            for (int v = 0; v < V; ++v) row[v * P + sub] = 0.0f;
        }
        __syncwarp();
    }
    if (bad) status_set(a.status, MOE_STATUS_BAD_EXPERT_ID);
}

template <class T, int V, int L, bool SIGMOID>
cudaError_t forward_v(RouterArgs a, int blocks, cudaStream_t stream) {
    // whole vectors of each lane's experts: groups of a multiple of V
    a.vector = (a.E / a.groups) % V == 0 && router_vectors<T>(a.logits, a.ld, a.E, V);
    const dim3 grid(static_cast<unsigned>(blocks)), block(router_warps(V, L) * 32);
    const size_t smem = router_smem<V, L>(a.part_share != nullptr);
    static_assert(router_smem<V, L>(true) <= 47 * 1024, "more shared memory than a block has unasked");
    if constexpr (L == 32)
        return a.part_share ? launch_pdl(router_warp_kernel<T, V, true, SIGMOID>, grid, block, smem, stream, a)
                            : launch_pdl(router_warp_kernel<T, V, false, SIGMOID>, grid, block, smem, stream, a);
    else
        return a.part_share ? launch_pdl(router_kernel<T, V, L, true, SIGMOID>, grid, block, smem, stream, a)
                            : launch_pdl(router_kernel<T, V, L, false, SIGMOID>, grid, block, smem, stream, a);
}
// Eight lanes to a token where they hold its experts and there are tokens for all warps of the GPU (65536 x 128: 19 us in place of
// 29 with 32 lanes; 152 x 128: 3.8 in place of 2.7; 16 lanes for 256 experts: 32 and 35), else 32.
template <class T, bool SIGMOID>
cudaError_t forward_scoring(RouterArgs a, int blocks, cudaStream_t stream) {
    int groups = 1;   // a power of two of lanes to each
    while (groups < a.groups) groups <<= 1;
    const int G = a.E / a.groups;
    const auto experts = [&](int L) { return (G + L / groups - 1) / (L / groups); };   // of a lane
    if (a.T > kPlanSms * 32 && groups <= 8 && experts(8) <= 16) {
        a.lanes = 8 / groups;
        if (experts(8) <= 4) return forward_v<T, 4, 8, SIGMOID>(a, blocks, stream);
        if (experts(8) <= 8) return forward_v<T, 8, 8, SIGMOID>(a, blocks, stream);
        return forward_v<T, 16, 8, SIGMOID>(a, blocks, stream);
    }
    a.lanes = 32 / groups;
    const int V = experts(32);
    if (V <= 4) return forward_v<T, 4, 32, SIGMOID>(a, blocks, stream);
    if (V <= 8) return forward_v<T, 8, 32, SIGMOID>(a, blocks, stream);
    if (V <= 16) return forward_v<T, 16, 32, SIGMOID>(a, blocks, stream);
    if (V <= 32) return forward_v<T, 32, 32, SIGMOID>(a, blocks, stream);
    return forward_v<T, 64, 32, SIGMOID>(a, blocks, stream);   // groups that leave lanes without an expert; E <= 1024
}

template <class T, int V, int L, bool SIGMOID>
cudaError_t backward_v(RouterBackwardArgs a, cudaStream_t stream) {
    a.vector = router_vectors<T>(a.logits, a.ld, a.E, V);
    a.vector_out = router_vectors<T>(a.dlogits, a.E, a.E, V);
    constexpr int TOKENS = kBackwardWarps * 32 / L;
    const int64_t blocks = (static_cast<int64_t>(a.T) + TOKENS - 1) / TOKENS, most = kPlanSms * 8;
    return launch_pdl(router_backward_kernel<T, V, L, SIGMOID>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                      dim3(kBackwardWarps * 32), static_cast<size_t>(TOKENS + 1) * (L + 1) * V * sizeof(float), stream, a);
}
// 8 lanes to a token up to 128 experts, 16 up to 256.
template <class T, bool SIGMOID>
cudaError_t backward_scoring(const RouterBackwardArgs& a, cudaStream_t stream) {
    if (a.E <= 16) return backward_v<T, 2, 8, SIGMOID>(a, stream);
    if (a.E <= 64) return backward_v<T, 8, 8, SIGMOID>(a, stream);
    if (a.E <= 128) return backward_v<T, 16, 8, SIGMOID>(a, stream);
    if (a.E <= 256) return backward_v<T, 16, 16, SIGMOID>(a, stream);
    if (a.E <= 512) return backward_v<T, 16, 32, SIGMOID>(a, stream);
    return backward_v<T, 32, 32, SIGMOID>(a, stream);
}

}  // namespace

template <class T>
cudaError_t router_forward(const RouterArgs& a, int blocks, cudaStream_t stream) {
    return a.sigmoid ? forward_scoring<T, true>(a, blocks, stream) : forward_scoring<T, false>(a, blocks, stream);
}
template <class T>
cudaError_t router_backward(const RouterBackwardArgs& a, cudaStream_t stream) {
    return a.sigmoid ? backward_scoring<T, true>(a, stream) : backward_scoring<T, false>(a, stream);
}
#endif  // MOE_ROUTER_KERNELS

}  // namespace mfp8
