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
// The choice is that of the real numbers: keys are formed in fp32, and where two of them that a decision compares are
// closer than their error (and not of the same logit and bias) the token's choice is repeated on fp64 keys.
//
// Lane i holds experts i V .. i V + V - 1 in registers (V = 1 to 32, E <= 32 V), the next token's logits are under way while
// one is chosen for.  A round of the top-k is a maximum over a lane's keys, one over the warp (as ordered integers) and
// a ballot.  Loads and score sums stay in registers over a warp's tokens, are added across a block's warps in
// order, and a last small launch adds the blocks' sums: no atomics, the same result every time.
#pragma once

#include <type_traits>

#include "train.cuh"

namespace mfp8 {

constexpr int kRouterWarps = 8;      // tokens under way in a block

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
cudaError_t router_backward(const RouterBackwardArgs& a, int blocks, cudaStream_t stream);

#ifdef MOE_ROUTER_KERNELS
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kNone = -INFINITY;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
// fp32 as integers of the same order, both zeros alike; 0 stands for no candidate.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_ordered(uint32_t u) {
    return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}

// V logits from p on, those past `count` kNone.
template <class T, int V>
struct Logits {
    static constexpr int kBytes = V * static_cast<int>(sizeof(T));
    static constexpr int kWords = kBytes >= 16 ? kBytes / 16 : 1;
    using Word = typename std::conditional<kBytes >= 16, uint4,
                 typename std::conditional<kBytes == 8, uint2, typename std::conditional<kBytes == 4, uint32_t, uint16_t>::type>::type>::type;
    union {
        Word w[kWords];
        T e[V];
    };
    __device__ __forceinline__ Logits() {}
    __device__ __forceinline__ void load(const T* p, int count, bool vector) {
        if (vector) {
            if (count > 0) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const Word*>(p) + i);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v < count) e[v] = p[v];
        }
    }
    __device__ __forceinline__ void store(T* p, int count, bool vector) const {
        if (vector) {
            if (count > 0) {
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

// A lane's logits; one that is not finite counts as -inf (true in *odd unless it is -inf).
template <class T, int V>
__device__ __forceinline__ void finite_logits(const Logits<T, V>& raw, int count, float (&l)[V], bool* odd) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float x = v < count ? to_f32(raw.e[v]) : kNone;
        l[v] = fabsf(x) < INFINITY ? x : kNone;
        *odd |= !(fabsf(x) < INFINITY) && x != kNone;
    }
}

// Accurate where it vanishes, too.
__device__ __forceinline__ float sigmoid32(float l) {
    const float e = expf(-fabsf(l));
    return __fdividef(l < 0.0f ? e : 1.0f, 1.0f + e);
}

// The choice on fp64 keys.  Returns on lane j < k the j-th expert or -1.
template <int V>
__device__ __noinline__ int choose_exact(const float* l, const RouterArgs& a, int first, int count) {
    const int lane = threadIdx.x & 31;
    double key[V];
    double m = kNone;
    for (int v = 0; v < V; ++v) m = fmax(m, static_cast<double>(l[v]));
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kAll, m, o));
    double z = 0.0;
    for (int v = 0; v < V; ++v) {
        const double x = l[v];
        key[v] = l[v] == kNone ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m);
        z += key[v];
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
    if (a.sigmoid) z = 1.0;
    for (int v = 0; v < V; ++v)
        key[v] = l[v] == kNone ? static_cast<double>(kNone) : key[v] / z + (a.bias ? static_cast<double>(a.bias[first + v]) : 0.0);
    if (a.groups > 1) {
        const int G = a.E / a.groups;
        double mine = kNone;   // lane g: value of group g
        for (int g = 0; g < a.groups; ++g) {
            double t1 = kNone, t2 = kNone;
            for (int v = 0; v < V; ++v)
                if (v < count && (first + v) / G == g) {
                    t2 = fmax(t2, fmin(t1, key[v]));
                    t1 = fmax(t1, key[v]);
                }
            for (int o = 16; o > 0; o >>= 1) {
                const double u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
                t2 = fmax(fmin(t1, u1), fmax(t2, u2));
                t1 = fmax(t1, u1);
            }
            if (a.top2 && t2 > kNone) t1 += t2;
            if (lane == g) mine = t1;
        }
        int place = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double o = __shfl_sync(kAll, mine, g);
            place += o > mine || (o == mine && g < lane);
        }
        const uint32_t stay = __ballot_sync(kAll, lane < a.groups && place < a.kept);
        for (int v = 0; v < V; ++v)
            if (v < count && !((stay >> ((first + v) / G)) & 1u)) key[v] = kNone;
    }
    int id = -1;
    for (int j = 0; j < a.k; ++j) {
        double best = kNone;
        int at = 0;
        for (int v = 0; v < V; ++v)
            if (key[v] > best) best = key[v], at = v;
        double top = best;
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kAll, top, o));
        if (top == kNone) break;
        const int src = __ffs(static_cast<int>(__ballot_sync(kAll, best == top))) - 1;
        const int e = __shfl_sync(kAll, first + at, src);
        if (lane == src) key[at] = kNone;
        if (lane == j) id = e;
    }
    return id;
}

template <class T, int V, bool STATS>
__global__ void __launch_bounds__(kRouterWarps * 32) router_kernel(const RouterArgs a) {
    grid_dependency_wait();
    extern __shared__ float s_share[];   // STATS: [E] sums, [E] counts, z, live
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = lane * V, count = min(max(a.E - first, 0), V);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouterWarps;
    const T* logits = static_cast<const T*>(a.logits);
    float b[V];
    float b_most = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        b[v] = a.bias && v < count ? __ldg(a.bias + first + v) : 0.0f;
        b_most = fmaxf(b_most, fabsf(b[v]));
    }
    if (a.bias) b_most = warp_max(b_most);
    const bool scored = a.bias || (a.groups > 1 && a.top2);   // keys are needed as numbers, not only their order
    const int G = a.E / a.groups;
    // groups of whole lanes, a power of two of them: by shuffles among them; other groups one after the other
    const int lanes = G % V == 0 && ((G / V) & (G / V - 1)) == 0 ? G / V : 0;
    float share[V];
    int loads[V];
    float z_sum = 0.0f;
    int live = 0;
    if constexpr (STATS) {
#pragma unroll
        for (int v = 0; v < V; ++v) share[v] = 0.0f, loads[v] = 0;
    }
    bool odd = false;

    int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWarps + warp;
    Logits<T, V> raw, next;
    if (t < a.T) next.load(logits + t * a.ld + first, count, a.vector);
    for (; t < a.T; t += step) {
        raw = next;
        if (t + step < a.T) next.load(logits + (t + step) * a.ld + first, count, a.vector);
        const bool wanted = !a.valid || a.valid[t] != 0;
        float l[V];
        bool any = false;
        finite_logits(raw, wanted ? count : 0, l, &any);
        odd |= any;
        float m = l[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
        m = warp_max(m);
        int id = -1;
        float w = 0.0f;
        if (m > kNone) {   // some expert can be chosen
            float s[V], z = 1.0f;
            if (scored || STATS || (!a.sigmoid && !a.renorm)) {
                z = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    s[v] = l[v] == kNone ? 0.0f : a.sigmoid ? sigmoid32(l[v]) : expf(l[v] - m);
                    z += s[v];
                }
                z = warp_sum(z);
            }
            const float per = __fdividef(1.0f, z);
            // keys, as ordered integers
            uint32_t key[V];
            // more than the error of a difference of keys, less 2^-19 of the keys: a score is off by 2^-20 of itself (two
            // ulp of expf and of the quotient; with softmax also of the distance to the largest logit, which
            // is at most 2^-24 of the largest score) and, with softmax, by a factor that all share (37 roundings)
            const float slack = 0x1p-17f * b_most + (a.sigmoid ? 0.0f : 0x1p-22f * per);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float x = a.bias ? (a.sigmoid ? s[v] : s[v] * per) + b[v] : l[v];
                key[v] = l[v] == kNone ? 0u : ordered(x);
            }
            bool close = false;
            if (a.groups > 1) {
                // a group's value; for groups of whole lanes in its lanes, else in lane g
                float mine = kNone;
                const auto number = [&](int v) {
                    return l[v] == kNone ? kNone : scored ? (a.sigmoid ? s[v] : s[v] * per) + b[v] : l[v];
                };
                const auto join = [](float& t1, float& t2, float u1, float u2) {
                    t2 = fmaxf(fminf(t1, u1), fmaxf(t2, u2));
                    t1 = fmaxf(t1, u1);
                };
                if (lanes > 0) {
                    float t1 = kNone, t2 = kNone;
#pragma unroll
                    for (int v = 0; v < V; ++v) join(t1, t2, number(v), kNone);
                    for (int o = 1; o < lanes; o <<= 1) {
                        const float u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
                        join(t1, t2, u1, u2);
                    }
                    mine = a.top2 && t2 > kNone ? t1 + t2 : t1;
                } else {
                    for (int g = 0; g < a.groups; ++g) {
                        float t1 = kNone, t2 = kNone;
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            if (v < count && (first + v) / G == g) join(t1, t2, number(v), kNone);
                        for (int o = 16; o > 0; o >>= 1) {
                            const float u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
                            join(t1, t2, u1, u2);
                        }
                        if (lane == g) mine = a.top2 && t2 > kNone ? t1 + t2 : t1;
                    }
                }
                const int apart = lanes > 0 ? lanes : 1, own = lane / apart;
                int place = 0;
                for (int g = 0; g < a.groups; ++g) {
                    const float o = __shfl_sync(kAll, mine, g * apart);
                    place += o > mine || (o == mine && g < own);
                }
                const bool real = own < a.groups;
                if (scored && a.kept < a.groups) {
                    const float last = warp_max(real && place == a.kept - 1 ? mine : kNone);
                    const float out = warp_max(real && place == a.kept ? mine : kNone);
                    close = out > kNone && last - out <= 4.0f * slack + 0x1p-18f * fmaxf(fabsf(last), fabsf(out));
                }
                const uint32_t stay = __ballot_sync(kAll, real && place < a.kept);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int g = lanes > 0 ? lane : (first + v) / G;
                    if (v >= count || !((stay >> (g & 31)) & 1u)) key[v] = 0u;
                }
            }
            // the k largest (and, with keys in fp32, one more to see how near it is)
            uint32_t taken = 0;
            float before = 0.0f;
            int before_id = -1;
            const int rounds = a.bias ? a.k + 1 : a.k;
            for (int j = 0; j < rounds; ++j) {
                uint32_t most = key[0];
#pragma unroll
                for (int v = 1; v < V; ++v) most = max(most, key[v]);
                const uint32_t top = __reduce_max_sync(kAll, most);
                if (top == 0u) break;
                const int src = __ffs(static_cast<int>(__ballot_sync(kAll, most == top))) - 1;
                int at = 0;
#pragma unroll
                for (int v = V - 1; v >= 0; --v)
                    if (key[v] == top) at = v;
                const int e = __shfl_sync(kAll, first + at, src);
                if (a.bias) {
                    const float now = of_ordered(top);
                    if (j > 0 && before - now <= slack + 0x1p-19f * fmaxf(fabsf(before), fabsf(now)))
                        close |= to_f32(logits[t * a.ld + e]) != to_f32(logits[t * a.ld + before_id]) ||
                                 a.bias[e] != a.bias[before_id];
                    before = now;
                    before_id = e;
                }
                if (j >= a.k) break;
                if (lane == src) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (v == at) key[v] = 0u;
                    taken |= 1u << at;
                }
                if (lane == j) id = e;
            }
            if (close) {   // (the same in every lane)
                float copy[V];   // (so that l itself stays in registers)
#pragma unroll
                for (int v = 0; v < V; ++v) copy[v] = l[v];
                id = choose_exact<V>(copy, a, first, count);
                taken = 0;
                for (int j = 0; j < a.k; ++j) {
                    const int e = __shfl_sync(kAll, id, j);
                    if (e >= first && e < first + V) taken |= 1u << (e - first);
                }
            }
            // weights, on lane j
            const bool chose = id >= 0;
            const float x = chose ? to_f32(logits[t * a.ld + id]) : kNone;
            if (a.renorm) {
                if (a.sigmoid) {
                    w = chose ? sigmoid32(x) : 0.0f;
                    const float sum = warp_sum(w), most = warp_max(x);
                    if (sum > 1e-30f) {
                        w = __fdividef(w, sum);
                    } else {   // all far below: s ~ exp(l)
                        w = chose ? expf(x - most) : 0.0f;
                        w /= warp_sum(w);
                    }
                } else {
                    const float most = warp_max(x);
                    w = chose ? expf(x - most) : 0.0f;
                    w = __fdividef(w, warp_sum(w));
                }
            } else {
                w = !chose ? 0.0f : a.sigmoid ? sigmoid32(x) : expf(x - m) * per;
            }
            if constexpr (STATS) {
                const float by = __fdividef(1.0f, fmaxf(z, 1e-37f));
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    share[v] = fmaf(s[v], by, share[v]);
                    loads[v] += static_cast<int>((taken >> v) & 1u);
                }
                const float lse = a.sigmoid ? 0.0f : m + logf(z);
                z_sum = fmaf(lse, lse, z_sum);
                ++live;
            }
        }
        if (lane < a.k) {
            a.ids[t * a.k + lane] = id;
            a.weights[t * a.k + lane] = w * a.scaling;
        }
    }
    if (odd) status_set(a.status, MOE_STATUS_BAD_LOGIT);
    if constexpr (STATS) {
        int* s_loads = reinterpret_cast<int*>(s_share + a.E);
        float* s_z = s_share + 2 * a.E;
        int* s_live = reinterpret_cast<int*>(s_z + 1);
        for (int i = 0; i < kRouterWarps; ++i) {
            if (warp == i) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v < count) {
                        s_share[first + v] = share[v] + (i ? s_share[first + v] : 0.0f);
                        s_loads[first + v] = loads[v] + (i ? s_loads[first + v] : 0);
                    }
                if (lane == 0) {
                    *s_z = z_sum + (i ? *s_z : 0.0f);
                    *s_live = live + (i ? *s_live : 0);
                }
            }
            __syncthreads();
        }
        for (int e = threadIdx.x; e < a.E; e += kRouterWarps * 32) {
            a.part_share[static_cast<int64_t>(blockIdx.x) * a.E + e] = s_share[e];
            a.part_count[static_cast<int64_t>(blockIdx.x) * a.E + e] = s_loads[e];
        }
        if (threadIdx.x == 0) {
            a.part_z[blockIdx.x] = *s_z;
            a.part_live[blockIdx.x] = *s_live;
        }
    }
}

template <class T, int V>
__global__ void __launch_bounds__(kRouterWarps * 32) router_backward_kernel(const RouterBackwardArgs a) {
    grid_dependency_wait();
    extern __shared__ float s_rows[];   // [warps][32 V]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = lane * V, count = min(max(a.E - first, 0), V);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouterWarps;
    const T* logits = static_cast<const T*>(a.logits);
    float* row = s_rows + warp * (32 * V);
    const bool shares = a.balance != 0.0f;
    const bool dense = shares || a.z != 0.0f || (!a.sigmoid && !a.renorm);   // every logit has a gradient
    float h[V];
    float z_by = 0.0f;
    if (shares || a.z != 0.0f) {
        const float n = fmaxf(static_cast<float>(*a.live), 1.0f);
        z_by = 2.0f * a.z / n;
        const float by = a.balance * static_cast<float>(a.E) / (static_cast<float>(a.k) * n) / n;
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = shares && v < count ? by * static_cast<float>(a.counts[first + v]) : 0.0f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) row[v * 32 + lane] = 0.0f;
    bool bad = false;

    int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWarps + warp;
    Logits<T, V> raw, next;
    int next_id = -1;
    float next_dw = 0.0f;
    const auto fetch = [&](int64_t u) {
        if (u >= a.T) return;
        next.load(logits + u * a.ld + first, dense ? count : 0, a.vector);
        if (lane < a.k) {
            next_id = __ldg(a.ids + u * a.k + lane);
            next_dw = __ldg(a.dweights + u * a.k + lane);
        }
    };
    fetch(t);
    for (; t < a.T; t += step) {
        raw = next;
        int id = lane < a.k ? next_id : -1;
        const float dw = next_dw;
        fetch(t + step);
        if (id >= a.E) bad = true, id = -1;
        const bool chose = id >= 0;
        Logits<T, V> out;
        if (__any_sync(kAll, chose)) {
            const float x = chose ? to_f32(logits[t * a.ld + id]) : kNone;
            const float g = chose ? a.scaling * dw : 0.0f;
            float l[V], s[V], m = 0.0f, z = 1.0f;
            if (dense) {
                bool odd = false;
                finite_logits(raw, count, l, &odd);
                m = l[0];
#pragma unroll
                for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
                m = warp_max(m);
                z = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    s[v] = l[v] == kNone ? 0.0f : a.sigmoid ? sigmoid32(l[v]) : expf(l[v] - m);
                    z += s[v];
                }
                z = warp_sum(z);
            }
            const float per = __fdividef(1.0f, fmaxf(z, 1e-37f));
            // the chosen experts' part, on lane j
            float d = 0.0f, sum_g = 0.0f;
            if (a.renorm) {
                float q;
                if (a.sigmoid) {
                    q = chose ? sigmoid32(x) : 0.0f;
                    const float sum = warp_sum(q), most = warp_max(x);
                    if (sum > 1e-30f) {
                        q = __fdividef(q, sum);
                    } else {
                        q = chose ? expf(x - most) : 0.0f;
                        q /= warp_sum(q);
                    }
                } else {
                    const float most = warp_max(x);
                    q = chose ? expf(x - most) : 0.0f;
                    q = __fdividef(q, warp_sum(q));
                }
                d = q * (g - warp_sum(q * g));
                if (a.sigmoid) d *= sigmoid32(-x);
            } else if (a.sigmoid) {
                d = g * sigmoid32(x) * sigmoid32(-x);
            } else {
                const float p = chose ? expf(x - m) * per : 0.0f;
                d = p * g;
                sum_g = warp_sum(p * g);
            }
            if (chose) row[id % V * 32 + id / V] = d;
            __syncwarp();
            float mean_h = 0.0f;
            if (shares) {
#pragma unroll
                for (int v = 0; v < V; ++v) mean_h = fmaf(s[v], h[v], mean_h);
                mean_h = warp_sum(mean_h) * per;
            }
            const float z_part = a.z != 0.0f ? z_by * (m + logf(z)) : 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float r = row[v * 32 + lane];
                if (dense && v < count) {
                    const float p = s[v] * per;
                    if (shares) r += p * (h[v] - mean_h) * (a.sigmoid ? sigmoid32(-l[v]) : 1.0f);
                    if (!a.sigmoid) r += p * (z_part - sum_g);
                }
                out.e[v] = from_f32<T>(r);
            }
            __syncwarp();
            if (chose) row[id % V * 32 + id / V] = 0.0f;
            __syncwarp();
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) out.e[v] = from_f32<T>(0.0f);
        }
        out.store(static_cast<T*>(a.dlogits) + t * a.E + first, count, a.vector_out);
    }
    if (bad) status_set(a.status, MOE_STATUS_BAD_EXPERT_ID);
}

template <class T, int V>
cudaError_t forward_v(const RouterArgs& a, int blocks, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(blocks)), block(kRouterWarps * 32);
    if (!a.part_share) return launch_pdl(router_kernel<T, V, false>, grid, block, 0, stream, a);
    return launch_pdl(router_kernel<T, V, true>, grid, block, (2 * static_cast<size_t>(a.E) + 2) * 4, stream, a);
}
template <class T, int V>
cudaError_t backward_v(const RouterBackwardArgs& a, int blocks, cudaStream_t stream) {
    return launch_pdl(router_backward_kernel<T, V>, dim3(static_cast<unsigned>(blocks)), dim3(kRouterWarps * 32),
                      static_cast<size_t>(kRouterWarps) * 32 * V * 4, stream, a);
}

}  // namespace

// Rows that can be loaded V elements at a time: E a multiple of V, addresses of the vectors (16 bytes at most).
template <class T>
bool router_vectors(const void* p, int64_t ld, int E, int V) {
    const int64_t bytes = V * static_cast<int64_t>(sizeof(T)) < 16 ? V * static_cast<int64_t>(sizeof(T)) : 16;
    return E % V == 0 && address(p) % bytes == 0 && ld * static_cast<int64_t>(sizeof(T)) % bytes == 0;
}
inline int router_v(int E) { return E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : E <= 256 ? 8 : E <= 512 ? 16 : 32; }

template <class T>
cudaError_t router_forward(const RouterArgs& args, int blocks, cudaStream_t stream) {
    RouterArgs a = args;
    const int V = router_v(a.E);
    a.vector = router_vectors<T>(a.logits, a.ld, a.E, V);
    switch (V) {
        case 1: return forward_v<T, 1>(a, blocks, stream);
        case 2: return forward_v<T, 2>(a, blocks, stream);
        case 4: return forward_v<T, 4>(a, blocks, stream);
        case 8: return forward_v<T, 8>(a, blocks, stream);
        case 16: return forward_v<T, 16>(a, blocks, stream);
        default: return forward_v<T, 32>(a, blocks, stream);
    }
}
template <class T>
cudaError_t router_backward(const RouterBackwardArgs& args, int blocks, cudaStream_t stream) {
    RouterBackwardArgs a = args;
    const int V = router_v(a.E);
    a.vector = router_vectors<T>(a.logits, a.ld, a.E, V);
    a.vector_out = router_vectors<T>(a.dlogits, a.E, a.E, V);
    switch (V) {
        case 1: return backward_v<T, 1>(a, blocks, stream);
        case 2: return backward_v<T, 2>(a, blocks, stream);
        case 4: return backward_v<T, 4>(a, blocks, stream);
        case 8: return backward_v<T, 8>(a, blocks, stream);
        case 16: return backward_v<T, 16>(a, blocks, stream);
        default: return backward_v<T, 32>(a, blocks, stream);
    }
}
#endif  // MOE_ROUTER_KERNELS

}  // namespace mfp8
