// route_scores.cu — routing to experts by softmax or sigmoid scores, with a bias for balance, groups and weights with
// or without renormalisation; and the gradient of the logits.  Per token, over E experts in G equal groups:
//
//   s[e] = exp(l[e]) / sum exp(l)  or  1 / (1 + exp(-l[e]))          scores
//   c[e] = s[e] + bias[e]                                            what the choice goes by
//   kept groups: the topk_group largest sums of a group's q = max(1, k / topk_group) largest c
//   idx  = the k largest c in the kept groups, falling;  w = scale s[idx] / (sum of the chosen s, or 1)
//
//   gradient, from dw and ds (of all scores, or none), u = scale dw:
//     D[e] = ds[e] + sum over the slots j with idx[j] = e of  u[j]   (renormalised: (u[j] - sum_i r[i] u[i]) / S,
//                                                                     r = s[idx] / S,  S = sum of the chosen s)
//     softmax  dl = s (D - sum_e s D)        sigmoid  dl = s (1 - s) D
//
// The choice is that of the definition in 64 bits, whatever 32 bits make of it: without bias and groups the logits
// themselves are compared; else c is computed in fp32, and where two neighbours of the order are closer than the
// errors of their fp32 values (a few rows in a thousand), the token is done again in fp64.  So the choice does not
// depend on how a compiler rounds an exp.  Equal c: the lower expert.
//
// LANES threads to a token (8 for up to 64 experts, else 32), each with EPL neighbouring experts of one group, so
// that lower lanes hold lower experts and a tie goes to the lowest lane.  A choice is a maximum over the lanes of an
// integer with the order of c (one instruction for a warp), and the lane that holds it looks for its next one.
// Bound by instructions, not by the T E logits that are read.
#include <climits>
#include <cmath>

#include "train_util.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;  // of a block
constexpr unsigned kAll = 0xffffffffu;
// Bounds on the relative error of an fp32 score.  expf is off by 2 units in the last place at the most (2.4e-7).
//   sigmoid  the addition and the division half a unit each: 3.6e-7
//   softmax  a term of the sum: expf and its argument's rounding, 6e-8 |l - top|, whose mean over the softmax is below
//            6e-8 ln 256; up to 21 additions of 6e-8: 1.9e-6 for the sum, and expf and the division of the score itself
//            (its argument's rounding is added where it is used)
constexpr float kSigmoidOff = 4.5e-7f, kSoftmaxOff = 2.5e-6f;

template <typename L>
__device__ __forceinline__ float logit(const L* p) {
    if constexpr (sizeof(L) == 2) return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
    else return __ldg(p);
}
template <typename L>
__device__ __forceinline__ void store_grad(L* p, float v) {
    if constexpr (sizeof(L) == 2) *p = __float2bfloat16_rn(v);
    else *p = v;
}

// Integers in the order of the values: above 1 for a number (-0 as 0), 1 for NaN, 0 for none.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return v != v ? 1u : u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
template <int LANES>
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {  // of a NaN and a number: either
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (LANES == 32) {
        return __reduce_max_sync(kAll, v);
    } else {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
        return v;
    }
}

// Where a token's experts lie: lane `sub` of LANES has `count` of them from `first` on, all of group `group`.
struct Place {
    int sub, per_group, group, first, count;  // per_group: lanes of a group
    __device__ __forceinline__ Place(int lanes, int E, int G) {
        sub = threadIdx.x & (lanes - 1);
        int slots = 1;  // groups, up to a power of two
        while (slots < G) slots *= 2;
        per_group = lanes / slots;
        group = sub / per_group;
        const int size = E / G, each = (size + per_group - 1) / per_group, at = (sub - group * per_group) * each;
        first = group * size + at;
        count = group < G ? max(0, min(each, size - at)) : 0;
    }
};

struct RouteArgs {
    const float* bias;
    int T, E, k, sigmoid, G, kept, renorm;
    float scale;
    int32_t* idx;
    float *w, *scores;
};

// ---------------------------------------------------------------------------------------------
// The choice in fp64: c[] of each lane -> the slots' experts, slot j's in lane j.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ bool before(double a, int ai, double b, int bi) {  // strict order; INT_MAX: none
    if (ai == INT_MAX) return false;
    if (bi == INT_MAX) return true;
    const bool an = a != a, bn = b != b;
    if (an != bn) return bn;
    return a > b || ((a == b || an) && ai < bi);
}
template <int LANES, int EPL, typename L>
__device__ __noinline__ int choose64(const L* row, const RouteArgs& a, const Place& p) {
    double c[EPL];
    float top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const float l = i < p.count ? logit(row + p.first + i) : -INFINITY;
        c[i] = l;
        nan |= l != l;
        top = fmaxf(top, l);
    }
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = 1.0 / (1.0 + exp(-c[i]));
    } else {
        top = lanes_max<LANES>(top);
        double s = nan ? static_cast<double>(NAN) : 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            c[i] = top == -INFINITY ? 0.0 : exp(c[i] - static_cast<double>(top));
            s += i < p.count ? c[i] : 0.0;
        }
        s = lanes_sum<LANES>(s);
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = top == -INFINITY && s == s ? 0.0 : c[i] / s;
    }
    unsigned left = 0;  // bit i: expert i of this lane may be chosen
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (i < p.count) {
            left |= 1u << i;
            if (a.bias) c[i] += static_cast<double>(__ldg(a.bias + p.first + i));
        }
    // The best of the lanes that differ in the bits below `lanes`, and its expert (INT_MAX: none).
    auto best = [&](unsigned open, int lanes, double& v, int& e) {
        v = 0.0;
        e = INT_MAX;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if ((open >> i & 1u) && before(c[i], p.first + i, v, e)) {
                v = c[i];
                e = p.first + i;
            }
        for (int o = lanes / 2; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(kAll, v, o);
            const int oe = __shfl_xor_sync(kAll, e, o);
            if (before(ov, oe, v, e)) {
                v = ov;
                e = oe;
            }
        }
    };
    if (a.G > 1) {
        const int q = min(a.E / a.G, max(1, a.k / a.kept));
        unsigned open = left;
        double score = 0.0;
        for (int r = 0; r < q; ++r) {
            double v;
            int e;
            best(open, p.per_group, v, e);
            score += v;
            if (e >= p.first && e < p.first + p.count) open &= ~(1u << (e - p.first));
        }
        int rank = 0;
        for (int g = 0; g < a.G; ++g) {
            const double v = __shfl_sync(kAll, score, g * p.per_group, LANES);
            rank += before(v, g, score, p.group) ? 1 : 0;
        }
        if (rank >= a.kept) left = 0;
    }
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
        double v;
        int e;
        best(left, LANES, v, e);
        if (e >= p.first && e < p.first + p.count) left &= ~(1u << (e - p.first));
        if (p.sub == j) mine = e;
    }
    return mine;
}

// The weights of the chosen experts, slot j's in lane j (8 lanes at least): s from its logit.
//   softmax     exp(l - top), renormalised over the slots, or over `sum` of the row
//   sigmoid     1 / (1 + exp(-l)); renormalised by logarithms where the sum is too small for a float
__device__ __forceinline__ float eight_sum(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float eight_max(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Shares of the chosen scores in their sum (`in`: this lane has a slot), and 1 / sum for the gradient's use.
__device__ __forceinline__ float share_of_chosen(float l, bool in, bool sig) {
    if (sig) {
        const float s = in ? sigmoid(l) : 0.0f, S = eight_sum(s);
        // Far below 0 (or NaN): from the logarithms of the scores, which 1 / (1 + e^-l) has lost.
        const bool small = !(S > 1e-30f);
        if (!__any_sync(kAll, in && small)) return s / S;
        const float ls = in ? fminf(l, 0.0f) - log1pf(expf(-fabsf(l))) : -INFINITY;
        const float top = eight_max(ls);
        const float e = in && top > -INFINITY ? expf(ls - top) : 0.0f, Z = eight_sum(e);
        const float r = Z > 0.0f ? e / Z : (Z != Z ? Z : 0.0f);
        return small ? (S != S ? S : r) : s / S;
    }
    const float top = eight_max(in ? l : -INFINITY);
    const float e = in ? (top == -INFINITY && l == l ? 0.0f : expf(l - top)) : 0.0f, Z = eight_sum(e);
    return Z > 0.0f ? e / Z : (Z != Z ? Z : 0.0f);
}

template <int LANES, int EPL, typename L>
__global__ void __launch_bounds__(kWarps * 32) route_scores_kernel(const L* __restrict__ logits, RouteArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int kTokens = 32 / LANES;
    const Place p(LANES, a.E, a.G);
    const int lane = threadIdx.x & 31, base = lane & ~(LANES - 1);  // the token's first lane
    const long long warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (warp * kTokens >= a.T) return;  // whole warps leave
    const long long want = warp * kTokens + lane / LANES;
    const bool there = want < a.T;
    const size_t t = static_cast<size_t>(there ? want : a.T - 1);
    const L* row = logits + t * a.E;
    const bool plain = !a.bias && a.G == 1;  // the order of the logits themselves

    float l[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = i < p.count ? logit(row + p.first + i) : -INFINITY;
    float top = 0.0f, total = 1.0f;
    if (!a.sigmoid && (!plain || !a.renorm || a.scores)) {
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) top = fmaxf(top, l[i]);
        top = lanes_max<LANES>(top);
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i < p.count) total += top == -INFINITY && l[i] == l[i] ? 0.0f : expf(l[i] - top);
        total = lanes_sum<LANES>(total);
    }
    auto score = [&](float v) {
        if (a.sigmoid) return sigmoid(v);
        return top == -INFINITY && total == 0.0f ? 0.0f : expf(v - top) / total;
    };
    uint32_t key[EPL];
    if (plain && !a.scores) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = i < p.count ? ordered(l[i]) : 0u;
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            key[i] = 0u;
            if (i < p.count) {
                const float s = score(l[i]);
                if (a.scores && there) a.scores[t * a.E + p.first + i] = s;
                key[i] = ordered(plain ? l[i] : a.bias ? s + __ldg(a.bias + p.first + i) : s);
            }
        }
    }
    auto value = [](uint32_t k) {  // of a key above 1
        return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
    };
    bool sure = true;  // the fp32 order is that of the definition
    if (a.G > 1) {
        // A group's score: its q largest, all groups at once.
        const int q = min(a.E / a.G, max(1, a.k / a.kept));
        unsigned open = (1u << EPL) - 1;
        float sum = 0.0f, size = 0.0f;
        for (int r = 0; r < q; ++r) {
            uint32_t m = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if ((open >> i & 1u) && key[i] > m) {
                    m = key[i];
                    at = i;
                }
            uint32_t all = m;
            for (int o = p.per_group / 2; o > 0; o >>= 1) all = max(all, __shfl_xor_sync(kAll, all, o));
            // (of equal ones the lowest lane's is taken out)
            const unsigned has = __ballot_sync(kAll, m == all) >> (lane & ~(p.per_group - 1));
            if ((lane & (p.per_group - 1)) == __ffs(has) - 1) open &= ~(1u << at);
            const float c = all > 1 ? value(all) : NAN;
            sum += c;
            size += fabsf(c);
        }
        // The error of sum: its scores' (see below; a softmax's add up to 1 at most), its additions'.
        const float off = (a.sigmoid ? q * kSigmoidOff : kSoftmaxOff) + size * (q + 1) * 6e-8f;
        int rank = 0;
        const uint32_t mine = ordered(sum);
        unsigned close = 0;  // groups whose scores may be in another order than their fp32 values
        for (int g = 0; g < a.G; ++g) {
            const float v = __shfl_sync(kAll, sum, g * p.per_group, LANES), vo = __shfl_sync(kAll, off, g * p.per_group, LANES);
            const uint32_t u = ordered(v);
            if (g != p.group) {
                rank += u > mine || (u == mine && g < p.group);
                if (!(fabsf(v - sum) > vo + off)) close |= 1u << g;
            }
        }
        const bool kept = p.group < a.G && rank < a.kept;
        const unsigned lanes_kept = __ballot_sync(kAll, kept) >> base;
        for (int g = 0; g < a.G; ++g)  // (only a kept one and another matter)
            if ((close >> g & 1u) && ((lanes_kept >> (g * p.per_group) & 1u) != 0) != kept && p.group < a.G) sure = false;
        if (!kept) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = 0u;
        }
    }
    // The slots, one by one (and the first that is not chosen, to see that it is not).
    const int rounds = plain ? a.k : a.k + 1;
    float last = INFINITY, last_off = 0.0f, my_l = 0.0f;
    int my_e = 0;
    uint32_t m = 0;
    int at = 0;
    auto next = [&] {
        m = 0;
        at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > m) {
                m = key[i];
                at = i;
            }
    };
    next();
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) {
        const uint32_t all = lanes_max<LANES>(m);
        const unsigned has = __ballot_sync(kAll, m == all) >> base;
        const int winner = __ffs(LANES == 32 ? has : has & ((1u << (LANES & 31)) - 1)) - 1;
        float wl = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i == at) wl = l[i];
        wl = __shfl_sync(kAll, wl, winner, LANES);
        const int e = __shfl_sync(kAll, p.first + at, winner, LANES);
        if (j < a.k && p.sub == j) {
            my_e = e;
            my_l = wl;
        }
        if (!plain) {
            const float c = all > 1 ? value(all) : NAN, sc = a.bias ? fabsf(c - __ldg(a.bias + e)) : fabsf(c);
            const float off = sc * (a.sigmoid ? kSigmoidOff : kSoftmaxOff + 6e-8f * fabsf(wl - top)) + fabsf(c) * 1.2e-7f + 1e-30f;
            if (all != 0 && j > 0 && !(last - c > last_off + off)) sure = false;
            last = c;
            last_off = off;
        }
        if (p.sub == winner) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == at) key[i] = 0u;
            next();
        }
    }
    if (!plain && __any_sync(kAll, !sure)) {
        const int e = choose64<LANES, EPL>(row, a, p);
        my_e = e;
        my_l = p.sub < a.k ? logit(row + e) : 0.0f;
    }
    const bool in = p.sub < a.k;
    float w;
    if (a.renorm) w = share_of_chosen(my_l, in, a.sigmoid);
    else w = in ? score(my_l) : 0.0f;
    if (in && there) {
        a.idx[t * a.k + p.sub] = my_e;
        a.w[t * a.k + p.sub] = a.scale * w;
    }
}

struct RouteGradArgs {
    const int32_t* idx;
    const float *dw, *dscores;
    int T, E, k, sigmoid, renorm, per_token;
    float scale;
};

template <int LANES, int EPL, typename L>
__global__ void __launch_bounds__(kWarps * 32)
route_scores_backward_kernel(const L* __restrict__ logits, RouteGradArgs a, L* __restrict__ dlogits) {
    pdl_wait();
    pdl_trigger();
    constexpr int kTokens = 32 / LANES;
    const Place p(LANES, a.E, 1);
    const int lane = threadIdx.x & 31;
    const long long warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (warp * kTokens >= a.T) return;
    const long long want = warp * kTokens + lane / LANES;
    const bool there = want < a.T;
    const size_t t = static_cast<size_t>(there ? want : a.T - 1);
    const L* row = logits + t * a.E;
    // Of all scores only those that a gradient reaches are needed: the chosen ones, but for a softmax that is not
    // renormalised or whose scores have a gradient of their own.
    const bool dense = a.dscores || (!a.sigmoid && !a.renorm);

    // Slot j in lane j; an expert that there is none of takes part in nothing.
    int e = -1;
    float u = 0.0f, l = 0.0f;
    if (a.dw && p.sub < a.k) {
        e = __ldg(a.idx + t * a.k + p.sub);
        if (e < 0 || e >= a.E) e = -1;
        else {
            u = a.scale * __ldg(a.dw + t * a.k + p.sub);
            l = logit(row + e);
        }
    }
    float direct = 0.0f;  // this slot's part of dl itself (not through D)
    float D = u;
    if (a.renorm) {  // d(share)/dl needs the shares alone: s (1/S) = r
        const float r = share_of_chosen(l, e >= 0, a.sigmoid);
        const float mean = eight_sum(e >= 0 ? r * u : 0.0f);
        direct = e >= 0 ? r * (u - mean) : 0.0f;
        if (a.sigmoid) direct *= sigmoid(-l);
        D = 0.0f;
    } else if (a.sigmoid) {
        direct = e >= 0 ? sigmoid(l) * sigmoid(-l) * u : 0.0f;
        D = 0.0f;
    }
    float g[EPL], s[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) g[i] = 0.0f;
    if (dense) {
        float v[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = i < p.count ? logit(row + p.first + i) : -INFINITY;
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] = sigmoid(v[i]) * sigmoid(-v[i]);
        } else {
            float top = -INFINITY, total = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) top = fmaxf(top, v[i]);
            top = lanes_max<LANES>(top);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                s[i] = i < p.count ? (top == -INFINITY && v[i] == v[i] ? 0.0f : expf(v[i] - top)) : 0.0f;
                total += s[i];
            }
            total = lanes_sum<LANES>(total);
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] *= inv;
        }
        if (a.dscores) {
            const float* ds = a.dscores + (a.per_token ? t * a.E : 0);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i < p.count) g[i] = __ldg(ds + p.first + i);
        }
        if (!a.sigmoid && !a.renorm && a.dw)
            for (int j = 0; j < a.k; ++j) {
                const int at = __shfl_sync(kAll, e, j, LANES) - p.first;
                const float add = __shfl_sync(kAll, D, j, LANES);
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (at == i && i < p.count) g[i] += add;
            }
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) g[i] *= s[i];
        } else {
            float mean = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) mean = fmaf(s[i], g[i], mean);
            mean = lanes_sum<LANES>(mean);
#pragma unroll
            for (int i = 0; i < EPL; ++i) g[i] = s[i] * (g[i] - mean);
        }
    }
    if (a.dw && (a.sigmoid || a.renorm))
        for (int j = 0; j < a.k; ++j) {
            const int at = __shfl_sync(kAll, e, j, LANES) - p.first;
            const float add = __shfl_sync(kAll, direct, j, LANES);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (at == i && i < p.count) g[i] += add;
        }
    if (there)
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i < p.count) store_grad(dlogits + t * a.E + p.first + i, g[i]);
}

// Experts of a lane, at most: groups up to a power of two share the lanes.
int experts_per_lane(int lanes, int E, int G) {
    int slots = 1;
    while (slots < G) slots *= 2;
    if (slots > lanes) return 1 << 30;
    const int per = lanes / slots;
    return (E / G + per - 1) / per;
}

#define MOE_BY_WIDTH(CALL)                                                                  \
    do {                                                                                    \
        const int n8 = E <= 64 ? experts_per_lane(8, E, G) : 1 << 30;                       \
        if (n8 <= 2) return CALL(8, 2);                                                     \
        if (n8 <= 8) return CALL(8, 8);                                                     \
        const int n32 = experts_per_lane(32, E, G);                                         \
        if (n32 <= 2) return CALL(32, 2);                                                   \
        if (n32 <= 4) return CALL(32, 4);                                                   \
        if (n32 <= 8 || G == 1) return CALL(32, 8);  /* (256 experts at most) */            \
        MOE_WIDER(CALL)                                                                     \
    } while (0)

template <typename L>
cudaError_t forward_as(const L* logits, const RouteArgs& a, cudaStream_t s) {
    const int E = a.E, G = a.G;
#define MOE_CALL(LANES, EPL)                                                                                              \
    launch_k(kPdlTrain, route_scores_kernel<LANES, EPL, L>, dim3((a.T - 1) / (kWarps * (32 / LANES)) + 1), dim3(kWarps * 32), \
             0, s, logits, a)
#define MOE_WIDER(CALL) return CALL(32, 16);
    MOE_BY_WIDTH(MOE_CALL);
#undef MOE_WIDER
#undef MOE_CALL
}
template <typename L>
cudaError_t backward_as(const L* logits, const RouteGradArgs& a, L* dlogits, cudaStream_t s) {
    const int E = a.E, G = 1;
#define MOE_CALL(LANES, EPL)                                                                                       \
    launch_k(kPdlTrain, route_scores_backward_kernel<LANES, EPL, L>, dim3((a.T - 1) / (kWarps * (32 / LANES)) + 1), \
             dim3(kWarps * 32), 0, s, logits, a, dlogits)
#define MOE_WIDER(CALL)
    MOE_BY_WIDTH(MOE_CALL);
#undef MOE_WIDER
#undef MOE_CALL
}

}  // namespace

cudaError_t launch_route_scores(const void* logits, bool bf16, const float* bias, int T, int E, int k, bool sigmoid,
                                int n_group, int topk_group, bool renorm, float scale, int32_t* idx, float* w,
                                float* scores, cudaStream_t s) {
    const RouteArgs a{bias, T, E, k, sigmoid, n_group, topk_group, renorm, scale, idx, w, scores};
    return bf16 ? forward_as(static_cast<const __nv_bfloat16*>(logits), a, s)
                : forward_as(static_cast<const float*>(logits), a, s);
}

cudaError_t launch_route_scores_backward(const void* logits, bool bf16, const int32_t* idx, const float* dw,
                                         const float* dscores, bool per_token, int T, int E, int k, bool sigmoid,
                                         bool renorm, float scale, void* dlogits, cudaStream_t s) {
    const RouteGradArgs a{idx, dw, dscores, T, E, k, sigmoid, renorm, per_token, scale};
    return bf16 ? backward_as(static_cast<const __nv_bfloat16*>(logits), a, static_cast<__nv_bfloat16*>(dlogits), s)
                : backward_as(static_cast<const float*>(logits), a, static_cast<float*>(dlogits), s);
}

}  // namespace moe
