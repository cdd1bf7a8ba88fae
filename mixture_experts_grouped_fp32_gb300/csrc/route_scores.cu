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
// errors of their fp32 values, the token is done again in fp64.  So the choice does not depend on how a compiler rounds an
// exp.  Equal c: the lower expert.  Of random fp32 logits over 256 experts 0.03 to 0.15 % of the rows are done again.
// Equal scores are too, though no precision tells them apart: of bf16 logits without a bias (in groups), or with a bias
// of zeros, that is every third row (16384 x 256, sigmoid 30 us, softmax 76; of fp32 logits 19 and 23), and where half of
// the rows are zeros, every one of those (150 and 220 us).  With a bias of unequal values they are no more than in fp32.
//
// LANES threads to a token (8 for up to 64 experts, else 32), each with up to EPL neighbouring experts of one group, so
// that lower lanes hold lower experts and a tie goes to the lowest lane.  A lane sorts its experts once, as integers
// with the order of c; a slot then costs one maximum over the lanes' first ones (one instruction for a warp), and the
// lane that held it reads its next one.  Which expert a slot's integer belongs to is looked up for all slots at once.
// Bound by instructions, not by the T E logits that are read: 780 of a warp for a token of 256 experts in 8 groups
// (sigmoid, bias; 16384 tokens 16 to 23 us by the inputs, 72 % of the issue slots while it runs, and the last contested token's fp64
// behind the others), 10.3 us without groups and bias, 7.2 us for 64 experts (sigmoid, bias).
//
// The gradient takes eight or sixteen threads to a token where the experts are fours: fewer steps of a reduction, wide
// loads (16001 x 160 softmax with all scores' gradient 6.2 us; with a warp to a token and one expert at a time 11.8).
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "train_util.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;  // of a block
constexpr unsigned kAll = 0xffffffffu;
// Bounds on the error of the fp32 scores that the choice goes by: 2.4e-7 of a value for the instructions 2^x and 1 / x
// (over all floats they are off by 1.5e-7 and 1.0e-7 at the most), 6e-8 for each rounding.
//   sigmoid  1 / (1 + e), e = exp(-l) is off by (1 - s) (2.4e-7 + 1.4e-7 |l|) of s; s (1 - s) |l| is below 0.28: with the
//            addition and the division 5.5e-7 s + 4e-8
//   softmax  a term of the sum by 2.4e-7 + 2e-7 |l - top| (its argument is rounded too), whose mean over the softmax is
//            below 2.4e-7 + 2e-7 ln 256, up to 21 additions, the quotient: 3e-6 + 2e-7 |l - top| of s
// Values below 2^-126 count as 0 there.
constexpr float kSigmoidRel = 5.5e-7f, kSigmoidAbs = 4e-8f, kSoftmaxRel = 3e-6f, kSoftmaxArg = 2e-7f;

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

// The same of a score with its bias, where NaN is dealt with elsewhere and -0 cannot be.
__device__ __forceinline__ uint32_t ordered_score(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ unsigned long long ordered(double v) {
    const long long u = __double_as_longlong(v + 0.0);
    return v != v ? 1ull : static_cast<unsigned long long>(u ^ ((u >> 63) | static_cast<long long>(0x8000000000000000ull)));
}
__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }
__device__ __forceinline__ float quick_exp(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
__device__ __forceinline__ float quick_inverse(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float sigmoid_slope(float l) {  // s (1 - s), small on both sides
    const float e = expf(-fabsf(l)), q = 1.0f + e;
    return e / (q * q);
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

// How a token's experts lie in its lanes: groups of `size` experts in 2^lanes_log2 lanes each, `each` to a lane.  Set on
// the host (divisions).
struct Layout {
    int G, size, each, lanes_log2;
    Layout() = default;
    Layout(int lanes, int E, int groups) : G(groups), size(E / groups), lanes_log2(0) {
        int slots = 1;  // groups, up to a power of two
        while (slots < G) slots *= 2;
        while ((slots << (lanes_log2 + 1)) <= lanes) ++lanes_log2;
        each = (size + (1 << lanes_log2) - 1) >> lanes_log2;
    }
};
// Lane `sub` has `count` experts from `first` on, all of group `group`.
struct Place {
    int sub, per_group, group, first, count;  // per_group: lanes of a group
    __device__ __forceinline__ Place(int lanes, const Layout& l) {
        sub = threadIdx.x & (lanes - 1);
        per_group = 1 << l.lanes_log2;
        group = sub >> l.lanes_log2;
        const int at = (sub & (per_group - 1)) * l.each;
        first = group * l.size + at;
        count = group < l.G ? max(0, min(l.each, l.size - at)) : 0;
    }
};

struct RouteArgs {
    const float* bias;
    Layout layout;  // set at the launch, by the lanes of a token
    int T, E, k, q, sigmoid, G, kept, renorm;  // q: experts whose c make a group's score
    float scale;
    int32_t* idx;
    float *w, *scores;
};

// ---------------------------------------------------------------------------------------------
// The k best of a few experts in fp64, for the tokens of the warp that are `unsure`: of the experts whose fp32 value is
// `from` at least (the k best are among them), one to a lane; slot j's in lane j, or -1 in all lanes where they are more
// than 32 or one is NaN.  `open`: this lane's may be chosen.
// ---------------------------------------------------------------------------------------------
template <int LANES, int EPL, typename L>
__device__ __noinline__ int choose_few64(const L* logits, size_t t, int E, const float* bias, int first, int count, bool open,
                                         bool unsure, float from, float top, float inv, int sigmoid_) {
    using Key = unsigned long long;
    __shared__ int list[kWarps][32];
    constexpr int kTokens = 32 / LANES;
    int* const own = list[threadIdx.x >> 5];
    const int lane = threadIdx.x & 31;
    unsigned todo = 0u;
    bool few = true;
    if (unsure && open) {
#pragma unroll 2
        for (int i = 0; i < count; ++i) {
            const float l = logit(logits + t * E + first + i), b = bias ? __ldg(bias + first + i) : 0.0f;
            const float c = (sigmoid_ ? quick_inverse(1.0f + quick_exp(-l)) : quick_exp(l - top) * inv) + b;
            if (!(c < from)) todo |= 1u << i;
            few &= c == c;
        }
    }
    const int n = __popc(todo);
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(kAll, upto, o);
        if (lane >= o) upto += v;
    }
    const int all = __shfl_sync(kAll, upto, 31);
    if (!__all_sync(kAll, few) || all > 32) return -1;
    for (int at = upto - n; todo; todo &= todo - 1) own[at++] = (first + __ffs(todo) - 1) | (lane / LANES) << 16;
    __syncwarp();
    const int e = lane < all ? own[lane] & 0xffff : 0, token = lane < all ? own[lane] >> 16 : -1;
    const size_t my_t = __shfl_sync(kAll, static_cast<unsigned long long>(t), max(token, 0) * LANES);
    const double my_top = __shfl_sync(kAll, top, max(token, 0) * LANES);
    double total = 1.0;
    if (!sigmoid_) {
        const unsigned which = __ballot_sync(kAll, unsure);
#pragma unroll 1
        for (int u = 0; u < kTokens; ++u) {
            if (!(which >> (u * LANES) & 1u)) continue;
            const L* row = logits + __shfl_sync(kAll, static_cast<unsigned long long>(t), u * LANES) * E;
            const double row_top = __shfl_sync(kAll, top, u * LANES);
            double sum = 0.0;
#pragma unroll 4
            for (int i = lane; i < E; i += 32) sum += exp(logit(row + i) - row_top);
            sum = lanes_sum<32>(sum);
            if (token == u) total = sum;
        }
    }
    Key key = 0ull;
    if (token >= 0) {
        const double l = logit(logits + my_t * E + e);
        double c = exp(sigmoid_ ? -l : l - my_top);
        c = (sigmoid_ ? 1.0 : c) / (sigmoid_ ? 1.0 + c : total);
        key = ordered(bias ? c + static_cast<double>(__ldg(bias + e)) : c);
    }
    // An expert's slot is the number of those before it.
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < all; ++i) {
        const Key v = __shfl_sync(kAll, key, i);
        const int other = __shfl_sync(kAll, e, i);
        rank += __shfl_sync(kAll, token, i) == token && (v > key || (v == key && other < e));
    }
    __syncwarp();
    own[lane] = 0;
    __syncwarp();
    if (token >= 0 && rank < 8) own[token * LANES + rank] = e;
    __syncwarp();
    return own[lane];
}

// ---------------------------------------------------------------------------------------------
// The same of any, groups among them.  Only the experts that the fp32 values leave in question are computed
// again, a lane's one after another: in each group those that may be of its q largest, and then in the kept groups those
// that may be of the k largest.  (Seldom run, so kept small: cold instructions take as long as the arithmetic.)
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ double key_value64(unsigned long long k) {
    return k == 1ull ? static_cast<double>(NAN) : __longlong_as_double(static_cast<long long>(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}
template <int LANES, int EPL, typename L>
__device__ __noinline__ int choose64(const L* row, const float* bias, int size, int each, int lanes_log2, int many, int sigmoid_) {
    using Key = unsigned long long;
    struct {
        int G, kept, k, q, sigmoid;
    } a = {many & 63, many >> 6 & 63, many >> 12 & 15, many >> 16, sigmoid_};
    Layout layout;
    layout.G = a.G, layout.size = size, layout.each = each, layout.lanes_log2 = lanes_log2;
    const Place p(LANES, layout);
    const int lane = threadIdx.x & 31;
    float top = -INFINITY;
    bool bad = false, nan = false;  // a logit is NaN (or +inf: a softmax over it is NaN throughout); one of c is
    double total = 1.0;
#pragma unroll 1
    for (int i = 0; i < p.count; ++i) {
        const float l = logit(row + p.first + i);
        bad |= l != l;
        nan |= bias && bias[p.first + i] != bias[p.first + i];  // (of that expert alone)
        top = fmaxf(top, l);
    }
    if (!a.sigmoid) {
        top = lanes_max<LANES>(top);
        bad |= top == INFINITY;
        total = bad ? static_cast<double>(NAN) : 0.0;
#pragma unroll 2
        for (int i = 0; i < p.count; ++i) {
            const float l = logit(row + p.first + i);
            if (top > -INFINITY) total += exp(static_cast<double>(l) - static_cast<double>(top));
        }
        total = lanes_sum<LANES>(total);
    }
    auto exactly = [&](int e) {
        const float l = logit(row + e);
        double c;
        if (a.sigmoid) c = 1.0 / (1.0 + exp(-static_cast<double>(l)));
        else c = top == -INFINITY && total == total ? 0.0 : exp(static_cast<double>(l) - static_cast<double>(top)) / total;
        return bias ? c + static_cast<double>(__ldg(bias + e)) : c;
    };
    // In fp32, and how far off that may be.
    float c[EPL], bulk = 0.0f, score = 0.0f;
    const float inv = 1.0f / static_cast<float>(total);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        c[i] = -INFINITY;
        if (i < p.count) {
            const float l = logit(row + p.first + i), s = a.sigmoid ? sigmoid(l) : top == -INFINITY ? 0.0f : expf(l - top) * inv;
            c[i] = bias ? s + __ldg(bias + p.first + i) : s;
            bulk = fmaxf(bulk, fabsf(c[i]));
            score = fmaxf(score, s);
        }
    }
    const float off = a.sigmoid ? kSigmoidRel + kSigmoidAbs : kSoftmaxRel * lanes_max<LANES>(score) + 0.37f * kSoftmaxArg;
    const float margin = 2.0f * (off + 1.2e-7f * lanes_max<LANES>(bulk));
    nan = __any_sync(kAll, nan || bad);  // then every expert of the warp's tokens is in question
    Key key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = 0ull;
    unsigned open = (1u << p.count) - 1, known = 0u;  // experts that may be chosen; that are computed
    // The n-th largest fp32 value of the open experts of `lanes` lanes.
    auto nth = [&](int n, int lanes) {
        unsigned left = open;
        uint32_t all = 0u;
#pragma unroll 1
        for (int r = 0; r < n; ++r) {
            uint32_t m = 0u;
            int at = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if ((left >> i & 1u) && ordered(c[i]) > m) {
                    m = ordered(c[i]);
                    at = i;
                }
            all = m;
            for (int o = lanes / 2; o > 0; o >>= 1) all = max(all, __shfl_xor_sync(kAll, all, o));
            const unsigned has = __ballot_sync(kAll, m == all) >> (lane & ~(lanes - 1));
            if ((lane & (lanes - 1)) == __ffs(has) - 1) left &= ~(1u << at);
        }
        return all <= 1u ? -INFINITY : __uint_as_float(all & 0x80000000u ? all ^ 0x80000000u : ~all);
    };
    auto compute = [&](float from) {  // the open experts whose fp32 value is `from` at least
        unsigned todo = 0u;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (((open & ~known) >> i & 1u) && (nan || !(c[i] < from))) todo |= 1u << i;
        known |= todo;
#pragma unroll 1
        while (__any_sync(kAll, todo != 0u)) {
            const int at = todo ? __ffs(todo) - 1 : -1;
            const Key v = todo ? ordered(exactly(p.first + at)) : 0ull;
            todo &= todo - 1;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == at) key[i] = v;
        }
    };
    // The largest key of `lanes` neighbouring lanes, taken out where the first lane and place hold it (that expert, there).
    unsigned out = 0u;
    auto best = [&](int lanes, bool& mine, int& at) {
        Key m = 0ull;
        at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (((open & ~out) >> i & 1u) && key[i] > m) {
                m = key[i];
                at = i;
            }
        Key all = m;
        for (int o = lanes / 2; o > 0; o >>= 1) all = max(all, __shfl_xor_sync(kAll, all, o));
        const unsigned has = __ballot_sync(kAll, m == all) >> (lane & ~(lanes - 1));
        mine = (lane & (lanes - 1)) == __ffs(has) - 1;
        if (mine) out |= 1u << at;
        return all;
    };
    bool mine;
    int at;
    if (a.kept < a.G) {
        compute(nth(a.q, p.per_group) - margin);
        double sum = 0.0;
#pragma unroll 1
        for (int r = 0; r < a.q; ++r) sum += key_value64(best(p.per_group, mine, at));
        const Key own = ordered(sum);
        int rank = 0;
#pragma unroll 1
        for (int g = 0; g < a.G; ++g) {
            const Key v = __shfl_sync(kAll, own, g * p.per_group, LANES);
            rank += v > own || (v == own && g < p.group);
        }
        if (rank >= a.kept || p.group >= a.G) open = 0u;
        out = 0u;
    }
    compute(nth(a.k, LANES) - margin);
    int slot = 0;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
        best(LANES, mine, at);
        const unsigned who = __ballot_sync(kAll, mine) >> (lane & ~(LANES - 1));
        const int e = __shfl_sync(kAll, p.first + at, __ffs(who) - 1, LANES);
        if (p.sub == j) slot = e;
    }
    return slot;
}

// ---------------------------------------------------------------------------------------------
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

// Batcher's odd-even merge sort of a lane's keys, the largest first.
template <int N>
__device__ __forceinline__ void sort_falling(uint32_t (&k)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(k[i + j], k[i + j + q]), lo = min(k[i + j], k[i + j + q]);
                        k[i + j] = hi;
                        k[i + j + q] = lo;
                    }
}
// The value of a key (-inf of none, NaN as none: rows with NaN are done in fp64).
__device__ __forceinline__ float key_value(uint32_t k) {
    return k <= 1u ? -INFINITY : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A lane's values of a row, four at a time where `vec` (all lanes' experts are fours of a row aligned for them).
template <int EPL>
__device__ __forceinline__ void read_row(float (&l)[EPL], const float* p, int count, bool vec, float none) {
    if (EPL % 4 == 0 && vec) {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
            float4 v = make_float4(none, none, none, none);
            if (i < count) v = __ldg(reinterpret_cast<const float4*>(p + i));
            l[i] = v.x;
            if (i + 3 < EPL) l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = i < count ? __ldg(p + i) : none;
}
template <int EPL>
__device__ __forceinline__ void read_row(float (&l)[EPL], const __nv_bfloat16* p, int count, bool vec, float none) {
    if (EPL % 4 == 0 && vec) {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
            float v[4] = {none, none, none, none};
            if (i < count) {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + i));
                unpack_bf16x2(u.x, v[0], v[1]);
                unpack_bf16x2(u.y, v[2], v[3]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < EPL) l[i + j] = v[j];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = i < count ? logit(p + i) : none;
}

template <int LANES, int EPL, typename L>
__global__ void __launch_bounds__(kWarps * 32) route_scores_kernel(const L* __restrict__ logits, RouteArgs a) {
    __shared__ uint2 slots[kWarps][32];          // of each token up to 8: key, and place in the lists
    __shared__ uint32_t lists[kWarps][EPL][32];  // each lane's keys, the largest first, then 0 (read by that lane alone)
    pdl_wait();
    pdl_trigger();
    constexpr int kTokens = 32 / LANES;
    const Place p(LANES, a.layout);
    const int lane = threadIdx.x & 31, base = lane & ~(LANES - 1);  // the token's first lane
    const unsigned own_lanes = LANES == 32 ? kAll : (1u << (LANES & 31)) - 1;
    const long long warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (warp * kTokens >= a.T) return;  // whole warps leave
    const long long want = warp * kTokens + lane / LANES;
    const bool there = want < a.T;
    const size_t t = static_cast<size_t>(there ? want : a.T - 1);
    const L* row = logits + t * a.E;
    const bool plain = !a.bias && a.G == 1;  // the order of the logits themselves
    const bool fours = ((a.layout.size | a.layout.each) & 3) == 0;
    const auto words = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(a.bias) |
                       reinterpret_cast<uintptr_t>(a.scores);
    const bool vec = fours && (words & 15) == 0;

    float l[EPL];
    read_row<EPL>(l, row + p.first, p.count, vec, -INFINITY);
    float top = 0.0f, total = 1.0f, c[EPL];
    const bool exactly = a.scores != nullptr;  // (scores that leave the kernel come from expf)
    if (!a.sigmoid && (!plain || !a.renorm || exactly)) {
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) top = fmaxf(top, l[i]);
        top = lanes_max<LANES>(top);
        total = 0.0f;
        // (weights that are parts of the sum have it from expf, too)
        if (a.renorm && !exactly) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                c[i] = i < p.count && !(top == -INFINITY && l[i] == l[i]) ? quick_exp(l[i] - top) : 0.0f;
                total += c[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                c[i] = i < p.count && !(top == -INFINITY && l[i] == l[i]) ? expf(l[i] - top) : 0.0f;
                total += c[i];
            }
        }
        total = lanes_sum<LANES>(total);
    }
    auto score = [&](float v) {
        if (a.sigmoid) return sigmoid(v);
        return top == -INFINITY && total == 0.0f ? 0.0f : expf(v - top) / total;
    };
    uint32_t key[EPL];
    bool nan = false;
    if (exactly) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = score(l[i]);
        float* out = a.scores + t * a.E + p.first;
        if (there) {
            if (EPL % 4 == 0 && vec) {
#pragma unroll
                for (int i = 0; i + 3 < EPL; i += 4)
                    if (i < p.count) *reinterpret_cast<float4*>(out + i) = make_float4(c[i], c[i + 1], c[i + 2], c[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (i < p.count) out[i] = c[i];
            }
        }
    }
    if (plain) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = i < p.count ? ordered(l[i]) : 0u;
    } else {
        float b[EPL];
        if (a.bias) read_row<EPL>(b, a.bias + p.first, p.count, vec, 0.0f);
        if (!exactly && a.sigmoid) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = quick_inverse(1.0f + quick_exp(-l[i]));
        } else if (!exactly) {
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] *= inv;
        }
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] += b[i];
        }
        float all = 0.0f;  // NaN where one of them is (or infinities of both signs are there); no expert's c is 0
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            all += c[i];
            key[i] = i < p.count ? ordered_score(c[i]) : 0u;
        }
        nan = all != all;
    }
    bool sure = plain || !nan;  // the fp32 order is that of the definition
    bool open = true;           // this lane's group is kept
    uint32_t head;  // the largest that is left of this lane's keys, at `pos` of its list
    float t1, t2;   // the largest two
    {
        uint32_t sorted[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) sorted[i] = key[i];
        sort_falling<EPL>(sorted);
        head = sorted[0];
        t1 = key_value(sorted[0]);
        t2 = EPL > 1 ? key_value(sorted[EPL > 1 ? 1 : 0]) : -INFINITY;
#pragma unroll
        for (int i = 1; i < EPL; ++i) lists[threadIdx.x >> 5][i - 1][lane] = sorted[i];
        lists[threadIdx.x >> 5][EPL - 1][lane] = 0u;
    }
    auto next_of = [&](int& pos) { return lists[threadIdx.x >> 5][min(pos++, EPL - 1)][lane]; };
    if (a.G > 1 && a.kept < a.G) {
        // A group's score: its q largest, all groups at once.  In eighths, exact but below 2^-123: the sum of up to eight
        // masks of the lowest float is a number, too.  A mask of -inf has no error.
        const int q = a.q;
        float sum = 0.0f, bulk = 0.0f;  // bulk: sum of sizes
        auto add = [&](float v) {
            sum = fmaf(v, 0.125f, sum);
            bulk += v == -INFINITY ? 0.0f : fabsf(v) * 0.125f;
        };
        if (q <= 2) {
            for (int o = p.per_group / 2; o > 0; o >>= 1) {
                const float o1 = __shfl_xor_sync(kAll, t1, o), o2 = __shfl_xor_sync(kAll, t2, o);
                t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
                t1 = fmaxf(t1, o1);
            }
            add(t1);
            if (q == 2) add(t2);
        } else {
            uint32_t rest = head;
            int pos = 0;
            for (int r = 0; r < q; ++r) {
                uint32_t all = rest;
                for (int o = p.per_group / 2; o > 0; o >>= 1) all = max(all, __shfl_xor_sync(kAll, all, o));
                const unsigned has = __ballot_sync(kAll, rest == all) >> (lane & ~(p.per_group - 1));
                if ((lane & (p.per_group - 1)) == __ffs(has) - 1) rest = next_of(pos);
                add(key_value(all));
            }
        }
        // The error of a sum: its scores' and its additions'.
        const bool real = p.group < a.G;
        const float inv = 1.0f / total;  // (no score is above it)
        const float off = 0.125f * (a.sigmoid ? q * (kSigmoidRel + kSigmoidAbs) : fminf(1.0f, q * inv) * kSoftmaxRel + q * inv * 0.37f * kSoftmaxArg) +
                          bulk * ((q + 2) * 6e-8f);
        const uint32_t g = real ? ordered(sum) : 0u;
        int rank = 0;  // groups with a larger sum
#pragma unroll 4
        for (int o = 0; o < a.G; ++o) rank += __shfl_sync(kAll, g, o << a.layout.lanes_log2, LANES) > g;
        const bool kept = real && rank < a.kept;
        const int many = __popc(__ballot_sync(kAll, kept) >> base & own_lanes);  // more than asked for where sums are equal
        const uint32_t least = ~lanes_max<LANES>(kept ? ~ordered(sum - off) : 0u), next = lanes_max<LANES>(real && !kept ? ordered(sum + off) : 0u);
        if (many != a.kept << a.layout.lanes_log2 || least <= next || least <= 1u) sure = false;
        open = kept;
        head = kept ? head : 0u;
    }
    const bool groups_sure = sure;
    // The slots: the lane whose key is the largest writes its key and where it took it from.
    const uint32_t* const list = &lists[threadIdx.x >> 5][0][0];
    int place = lane;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
        const uint32_t all = lanes_max<LANES>(head);
        const int winner = __ffs(__ballot_sync(kAll, head == all) >> base & own_lanes) - 1;
        if (p.sub == winner) {
            slots[threadIdx.x >> 5][base + j] = make_uint2(all, place);
            head = list[min(place, 32 * (EPL - 1) + lane)];
            place += 32;
        }
    }
    __syncwarp();
    const uint2 slot = slots[threadIdx.x >> 5][base + min(p.sub, a.k - 1)];
    const uint32_t my_key = slot.x;
    const int my_lane = slot.y & (LANES - 1);
    // How often a slot's key of its lane came before: equal ones follow one another.  (Equal scores are done in fp64.)
    int my_rep = 0;
    if (plain) {
        const uint32_t key_before = __shfl_up_sync(kAll, my_key, 1, LANES);
        const int lane_before = __shfl_up_sync(kAll, my_lane, 1, LANES);
        const unsigned again = __ballot_sync(kAll, p.sub > 0 && my_key == key_before && my_lane == lane_before) >> base;
        my_rep = __clz(~(again << (31 - p.sub)));
    }
    int at = 0, seen = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const uint32_t v = __shfl_sync(kAll, key[i], my_lane, LANES);
        if (v == my_key) {
            if (seen == my_rep) at = i;
            ++seen;
        }
    }
    const bool in = p.sub < a.k;
    int my_e = __shfl_sync(kAll, p.first, my_lane, LANES) + at;
    if (!in) my_e = 0;
    float my_l = logit(row + my_e);
    if (!plain) {
        // Neighbours in the order have to be further apart than their errors; the last slot's is the best that is left.
        const float inv = 1.0f / total, c = key_value(my_key), x = my_l - top, e = quick_exp(x);  // (e |x| is below 0.37)
        const uint32_t left = lanes_max<LANES>(head);
        const float off = fabsf(c) * 1.2e-7f + (a.sigmoid ? kSigmoidRel + kSigmoidAbs
                                                         : inv * (e * kSoftmaxRel + kSoftmaxArg * fminf(e * fabsf(x), 0.37f)) + 1e-30f);
        const float left_off = fabsf(fmaxf(key_value(left), -FLT_MAX)) * 1.2e-7f +
                               (a.sigmoid ? kSigmoidRel + kSigmoidAbs : inv * (kSoftmaxRel + 0.37f * kSoftmaxArg));
        float next_c = __shfl_down_sync(kAll, c, 1, LANES), next_off = __shfl_down_sync(kAll, off, 1, LANES);
        if (p.sub == a.k - 1) {
            next_c = key_value(left);
            next_off = left_off;
        }
        const bool none_left = p.sub == a.k - 1 && left == 0u;
        if (in && !none_left && !(c - next_c > off + next_off)) sure = false;
        const unsigned unsure = __ballot_sync(kAll, !sure);
        if (unsure) {
            const bool mine = unsure >> base & own_lanes;  // the token is
            int e = -1;
            if (__all_sync(kAll, groups_sure)) {
                const float least = __shfl_sync(kAll, c, a.k - 1, LANES);
                const float most = fabsf(least) * 1.2e-7f + (a.sigmoid ? kSigmoidRel + kSigmoidAbs : inv * (kSoftmaxRel + 0.37f * kSoftmaxArg));
                e = choose_few64<LANES, EPL>(logits, t, a.E, a.bias, p.first, p.count, open, mine, least - 2.1f * most, top, inv, a.sigmoid);
            }
            if (__any_sync(kAll, e < 0))
                e = choose64<LANES, EPL>(row, a.bias, a.layout.size, a.layout.each, a.layout.lanes_log2,
                                         a.G | a.kept << 6 | a.k << 12 | a.q << 16, a.sigmoid);
            if (in && mine) my_e = e;
            my_l = logit(row + my_e);
        }
    }
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

// Fours of a row.
__device__ __forceinline__ void read4(float* v, const float* p) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}
__device__ __forceinline__ void read4(float* v, const __nv_bfloat16* p) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    unpack_bf16x2(u.x, v[0], v[1]);
    unpack_bf16x2(u.y, v[2], v[3]);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// A lane has every LANES-th expert of its token, or (U = 4) every LANES-th four of them.  What the slots add to their
// experts goes through shared memory.
template <int LANES, int EPL, int U, typename L>
__global__ void __launch_bounds__(kWarps * 32)
route_scores_backward_kernel(const L* __restrict__ logits, RouteGradArgs a, L* __restrict__ dlogits) {
    constexpr int kTokens = 32 / LANES;
    __shared__ __align__(16) float sums[kWarps][kTokens][LANES * EPL];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = lane & (LANES - 1);
    const long long warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (warp * kTokens >= a.T) return;
    const long long want = warp * kTokens + lane / LANES;
    const bool there = want < a.T;
    const size_t t = static_cast<size_t>(there ? want : a.T - 1);
    const L* row = logits + t * a.E;
    auto expert = [&](int i) { return (sub + i / U * LANES) * U + i % U; };
    // Of all scores only those that a gradient reaches are needed: the chosen ones, but for a softmax that is not
    // renormalised or whose scores have a gradient of their own.
    const bool dense = a.dscores || (!a.sigmoid && !a.renorm);
    float v[EPL], g[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) g[i] = 0.0f;
    if (dense) {
        const float* ds = a.dscores + (a.per_token ? t * a.E : 0);
#pragma unroll
        for (int i = 0; i < EPL; i += U) {
#pragma unroll
            for (int j = 0; j < U; ++j) v[i + j] = -INFINITY;
            if (expert(i) >= a.E) continue;
            if constexpr (U == 4) {
                read4(v + i, row + expert(i));
                if (a.dscores) read4(g + i, ds + expert(i));
            } else {
                v[i] = logit(row + expert(i));
                if (a.dscores) g[i] = __ldg(ds + expert(i));
            }
        }
    }
    // Slot j in lane j; an expert that there is none of takes part in nothing.
    int e = -1;
    float u = 0.0f, l = 0.0f;
    if (a.dw && sub < a.k) {
        e = __ldg(a.idx + t * a.k + sub);
        u = a.scale * __ldg(a.dw + t * a.k + sub);
        if (e < 0 || e >= a.E) e = -1;
        else l = logit(row + e);
    }
    // What a slot adds to its expert: to dl itself, or (a softmax that is not renormalised) to D.
    float add = e >= 0 ? u : 0.0f;
    const bool to_dl = a.sigmoid || a.renorm;
    if (a.renorm) {  // d(share)/dl needs the shares alone: s / S = r
        const float r = share_of_chosen(l, e >= 0, a.sigmoid);
        const float mean = eight_sum(e >= 0 ? r * u : 0.0f);
        add = e >= 0 ? r * (u - mean) : 0.0f;
        if (a.sigmoid) add *= sigmoid(-l);
    } else if (a.sigmoid) {
        add = e >= 0 ? sigmoid_slope(l) * u : 0.0f;
    }
    float* sum = sums[threadIdx.x >> 5][lane / LANES];  // of the token's experts
    auto scatter = [&] {
        if constexpr (U == 4) {
#pragma unroll
            for (int i = 0; i < EPL; i += 4) *reinterpret_cast<float4*>(sum + expert(i)) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) sum[expert(i)] = 0.0f;
        }
        __syncwarp();
        // Whether an expert is in two slots (a caller's own choice): then one slot after another.
        int* mark = reinterpret_cast<int*>(sum);
        if (e >= 0) mark[e] = lane;
        __syncwarp();
        const bool first = e >= 0 && mark[e] == lane;
        const bool twice = __any_sync(kAll, e >= 0 && !first);
        __syncwarp();
        if (first) sum[e] = twice ? 0.0f : add;
        __syncwarp();
        if (twice)
            for (int j = 0; j < a.k; ++j) {
                if (sub == j && e >= 0) sum[e] += add;
                __syncwarp();
            }
        if constexpr (U == 4) {
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(sum + expert(i));
                g[i] += f.x, g[i + 1] += f.y, g[i + 2] += f.z, g[i + 3] += f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) g[i] += sum[expert(i)];
        }
    };
    if (dense && a.sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) g[i] *= sigmoid_slope(v[i]);
    } else if (dense) {
        if (!to_dl && a.dw) scatter();
        float top = -INFINITY, total = 0.0f, mean = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) top = fmaxf(top, v[i]);
        top = lanes_max<LANES>(top);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool none = expert(i) >= a.E || (top == -INFINITY && v[i] == v[i]);
            v[i] = none ? 0.0f : expf(v[i] - top);
            total += v[i];
            mean = fmaf(v[i], g[i], mean);
        }
        total = lanes_sum<LANES>(total);
        mean = lanes_sum<LANES>(mean);
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        mean *= inv;
#pragma unroll
        for (int i = 0; i < EPL; ++i) g[i] = v[i] * inv * (g[i] - mean);
    }
    if (to_dl && a.dw) scatter();
    if (!there) return;
#pragma unroll
    for (int i = 0; i < EPL; i += U) {
        if (expert(i) >= a.E) continue;
        if constexpr (U == 4) store4(dlogits + t * a.E + expert(i), g + i);
        else store_grad(dlogits + t * a.E + expert(i), g[i]);
    }
}

// Experts of a lane; far too many where the lanes are fewer than the groups.
int experts_per_lane(int lanes, int E, int G) {
    int slots = 1;
    while (slots < G) slots *= 2;
    return slots > lanes ? 1 << 30 : Layout(lanes, E, G).each;
}
template <int LANES, int EPL, typename L>
cudaError_t forward_with(const L* logits, RouteArgs a, cudaStream_t s) {
    a.layout = Layout(LANES, a.E, a.G);
    return launch_k(kPdlTrain, route_scores_kernel<LANES, EPL, L>, dim3((a.T - 1) / (kWarps * (32 / LANES)) + 1),
                    dim3(kWarps * 32), 0, s, logits, a);
}
template <typename L>
cudaError_t forward_as(const L* logits, const RouteArgs& a, cudaStream_t s) {
    const int n8 = a.E <= 64 ? experts_per_lane(8, a.E, a.G) : 1 << 30, n32 = experts_per_lane(32, a.E, a.G);
    if (n8 <= 2) return forward_with<8, 2>(logits, a, s);
    if (n8 <= 8) return forward_with<8, 8>(logits, a, s);
    if (n32 <= 2) return forward_with<32, 2>(logits, a, s);
    if (n32 <= 4) return forward_with<32, 4>(logits, a, s);
    if (n32 <= 8) return forward_with<32, 8>(logits, a, s);
    return forward_with<32, 16>(logits, a, s);
}
template <int LANES, int EPL, int U, typename L>
cudaError_t backward_with(const L* logits, const RouteGradArgs& a, L* dlogits, cudaStream_t s) {
    return launch_k(kPdlTrain, route_scores_backward_kernel<LANES, EPL, U, L>, dim3((a.T - 1) / (kWarps * (32 / LANES)) + 1),
                    dim3(kWarps * 32), 0, s, logits, a, dlogits);
}
template <typename L>
cudaError_t backward_as(const L* logits, const RouteGradArgs& a, L* dlogits, cudaStream_t s) {
    // Fours where the experts are fours and the tensors aligned for them.
    if (a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits)) % (4 * sizeof(L)) == 0 &&
        reinterpret_cast<uintptr_t>(a.dscores) % 16 == 0) {
        if (a.E <= 32) return backward_with<8, 4, 4>(logits, a, dlogits, s);
        if (a.E <= 64) return backward_with<8, 8, 4>(logits, a, dlogits, s);
        if (a.E <= 128) return backward_with<16, 8, 4>(logits, a, dlogits, s);
        if (a.E <= 192) return backward_with<16, 12, 4>(logits, a, dlogits, s);
        return backward_with<16, 16, 4>(logits, a, dlogits, s);
    }
    if (a.E <= 8) return backward_with<8, 1, 1>(logits, a, dlogits, s);
    if (a.E <= 16) return backward_with<8, 2, 1>(logits, a, dlogits, s);
    if (a.E <= 32) return backward_with<8, 4, 1>(logits, a, dlogits, s);
    if (a.E <= 64) return backward_with<8, 8, 1>(logits, a, dlogits, s);
    if (a.E <= 128) return backward_with<32, 4, 1>(logits, a, dlogits, s);
    if (a.E <= 192) return backward_with<32, 6, 1>(logits, a, dlogits, s);
    return backward_with<32, 8, 1>(logits, a, dlogits, s);
}

}  // namespace

cudaError_t launch_route_scores(const void* logits, bool bf16, const float* bias, int T, int E, int k, bool sigmoid,
                                int n_group, int topk_group, bool renorm, float scale, int32_t* idx, float* w,
                                float* scores, cudaStream_t s) {
    const RouteArgs a{bias, Layout(), T, E, k, std::min(E / n_group, std::max(1, k / topk_group)), sigmoid, n_group,
                      topk_group, renorm, scale, idx, w, scores};
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
