// layer_norm.cu — layer norm of a residual stream after a block's output was added to it.  Per row t of d values:
//
//   y = x + drop(h)                                rounded to the stream's type: n is the norm of what is stored
//   mean = sum(y) / d,  r = 1 / sqrt(sum((y - mean)^2) / d + eps)
//   n = weight (y - mean) r + bias
//
// y is bf16 or fp32, h and n bf16, weight, bias and the stats (mean, r) fp32.  layer_norm_backward.cu is its gradient.
//
// One pass over memory; bound by it.  A thread holds its values of a row in registers, with those of its next row on
// their way into shared memory (cp.async: a thread copies just the words that it will use, so no barrier is needed for
// them).  The variance is the sum of squared distances from the mean (no difference of large sums): two reductions,
// one after the other, which other blocks of the SM fill.  The second one also sums the distances themselves, which is
// what the first was off by: the mean is then right to its own rounding, and a constant row's distances are 0 (without
// that 1000.1 gave n = 0.02 for some widths; it costs 0 to 4 %, 8192 x 4096 bf16 26.9 -> 27.7 us, and 0.1 us of a token).
// Rows of up to 256 values are eight lanes' each, rows of up to 1024 eights a block's; wider ones lie in the blocks of a
// cluster, which exchange their warps' sums through each other's shared memory.
#include "layer_norm.cuh"

namespace moe {
namespace {

struct Forward {
    const void* x;
    const __nv_bfloat16* h;
    const float *weight, *bias;
    int T, d;
    float eps;
    DropArgs drop;
    void* y;
    __nv_bfloat16* n;
    float2* stats;
    int blocks, vec, keep;  // blocks of a cluster; keep: the weights lie behind the row
};

// VPT eights to a thread, blockDim.x apart.  LANES: 32 and a block's threads for a row (or those of a cluster), or as many
// lanes of a warp, blockDim.y rows side by side.  WIDE: eight weights as one word.
template <typename X, bool H, bool EDGE, int VPT, int LANES, bool CLUSTER, bool WIDE>
__global__ void __launch_bounds__(LANES == 32 ? 1024 / VPT : 256, LANES == 32 ? VPT : 3)
layer_norm_kernel(const __grid_constant__ Forward a) {
    __shared__ float red[2 * 2 * (CLUSTER ? kMostBlocks * 32 / VPT : 32 / VPT)];
    constexpr bool SIDE = LANES < 32;
    extern __shared__ uint4 next_row[];
    constexpr int W = words<X>() + (H ? 1 : 0);
    const int tid = threadIdx.x, nt = blockDim.x, d = a.d;  // (of a row)
    const float inv_d = 1.0f / static_cast<float>(d);
    const X* x = static_cast<const X*>(a.x);
    X* y = static_cast<X*>(a.y);
    const long long T = a.T, total = T * d, side = SIDE ? blockDim.y : 1, step = gridDim.x / a.blocks * side;
    const long long row0 = blockIdx.x / a.blocks * side + (SIDE ? threadIdx.y : 0), row = step * d;
    // (side by side: as many as the block's first row has, so that a warp's lanes stay together)
    const int rows = static_cast<int>((T - (SIDE ? blockIdx.x * side : row0) - 1) / step) + 1;
    const int own = SIDE ? (row0 < T ? static_cast<int>((T - row0 - 1) / step) + 1 : 0) : rows;
    if (CLUSTER) ptx::cluster_arrive();  // (the other blocks' memory is there once all have begun)
    pdl_wait();
    pdl_trigger();
    if (CLUSTER) ptx::cluster_wait();
    RowSums<CLUSTER, 2> row_sums(red, nt >> 5, 0, a.blocks);
    auto sum_row = [&](auto& s) {
        if constexpr (SIDE) {
            for (float& v : s) v = lanes_sum<LANES>(v);
        } else {
            row_sums(s);
        }
    };
    const int shift = EDGE ? static_cast<int>(row0 * d & 7) : 0, q0 = (CLUSTER ? row_sums.rank * nt * VPT : 0) + tid;
    auto eight = [&](int v) { return Eight<EDGE>(q0 + v * nt, shift, d, a.vec != 0); };
    long long at = row0 * d - shift;  // where the row begins
    uint4* const word = next_row + (SIDE ? threadIdx.y * (VPT * W * nt) : 0) + tid;
    const int span = 8 * ((d + shift + 7) / 8);  // of the eights that a row lies in
    auto fetch = [&](long long base) {
        const long long end = EDGE && base + span > total ? total : 0;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const Eight<EDGE> e = eight(v);
            if (e.some()) {
                e.copy(word + v * W * nt, nt, x, base, end);
                if (H) e.copy(word + (v * W + words<X>()) * nt, nt, a.h, base, end);
            }
        }
        ptx::cp_async_commit();
    };
    if (own > 0) fetch(at);
    // A thread's own words: no barrier.
    float4* const kept = reinterpret_cast<float4*>(next_row + VPT * W * nt) + tid;
    if (EDGE && !SIDE && a.keep) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const Eight<EDGE> e = eight(v);
            if (e.some()) {
                const Vec8 w = e.column(a.weight, 1.0f), b = e.column(a.bias, 0.0f);
                float4* k = kept + 4 * v * nt;
                k[0] = make_float4(w.v[0], w.v[1], w.v[2], w.v[3]);
                k[nt] = make_float4(w.v[4], w.v[5], w.v[6], w.v[7]);
                k[2 * nt] = make_float4(b.v[0], b.v[1], b.v[2], b.v[3]);
                k[3 * nt] = make_float4(b.v[4], b.v[5], b.v[6], b.v[7]);
            }
        }
    }
    const Drop drop(a.drop);
    float2* stats = a.stats + row0;
    for (int k = 0; k < rows; ++k) {
        Vec8 val[VPT];
        const bool here = !SIDE || k < own;
        float2 sum = make_float2(0.0f, 0.0f);
        ptx::cp_async_wait<0>();
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const Eight<EDGE> e = eight(v);
            if (here && e.some()) {
                Vec8& c = val[v];
                c = ring8<X>(word + v * W * nt, nt);
                if (H) {
                    Vec8 hv = ring8<__nv_bfloat16>(word + (v * W + words<X>()) * nt, nt);
                    if (drop.on()) drop.apply(hv, at + e.off);
#pragma unroll
                    for (int j = 0; j < 4; ++j) c.set(j, add2(c.pair(j), hv.pair(j)));
                    c = rounded(c, static_cast<const X*>(nullptr));
                    e.store(y, at, c);
                }
                e.mask(c);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = add2(sum, c.pair(j));
            }
        }
        if (k + 1 < own) fetch(at + row);
        float about[1] = {sum.x + sum.y};  // the mean, but for the errors of its sum
        sum_row(about);
        about[0] *= inv_d;
        float2 back = make_float2(-about[0], -about[0]), square = make_float2(0.0f, 0.0f);
        sum = square;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const Eight<EDGE> e = eight(v);
            if (here && e.some()) {
#pragma unroll
                for (int j = 0; j < 4; ++j) val[v].set(j, add2(val[v].pair(j), back));
                e.mask(val[v]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum = add2(sum, val[v].pair(j));
                    square = fma2(val[v].pair(j), val[v].pair(j), square);
                }
            }
        }
        // The mean with the mean of what it leaves, and the variance about that.  `shift_by` is what the distances change by,
        // exactly where the mean is not near 0 (a difference of close floats): those of a constant row become 0, and its
        // mean the constant.
        float second[2] = {sum.x + sum.y, square.x + square.y};
        sum_row(second);
        const float left = second[0] * inv_d, mean = about[0] + left, shift_by = mean - about[0];
        const float var = second[1] * inv_d - shift_by * (2.0f * left - shift_by);
        const float r = rsqrtf((var < 0.0f ? 0.0f : var) + a.eps);  // (NaN stays)
        back = make_float2(-shift_by, -shift_by);
        if (here && tid == 0 && row_sums.rank == 0) *stats = make_float2(mean, r);
        stats += step;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const Eight<EDGE> e = eight(v);
            if (here && e.some()) {
                Vec8 w, b;
                if (EDGE && !SIDE && a.keep) {
                    const float4* k4 = kept + 4 * v * nt;
                    const float4 p = k4[0], q = k4[nt], f = k4[2 * nt], g = k4[3 * nt];
                    w = Vec8{{p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w}};
                    b = Vec8{{f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w}};
                } else {
                    w = e.template column<WIDE>(a.weight, 1.0f);
                    b = e.template column<WIDE>(a.bias, 0.0f);
                }
                Vec8 o;
#pragma unroll
                for (int j = 0; j < 4; ++j) o.set(j, fma2(mul2(add2(val[v].pair(j), back), r), w.pair(j), b.pair(j)));
                e.store(a.n, at, o);
            }
        }
        at += row;
    }
}

constexpr size_t kSmSmem = 212 * 1024;  // of an SM, for its blocks' rows and weights

// word_bytes: of a row's eight in shared memory; keep: 64 more for its weights.
//   Rows of up to 32 eights: eight lanes each, 32 rows side by side (16384 rows of 256 values: 12 us with a warp each).
//   Others: two eights to a thread (8192 x 7168, fp32 stream with h and dropout: 106 us; with one 131, with four 117), one
//   for up to 64 eights (4000 x 512: 7.7 us against 9.3) and where each block has one row, whose latency counts.
Shape forward_shape(int T, int d, int word_bytes, bool keep) {
    const int eights = eights_of(d);
    Shape s;
    s.groups = 1;
    s.blocks = 1;
    if (eights <= 32) {
        s.vpt = 4;
        s.threads = 8;
        s.groups = 32;
        s.clusters = std::min((T - 1) / 32 + 1, kSms * 3);
        return s;
    }
    while (s.blocks < kMostBlocks && s.blocks * 1024 < eights) s.blocks *= 2;
    const int own = (eights + s.blocks - 1) / s.blocks;  // of a block
    const int fit = static_cast<int>(kSmSmem / (static_cast<size_t>(own) * (word_bytes + (keep ? 64 : 0))));
    for (s.vpt = own <= 64 ? 1 : 2;; s.vpt = 1) {
        s.threads = ((own + s.vpt - 1) / s.vpt + 31) / 32 * 32;
        s.clusters = clusters_for(T, std::max(1, std::min({32, 1024 / s.threads, fit})), s.blocks);
        if (s.vpt == 1 || T > s.clusters) return s;
    }
}

template <typename X, bool H, bool EDGE, int VPT, int LANES, bool CLUSTER, bool WIDE = true>
cudaError_t forward_with(const Forward& a, const Shape& f, int word_bytes, cudaStream_t s) {
    const size_t smem = static_cast<size_t>(f.threads) * f.groups * VPT * (word_bytes + (a.keep ? 64 : 0));
    return launch_rows(layer_norm_kernel<X, H, EDGE, VPT, LANES, CLUSTER, WIDE>, f, smem, s, a);
}
template <typename X, bool H, bool EDGE>
cudaError_t forward_as(Forward a, cudaStream_t s) {
    const int word_bytes = 16 * (words<X>() + (H ? 1 : 0));
    const Shape f = forward_shape(a.T, a.d, word_bytes, EDGE);
    // Weights whose loads would be one by one are read once, where a block has more than one row after another.
    a.keep = EDGE && f.groups == 1 && a.T > f.clusters;
    a.blocks = f.blocks;
    // Weights as two words of four: for an fp32 stream with h whose rows fill a block each, many to a block.  These streams
    // are at the memory's rate, and slower where the weights come faster (us, as two words / as one, with dropout; the
    // cause is not known):
    //   8192 rows of   4096 70/73, 4608 84/82, 5120 81/88, 6144 125/113, 6656 100/108, 7168 105/119, 7680 114/128, 8192 127/139
    //   2000 rows of   4096 17.8/16.6, 5120 23.0/22.6, 6656 28.4/27.3, 7168 30.2/29.7, 8192 33.5/34.8
    // and rows in less than a block or in a cluster: 8192 x 512 11.7/11.1, x 10240 202/194, x 16384 314/305.
    if constexpr (sizeof(X) == 4 && H && !EDGE)
        if (f.blocks == 1 && f.vpt == 2 && a.d >= 5120 && a.T >= 8 * f.clusters) return forward_with<X, H, EDGE, 2, 32, false, false>(a, f, word_bytes, s);
    if (f.threads < 32) return forward_with<X, H, EDGE, 4, 8, false>(a, f, word_bytes, s);
    if (f.blocks > 1)
        return f.vpt == 2 ? forward_with<X, H, EDGE, 2, 32, true>(a, f, word_bytes, s) : forward_with<X, H, EDGE, 1, 32, true>(a, f, word_bytes, s);
    return f.vpt == 2 ? forward_with<X, H, EDGE, 2, 32, false>(a, f, word_bytes, s) : forward_with<X, H, EDGE, 1, 32, false>(a, f, word_bytes, s);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& g, cudaStream_t s) {
    Forward a{g.x, g.h, g.weight, g.bias, g.T, g.d, g.eps, g.drop, g.y, g.n, reinterpret_cast<float2*>(g.stats), 1, 0, 0};
    a.vec = aligned({g.x, g.h, g.y, g.n});
    const bool edge = g.d % 8 != 0 || !a.vec || !aligned({g.weight, g.bias}, 31);
    using B = __nv_bfloat16;
    if (g.x_fp32) {
        if (g.h) return edge ? forward_as<float, true, true>(a, s) : forward_as<float, true, false>(a, s);
        return edge ? forward_as<float, false, true>(a, s) : forward_as<float, false, false>(a, s);
    }
    if (g.h) return edge ? forward_as<B, true, true>(a, s) : forward_as<B, true, false>(a, s);
    return edge ? forward_as<B, false, true>(a, s) : forward_as<B, false, false>(a, s);
}

}  // namespace moe
