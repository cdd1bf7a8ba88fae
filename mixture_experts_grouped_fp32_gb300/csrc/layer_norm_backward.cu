// layer_norm_backward.cu — the gradient of layer_norm.cu.  Given dn and dy, with yh = (y - mean) r and g = dn weight:
//
//   dx = dy + r (g - mean(g) - yh mean(g yh)),  dh = drop(dx) with the same mask
//   dweight = sum_t dn yh,  dbias = sum_t dn
//
// One pass over memory.  A thread holds two eights, of two rows or of one, and the column sums of its columns, with the
// next eights on their way into shared memory (cp.async).  A row that is wider than a block's threads hold lies in the
// blocks of a cluster, which exchange their warps' sums through each other's shared memory.  The column sums of a
// block's rows are written once, and a second kernel adds the blocks in a fixed order: no atomics, the same result on
// every run.  They are fp32 sums of a block's rows one after another: off by as many 2^-24 of the terms' sizes at the most
// as a block has rows (8192 x 4096 27, 16384 x 65536 1024; by about the root of that in earnest), and by some 40 more for
// the join.  A second sum for each column would cost the registers that hold two eights.
//
// What bounds it: memory, with about 300 instructions to a warp's two eights close behind.  In a graph, with dh:
// 8192 x 4096 bf16 57 us (86 % of the copy rate), fp32 84 us (94 %), 2932 x 8192 bf16 44 us (80 %).  Rows of odd widths
// pay for the masks and the single values at both ends: 16000 x 2891 105 us (65 %).  In a cluster each row waits for the
// others' sums: 1422 x 16384 bf16 58 us (59 %), 4000 x 12288 fp32 160 us (73 %).
#include "layer_norm.cuh"

namespace moe {
namespace {

// Pairs of eights in a thread's ring (512 threads: 147 KB, 164 KB with an fp32 stream).
template <typename X>
constexpr int pair_stages() { return sizeof(X) == 4 ? 2 : 3; }

struct Backward {
    const void* x;
    const float2* stats;
    const __nv_bfloat16* dn;
    const void* dy;
    const float* weight;
    int T, d;
    DropArgs drop;
    void* dx;
    __nv_bfloat16* dh;
    float* partial;  // [clusters, 2, 8 eights], or null
    int blocks, vec, eights;
};

// Two eights to a thread: of two rows (VPT 1), whose four sums share a reduction, or of one (VPT 2).  The column sums
// dweight and dbias of the rows that a block visits stay in registers and are written once; rows that are narrower than
// the block lie side by side in it (threadIdx.y), each with its barrier, and their sums are added up first.
template <typename X, bool EDGE, int VPT, bool CLUSTER>
__global__ void __launch_bounds__(512, 1) layer_norm_backward_kernel(const __grid_constant__ Backward a) {
    __shared__ float red[2 * 4 * (CLUSTER ? kMostBlocks * 16 : 16)];
    extern __shared__ uint4 ring_all[];
    constexpr int R = 2 / VPT;  // rows at a time
    using B = __nv_bfloat16;
    const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, d = a.d, groups = CLUSTER ? 1 : blockDim.y, group = threadIdx.y;
    const float inv_d = 1.0f / static_cast<float>(d);
    const X *x = static_cast<const X*>(a.x), *dy = static_cast<const X*>(a.dy);
    X* dx = static_cast<X*>(a.dx);
    const long long T = a.T, total = T * d, clusters = gridDim.x / a.blocks, cluster = blockIdx.x / a.blocks;
    const long long row0 = cluster + clusters * group, step = clusters * groups;
    const int rows = row0 < T ? static_cast<int>((T - row0 - 1) / step) + 1 : 0;
    if (CLUSTER) ptx::cluster_arrive();
    pdl_wait();
    pdl_trigger();
    if (CLUSTER) ptx::cluster_wait();
    RowSums<CLUSTER, 2 * R> row_sum(red + (CLUSTER ? 0 : 4 * R * warps * group), warps, groups > 1 ? 1 + group : 0, a.blocks);
    const Drop drop(a.drop);
    const int shift = EDGE ? static_cast<int>(cluster * d & 7) : 0;
    const int q0 = (CLUSTER ? row_sum.rank * nt * VPT : 0) + tid;
    auto eight = [&](int v) { return Eight<EDGE>(q0 + v * nt, shift, d, a.vec != 0); };
    // Words of a row: x, dn, dy.
    constexpr int o_dn = words<X>(), o_dy = o_dn + 1, W = o_dy + words<X>(), S = pair_stages<X>();
    const long long row = step * d;
    long long in = row0 * d - shift, out = in;  // where the row to copy next begins, and the one to write
    uint4* const first = ring_all + group * (S * 2 * W * nt) + tid;
    uint4* const last = first + (S - 1) * 2 * W * nt;
    uint4* slot = first;  // the words of the rows to copy next, of the rows to work on
    const uint4* word = first;
    int copied = 0;
    const int span = 8 * ((d + shift + 7) / 8);  // of the eights that a row lies in
    auto fetch = [&] {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const Eight<EDGE> e = eight(m / R);
            if (copied < rows && e.some()) {
                uint4* w = slot + m * W * nt;
                const long long end = EDGE && in + span > total ? total : 0;
                e.copy(w, nt, x, in, end);
                e.copy(w + o_dn * nt, nt, a.dn, in, end);
                if (dy) e.copy(w + o_dy * nt, nt, dy, in, end);
            }
            if (R == 2 || m == 1) {
                in += row;
                ++copied;
            }
        }
        ptx::cp_async_commit();
        slot = slot == last ? first : slot + 2 * W * nt;
    };
    float2 st[R] = {}, next[R] = {};
    const float2* stats = a.stats + row0;  // of the rows to read next
    int stats_left = rows;
    auto read_stats = [&] {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (stats_left > 0) next[i] = __ldg(stats);
            stats += step;
            --stats_left;
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < S; ++k) fetch();
    read_stats();
    // The weights: in registers, or (VPT 2) a thread's own words behind the ring.
    float4* const kept = reinterpret_cast<float4*>(ring_all + groups * (S * 2 * W * nt)) + group * (4 * nt) + tid;
    Vec8 w0{};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const Eight<EDGE> e = eight(v);
        if (!e.some()) continue;
        w0 = e.column(a.weight, 1.0f);
        if (VPT == 2) {
            kept[2 * v * nt] = make_float4(w0.v[0], w0.v[1], w0.v[2], w0.v[3]);
            kept[(2 * v + 1) * nt] = make_float4(w0.v[4], w0.v[5], w0.v[6], w0.v[7]);
        }
    }
    auto weight = [&](int v) {
        if (VPT == 1) return w0;
        const float4 f = kept[2 * v * nt], h = kept[(2 * v + 1) * nt];
        return Vec8{{f.x, f.y, f.z, f.w, h.x, h.y, h.z, h.w}};
    };
    Vec8 sw[VPT] = {}, sb[VPT] = {};
    for (int k = 0; k < rows; k += R) {
        fetch();
#pragma unroll
        for (int i = 0; i < R; ++i) st[i] = next[i];
        read_stats();
        ptx::cp_async_wait<S - 1>();
        const bool two = k + 1 < rows;
        Vec8 yh[2], g[2];
        float s[2 * R];
#pragma unroll
        for (int i = 0; i < 2 * R; ++i) s[i] = 0.0f;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int i = R == 2 ? m : 0, v = R == 2 ? 0 : m;  // row, eight
            const Eight<EDGE> e = eight(v);
            if (e.some() && (i == 0 || two)) {
                const float r = st[i].y;
                const float2 back = make_float2(-st[i].x, -st[i].x);
                const Vec8 w = weight(v);
                float2 sg, sy;
                yh[m] = ring8<X>(word + m * W * nt, nt);
                Vec8 nv = ring8<B>(word + (m * W + o_dn) * nt, nt);
                e.mask(yh[m]);
                e.mask(nv);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    yh[m].set(j, mul2(add2(yh[m].pair(j), back), r));
                    g[m].set(j, mul2(nv.pair(j), w.pair(j)));
                    sg = j ? add2(sg, g[m].pair(j)) : g[m].pair(j);
                    sy = j ? fma2(g[m].pair(j), yh[m].pair(j), sy) : mul2(g[m].pair(j), yh[m].pair(j));
                    sw[v].set(j, fma2(nv.pair(j), yh[m].pair(j), sw[v].pair(j)));
                    sb[v].set(j, add2(sb[v].pair(j), nv.pair(j)));
                }
                s[2 * i] += sg.x + sg.y;
                s[2 * i + 1] += sy.x + sy.y;
            }
        }
        row_sum(s);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int i = R == 2 ? m : 0, v = R == 2 ? 0 : m;
            const Eight<EDGE> e = eight(v);
            if (e.some() && (i == 0 || two)) {
                // (r taken into the means: r (g - mg - yh my) + dy)
                const float r = st[i].y, mg = -s[2 * i] * inv_d * r, my = -s[2 * i + 1] * inv_d * r;
                Vec8 o;
                if (dy) {
                    o = ring8<X>(word + (m * W + o_dy) * nt, nt);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o.set(j, add2(o.pair(j), make_float2(mg, mg)));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o.v[j] = mg;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) o.set(j, fma2(g[m].pair(j), r, fma2(yh[m].pair(j), my, o.pair(j))));
                e.store(dx, out, o);
                if (a.dh) {
                    if (drop.on()) drop.apply(o, out + e.off);
                    e.store(a.dh, out, o);
                }
            }
            if (R == 2 || m == 1) out += row;
        }
        word = word == last ? first : word + 2 * W * nt;
    }
    ptx::cp_async_wait_all();
    if (!a.partial) return;
    // In eights of this cluster's shift, as wide as any.
    const size_t width = 8 * static_cast<size_t>(a.eights);
    float* p = a.partial + static_cast<size_t>(cluster) * 2 * width;
    float* sums = reinterpret_cast<float*>(ring_all);  // [rows side by side][8][threads of a row], once all are done
#pragma unroll
    for (int k = 0; k < 2 * VPT; ++k) {  // dweight, then dbias
        const Vec8& own = k < VPT ? sw[k % VPT] : sb[k % VPT];
        const Eight<EDGE> e = eight(k % VPT);
        float* to = p + (k / VPT) * width + e.off;
        if (groups == 1) {
            if (e.some()) store8(to, 0, own);
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[(group * 8 + j) * nt + tid] = own.v[j];
        __syncthreads();
        if (group == 0 && e.some()) {
            Vec8 v = own;
            for (int o = 1; o < groups; ++o)
#pragma unroll
                for (int j = 0; j < 8; ++j) v.v[j] += sums[(o * 8 + j) * nt + tid];
            store8(to, 0, v);
        }
    }
}

// Adds the blocks' column sums in block order (16 runs of blocks, then the runs).
__global__ void __launch_bounds__(512)
layer_norm_join_kernel(const float* __restrict__ partial, int blocks, int d, int eights, float* __restrict__ dweight,
                       float* __restrict__ dbias) {
    __shared__ float part[16][33];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int c = (blockIdx.x >> 1) * 32 + lane, which = blockIdx.x & 1;  // column, of dweight or dbias
    const size_t width = 8 * static_cast<size_t>(eights);
    const int per = (blocks + 15) / 16, b0 = min(run * per, blocks), b1 = min(b0 + per, blocks);
    pdl_wait();
    pdl_trigger();
    float s = 0.0f;
    if (c < d) {
        const float* p = partial + which * width + c;
#pragma unroll 10
        for (int b = b0; b < b1; ++b)  // (where a block's rows start inside their first eight)
            s += __ldcg(p + b * 2 * width + (static_cast<unsigned>(b) * static_cast<unsigned>(d) & 7));
    }
    part[run][lane] = s;
    __syncthreads();
    if (run == 0 && c < d) {
        float a = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) a += part[k][lane];
        float* out = which ? dbias : dweight;
        if (out) out[c] = a;
    }
}

Shape backward_shape(int T, int d) {
    const int most = 512, eights = eights_of(d);  // threads of an SM, all of its blocks together
    Shape s;
    s.blocks = 1;
    // Two eights of one row halve a wide row's threads: 8192 x 4096 bf16 58 -> 56 us, 16000 x 2891 118 -> 105 us.  Two
    // rows at a time win where a block has few of them (160 x 3261 8.2 us, not 9.3) and for narrow rows (1000 x 1024 7.7
    // us, not 10.3).
    s.vpt = eights > most || (eights > most / 2 && T >= 8 * kSms) ? 2 : 1;
    auto blocks_of = [&](int threads) {
        int b = 1;
        while (b < kMostBlocks && b * threads * s.vpt < eights) b *= 2;
        return b;
    };
    // Clusters of twice the blocks of half the threads, two blocks to an SM, where these are mostly filled: one row's
    // exchange runs while the other's threads work (4000 x 12288 139 -> 131 us, x 16384 164 -> 145; 1422 x 9739, whose
    // threads would be 60 % filled, 57 -> 63).
    const int half = blocks_of(most / 2);
    s.blocks = half > 2 && 4 * eights >= 3 * half * (most / 2) * s.vpt ? half : blocks_of(most);
    s.threads = ((eights + s.blocks * s.vpt - 1) / (s.blocks * s.vpt) + 31) / 32 * 32;
    s.groups = 1;
    int per_sm = std::min(32, most / s.threads);
    if (s.blocks == 1) {
        s.groups = std::max(1, std::min({per_sm, s.threads == 32 ? 16 : 8, (T - 1) / kSms + 1}));
        per_sm = std::max(1, most / (s.threads * s.groups));
    }
    if (s.blocks > 1) per_sm = std::min(per_sm, 2);
    s.clusters = clusters_for((T - 1) / s.groups + 1, per_sm, s.blocks);
    if (s.groups > 1 && d % 8) s.clusters = (s.clusters + 7) / 8 * 8;
    return s;
}
template <typename X, bool EDGE>
cudaError_t backward_as(Backward a, const Shape& f, cudaStream_t s) {
    a.blocks = f.blocks;
    const size_t ring = pair_stages<X>() * 2 * (2 * words<X>() + 1), weights = f.vpt == 2 ? 4 : 0;  // words of a thread
    const size_t smem = sizeof(uint4) * (ring + weights) * f.threads * f.groups;
    const auto kernel = f.vpt == 1   ? layer_norm_backward_kernel<X, EDGE, 1, false>
                        : f.blocks > 1 ? layer_norm_backward_kernel<X, EDGE, 2, true>
                                       : layer_norm_backward_kernel<X, EDGE, 2, false>;
    return launch_rows(kernel, f, smem, s, a);
}

}  // namespace

// Blocks' sums of the backward pass on GB300's 152 SMs (the workspace depends on the shape alone).
int layer_norm_blocks(int T, int d) { return T == 0 ? 0 : backward_shape(T, d).clusters; }
int layer_norm_width(int d) { return 8 * eights_of(d); }

cudaError_t launch_layer_norm_backward(const LayerNormArgs& g, cudaStream_t s) {
    Backward a{g.x, reinterpret_cast<const float2*>(g.stats), g.dn, g.dy, g.weight, g.T, g.d, g.drop, g.dx, g.dh, nullptr, 1, 0, eights_of(g.d)};
    const bool sums = g.dweight || g.dbias;
    if (sums) a.partial = g.partial;
    a.vec = aligned({g.x, g.dn, g.dy, g.dx, g.dh});
    const bool edge = g.d % 8 != 0 || !a.vec || !aligned({g.weight}, 31);
    const Shape f = backward_shape(g.T, g.d);
    using B = __nv_bfloat16;
    const cudaError_t e = g.x_fp32 ? (edge ? backward_as<float, true>(a, f, s) : backward_as<float, false>(a, f, s))
                                   : (edge ? backward_as<B, true>(a, f, s) : backward_as<B, false>(a, f, s));
    if (e != cudaSuccess || !sums) return e;
    return launch_k(kPdlTrain, layer_norm_join_kernel, dim3(2 * ((g.d + 31) / 32)), dim3(512), 0, s,
                    static_cast<const float*>(g.partial), f.clusters, g.d, eights_of(g.d), g.dweight, g.dbias);
}

}  // namespace moe
