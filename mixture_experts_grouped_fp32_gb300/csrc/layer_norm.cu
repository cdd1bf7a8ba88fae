// layer_norm.cu — layer norm of a residual stream after a block's output was added to it, forward and backward.
// Per row t of d values:
//
//   forward    y = x + drop(h)                                  rounded to the stream's type: n is the norm of what
//              mean = sum(y) / d,  r = 1 / sqrt(sum((y - mean)^2) / d + eps)                  is stored
//              n = weight (y - mean) r + bias
//   backward   given dn and dy, with yh = (y - mean) r and g = dn weight:
//              dx = dy + r (g - mean(g) - yh mean(g yh)),  dh = drop(dx) with the same mask
//              dweight = sum_t dn yh,  dbias = sum_t dn
//
// y is bf16 or fp32, h, n, dn and dh bf16, weight, bias, their gradients and the stats (mean, r) fp32.
//
// One pass over memory each way; bound by it.  Each thread holds eight values of a row.  The variance is the sum of
// squared distances from the mean (no difference of large sums), so a row needs two sums one after the other; the
// second of row k is taken in the same reduction as the first of row k + 1, one barrier a row, with the loads of row
// k + 2 under way.  A row that is wider than a block's threads hold lies in the blocks of a cluster, which exchange
// their warps' sums through each other's shared memory.
//
// Rows of any width: the eights are those of the tensor in memory order, aligned whatever the row, so a row starts
// in the middle of one (at s = t d mod 8) and its first and last eights are shared with its neighbours: loaded whole,
// their other values masked, and stored value by value.  A block takes rows whose distance is a multiple of 8, which
// have the same s, so a thread's columns, its weights and its column sums stay the same from row to row.
#include <algorithm>
#include <initializer_list>

#include "stack_ops.cuh"
#include "train_ptx.cuh"

namespace moe {
namespace {

constexpr int kSms = 152;  // of a GB300
constexpr int kMostBlocks = 16;  // of a cluster

// Two sums over a warp, in every lane: a half-warp takes each after the first exchange.
__device__ __forceinline__ float2 warp_sum2(float2 v) {
    const bool up = threadIdx.x & 16;
    float a = up ? v.y : v.x;
    a += __shfl_xor_sync(0xffffffffu, up ? v.x : v.y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    const float b = __shfl_xor_sync(0xffffffffu, a, 16);
    return up ? make_float2(b, a) : make_float2(a, b);
}

// Sums over the threads that hold a row.  One barrier each; the buffers alternate, so that none is needed behind it.
template <bool CLUSTER>
struct RowSums {
    float2* red;  // [2][blocks of the cluster x warps]
    int warps, barrier, blocks, rank, parity = 0;
    __device__ __forceinline__ RowSums(float2* red_, int warps_, int barrier_, int blocks_)
        : red(red_), warps(warps_), barrier(barrier_), blocks(blocks_), rank(CLUSTER ? ptx::cluster_ctarank() : 0) {}
    __device__ __forceinline__ float2 operator()(float2 v) {
        v = warp_sum2(v);
        if (!CLUSTER && warps == 1) return v;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, all = CLUSTER ? blocks * warps : warps;
        float2* buf = red + parity * all;
        parity ^= 1;
        if (CLUSTER) {
            if (lane < blocks) {
                const uint32_t to = ptx::map_to_cta(ptx::smem_u32(buf + rank * warps + warp), lane);
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v.x), "f"(v.y) : "memory");
            }
            ptx::cluster_arrive();
            ptx::cluster_wait();
            v = make_float2(0.0f, 0.0f);
            for (int i = lane; i < all; i += 32) v = add2(v, buf[i]);
        } else {
            if (lane == 0) buf[warp] = v;
            if (barrier == 0) __syncthreads();
            else asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(warps * 32) : "memory");
            v = lane < warps ? buf[lane] : make_float2(0.0f, 0.0f);
        }
        return warp_sum2(v);
    }
};

// A thread's eight of a row: the columns c .. c + 7, of which those from lo to hi - 1 are the row's.
template <bool EDGE>
struct Eight {
    int c, lo, hi;
    bool vec;  // the tensors are aligned for vectors
    __device__ __forceinline__ Eight(int q, int shift, int d, bool vectors) : c(8 * q - shift), vec(vectors) {
        lo = EDGE ? max(0, -c) : 0;
        hi = min(8, d - c);
    }
    __device__ __forceinline__ bool some() const { return hi > lo; }
    __device__ __forceinline__ bool whole() const { return !EDGE || (lo == 0 && hi == 8); }
    // `at`: the first value's place in the tensor of `total` values.  Values that are not the row's may be any.
    template <typename X>
    __device__ __forceinline__ void load(Raw8<X>& r, const X* p, long long at, long long total) const {
        if (!EDGE || (vec && at + 8 <= total)) {
            fetch_raw<true>(r, p + at, 8);
        } else {
            Vec8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v.v[j] = j >= lo && j < hi ? to_float(p[at + j]) : 0.0f;
            set_values(r, v);
        }
    }
    __device__ __forceinline__ void mask(Vec8& v) const {
        if (!whole()) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < lo || j >= hi) v.v[j] = 0.0f;
        }
    }
    template <typename X>
    __device__ __forceinline__ void store(X* p, long long at, const Vec8& v) const {
        if (!EDGE || (vec && whole())) {
            store8(p + at, 0, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= lo && j < hi) put(p + at + j, v.v[j]);
        }
    }
    // Of a vector over the columns, or `none` without it.
    __device__ __forceinline__ Vec8 column(const float* p, float none) const {
        if (!EDGE && p) return load8_cached(p + c, 0);
        Vec8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v.v[j] = p && j >= lo && j < hi ? __ldg(p + c + j) : none;
        return v;
    }
};

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
    int blocks, vec, keep;  // blocks of a cluster; keep: the weights go through shared memory
};

template <typename X, bool H, bool EDGE, bool CLUSTER>
__global__ void __launch_bounds__(1024, 1) layer_norm_kernel(Forward a) {
    __shared__ float2 red[2 * (CLUSTER ? kMostBlocks * 32 : 32)];
    extern __shared__ float4 kept[];  // weight and bias, two words a thread each
    const int tid = threadIdx.x, nt = blockDim.x, d = a.d;
    const float fd = static_cast<float>(d);  // divided by, so that a constant row has deviations of 0
    const X* x = static_cast<const X*>(a.x);
    X* y = static_cast<X*>(a.y);
    const long long T = a.T, total = T * d, step = gridDim.x / a.blocks, row0 = blockIdx.x / a.blocks;
    if (CLUSTER) ptx::cluster_arrive();  // (the other blocks' memory is there once all have begun)
    pdl_wait();
    pdl_trigger();
    if (CLUSTER) ptx::cluster_wait();
    RowSums<CLUSTER> row_sum(red, nt >> 5, 0, a.blocks);
    const Drop drop(a.drop);
    const int shift = EDGE ? static_cast<int>(row0 * d & 7) : 0;
    const Eight<EDGE> e((CLUSTER ? row_sum.rank * nt : 0) + tid, shift, d, a.vec != 0);
    const bool some = e.some();
    Raw8<X> xr;
    Raw8<__nv_bfloat16> hr;
    auto fetch = [&](long long t) {
        if (some) {
            e.load(xr, x, t * d + e.c, total);
            if (H) e.load(hr, a.h, t * d + e.c, total);
        }
    };
    auto take = [&](Vec8& row, long long t) {  // the stream's values from the raw ones, stored with H; their sum
        if (!some) return 0.0f;
        row = values(xr);
        if (H) {
            Vec8 hv = values(hr);
            if (drop.on()) drop.apply(hv, t * d + e.c);
#pragma unroll
            for (int j = 0; j < 4; ++j) row.set(j, add2(row.pair(j), hv.pair(j)));
            row = rounded(row, static_cast<const X*>(nullptr));
            e.store(y, t * d + e.c, row);
        }
        e.mask(row);
        float2 s = row.pair(0);
#pragma unroll
        for (int j = 1; j < 4; ++j) s = add2(s, row.pair(j));
        return s.x + s.y;
    };
    Vec8 cur, nxt;
    fetch(row0);
    if (a.keep && some) {
        const Vec8 w = e.column(a.weight, 1.0f), b = e.column(a.bias, 0.0f);
        kept[tid] = make_float4(w.v[0], w.v[1], w.v[2], w.v[3]);
        kept[nt + tid] = make_float4(w.v[4], w.v[5], w.v[6], w.v[7]);
        kept[2 * nt + tid] = make_float4(b.v[0], b.v[1], b.v[2], b.v[3]);
        kept[3 * nt + tid] = make_float4(b.v[4], b.v[5], b.v[6], b.v[7]);
    }
    auto kept8 = [&](int k) {  // (a thread's own words: no barrier)
        const float4 p = kept[2 * k * nt + tid], q = kept[(2 * k + 1) * nt + tid];
        return Vec8{{p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w}};
    };
    float mean = take(cur, row0);
    if (row0 + step < T) fetch(row0 + step);
    mean = row_sum(make_float2(mean, 0.0f)).x / fd;
    for (long long t = row0; t < T; t += step) {
        float next_sum = 0.0f;
        if (t + step < T) {
            next_sum = take(nxt, t + step);
            if (t + 2 * step < T) fetch(t + 2 * step);
        }
        float2 q = make_float2(0.0f, 0.0f);
        if (some) {
#pragma unroll
            for (int j = 0; j < 4; ++j) cur.set(j, add2(cur.pair(j), make_float2(-mean, -mean)));
            e.mask(cur);
#pragma unroll
            for (int j = 0; j < 4; ++j) q = fma2(cur.pair(j), cur.pair(j), q);
        }
        const float2 s = row_sum(make_float2(q.x + q.y, next_sum));
        const float r = 1.0f / sqrtf(s.x / fd + a.eps);
        if (tid == 0 && row_sum.rank == 0) a.stats[t] = make_float2(mean, r);
        if (some) {
            const Vec8 w = a.keep ? kept8(0) : e.column(a.weight, 1.0f), b = a.keep ? kept8(1) : e.column(a.bias, 0.0f);
            Vec8 o;
#pragma unroll
            for (int j = 0; j < 4; ++j) o.set(j, fma2(mul2(cur.pair(j), r), w.pair(j), b.pair(j)));
            e.store(a.n, t * d + e.c, o);
        }
        mean = s.y / fd;
        cur = nxt;
    }
}

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
    float* partial;  // [clusters, 2, d], or null
    int blocks, vec;
};

// One reduction a row.  The column sums dweight and dbias of the rows that a block visits stay in registers and are
// written once; rows that are narrower than the block lie side by side in it (threadIdx.y), each with its barrier, and
// their sums are added up first.
template <typename X, bool EDGE, bool CLUSTER>
__global__ void __launch_bounds__(512, 1) layer_norm_backward_kernel(Backward a) {
    __shared__ float2 red[2 * (CLUSTER ? kMostBlocks * 16 : 16)];
    extern __shared__ float sums[];  // [rows side by side][8][threads of a row]
    using B = __nv_bfloat16;
    const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, d = a.d, groups = CLUSTER ? 1 : blockDim.y, group = threadIdx.y;
    const float inv_d = 1.0f / static_cast<float>(d);
    const X *x = static_cast<const X*>(a.x), *dy = static_cast<const X*>(a.dy);
    X* dx = static_cast<X*>(a.dx);
    const long long T = a.T, total = T * d, clusters = gridDim.x / a.blocks, cluster = blockIdx.x / a.blocks;
    const long long row0 = cluster + clusters * group, step = clusters * groups;
    if (CLUSTER) ptx::cluster_arrive();
    pdl_wait();
    pdl_trigger();
    if (CLUSTER) ptx::cluster_wait();
    RowSums<CLUSTER> row_sum(red + (CLUSTER ? 0 : 2 * warps * group), warps, groups > 1 ? 1 + group : 0, a.blocks);
    const Drop drop(a.drop);
    const int shift = EDGE ? static_cast<int>(cluster * d & 7) : 0;
    const Eight<EDGE> e((CLUSTER ? row_sum.rank * nt : 0) + tid, shift, d, a.vec != 0);
    const bool some = e.some();
    Raw8<X> xr, er;
    Raw8<B> nr;
    float2 st = make_float2(0.0f, 0.0f);
    auto fetch = [&](long long t) {
        st = __ldg(a.stats + t);
        if (some) {
            const long long at = t * d + e.c;
            e.load(xr, x, at, total);
            e.load(nr, a.dn, at, total);
            if (dy) e.load(er, dy, at, total);
        }
    };
    const Vec8 w = some ? e.column(a.weight, 1.0f) : Vec8{};
    Vec8 sw{}, sb{};
    if (row0 < T) fetch(row0);
    for (long long t = row0; t < T; t += step) {
        const float r = st.y, back = -st.x;
        Vec8 yh, g, o;
        float2 sg = make_float2(0.0f, 0.0f), sy = sg;
        if (some) {
            yh = values(xr);
            Vec8 nv = values(nr);
            e.mask(yh);
            e.mask(nv);
            o = dy ? values(er) : Vec8{};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                yh.set(j, mul2(add2(yh.pair(j), make_float2(back, back)), r));
                g.set(j, mul2(nv.pair(j), w.pair(j)));
                sg = add2(sg, g.pair(j));
                sy = fma2(g.pair(j), yh.pair(j), sy);
                sw.set(j, fma2(nv.pair(j), yh.pair(j), sw.pair(j)));
                sb.set(j, add2(sb.pair(j), nv.pair(j)));
            }
        }
        if (t + step < T) fetch(t + step);
        const float2 s = row_sum(make_float2(sg.x + sg.y, sy.x + sy.y));
        const float mg = s.x * inv_d, my = s.y * inv_d;
        if (some) {
            const long long at = t * d + e.c;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 b = fma2(yh.pair(j), make_float2(-my, -my), add2(g.pair(j), make_float2(-mg, -mg)));
                o.set(j, fma2(b, r, o.pair(j)));
            }
            e.store(dx, at, o);
            if (a.dh) {
                if (drop.on()) drop.apply(o, at);
                e.store(a.dh, at, o);
            }
        }
    }
    if (!a.partial) return;
    float* p = a.partial + static_cast<size_t>(cluster) * 2 * d;
    const Eight<EDGE> column(some ? (e.c + shift) / 8 : 0, shift, d, false);  // (the rows of `partial` start anywhere)
    auto write = [&](float* to, const Vec8& v) {
        if (!EDGE) {
            store8(to + e.c, 0, v);
            return;
        }
        column.store(to, e.c, v);
    };
    if (groups > 1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // dweight, then dbias
            const Vec8& own = k ? sb : sw;
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[(group * 8 + j) * nt + tid] = own.v[j];
            __syncthreads();
            if (group == 0 && some) {
                Vec8 v = own;
                for (int g = 1; g < groups; ++g)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v.v[j] += sums[(g * 8 + j) * nt + tid];
                write(p + k * static_cast<size_t>(d), v);
            }
            __syncthreads();
        }
    } else if (some) {
        write(p, sw);
        write(p + d, sb);
    }
}

// Adds the blocks' column sums in block order (16 runs of blocks, then the runs).
__global__ void __launch_bounds__(512)
layer_norm_join_kernel(const float* __restrict__ partial, int blocks, int d, float* __restrict__ dweight,
                       float* __restrict__ dbias) {
    __shared__ float part[16][33];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const size_t col = static_cast<size_t>(blockIdx.x) * 32 + lane, width = 2 * static_cast<size_t>(d);
    const int per = (blocks + 15) / 16, b0 = min(run * per, blocks), b1 = min(b0 + per, blocks);
    pdl_wait();
    pdl_trigger();
    float s = 0.0f;
    if (col < width)
#pragma unroll 10
        for (int b = b0; b < b1; ++b) s += __ldcg(partial + b * width + col);
    part[run][lane] = s;
    __syncthreads();
    if (run == 0 && col < width) {
        float a = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) a += part[k][lane];
        float* out = col < static_cast<size_t>(d) ? dweight : dbias;
        if (out) out[col < static_cast<size_t>(d) ? col : col - d] = a;
    }
}

bool aligned(std::initializer_list<const void*> ps) {
    uintptr_t all = 0;
    for (const void* p : ps) all |= reinterpret_cast<uintptr_t>(p);
    return (all & 15) == 0;
}

// How a pass is launched: blocks of a row's cluster, threads of a row in a block, rows side by side, clusters.
struct Shape {
    int blocks, threads, groups, clusters;
};
Shape shape_of(int T, int d, bool bwd) {
    const int most = bwd ? 512 : 1024, eights = (d + 7) / 8 + (d % 8 ? 1 : 0);  // (an eight more where rows start inside one)
    Shape s;
    s.blocks = 1;
    while (s.blocks < kMostBlocks && s.blocks * most < eights) s.blocks *= 2;
    s.threads = ((eights + s.blocks - 1) / s.blocks + 31) / 32 * 32;
    s.groups = 1;
    int per_sm = std::min(32, most / s.threads);
    if (bwd && s.blocks == 1) {
        s.groups = std::max(1, std::min({per_sm, s.threads == 32 ? 16 : 8, (T - 1) / kSms + 1}));
        per_sm = std::max(1, most / (s.threads * s.groups));
    }
    const int rows = (T - 1) / s.groups + 1;
    s.clusters = std::max(8, kSms * per_sm / s.blocks / 8 * 8);  // a multiple of 8, or a row each
    if (rows <= s.clusters) s.clusters = s.groups == 1 ? rows : std::min(rows, s.clusters);
    if (s.groups > 1 && s.clusters % 8 && d % 8) s.clusters = (s.clusters + 7) / 8 * 8;
    return s;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kernel)(KArgs...), const Shape& f, size_t smem, cudaStream_t s, Args&&... args) {
    if (f.blocks > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(f.clusters * f.blocks);
    cfg.blockDim = dim3(f.threads, f.groups);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = f.blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled(kPdlTrain) ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <typename X, bool H, bool EDGE>
cudaError_t forward_as(Forward a, cudaStream_t s) {
    const Shape f = shape_of(a.T, a.d, false);
    a.blocks = f.blocks;
    // Weights whose loads would be one by one are read once for all rows of a block.
    a.keep = EDGE && a.T > f.clusters;
    const size_t smem = a.keep ? sizeof(float4) * 4 * f.threads : 0;
    const auto kernel = f.blocks > 1 ? layer_norm_kernel<X, H, EDGE, true> : layer_norm_kernel<X, H, EDGE, false>;
    if (smem) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
        if (e != cudaSuccess) return e;
    }
    return launch_rows(kernel, f, smem, s, a);
}
template <typename X, bool EDGE>
cudaError_t backward_as(Backward a, const Shape& f, cudaStream_t s) {
    a.blocks = f.blocks;
    const size_t smem = f.groups > 1 && a.partial ? sizeof(float) * 8 * f.threads * f.groups : 0;
    const auto kernel = f.blocks > 1 ? layer_norm_backward_kernel<X, EDGE, true> : layer_norm_backward_kernel<X, EDGE, false>;
    return launch_rows(kernel, f, smem, s, a);
}

}  // namespace

// Blocks' sums of the backward pass on GB300's 152 SMs (the workspace depends on the shape alone).
int layer_norm_blocks(int T, int d) { return T == 0 ? 0 : shape_of(T, d, true).clusters; }

cudaError_t launch_layer_norm(const LayerNormArgs& g, cudaStream_t s) {
    Forward a{g.x, g.h, g.weight, g.bias, g.T, g.d, g.eps, g.drop, g.y, g.n, reinterpret_cast<float2*>(g.stats), 1, 0, 0};
    a.vec = aligned({g.x, g.h, g.y, g.n});
    const bool edge = g.d % 8 != 0 || !a.vec || !aligned({g.weight, g.bias});
    using B = __nv_bfloat16;
    if (g.x_fp32) {
        if (g.h) return edge ? forward_as<float, true, true>(a, s) : forward_as<float, true, false>(a, s);
        return edge ? forward_as<float, false, true>(a, s) : forward_as<float, false, false>(a, s);
    }
    if (g.h) return edge ? forward_as<B, true, true>(a, s) : forward_as<B, true, false>(a, s);
    return edge ? forward_as<B, false, true>(a, s) : forward_as<B, false, false>(a, s);
}

cudaError_t launch_layer_norm_backward(const LayerNormArgs& g, cudaStream_t s) {
    Backward a{g.x, reinterpret_cast<const float2*>(g.stats), g.dn, g.dy, g.weight, g.T, g.d, g.drop, g.dx, g.dh, nullptr, 1, 0};
    const bool sums = g.dweight || g.dbias;
    if (sums) a.partial = g.partial;
    a.vec = aligned({g.x, g.dn, g.dy, g.dx, g.dh});
    const bool edge = g.d % 8 != 0 || !a.vec || !aligned({g.weight, g.partial});
    const Shape f = shape_of(g.T, g.d, true);
    using B = __nv_bfloat16;
    const cudaError_t e = g.x_fp32 ? (edge ? backward_as<float, true>(a, f, s) : backward_as<float, false>(a, f, s))
                                   : (edge ? backward_as<B, true>(a, f, s) : backward_as<B, false>(a, f, s));
    if (e != cudaSuccess || !sums) return e;
    return launch_k(kPdlTrain, layer_norm_join_kernel, dim3((2 * g.d + 31) / 32), dim3(512), 0, s,
                    static_cast<const float*>(g.partial), f.clusters, g.d, g.dweight, g.dbias);
}

}  // namespace moe
