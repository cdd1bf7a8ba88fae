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
// One pass over memory each way; bound by it.  Each thread holds eight values of a row, with the next rows on their way
// into shared memory (cp.async: a thread copies just the words that it will use, so the ring of rows needs no barrier).
// The variance is the sum of squared distances from the mean (no difference of large sums), so a row needs two sums one
// after the other; the second of row k is taken in the same reduction as the first of row k + 1, one barrier a row.
// The backward pass takes two rows at a time, whose four sums share a reduction.  A row that is wider than a block's
// threads hold lies in the blocks of a cluster, which exchange their warps' sums through each other's shared memory.
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

// Four sums over a warp: lane l holds that of s[l / 8].
__device__ __forceinline__ float warp_sum4(const float (&s)[4]) {
    const bool up = threadIdx.x & 16, up8 = threadIdx.x & 8;
    const float a = (up ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, up ? s[0] : s[2], 16);
    const float b = (up ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, up ? s[1] : s[3], 16);
    float v = (up8 ? b : a) + __shfl_xor_sync(0xffffffffu, up8 ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// N = 2 or 4 sums over the threads that hold a row.  One barrier each; the buffers alternate, so that none is needed
// behind it.
template <bool CLUSTER, int N>
struct RowSums {
    float* red;  // [2][blocks of the cluster x warps][N]
    int warps, barrier, blocks, rank, parity = 0;
    __device__ __forceinline__ RowSums(float* red_, int warps_, int barrier_, int blocks_)
        : red(red_), warps(warps_), barrier(barrier_), blocks(blocks_), rank(CLUSTER ? ptx::cluster_ctarank() : 0) {}
    __device__ __forceinline__ void operator()(float (&s)[N]) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, all = (CLUSTER ? blocks : 1) * warps;
        float mine;  // this lane's part of sum lane / (32 / N)
        if constexpr (N == 4) {
            mine = warp_sum4(s);
        } else {
            const float2 v = warp_sum2(make_float2(s[0], s[1]));
            mine = lane & 16 ? v.y : v.x;
        }
        if (CLUSTER || warps > 1) {
            float* buf = red + parity * all * N;
            parity ^= 1;
            if (CLUSTER) {
                // Lane l sends sum l mod N to block l / N, and to those 32 / N further on.
                const float v = __shfl_sync(0xffffffffu, mine, (lane & (N - 1)) * (32 / N));
                for (int to = lane / N; to < blocks; to += 32 / N)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(ptx::map_to_cta(
                                     ptx::smem_u32(buf + (rank * warps + warp) * N + (lane & (N - 1))), to)),
                                 "f"(v)
                                 : "memory");
                ptx::cluster_arrive();
                ptx::cluster_wait();
            } else {
                if (lane % (32 / N) == 0) buf[warp * N + lane / (32 / N)] = mine;
                if (barrier == 0) __syncthreads();
                else asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(warps * 32) : "memory");
            }
            // Lane l adds up sum l mod N of the warps l / N, l / N + 32 / N, ..
            mine = 0.0f;
            for (int w = lane / N; w < all; w += 32 / N) mine += buf[w * N + (lane & (N - 1))];
#pragma unroll
            for (int o = 16; o >= N; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
#pragma unroll
            for (int k = 0; k < N; ++k) s[k] = __shfl_sync(0xffffffffu, mine, k);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) s[k] = __shfl_sync(0xffffffffu, mine, k * (32 / N));
        }
    }
};

// 16-byte words of eight values of X, and a thread's words in a ring of rows.
template <typename X>
constexpr int words() { return sizeof(X) == 4 ? 2 : 1; }
__device__ __forceinline__ void copy_word(uint4* to, const void* from, int bytes) {  // zeros behind `bytes`
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(to)), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_word_l1(uint4* to, const void* from, int bytes) {  // (half a sector: through L1)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(to)), "l"(from), "r"(bytes) : "memory");
}
template <typename X>
__device__ __forceinline__ Vec8 ring8(const uint4* word, int nt) {  // (its words lie nt apart)
    const uint4 a = word[0];
    if constexpr (sizeof(X) == 2) {
        return unpack8(a);
    } else {
        const uint4 b = word[nt];
        return Vec8{{__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                     __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)}};
    }
}
// A thread's eight of a row: the columns c .. c + 7, of which those from lo to hi - 1 are the row's.  `base` below is
// where the row's first eight begins in a tensor of `total` values (the same for all threads of a row), `off` the
// thread's from there.
template <bool EDGE>
struct Eight {
    unsigned off;
    int c, lo, hi;
    bool vec;  // the tensors are aligned for vectors
    __device__ __forceinline__ Eight(int q, int shift, int d, bool vectors) : off(8 * q), c(8 * q - shift), vec(vectors) {
        lo = EDGE ? max(0, -c) : 0;
        hi = min(8, d - c);
    }
    __device__ __forceinline__ bool some() const { return hi > lo; }
    __device__ __forceinline__ bool whole() const { return !EDGE || (lo == 0 && hi == 8); }
    // On their way to `word`, words nt apart.  Values that are not the row's may be any.
    template <typename X>
    __device__ __forceinline__ void copy(uint4* word, int nt, const X* p, long long base, long long total) const {
        const X* from = p + base + off;
        if (!EDGE || vec) {
            // (only the tensor's last eight can reach behind its end: zeros are put there)
            const bool inside = !EDGE || base + off + 8 <= total;
            const int left = inside ? 32 : static_cast<int>(total - base - off) * static_cast<int>(sizeof(X));  // bytes
            if constexpr (sizeof(X) == 2) {
                copy_word(word, from, min(left, 16));
            } else {
                copy_word_l1(word, from, min(left, 16));
                copy_word_l1(word + nt, left > 16 ? from + 4 : from, max(0, min(left - 16, 16)));
            }
        } else {
            Vec8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v.v[j] = j >= lo && j < hi ? to_float(from[j]) : 0.0f;
            if constexpr (sizeof(X) == 2) {
                *word = pack8(v);
            } else {
                word[0] = make_uint4(__float_as_uint(v.v[0]), __float_as_uint(v.v[1]), __float_as_uint(v.v[2]), __float_as_uint(v.v[3]));
                word[nt] = make_uint4(__float_as_uint(v.v[4]), __float_as_uint(v.v[5]), __float_as_uint(v.v[6]), __float_as_uint(v.v[7]));
            }
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
    __device__ __forceinline__ void store(X* p, long long base, const Vec8& v) const {
        X* to = p + base + off;
        if (!EDGE || (vec && whole())) {
            store8(to, 0, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= lo && j < hi) put(to + j, v.v[j]);
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
    int blocks, vec, keep;  // blocks of a cluster; keep: the weights lie behind the ring
};

constexpr int kStages = 3;  // rows in the forward pass' ring
// Pairs of rows in the backward pass' (512 threads: 144 KB, 160 KB with an fp32 stream).
template <typename X>
constexpr int pair_stages() { return sizeof(X) == 4 ? 2 : 3; }

template <typename X, bool H, bool EDGE, bool CLUSTER>
__global__ void __launch_bounds__(1024, 1) layer_norm_kernel(const __grid_constant__ Forward a) {
    __shared__ float red[2 * 2 * (CLUSTER ? kMostBlocks * 32 : 32)];
    extern __shared__ uint4 ring[];
    constexpr int W = words<X>() + (H ? 1 : 0);
    const int tid = threadIdx.x, nt = blockDim.x, d = a.d;
    // The mean is divided for, so that a constant row has deviations of 0.
    const float fd = static_cast<float>(d), inv_d = 1.0f / fd;
    const X* x = static_cast<const X*>(a.x);
    X* y = static_cast<X*>(a.y);
    const long long T = a.T, total = T * d, step = gridDim.x / a.blocks, row0 = blockIdx.x / a.blocks, row = step * d;
    const int rows = static_cast<int>((T - row0 - 1) / step) + 1;
    if (CLUSTER) ptx::cluster_arrive();  // (the other blocks' memory is there once all have begun)
    pdl_wait();
    pdl_trigger();
    if (CLUSTER) ptx::cluster_wait();
    RowSums<CLUSTER, 2> row_sum(red, nt >> 5, 0, a.blocks);
    const int shift = EDGE ? static_cast<int>(row0 * d & 7) : 0;
    const Eight<EDGE> e((CLUSTER ? row_sum.rank * nt : 0) + tid, shift, d, a.vec != 0);
    const bool some = e.some();
    long long in = row0 * d - shift, out = in;  // where the row to copy next begins, and the one to write
    int copied = 0;
    uint4* const first = ring + tid;
    uint4* slot = first;  // the words of the row to copy next, of the row to take next
    const uint4* word = first;
    uint4* const last = first + (kStages - 1) * W * nt;
    auto fetch = [&] {
        if (copied < rows && some) {
            e.copy(slot, nt, x, in, total);
            if (H) e.copy(slot + words<X>() * nt, nt, a.h, in, total);
        }
        ptx::cp_async_commit();
        in += row;
        slot = slot == last ? first : slot + W * nt;
        ++copied;
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) fetch();
    float4* const kept = reinterpret_cast<float4*>(ring + kStages * W * nt) + tid;  // a thread's own words: no barrier
    if (a.keep && some) {
        const Vec8 w = e.column(a.weight, 1.0f), b = e.column(a.bias, 0.0f);
        kept[0] = make_float4(w.v[0], w.v[1], w.v[2], w.v[3]);
        kept[nt] = make_float4(w.v[4], w.v[5], w.v[6], w.v[7]);
        kept[2 * nt] = make_float4(b.v[0], b.v[1], b.v[2], b.v[3]);
        kept[3 * nt] = make_float4(b.v[4], b.v[5], b.v[6], b.v[7]);
    }
    auto kept8 = [&](int k) {
        const float4 p = kept[2 * k * nt], q = kept[(2 * k + 1) * nt];
        return Vec8{{p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w}};
    };
    const Drop drop(a.drop);
    auto take = [&](Vec8& v, long long base) {  // the stream's values, stored with H; their sum
        float2 s = make_float2(0.0f, 0.0f);
        if (some) {
            v = ring8<X>(word, nt);
            if (H) {
                Vec8 hv = ring8<__nv_bfloat16>(word + words<X>() * nt, nt);
                if (drop.on()) drop.apply(hv, base + e.off);
#pragma unroll
                for (int j = 0; j < 4; ++j) v.set(j, add2(v.pair(j), hv.pair(j)));
                v = rounded(v, static_cast<const X*>(nullptr));
                e.store(y, base, v);
            }
            e.mask(v);
            s = v.pair(0);
#pragma unroll
            for (int j = 1; j < 4; ++j) s = add2(s, v.pair(j));
        }
        word = word == last ? first : word + W * nt;
        return s.x + s.y;
    };
    Vec8 cur, nxt;
    ptx::cp_async_wait<kStages - 1>();
    float s[2] = {0.0f, take(cur, out)};
    row_sum(s);
    float2* stats = a.stats + row0;
    for (int k = 0; k < rows; ++k) {
        const float mean = s[1] / fd;
        fetch();
        ptx::cp_async_wait<kStages - 1>();
        s[1] = k + 1 < rows ? take(nxt, out + row) : 0.0f;
        float2 q = make_float2(0.0f, 0.0f);
        if (some) {
            const float2 back = make_float2(-mean, -mean);
#pragma unroll
            for (int j = 0; j < 4; ++j) cur.set(j, add2(cur.pair(j), back));
            e.mask(cur);
#pragma unroll
            for (int j = 0; j < 4; ++j) q = fma2(cur.pair(j), cur.pair(j), q);
        }
        s[0] = q.x + q.y;
        row_sum(s);
        const float r = rsqrtf(s[0] * inv_d + a.eps);
        if (tid == 0 && row_sum.rank == 0) *stats = make_float2(mean, r);
        stats += step;
        if (some) {
            const Vec8 w = a.keep ? kept8(0) : e.column(a.weight, 1.0f), b = a.keep ? kept8(1) : e.column(a.bias, 0.0f);
            Vec8 o;
#pragma unroll
            for (int j = 0; j < 4; ++j) o.set(j, fma2(mul2(cur.pair(j), r), w.pair(j), b.pair(j)));
            e.store(a.n, out, o);
        }
        out += row;
        cur = nxt;
    }
    ptx::cp_async_wait_all();
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

// Two rows at a time.  The column sums dweight and dbias of the rows that a block visits stay in registers and are
// written once; rows that are narrower than the block lie side by side in it (threadIdx.y), each with its barrier, and
// their sums are added up first.
template <typename X, bool EDGE, bool CLUSTER>
__global__ void __launch_bounds__(512, 1) layer_norm_backward_kernel(const __grid_constant__ Backward a) {
    __shared__ float red[2 * 4 * (CLUSTER ? kMostBlocks * 16 : 16)];
    extern __shared__ uint4 ring_all[];
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
    RowSums<CLUSTER, 4> row_sum(red + (CLUSTER ? 0 : 8 * warps * group), warps, groups > 1 ? 1 + group : 0, a.blocks);
    const Drop drop(a.drop);
    const int shift = EDGE ? static_cast<int>(cluster * d & 7) : 0;
    const Eight<EDGE> e((CLUSTER ? row_sum.rank * nt : 0) + tid, shift, d, a.vec != 0);
    const bool some = e.some();
    // Words of a row: x, dn, dy.
    constexpr int o_dn = words<X>(), o_dy = o_dn + 1, W = o_dy + words<X>(), S = pair_stages<X>();
    const long long row = step * d;
    long long in = row0 * d - shift, out = in;  // where the row to copy next begins, and the one to write
    uint4* const first = ring_all + group * (S * 2 * W * nt) + tid;
    uint4* const last = first + (S - 1) * 2 * W * nt;
    uint4* slot = first;  // the words of the rows to copy next, of the rows to work on
    const uint4* word = first;
    int copied = 0;
    auto fetch = [&] {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (copied < rows && some) {
                uint4* w = slot + i * W * nt;
                e.copy(w, nt, x, in, total);
                e.copy(w + o_dn * nt, nt, a.dn, in, total);
                if (dy) e.copy(w + o_dy * nt, nt, dy, in, total);
            }
            in += row;
            ++copied;
        }
        ptx::cp_async_commit();
        slot = slot == last ? first : slot + 2 * W * nt;
    };
    float2 st[2] = {}, next[2] = {};
    const float2* stats = a.stats + row0;  // of the rows to read next
    int stats_left = rows;
    auto read_stats = [&] {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (stats_left > 0) next[i] = __ldg(stats);
            stats += step;
            --stats_left;
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < S; ++k) fetch();
    read_stats();
    const Vec8 w = some ? e.column(a.weight, 1.0f) : Vec8{};
    Vec8 sw{}, sb{};
    for (int k = 0; k < rows; k += 2) {
        fetch();
        st[0] = next[0], st[1] = next[1];
        read_stats();
        ptx::cp_async_wait<S - 1>();
        const bool two = k + 1 < rows;
        Vec8 yh[2], g[2];
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (some && (i == 0 || two)) {
                const float r = st[i].y;
                const float2 back = make_float2(-st[i].x, -st[i].x);
                float2 sg, sy;
                yh[i] = ring8<X>(word + i * W * nt, nt);
                Vec8 nv = ring8<B>(word + (i * W + o_dn) * nt, nt);
                e.mask(yh[i]);
                e.mask(nv);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    yh[i].set(j, mul2(add2(yh[i].pair(j), back), r));
                    g[i].set(j, mul2(nv.pair(j), w.pair(j)));
                    sg = j ? add2(sg, g[i].pair(j)) : g[i].pair(j);
                    sy = j ? fma2(g[i].pair(j), yh[i].pair(j), sy) : mul2(g[i].pair(j), yh[i].pair(j));
                    sw.set(j, fma2(nv.pair(j), yh[i].pair(j), sw.pair(j)));
                    sb.set(j, add2(sb.pair(j), nv.pair(j)));
                }
                s[2 * i] = sg.x + sg.y;
                s[2 * i + 1] = sy.x + sy.y;
            }
        row_sum(s);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (some && (i == 0 || two)) {
                // (r taken into the means: r (g - mg - yh my) + dy)
                const float r = st[i].y, mg = -s[2 * i] * inv_d * r, my = -s[2 * i + 1] * inv_d * r;
                Vec8 o;
                if (dy) {
                    o = ring8<X>(word + (i * W + o_dy) * nt, nt);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o.set(j, add2(o.pair(j), make_float2(mg, mg)));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o.v[j] = mg;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) o.set(j, fma2(g[i].pair(j), r, fma2(yh[i].pair(j), my, o.pair(j))));
                e.store(dx, out, o);
                if (a.dh) {
                    if (drop.on()) drop.apply(o, out + e.off);
                    e.store(a.dh, out, o);
                }
            }
            out += row;
        }
        word = word == last ? first : word + 2 * W * nt;
    }
    ptx::cp_async_wait_all();
    if (!a.partial) return;
    float* p = a.partial + static_cast<size_t>(cluster) * 2 * d;
    const Eight<EDGE> column(some ? (e.c + shift) / 8 : 0, shift, d, false);  // (the rows of `partial` start anywhere)
    auto write = [&](float* to, const Vec8& v) {
        if (!EDGE) store8(to + e.c, 0, v);
        else column.store(to - shift, 0, v);
    };
    if (groups > 1) {
        float* sums = reinterpret_cast<float*>(ring_all);  // [rows side by side][8][threads of a row], once all are done
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // dweight, then dbias
            const Vec8& own = k ? sb : sw;
            __syncthreads();
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

constexpr size_t kMostSmem = 216 * 1024;  // of a block's ring and weights (1024 threads: 208 KB)

// Dynamic shared memory beyond what a launch gets unasked (48 KB with the static one).
template <typename... KArgs>
cudaError_t allow_smem(void (*kernel)(KArgs...), size_t smem) {
    if (smem <= 39 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostSmem));
}

template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kernel)(KArgs...), const Shape& f, size_t smem, cudaStream_t s, Args&&... args) {
    cudaError_t e = allow_smem(kernel, smem);
    if (e == cudaSuccess && f.blocks > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
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
    a.keep = a.T > f.clusters;  // more than one row to a block: the weights are read once
    const size_t words_of_row = words<X>() + (H ? 1 : 0);
    const size_t smem = sizeof(uint4) * f.threads * (kStages * words_of_row + (a.keep ? 4 : 0));
    const auto kernel = f.blocks > 1 ? layer_norm_kernel<X, H, EDGE, true> : layer_norm_kernel<X, H, EDGE, false>;
    return launch_rows(kernel, f, smem, s, a);
}
template <typename X, bool EDGE>
cudaError_t backward_as(Backward a, const Shape& f, cudaStream_t s) {
    a.blocks = f.blocks;
    const size_t smem = sizeof(uint4) * pair_stages<X>() * 2 * (2 * words<X>() + 1) * f.threads * f.groups;
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
