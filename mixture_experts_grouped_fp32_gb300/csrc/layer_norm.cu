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
// One pass over memory each way; bound by it.  The variance is the sum of squared distances from the mean (no
// difference of large sums), so a row needs two sums one after the other; the second of row k is taken in the same
// reduction as the first of row k + 1, one barrier a row, with the loads of row k + 2 under way (in registers: a
// thread's eight values of each tensor).
#include <algorithm>
#include <initializer_list>

#include "stack_ops.cuh"

namespace moe {
namespace {

constexpr int kSms = 152;  // of a GB300
constexpr int kMaxWarps = 32;

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
// Over the threads of a row (threadIdx.x): one barrier, none for a single warp; `red` alternates between calls.
__device__ __forceinline__ float2 row_sum2(float2 v, float2* red, int warps) {
    v = warp_sum2(v);
    if (warps > 1) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) red[warp] = v;
        __syncthreads();
        v = warp_sum2(lane < warps ? red[lane] : make_float2(0.0f, 0.0f));
    }
    return v;
}

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
};

// The stream's values of one vector: x, or x + drop(h) as it is stored (and stored here).
template <typename X, bool H, bool ALIGNED>
__device__ __forceinline__ Vec8 stream8(const Raw8<X>& xr, const Raw8<__nv_bfloat16>& hr, const Drop& drop, size_t at,
                                        int count, X* y) {
    Vec8 v = values(xr);
    if (H) {
        Vec8 hv = values(hr);
        if (drop.on()) {
            if (ALIGNED) drop.apply(hv, at);
            else drop.apply_any(hv, at);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v.set(j, add2(v.pair(j), hv.pair(j)));
        v = rounded(v, static_cast<const X*>(nullptr));
        if (y) put8<ALIGNED>(y + at, v, count);
    }
    return v;
}

// Rows of up to 8192 values in registers, VPT vectors of eight in each of the row's threads.  blockDim.y rows side
// by side where one warp holds a row.
template <typename X, int VPT, bool H, bool ALIGNED>
__global__ void __launch_bounds__(512, VPT == 1 ? 2 : 1) layer_norm_kernel(Forward a) {
    __shared__ float2 red[2][kMaxWarps];
    const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, d = a.d;
    const float fd = static_cast<float>(d);  // divided by, so that a constant row has deviations of 0
    const X* x = static_cast<const X*>(a.x);
    X* y = static_cast<X*>(a.y);
    const size_t row0 = static_cast<size_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const size_t step = static_cast<size_t>(gridDim.x) * blockDim.y;
    pdl_wait();
    pdl_trigger();
    if (row0 >= static_cast<size_t>(a.T)) return;  // (a whole warp, of a block without barriers)
    const Drop drop(a.drop);
    int count[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) count[v] = min(8, max(0, d - 8 * (tid + v * nt)));
    Raw8<X> xr[VPT];
    Raw8<__nv_bfloat16> hr[VPT];
    auto fetch = [&](size_t t) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (count[v] > 0) {
                const size_t at = t * d + 8 * (tid + v * nt);
                fetch_raw<ALIGNED>(xr[v], x + at, count[v]);
                if (H) fetch_raw<ALIGNED>(hr[v], a.h + at, count[v]);
            }
    };
    auto take = [&](Vec8 (&row)[VPT], size_t t) {  // the stream's row from the raw values; its sum
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (count[v] > 0) {
                row[v] = stream8<X, H, ALIGNED>(xr[v], hr[v], drop, t * d + 8 * (tid + v * nt), count[v], y);
#pragma unroll
                for (int j = 0; j < 4; ++j) s = add2(s, row[v].pair(j));
            }
        return s.x + s.y;
    };
    Vec8 cur[VPT], nxt[VPT];
    fetch(row0);
    float mean = take(cur, row0);
    if (row0 + step < static_cast<size_t>(a.T)) fetch(row0 + step);
    mean = row_sum2(make_float2(mean, 0.0f), red[1], warps).x / fd;
    int k = 0;
    for (size_t t = row0; t < static_cast<size_t>(a.T); t += step, ++k) {
        float next_sum = 0.0f;
        const bool more = t + step < static_cast<size_t>(a.T);
        if (more) {
            next_sum = take(nxt, t + step);
            if (t + 2 * step < static_cast<size_t>(a.T)) fetch(t + 2 * step);
        }
        float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (count[v] > 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 c = add2(cur[v].pair(j), make_float2(-mean, -mean));
                    cur[v].set(j, c);
                    if (!ALIGNED) {
                        if (2 * j >= count[v]) c.x = 0.0f;
                        if (2 * j + 1 >= count[v]) c.y = 0.0f;
                    }
                    q = fma2(c, c, q);
                }
            }
        const float2 s = row_sum2(make_float2(q.x + q.y, next_sum), red[k & 1], warps);
        const float r = 1.0f / sqrtf(s.x / fd + a.eps);
        if (tid == 0) a.stats[t] = make_float2(mean, r);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (count[v] > 0) {
                const int c = 8 * (tid + v * nt);
                Vec8 o;
#pragma unroll
                for (int j = 0; j < 4; ++j) o.set(j, mul2(cur[v].pair(j), r));
                if (a.weight) {
                    const Vec8 w = cached8<ALIGNED>(a.weight + c, count[v]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o.set(j, mul2(o.pair(j), w.pair(j)));
                }
                if (a.bias) {
                    const Vec8 b = cached8<ALIGNED>(a.bias + c, count[v]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o.set(j, add2(o.pair(j), b.pair(j)));
                }
                put8<ALIGNED>(a.n + t * d + c, o, count[v]);
            }
        mean = s.y / fd;
#pragma unroll
        for (int v = 0; v < VPT; ++v) cur[v] = nxt[v];
    }
}

// Rows of any width: a block reads its row three times, from the caches after the first.
template <typename X, bool H, bool ALIGNED>
__global__ void __launch_bounds__(1024) layer_norm_wide_kernel(Forward a) {
    __shared__ float2 red[2][kMaxWarps];
    const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, d = a.d, d8 = (d + 7) / 8;
    const float fd = static_cast<float>(d);  // divided by, so that a constant row has deviations of 0
    X* y = static_cast<X*>(a.y);
    pdl_wait();
    pdl_trigger();
    const Drop drop(a.drop);
    for (size_t t = blockIdx.x; t < static_cast<size_t>(a.T); t += gridDim.x) {
        const X* x = static_cast<const X*>(a.x) + t * d;
        const bool again = H && !y;  // the stream is not stored: it is computed each time
        auto row = [&](int c, int count, X* to, bool first) {
            Raw8<X> xr;
            Raw8<__nv_bfloat16> hr{};
            const size_t at = t * d + 8 * static_cast<size_t>(c);
            if (first || again || !H) {
                fetch_raw<ALIGNED>(xr, x + 8 * static_cast<size_t>(c), count);
                if (H) fetch_raw<ALIGNED>(hr, a.h + at, count);
                return stream8<X, H, ALIGNED>(xr, hr, drop, at, count, to);
            }
            fetch_raw<ALIGNED>(xr, y + at, count);  // (what this thread stored)
            return values(xr);
        };
        float2 s = make_float2(0.0f, 0.0f);
        for (int c = tid; c < d8; c += nt) {
            const Vec8 v = row(c, min(8, d - 8 * c), y, true);
#pragma unroll
            for (int j = 0; j < 4; ++j) s = add2(s, v.pair(j));
        }
        const float mean = row_sum2(make_float2(s.x + s.y, 0.0f), red[0], warps).x / fd;
        float2 q = make_float2(0.0f, 0.0f);
        for (int c = tid; c < d8; c += nt) {
            const int count = min(8, d - 8 * c);
            const Vec8 v = row(c, count, nullptr, false);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = j < count ? v.v[j] - mean : 0.0f;
                q.x = fmaf(e, e, q.x);
            }
        }
        const float r = 1.0f / sqrtf(row_sum2(q, red[1], warps).x / fd + a.eps);
        if (tid == 0) a.stats[t] = make_float2(mean, r);
        for (int c = tid; c < d8; c += nt) {
            const int count = min(8, d - 8 * c);
            Vec8 o = row(c, count, nullptr, false);
            const Vec8 w = a.weight ? cached8<ALIGNED>(a.weight + 8 * c, count) : Vec8{{1, 1, 1, 1, 1, 1, 1, 1}};
            const Vec8 b = a.bias ? cached8<ALIGNED>(a.bias + 8 * c, count) : Vec8{};
#pragma unroll
            for (int j = 0; j < 8; ++j) o.v[j] = (o.v[j] - mean) * r * w.v[j] + b.v[j];
            put8<ALIGNED>(a.n + t * d + 8 * static_cast<size_t>(c), o, count);
        }
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
    float* partial;  // [blocks, 2, d]
};

// One reduction a row; the column sums dweight and dbias of the rows that a block visits stay in registers and are
// written once a block.  Rows of up to 8192 values.
template <typename X, int VPT, bool ALIGNED>
__global__ void __launch_bounds__(512, 1) layer_norm_backward_kernel(Backward a) {
    __shared__ float2 red[2][kMaxWarps];
    using B = __nv_bfloat16;
    const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, d = a.d;
    const float inv_d = 1.0f / static_cast<float>(d);
    const X *x = static_cast<const X*>(a.x), *dy = static_cast<const X*>(a.dy);
    X* dx = static_cast<X*>(a.dx);
    const size_t T = static_cast<size_t>(a.T), step = gridDim.x;
    pdl_wait();
    pdl_trigger();
    const Drop drop(a.drop);
    int count[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) count[v] = min(8, max(0, d - 8 * (tid + v * nt)));
    Raw8<X> xr[VPT], gr[VPT];
    Raw8<B> nr[VPT];
    float2 st = make_float2(0.0f, 0.0f);
    auto fetch = [&](size_t t) {
        st = __ldg(a.stats + t);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (count[v] > 0) {
                const size_t at = t * d + 8 * (tid + v * nt);
                fetch_raw<ALIGNED>(xr[v], x + at, count[v]);
                fetch_raw<ALIGNED>(nr[v], a.dn + at, count[v]);
                if (dy) fetch_raw<ALIGNED>(gr[v], dy + at, count[v]);
            }
    };
    Vec8 w[VPT], sw[VPT], sb[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        w[v] = Vec8{{1, 1, 1, 1, 1, 1, 1, 1}};
        if (count[v] > 0 && a.weight) w[v] = cached8<ALIGNED>(a.weight + 8 * (tid + v * nt), count[v]);
        sw[v] = sb[v] = Vec8{};
    }
    fetch(blockIdx.x);
    int k = 0;
    for (size_t t = blockIdx.x; t < T; t += step, ++k) {
        const float r = st.y, back = -st.x;
        Vec8 yh[VPT], g[VPT], e[VPT];
        float2 sg = make_float2(0.0f, 0.0f), sy = sg;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (count[v] > 0) {
                const Vec8 xv = values(xr[v]), nv = values(nr[v]);
                e[v] = dy ? values(gr[v]) : Vec8{};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 h = mul2(add2(xv.pair(j), make_float2(back, back)), r), m = mul2(nv.pair(j), w[v].pair(j));
                    yh[v].set(j, h);
                    g[v].set(j, m);
                    sg = add2(sg, m);
                    sy = fma2(m, h, sy);
                    sw[v].set(j, fma2(nv.pair(j), h, sw[v].pair(j)));
                    sb[v].set(j, add2(sb[v].pair(j), nv.pair(j)));
                }
            }
        if (t + step < T) fetch(t + step);
        const float2 s = row_sum2(make_float2(sg.x + sg.y, sy.x + sy.y), red[k & 1], warps);
        const float mg = s.x * inv_d, my = s.y * inv_d;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (count[v] > 0) {
                const size_t at = t * d + 8 * (tid + v * nt);
                Vec8 o;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 b = fma2(yh[v].pair(j), make_float2(-my, -my), add2(g[v].pair(j), make_float2(-mg, -mg)));
                    o.set(j, fma2(b, r, e[v].pair(j)));
                }
                put8<ALIGNED>(dx + at, o, count[v]);
                if (a.dh) {
                    if (drop.on()) {
                        if (ALIGNED) drop.apply(o, at);
                        else drop.apply_any(o, at);
                    }
                    put8<ALIGNED>(a.dh + at, o, count[v]);
                }
            }
    }
    if (!a.partial) return;
    float* p = a.partial + static_cast<size_t>(blockIdx.x) * 2 * d;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        if (count[v] > 0) {
            const int c = 8 * (tid + v * nt);
            put8<ALIGNED>(p + c, sw[v], count[v]);
            put8<ALIGNED>(p + d + c, sb[v], count[v]);
        }
}

// Rows of any width: a block takes a range of rows and reads each twice; the column sums live in its slice of the
// workspace (a thread's own elements).
template <typename X, bool ALIGNED>
__global__ void __launch_bounds__(1024) layer_norm_backward_wide_kernel(Backward a) {
    __shared__ float2 red[2][kMaxWarps];
    using B = __nv_bfloat16;
    const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5, d = a.d, d8 = (d + 7) / 8;
    const float inv_d = 1.0f / static_cast<float>(d);
    pdl_wait();
    pdl_trigger();
    const Drop drop(a.drop);
    float* p = a.partial + static_cast<size_t>(blockIdx.x) * 2 * d;
    int k = 0;
    for (size_t t = blockIdx.x; t < static_cast<size_t>(a.T); t += gridDim.x, ++k) {
        const float2 st = __ldg(a.stats + t);
        auto row = [&](int c, int count, Vec8& yh, Vec8& nv, Vec8& g) {
            const size_t at = t * d + 8 * static_cast<size_t>(c);
            Raw8<X> xr;
            Raw8<B> nr;
            fetch_raw<ALIGNED>(xr, static_cast<const X*>(a.x) + at, count);
            fetch_raw<ALIGNED>(nr, a.dn + at, count);
            const Vec8 xv = values(xr), w = a.weight ? cached8<ALIGNED>(a.weight + 8 * c, count) : Vec8{{1, 1, 1, 1, 1, 1, 1, 1}};
            nv = values(nr);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                yh.v[j] = (xv.v[j] - st.x) * st.y;
                g.v[j] = nv.v[j] * w.v[j];
            }
        };
        float2 s = make_float2(0.0f, 0.0f);
        for (int c = tid; c < d8; c += nt) {
            Vec8 yh, nv, g;
            row(c, min(8, d - 8 * c), yh, nv, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s.x += g.v[j];
                s.y = fmaf(g.v[j], yh.v[j], s.y);
            }
        }
        s = row_sum2(s, red[k & 1], warps);
        const float mg = s.x * inv_d, my = s.y * inv_d;
        for (int c = tid; c < d8; c += nt) {
            const int count = min(8, d - 8 * c);
            const size_t at = t * d + 8 * static_cast<size_t>(c);
            Vec8 yh, nv, g, o, e{};
            row(c, count, yh, nv, g);
            if (a.dy) {
                Raw8<X> er;
                fetch_raw<ALIGNED>(er, static_cast<const X*>(a.dy) + at, count);
                e = values(er);
            }
            Vec8 sw{}, sb{};
            float *pw = p + 8 * static_cast<size_t>(c), *pb = pw + d;
            if (k > 0) {
                Raw8<float> f;
                fetch_raw<ALIGNED>(f, pw, count);
                sw = values(f);
                fetch_raw<ALIGNED>(f, pb, count);
                sb = values(f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o.v[j] = fmaf(g.v[j] - mg - yh.v[j] * my, st.y, e.v[j]);
                sw.v[j] = fmaf(nv.v[j], yh.v[j], sw.v[j]);
                sb.v[j] += nv.v[j];
            }
            put8<ALIGNED>(pw, sw, count);
            put8<ALIGNED>(pb, sb, count);
            put8<ALIGNED>(static_cast<X*>(a.dx) + at, o, count);
            if (a.dh) {
                if (drop.on()) {
                    if (ALIGNED) drop.apply(o, at);
                    else drop.apply_any(o, at);
                }
                put8<ALIGNED>(a.dh + at, o, count);
            }
        }
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
#pragma unroll 8
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

constexpr int kMostInRegisters = 8192;  // values of a row

// Threads of a row and rows side by side in a block.
struct Shape {
    int vpt, threads, rows, per_sm;
};
Shape shape_of(int d, bool bwd) {
    const int d8 = (d + 7) / 8;
    Shape s;
    if (d > kMostInRegisters) return Shape{0, 1024, 1, bwd ? 1 : 2};
    s.vpt = d8 <= 512 ? 1 : 2;
    s.threads = ((d8 + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    s.rows = s.threads == 32 && !bwd ? 4 : 1;
    s.per_sm = bwd ? std::min(8, 512 / s.threads) : (s.vpt == 1 ? 1024 : 512) / (s.threads * s.rows);
    return s;
}

template <typename X, bool H, bool ALIGNED>
cudaError_t forward_as(const Forward& a, int num_sms, cudaStream_t s) {
    const Shape f = shape_of(a.d, false);
    const dim3 block(f.threads, f.rows);
    const int most = (a.T - 1) / f.rows + 1;
    const dim3 grid(std::min(most, num_sms * f.per_sm));
    if (f.vpt == 0) return launch_k(kPdlTrain, layer_norm_wide_kernel<X, H, ALIGNED>, grid, block, 0, s, a);
    if (f.vpt == 1) return launch_k(kPdlTrain, layer_norm_kernel<X, 1, H, ALIGNED>, grid, block, 0, s, a);
    return launch_k(kPdlTrain, layer_norm_kernel<X, 2, H, ALIGNED>, grid, block, 0, s, a);
}
template <typename X, bool ALIGNED>
cudaError_t backward_as(const Backward& a, int blocks, cudaStream_t s) {
    const Shape f = shape_of(a.d, true);
    const dim3 grid(blocks), block(f.threads);
    if (f.vpt == 0) return launch_k(kPdlTrain, layer_norm_backward_wide_kernel<X, ALIGNED>, grid, block, 0, s, a);
    if (f.vpt == 1) return launch_k(kPdlTrain, layer_norm_backward_kernel<X, 1, ALIGNED>, grid, block, 0, s, a);
    return launch_k(kPdlTrain, layer_norm_backward_kernel<X, 2, ALIGNED>, grid, block, 0, s, a);
}

bool vectors(int d, std::initializer_list<const void*> ps) {
    uintptr_t all = 0;
    for (const void* p : ps) all |= reinterpret_cast<uintptr_t>(p);
    return d % 8 == 0 && (all & 15) == 0;
}

}  // namespace

// Blocks of the backward pass on GB300's 152 SMs (the workspace depends on the shape alone).
int layer_norm_blocks(int T, int d) { return std::min(T, kSms * shape_of(d, true).per_sm); }

cudaError_t launch_layer_norm(const LayerNormArgs& g, int num_sms, cudaStream_t s) {
    const Forward a{g.x, g.h, g.weight, g.bias, g.T, g.d, g.eps, g.drop, g.y, g.n, reinterpret_cast<float2*>(g.stats)};
    const bool al = vectors(g.d, {g.x, g.h, g.weight, g.bias, g.y, g.n});
    using B = __nv_bfloat16;
    if (g.x_fp32) {
        if (g.h) return al ? forward_as<float, true, true>(a, num_sms, s) : forward_as<float, true, false>(a, num_sms, s);
        return al ? forward_as<float, false, true>(a, num_sms, s) : forward_as<float, false, false>(a, num_sms, s);
    }
    if (g.h) return al ? forward_as<B, true, true>(a, num_sms, s) : forward_as<B, true, false>(a, num_sms, s);
    return al ? forward_as<B, false, true>(a, num_sms, s) : forward_as<B, false, false>(a, num_sms, s);
}

cudaError_t launch_layer_norm_backward(const LayerNormArgs& g, cudaStream_t s) {
    const Backward a{g.x, reinterpret_cast<const float2*>(g.stats), g.dn, g.dy, g.weight, g.T, g.d, g.drop, g.dx, g.dh, g.partial};
    const bool al = vectors(g.d, {g.x, g.dn, g.dy, g.weight, g.dx, g.dh, g.partial});
    const int blocks = layer_norm_blocks(g.T, g.d);
    using B = __nv_bfloat16;
    const cudaError_t e = g.x_fp32 ? (al ? backward_as<float, true>(a, blocks, s) : backward_as<float, false>(a, blocks, s))
                                   : (al ? backward_as<B, true>(a, blocks, s) : backward_as<B, false>(a, blocks, s));
    if (e != cudaSuccess || !(g.dweight || g.dbias)) return e;
    return launch_k(kPdlTrain, layer_norm_join_kernel, dim3((2 * g.d + 31) / 32), dim3(512), 0, s,
                    static_cast<const float*>(g.partial), blocks, g.d, g.dweight, g.dbias);
}

}  // namespace moe
