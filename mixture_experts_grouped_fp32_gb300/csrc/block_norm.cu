// block_norm.cu — the root-mean-square norms after and before a block, with the block's gate and the
// residual scale, forward and backward.  Per row t of d values:
//
//   forward    hh = h / rms(h),  rms(a) = sqrt(mean(a^2) + eps)
//              y = res * x + (gate * tgate[t]) * (w_post * hh)        the residual stream after the block
//              n = w_pre * y / rms(y)                                 the next block's input
//   backward   given dy and dn, with yh = y / rms(y) and e = dn * w_pre:
//              D  = dy + (e - yh mean(e yh)) / rms(y)                 the whole gradient of y
//              dx = res * D,  dres = sum_t D x,  dw_pre = sum_t dn yh
//              q  = D * gate * w_post,  S = sum over the row of q h
//              dh = tgate (q - hh mean(q hh)) / rms(h),  dtgate[t] = S / rms(h)
//              A  = sum_t D tgate hh:  dgate = w_post A,  dw_post = gate A
//
// w_pre, w_post, gate, res [d] and tgate [T] are fp32; x, y, dy, dx bf16 or fp32 (the residual stream),
// h, n, dn, dh bf16.  Without h: y = x.  Without w_pre: no n.  y is not kept for the backward pass: it
// is recomputed, in fp32, from x and h, which must be read anyway.
//
// One pass over memory each way: a row lives in the registers of one thread block (VPT vectors of eight
// per thread).  The backward pass keeps the column sums A, dres and dw_pre of all rows that a block
// visits in registers, writes them once per block, and a second kernel adds the blocks in a fixed order:
// no atomics, the same result on every run.
#include "train_util.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 32;

// Sum over the block, in every thread; `red` alternates between two halves so that one barrier is
// enough for each sum.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*red)[N], int warps) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) red[warp][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < warps ? red[lane][k] : 0.0f);
}

__device__ __forceinline__ Vec8 ones() { return Vec8{{1, 1, 1, 1, 1, 1, 1, 1}}; }

// Threads of a block by its vectors per thread (row_shape).
constexpr int max_threads(int vpt) { return vpt == 1 ? 256 : vpt == 8 ? 1024 : 512; }

template <typename X, int VPT>
__global__ void __launch_bounds__(max_threads(VPT))
block_norm_kernel(const X* __restrict__ x, const __nv_bfloat16* __restrict__ h,
                                  const float* __restrict__ w_pre, const float* __restrict__ w_post,
                                  const float* __restrict__ gate, const float* __restrict__ tgate,
                                  const float* __restrict__ res, int T, int d, float eps, X* __restrict__ y,
                                  __nv_bfloat16* __restrict__ n) {
    __shared__ float red[2][kMaxWarps][1];
    const int d8 = d / 8, warps = blockDim.x >> 5;
    const float inv_d = 1.0f / static_cast<float>(d);
    pdl_wait();
    pdl_trigger();
    for (long long t = blockIdx.x; t < T; t += gridDim.x) {
        const size_t base = static_cast<size_t>(t) * d8;
        Vec8 yv[VPT], hv[VPT];
        float ss[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = threadIdx.x + k * blockDim.x;
            if (c < d8) {
                yv[k] = load8(x, base + c);
                if (h) hv[k] = load8(h, base + c);
            }
        }
        if (h) {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (threadIdx.x + k * blockDim.x < d8)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss[0] += hv[k].v[j] * hv[k].v[j];
            block_sum<1>(ss, red[0], warps);
            const float scale = rsqrtf(ss[0] * inv_d + eps) * (tgate ? __ldg(tgate + t) : 1.0f);
            ss[0] = 0.0f;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = threadIdx.x + k * blockDim.x;
                if (c < d8) {
                    const Vec8 wp = load8_cached(w_post, c);
                    const Vec8 gv = gate ? load8_cached(gate, c) : ones();
                    const Vec8 rv = res ? load8_cached(res, c) : ones();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float a = rv.v[j] * yv[k].v[j] + gv.v[j] * wp.v[j] * (hv[k].v[j] * scale);
                        yv[k].v[j] = a;
                        ss[0] += a * a;
                    }
                    if (y) store8(y, base + c, yv[k]);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (threadIdx.x + k * blockDim.x < d8)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss[0] += yv[k].v[j] * yv[k].v[j];
        }
        if (n) {
            block_sum<1>(ss, red[1], warps);
            const float scale = rsqrtf(ss[0] * inv_d + eps);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = threadIdx.x + k * blockDim.x;
                if (c < d8) {
                    const Vec8 wv = load8_cached(w_pre, c);
                    Vec8 o;
#pragma unroll
                    for (int j = 0; j < 8; ++j) o.v[j] = wv.v[j] * (yv[k].v[j] * scale);
                    store8(n, base + c, o);
                }
            }
        }
        if (!(h && n)) __syncthreads();  // one sum per row: its buffer is written again in the next row
    }
}

// Column sums of a block go to partial[blockIdx][3][d]: A, dres, dw_pre.
template <typename X, int VPT>
__global__ void __launch_bounds__(max_threads(VPT))
block_norm_backward_kernel(const X* __restrict__ x, const __nv_bfloat16* __restrict__ h,
                                           const X* __restrict__ dy, const __nv_bfloat16* __restrict__ dn,
                                           const float* __restrict__ w_pre, const float* __restrict__ w_post,
                                           const float* __restrict__ gate, const float* __restrict__ tgate,
                                           const float* __restrict__ res, int T, int d, float eps, X* __restrict__ dx,
                                           __nv_bfloat16* __restrict__ dh, float* __restrict__ dtgate,
                                           float* __restrict__ partial) {
    __shared__ float red0[kMaxWarps][1], red1[kMaxWarps][2], red2[kMaxWarps][1];
    const int d8 = d / 8, warps = blockDim.x >> 5;
    const float inv_d = 1.0f / static_cast<float>(d);
    Vec8 sA[VPT], sR[VPT], sP[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) sA[k].v[j] = sR[k].v[j] = sP[k].v[j] = 0.0f;
    pdl_wait();
    pdl_trigger();
    for (long long t = blockIdx.x; t < T; t += gridDim.x) {
        const size_t base = static_cast<size_t>(t) * d8;
        Vec8 xv[VPT], hv[VPT], D[VPT], nv[VPT];
        float s0[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = threadIdx.x + k * blockDim.x;
            if (c < d8) {
                xv[k] = load8(x, base + c);
                if (h) hv[k] = load8(h, base + c);
                if (dn) nv[k] = load8(dn, base + c);
                D[k] = dy ? load8(dy, base + c) : Vec8{};
            }
        }
        const float tg = tgate ? __ldg(tgate + t) : 1.0f;
        float rh = 0.0f;
        if (h) {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (threadIdx.x + k * blockDim.x < d8)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s0[0] += hv[k].v[j] * hv[k].v[j];
            block_sum<1>(s0, red0, warps);
            rh = rsqrtf(s0[0] * inv_d + eps);
        }
        if (dn) {
            float s1[2] = {0.0f, 0.0f};  // sum of y^2, sum of dn w_pre y
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = threadIdx.x + k * blockDim.x;
                if (c < d8) {
                    const Vec8 wv = load8_cached(w_pre, c);
                    const Vec8 wp = h ? load8_cached(w_post, c) : ones();
                    const Vec8 gv = gate ? load8_cached(gate, c) : ones();
                    const Vec8 rv = res ? load8_cached(res, c) : ones();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float a = xv[k].v[j];
                        if (h) a = rv.v[j] * a + gv.v[j] * wp.v[j] * (hv[k].v[j] * (rh * tg));
                        s1[0] += a * a;
                        s1[1] += nv[k].v[j] * wv.v[j] * a;
                    }
                }
            }
            block_sum<2>(s1, red1, warps);
            const float ry = rsqrtf(s1[0] * inv_d + eps), mean = s1[1] * ry * inv_d;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = threadIdx.x + k * blockDim.x;
                if (c < d8) {
                    const Vec8 wv = load8_cached(w_pre, c);
                    const Vec8 wp = h ? load8_cached(w_post, c) : ones();
                    const Vec8 gv = gate ? load8_cached(gate, c) : ones();
                    const Vec8 rv = res ? load8_cached(res, c) : ones();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float a = xv[k].v[j];
                        if (h) a = rv.v[j] * a + gv.v[j] * wp.v[j] * (hv[k].v[j] * (rh * tg));
                        const float yh = a * ry;
                        sP[k].v[j] += nv[k].v[j] * yh;
                        D[k].v[j] += ry * (nv[k].v[j] * wv.v[j] - yh * mean);
                    }
                }
            }
        }
        float S[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = threadIdx.x + k * blockDim.x;
            if (c < d8) {
                const Vec8 rv = res ? load8_cached(res, c) : ones();
                Vec8 o;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o.v[j] = rv.v[j] * D[k].v[j];
                    sR[k].v[j] += D[k].v[j] * xv[k].v[j];
                }
                store8(dx, base + c, o);
                if (h) {
                    const Vec8 wp = load8_cached(w_post, c);
                    const Vec8 gv = gate ? load8_cached(gate, c) : ones();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        sA[k].v[j] += D[k].v[j] * (tg * (hv[k].v[j] * rh));
                        D[k].v[j] *= gv.v[j] * wp.v[j];
                        S[0] += D[k].v[j] * hv[k].v[j];
                    }
                }
            }
        }
        if (h) {
            block_sum<1>(S, red2, warps);
            const float mean = S[0] * rh * inv_d;  // mean of q hh
            if (dtgate && threadIdx.x == 0) dtgate[t] = S[0] * rh;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = threadIdx.x + k * blockDim.x;
                if (c < d8) {
                    Vec8 o;
#pragma unroll
                    for (int j = 0; j < 8; ++j) o.v[j] = tg * rh * (D[k].v[j] - hv[k].v[j] * rh * mean);
                    store8(dh, base + c, o);
                }
            }
        }
        if (!h || !dn) __syncthreads();  // fewer than two sums per row: a buffer is written again in the next row
    }
    float* p = partial + static_cast<size_t>(blockIdx.x) * 3 * d;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = threadIdx.x + k * blockDim.x;
        if (c < d8) {
            store8(p, c, sA[k]);
            store8(p + d, c, sR[k]);
            store8(p + 2 * static_cast<size_t>(d), c, sP[k]);
        }
    }
}

// Adds the blocks' column sums in block order (16 runs of blocks, then the runs).
__global__ void __launch_bounds__(512)
block_norm_join_kernel(const float* __restrict__ partial, int blocks, int d, const float* __restrict__ w_post,
                       const float* __restrict__ gate, float* __restrict__ dw_pre, float* __restrict__ dw_post,
                       float* __restrict__ dgate, float* __restrict__ dres) {
    __shared__ float part[16][33];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const size_t col = static_cast<size_t>(blockIdx.x) * 32 + lane, width = 3 * static_cast<size_t>(d);
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
        const int which = static_cast<int>(col / d), c = static_cast<int>(col - static_cast<size_t>(which) * d);
        if (which == 0) {
            if (dw_post) dw_post[c] = (gate ? gate[c] : 1.0f) * a;
            if (dgate) dgate[c] = w_post[c] * a;
        } else if (which == 1) {
            if (dres) dres[c] = a;
        } else if (dw_pre) {
            dw_pre[c] = a;
        }
    }
}

// Vectors of eight per thread, and threads (a multiple of 32, at most max_threads).
void row_shape(int d, int* vpt, int* threads) {
    const int d8 = d / 8;
    *vpt = d8 <= 256 ? 1 : d8 <= 1024 ? 2 : d8 <= 2048 ? 4 : 8;
    *threads = ((d8 + *vpt - 1) / *vpt + 31) / 32 * 32;
}

template <typename X, int VPT>
cudaError_t forward(const BlockNormArgs& a, int threads, int num_sms, cudaStream_t s) {
    const int most = num_sms * 16;
    return launch_k(kPdlTrain, block_norm_kernel<X, VPT>, dim3(a.T < most ? a.T : most), dim3(threads), 0, s,
                    static_cast<const X*>(a.x), a.h, a.w_pre, a.w_post, a.gate, a.tgate, a.res, a.T, a.d, a.eps,
                    static_cast<X*>(a.y), a.n);
}
template <typename X, int VPT>
cudaError_t backward(const BlockNormArgs& a, int threads, cudaStream_t s) {
    cudaError_t e = launch_k(kPdlTrain, block_norm_backward_kernel<X, VPT>, dim3(block_norm_blocks(a.T)), dim3(threads),
                             0, s, static_cast<const X*>(a.x), a.h, static_cast<const X*>(a.dy), a.dn, a.w_pre,
                             a.w_post, a.gate, a.tgate, a.res, a.T, a.d, a.eps, static_cast<X*>(a.dx), a.dh, a.dtgate,
                             a.partial);
    if (e != cudaSuccess || !(a.dw_pre || a.dw_post || a.dgate || a.dres)) return e;
    return launch_k(kPdlTrain, block_norm_join_kernel, dim3((3 * a.d + 31) / 32), dim3(512), 0, s,
                    static_cast<const float*>(a.partial), block_norm_blocks(a.T), a.d, a.w_post, a.gate, a.dw_pre,
                    a.dw_post, a.dgate, a.dres);
}

}  // namespace

// Blocks of the backward pass: two for each of the 152 SMs, or one per row.
int block_norm_blocks(int T) { return T < 304 ? T : 304; }

cudaError_t launch_block_norm(const BlockNormArgs& a, bool backward_pass, int num_sms, cudaStream_t s) {
    int vpt, threads;
    row_shape(a.d, &vpt, &threads);
#define MOE_NORM_CASE(V)                                                                            \
    if (vpt == V) {                                                                                 \
        if (backward_pass)                                                                          \
            return a.x_fp32 ? backward<float, V>(a, threads, s) : backward<__nv_bfloat16, V>(a, threads, s); \
        return a.x_fp32 ? forward<float, V>(a, threads, num_sms, s)                                 \
                        : forward<__nv_bfloat16, V>(a, threads, num_sms, s);                        \
    }
    MOE_NORM_CASE(1)
    MOE_NORM_CASE(2)
    MOE_NORM_CASE(4)
    MOE_NORM_CASE(8)
#undef MOE_NORM_CASE
    return cudaErrorInvalidValue;
}

}  // namespace moe
