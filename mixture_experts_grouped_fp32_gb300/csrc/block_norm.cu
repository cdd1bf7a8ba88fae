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
// One pass over memory each way; bound by it.  A thread block works through its rows (persistent, every
// gridDim-th row) with the next rows on their way into shared memory (cp.async): a thread copies just
// the vectors that it will use, so the ring of rows needs no barrier.  The row sums need one barrier per
// row: the sum over h of row k + 1, which that row starts with, is taken in the same reduction as the
// last sum of row k (forward: one reduction per row, backward: two).  Rows too wide for two of them in
// shared memory (d > 8192) take the plain kernels, which hold one row in registers.
//
// Measured: 4096 x 7168 with an fp32 stream 60 us (5.8 TB/s; 54 under ncu), gradient of 4096 x 4096 52 us
// (3.8 TB/s: 16 warps per SM, whose instruction latency shows; an earlier form that loaded tgate in the row
// that uses it took 78).
//
// The backward pass keeps the column sums A, dres and dw_pre of all rows that a block visits in
// registers, writes them once per block, and a second kernel adds the blocks in a fixed order: no
// atomics, the same result on every run.
#include <algorithm>
#include <atomic>

#include "train_ptx.cuh"
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

// Two sums over a warp, in every lane: a half-warp takes each after the first exchange, so both cost
// little more than the shuffles of one.
__device__ __forceinline__ float2 warp_pair_sum(float2 v) {
    const bool up = threadIdx.x & 16;
    float a = up ? v.y : v.x;
    a += __shfl_xor_sync(0xffffffffu, up ? v.x : v.y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    const float b = __shfl_xor_sync(0xffffffffu, a, 16);
    return up ? make_float2(b, a) : make_float2(a, b);
}
// Two sums over the threads of a row (threadIdx.x), in each of them, with one barrier (none for a single
// warp); the caller's buffers alternate between calls.  `barrier`: 0 if the block has no other threads, else
// one of the row's own.
__device__ __forceinline__ void pair_sum(float (&v)[2], float2* red, int warps, int barrier = 0) {
    float2 s = warp_pair_sum(make_float2(v[0], v[1]));
    if (warps > 1) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) red[warp] = s;
        if (barrier == 0) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(warps * 32) : "memory");
        s = warp_pair_sum(lane < warps ? red[lane] : make_float2(0.0f, 0.0f));
    }
    v[0] = s.x;
    v[1] = s.y;
}

// 16-byte words of eight values of X.
template <typename X>
constexpr int words() { return sizeof(X) == 4 ? 2 : 1; }

// A thread's part of the ring of rows in shared memory: word w of stage s at (s * words + w) * threads.
struct Ring {
    uint4* base;  // this thread's first word
    int per_stage, threads;
    __device__ __forceinline__ uint4* at(int s, int w) const { return base + (s * per_stage + w) * threads; }
};
__device__ __forceinline__ void fetch8(const Ring& r, int s, int w, const __nv_bfloat16* p, size_t i) {
    ptx::cp_async_16(ptx::smem_u32(r.at(s, w)), reinterpret_cast<const uint4*>(p) + i, 16);
}
__device__ __forceinline__ void fetch8(const Ring& r, int s, int w, const float* p, size_t i) {
    ptx::cp_async_16_l1(ptx::smem_u32(r.at(s, w)), reinterpret_cast<const uint4*>(p) + 2 * i);
    ptx::cp_async_16_l1(ptx::smem_u32(r.at(s, w + 1)), reinterpret_cast<const uint4*>(p) + 2 * i + 1);
}
template <typename X>
__device__ __forceinline__ Vec8 ring8(const Ring& r, int s, int w) {
    const uint4 a = *r.at(s, w);
    if constexpr (sizeof(X) == 2) {
        return unpack8(a);
    } else {
        const uint4 b = *r.at(s, w + 1);
        return Vec8{{__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                     __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)}};
    }
}
// tgate of a block's rows, read by a warp 32 rows at a time (a load per row would be waited for in each).
struct TokenGate {
    const float* p;
    int rows;
    float mine = 1.0f;
    template <typename RowOf>
    __device__ __forceinline__ float at(int k, const RowOf& row_of) {
        if (!p) return 1.0f;
        const int lane = threadIdx.x & 31;
        if ((k & 31) == 0) mine = k + lane < rows ? __ldg(p + row_of(k + lane)) : 0.0f;
        return __shfl_sync(0xffffffffu, mine, k & 31);
    }
};
// All but the newest `pending` rows have landed (pending = stages - 2).
__device__ __forceinline__ void wait_rows(int pending) {
    if (pending == 2) ptx::cp_async_wait<2>();
    else if (pending == 1) ptx::cp_async_wait<1>();
    else ptx::cp_async_wait<0>();
}

__device__ __forceinline__ Vec8 ones() { return Vec8{{1, 1, 1, 1, 1, 1, 1, 1}}; }

// H: with h (the block's output, its norm and gates);  N: with n (the next norm).
template <typename X, int VPT, bool H, bool N>
__global__ void __launch_bounds__(VPT == 1 ? 256 : 512, VPT == 1 ? 4 : 1)
norm_rows_kernel(const X* __restrict__ x, const __nv_bfloat16* __restrict__ h, const float* __restrict__ w_pre,
                 const float* __restrict__ w_post, const float* __restrict__ gate, const float* __restrict__ tgate,
                 const float* __restrict__ res, int T, int d, float eps, int stages, X* __restrict__ y,
                 __nv_bfloat16* __restrict__ n) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float2 red[2][kMaxWarps];
    constexpr int XW = words<X>();
    const int tid = threadIdx.x, nt = blockDim.x, d8 = d / 8, warps = nt >> 5;
    const float inv_d = 1.0f / static_cast<float>(d);
    const int per_vec = XW + (H ? 1 : 0);
    const Ring ring{ring_smem + tid, VPT * per_vec, nt};
    const int rows = (T - static_cast<int>(blockIdx.x) - 1) / static_cast<int>(gridDim.x) + 1;  // gridDim.x <= T
    pdl_wait();
    pdl_trigger();
    auto row_of = [&](int k) { return static_cast<size_t>(blockIdx.x) + static_cast<size_t>(k) * gridDim.x; };
    auto fetch = [&](int k, int s) {
        if (k < rows) {
            const size_t base = row_of(k) * d8;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * nt;
                if (c < d8) {
                    fetch8(ring, s, v * per_vec, x, base + c);
                    if (H) fetch8(ring, s, v * per_vec + XW, h, base + c);
                }
            }
        }
        ptx::cp_async_commit();
    };
    for (int k = 0; k < stages - 1; ++k) fetch(k, k);
    Vec8 wn[VPT], wg[VPT], rs[VPT];  // w_pre, gate w_post, res
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = tid + v * nt;
        wn[v] = wg[v] = rs[v] = ones();
        if (c < d8) {
            if (N) wn[v] = load8_cached(w_pre, c);
            if (H) wg[v] = load8_cached(w_post, c);
            if (gate) {
                const Vec8 g = load8_cached(gate, c);
#pragma unroll
                for (int j = 0; j < 4; ++j) wg[v].set(j, mul2(wg[v].pair(j), g.pair(j)));
            }
            if (res) rs[v] = load8_cached(res, c);
        }
    }
    auto sum_h = [&](int s) {
        float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (tid + v * nt < d8) {
                const Vec8 hv = ring8<__nv_bfloat16>(ring, s, v * per_vec + XW);
#pragma unroll
                for (int j = 0; j < 4; ++j) a = fma2(hv.pair(j), hv.pair(j), a);
            }
        return a.x + a.y;
    };
    float sums[2] = {0.0f, 0.0f};  // of y^2 in this row, of h^2 in the next
    TokenGate token{tgate, rows};
    if (H) {
        wait_rows(stages - 2);
        sums[1] = sum_h(0);
        pair_sum(sums, red[1], warps);
    }
    else wait_rows(stages - 2);
    int s = 0;
    for (int k = 0; k < rows; ++k) {
        const int free_stage = s == 0 ? stages - 1 : s - 1, next = s + 1 == stages ? 0 : s + 1;
        fetch(k + stages - 1, free_stage);
        const size_t t = row_of(k), base = t * d8;
        const float scale = H ? rsqrtf(sums[1] * inv_d + eps) * token.at(k, row_of) : 0.0f;
        Vec8 yv[VPT];
        float2 yy = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = tid + v * nt;
            if (c < d8) {
                yv[v] = ring8<X>(ring, s, v * per_vec);
                if (H) {
                    const Vec8 hv = ring8<__nv_bfloat16>(ring, s, v * per_vec + XW);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        yv[v].set(j, fma2(rs[v].pair(j), yv[v].pair(j), mul2(wg[v].pair(j), mul2(hv.pair(j), scale))));
                    if (y) store8(y, base + c, yv[v]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) yy = fma2(yv[v].pair(j), yv[v].pair(j), yy);
            }
        }
        wait_rows(stages - 2);  // the next row
        sums[0] = yy.x + yy.y;
        sums[1] = H && k + 1 < rows ? sum_h(next) : 0.0f;
        pair_sum(sums, red[k & 1], warps);
        if (N) {
            const float ry = rsqrtf(sums[0] * inv_d + eps);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * nt;
                if (c < d8) {
                    Vec8 o;
#pragma unroll
                    for (int j = 0; j < 4; ++j) o.set(j, mul2(wn[v].pair(j), mul2(yv[v].pair(j), ry)));
                    store8(n, base + c, o);
                }
            }
        }
        s = next;
    }
    ptx::cp_async_wait_all();
}

// Column sums of a block go to partial[blockIdx][3][d]: A, dres, dw_pre.  SIDE (narrow rows): the block works
// on blockDim.y of them side by side, each with its threads, ring and barrier, and adds up their column sums at
// the end: the SM's 512 threads are used whatever the width, and fewer blocks' sums remain to be joined (16384
// rows of 256 values 15 us, of 512 29, 4096 of 1024 18; as four blocks per SM 28, 42 and 20).
template <typename X, int VPT, bool H, bool N, bool SIDE>
__global__ void __launch_bounds__(512, 1)
norm_rows_backward_kernel(const X* __restrict__ x, const __nv_bfloat16* __restrict__ h, const X* __restrict__ dy,
                          const __nv_bfloat16* __restrict__ dn, const float* __restrict__ w_pre,
                          const float* __restrict__ w_post, const float* __restrict__ gate,
                          const float* __restrict__ tgate, const float* __restrict__ res, int T, int d, float eps,
                          int stages, int kept, X* __restrict__ dx, __nv_bfloat16* __restrict__ dh,
                          float* __restrict__ dtgate, float* __restrict__ partial) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float2 red1[2][kMaxWarps], red2[2][kMaxWarps];
    constexpr int XW = words<X>();
    using B = __nv_bfloat16;
    const int tid = threadIdx.x, nt = blockDim.x, d8 = d / 8, warps = nt >> 5;
    const int group = SIDE ? threadIdx.y : 0, groups = SIDE ? blockDim.y : 1;
    const int warp0 = group * warps, barrier = SIDE ? 1 + group : 0;
    const float inv_d = 1.0f / static_cast<float>(d);
    // Words of a vector: x, then dy, h, dn as given.
    const int o_dy = XW, o_h = o_dy + (dy ? XW : 0), o_dn = o_h + (H ? 1 : 0), per_vec = o_dn + (N ? 1 : 0);
    const Ring ring{ring_smem + group * (stages * VPT * per_vec * nt) + tid, VPT * per_vec, nt};
    const int first = static_cast<int>(blockIdx.x) * groups + group, step = static_cast<int>(gridDim.x) * groups;
    const int rows = first < T ? (T - first - 1) / step + 1 : 0;
    pdl_wait();
    pdl_trigger();
    auto row_of = [&](int k) { return static_cast<size_t>(first) + static_cast<size_t>(k) * step; };
    auto fetch = [&](int k, int s) {
        if (k < rows) {
            const size_t base = row_of(k) * d8;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * nt;
                if (c < d8) {
                    fetch8(ring, s, v * per_vec, x, base + c);
                    if (dy) fetch8(ring, s, v * per_vec + o_dy, dy, base + c);
                    if (H) fetch8(ring, s, v * per_vec + o_h, h, base + c);
                    if (N) fetch8(ring, s, v * per_vec + o_dn, dn, base + c);
                }
            }
        }
        ptx::cp_async_commit();
    };
    for (int k = 0; k < stages - 1; ++k) fetch(k, k);
    // One vector per thread: the weights stay in registers.  Two: they are read again where used (the
    // column sums take the registers), from shared memory behind the ring where they fit (`kept`; each thread
    // keeps its own), else from global memory, for which the ring leaves half of the SM's memory to L1.
    Vec8 kn[VPT], kg[VPT], kr[VPT];
    auto load_weights = [&](int c, Vec8& n_, Vec8& g_, Vec8& r_) {
        n_ = N ? load8_cached(w_pre, c) : ones();
        g_ = H ? load8_cached(w_post, c) : ones();
        if (gate) {
            const Vec8 g = load8_cached(gate, c);
#pragma unroll
            for (int j = 0; j < 4; ++j) g_.set(j, mul2(g_.pair(j), g.pair(j)));
        }
        r_ = res ? load8_cached(res, c) : ones();
    };
    if (VPT == 1 && tid < d8) load_weights(tid, kn[0], kg[0], kr[0]);
    // Word w of 6 of vector v: w_pre, gate w_post, res, two words each.
    uint4* const keep = ring_smem + stages * VPT * per_vec * nt + tid;
    auto keep_at = [&](int v, int w) { return reinterpret_cast<float4*>(keep + (v * 6 + w) * nt); };
    if (VPT > 1 && kept) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = tid + v * nt;
            if (c < d8) {
                Vec8 a, b, r;
                load_weights(c, a, b, r);
                const Vec8* all[3] = {&a, &b, &r};
#pragma unroll
                for (int w = 0; w < 6; ++w) {
                    const float* p = all[w / 2]->v + 4 * (w & 1);
                    *keep_at(v, w) = make_float4(p[0], p[1], p[2], p[3]);
                }
            }
        }
    }
    auto weights = [&](int v, int c, Vec8& n_, Vec8& g_, Vec8& r_) {
        if (VPT == 1) {
            n_ = kn[0], g_ = kg[0], r_ = kr[0];
        } else if (kept) {
            auto get = [&](int w, Vec8& o) {
                const float4 a = *keep_at(v, w), b = *keep_at(v, w + 1);
                o = Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
            };
            get(0, n_);
            get(2, g_);
            get(4, r_);
        } else {
            load_weights(c, n_, g_, r_);
        }
    };
    Vec8 sA[VPT], sR[VPT], sP[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) sA[v].v[j] = sR[v].v[j] = sP[v].v[j] = 0.0f;
    auto sum_h = [&](int s) {
        float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (tid + v * nt < d8) {
                const Vec8 hv = ring8<B>(ring, s, v * per_vec + o_h);
#pragma unroll
                for (int j = 0; j < 4; ++j) a = fma2(hv.pair(j), hv.pair(j), a);
            }
        return a.x + a.y;
    };
    // Pair j of the row's y (res x + gate w_post h tgate / rms(h)).
    auto stream = [&](const Vec8& xv, const Vec8& hv, const Vec8& wg, const Vec8& rs, float hs, int j) {
        return H ? fma2(rs.pair(j), xv.pair(j), mul2(wg.pair(j), mul2(hv.pair(j), hs))) : xv.pair(j);
    };
    float s2[2] = {0.0f, 0.0f};  // S of this row, sum of h^2 in the next
    TokenGate token{tgate, rows};
    if (H) {
        wait_rows(stages - 2);
        s2[1] = sum_h(0);
        pair_sum(s2, red2[1] + warp0, warps, barrier);
    }
    else wait_rows(stages - 2);
    int s = 0;
    for (int k = 0; k < rows; ++k) {
        const int free_stage = s == 0 ? stages - 1 : s - 1, next = s + 1 == stages ? 0 : s + 1;
        fetch(k + stages - 1, free_stage);
        const size_t t = row_of(k), base = t * d8;
        const float tg = token.at(k, row_of);
        const float rh = H ? rsqrtf(s2[1] * inv_d + eps) : 0.0f;
        const float hs = rh * tg;
        float ry = 0.0f, mean = 0.0f;
        if (N) {
            float2 yy = make_float2(0.0f, 0.0f), ey = yy;  // sums of y^2 and of dn w_pre y
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * nt;
                if (c < d8) {
                    Vec8 wn, wg, rs;
                    weights(v, c, wn, wg, rs);
                    const Vec8 xv = ring8<X>(ring, s, v * per_vec), nv = ring8<B>(ring, s, v * per_vec + o_dn);
                    Vec8 hv{};
                    if (H) hv = ring8<B>(ring, s, v * per_vec + o_h);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 a = stream(xv, hv, wg, rs, hs, j);
                        yy = fma2(a, a, yy);
                        ey = fma2(mul2(nv.pair(j), wn.pair(j)), a, ey);
                    }
                }
            }
            float s1[2] = {yy.x + yy.y, ey.x + ey.y};
            pair_sum(s1, red1[k & 1] + warp0, warps, barrier);
            ry = rsqrtf(s1[0] * inv_d + eps);
            mean = s1[1] * ry * inv_d;
        }
        Vec8 q[VPT];
        float2 qh = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = tid + v * nt;
            if (c < d8) {
                Vec8 wn, wg, rs;
                weights(v, c, wn, wg, rs);
                const Vec8 xv = ring8<X>(ring, s, v * per_vec);
                Vec8 D{}, hv{}, o;
                if (dy) D = ring8<X>(ring, s, v * per_vec + o_dy);
                if (H) hv = ring8<B>(ring, s, v * per_vec + o_h);
                if (N) {
                    const Vec8 nv = ring8<B>(ring, s, v * per_vec + o_dn);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 yh = mul2(stream(xv, hv, wg, rs, hs, j), ry);
                        sP[v].set(j, fma2(nv.pair(j), yh, sP[v].pair(j)));
                        D.set(j, fma2(fma2(yh, -mean, mul2(nv.pair(j), wn.pair(j))), ry, D.pair(j)));
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o.set(j, mul2(rs.pair(j), D.pair(j)));
                    sR[v].set(j, fma2(D.pair(j), xv.pair(j), sR[v].pair(j)));
                }
                store8(dx, base + c, o);
                if (H) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sA[v].set(j, fma2(D.pair(j), mul2(hv.pair(j), hs), sA[v].pair(j)));
                        q[v].set(j, mul2(D.pair(j), wg.pair(j)));
                        qh = fma2(q[v].pair(j), hv.pair(j), qh);
                    }
                }
            }
        }
        wait_rows(stages - 2);  // the next row
        if (H) {
            s2[0] = qh.x + qh.y;
            s2[1] = k + 1 < rows ? sum_h(next) : 0.0f;
            pair_sum(s2, red2[k & 1] + warp0, warps, barrier);
            const float qmean = s2[0] * rh * inv_d;  // mean of q hh
            if (dtgate && tid == 0) dtgate[t] = s2[0] * rh;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int c = tid + v * nt;
                if (c < d8) {
                    const Vec8 hv = ring8<B>(ring, s, v * per_vec + o_h);
                    Vec8 o;
#pragma unroll
                    for (int j = 0; j < 4; ++j) o.set(j, mul2(fma2(hv.pair(j), -rh * qmean, q[v].pair(j)), hs));
                    store8(dh, base + c, o);
                }
            }
        }
        s = next;
    }
    ptx::cp_async_wait_all();
    float* p = partial + static_cast<size_t>(blockIdx.x) * 3 * d;
    if constexpr (SIDE) {
        __syncthreads();  // the rings are done with
        float* all = reinterpret_cast<float*>(ring_smem);
        auto put = [&](int which, const Vec8& a) {  // (store8 is for global memory)
            float4* q = reinterpret_cast<float4*>(all + (group * 3 + which) * d) + 2 * tid;
            q[0] = make_float4(a.v[0], a.v[1], a.v[2], a.v[3]);
            q[1] = make_float4(a.v[4], a.v[5], a.v[6], a.v[7]);
        };
        if (tid < d8) {
            put(0, sA[0]);
            put(1, sR[0]);
            put(2, sP[0]);
        }
        __syncthreads();
        for (int c = group * nt + tid; c < 3 * d; c += groups * nt) {
            float a = all[c];
            for (int g = 1; g < groups; ++g) a += all[g * 3 * d + c];
            p[c] = a;
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = tid + v * nt;
        if (c < d8) {
            store8(p, c, sA[v]);
            store8(p + d, c, sR[v]);
            store8(p + 2 * static_cast<size_t>(d), c, sP[v]);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Wide rows (d > 8192): one row at a time in registers (or the compiler's spills of them).
// ---------------------------------------------------------------------------------------------
constexpr int max_threads(int vpt) { return vpt == 8 ? 1024 : 512; }

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

// How a pass is launched: vectors of eight per thread, threads (a multiple of 32), blocks per SM and rows
// in the ring; stages = 0: the plain kernels.
struct Shape {
    int vpt, threads, per_sm, stages;
    int groups;  // rows that a block works on side by side
    int kept;  // backward, two vectors per thread: the weights fit behind the ring
    size_t smem;
};
constexpr int kSms = 152;                 // of a GB300
constexpr size_t kMostSmem = 225 * 1024;  // dynamic shared memory of a block, at most

Shape shape_of(const BlockNormArgs& a, bool bwd) {
    const int d8 = a.d / 8;
    Shape s{};
    s.groups = 1;
    if (a.d > 8192) {
        s.vpt = d8 <= 2048 ? 4 : 8;
        s.threads = ((d8 + s.vpt - 1) / s.vpt + 31) / 32 * 32;
        s.per_sm = bwd ? 2 : 16;
        return s;
    }
    // Forward: up to 256 threads of one vector or 512 of two, 1024 threads per SM.  Backward: one vector
    // up to 512 threads, with up to 128 registers a thread 512 threads per SM; rows of up to 1024 values side by
    // side in one block, no more of them than leave each of the 152 SMs rows (of 2048 values, two blocks: 30.0
    // against 30.8 us for 4096 rows).
    s.vpt = d8 <= (bwd ? 512 : 256) ? 1 : 2;
    s.threads = ((d8 + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    if (bwd && s.threads <= 128) s.groups = std::max(1, std::min(512 / s.threads, (a.T - 1) / kSms + 1));
    s.per_sm = bwd ? (s.threads > 128 && s.threads <= 256 ? 2 : 1)
                   : (s.vpt == 2 ? (s.threads <= 256 ? 2 : 1) : s.threads <= 64 ? 16 : 1024 / s.threads);
    const int xw = a.x_fp32 ? 2 : 1;
    const int words = bwd ? xw * (a.dy ? 2 : 1) + (a.h ? 1 : 0) + (a.dn ? 1 : 0) : xw + (a.h ? 1 : 0);
    const size_t row = static_cast<size_t>(words) * s.vpt * s.threads * 16;
    // Up to four rows in 150 KB per SM (200 KB, a row more for the widest: 62 against 60 us for 4096 x 7168 with
    // an fp32 stream; 100 KB: 67).
    const size_t fit = (bwd && s.vpt == 2 ? 112 : 150) * 1024 / (row * s.per_sm * s.groups);
    s.stages = fit >= 4 ? 4 : fit >= 3 ? 3 : 2;
    s.smem = std::max(row * s.stages, s.groups > 1 ? sizeof(float) * 3 * a.d : 0) * s.groups;
    const size_t weights = static_cast<size_t>(6) * s.vpt * s.threads * 16;
    if (bwd && s.vpt == 2 && 2 * row + weights <= kMostSmem) {
        s.kept = 1;
        s.stages = 3 * row + weights <= kMostSmem ? 3 : 2;
        s.smem = s.stages * row + weights;
    }
    return s;
}

template <typename... KArgs>
cudaError_t allow_smem(void (*kernel)(KArgs...), std::atomic<bool>* done) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && done[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

template <typename X, int VPT, bool H, bool N>
cudaError_t forward_as(const BlockNormArgs& a, const Shape& s, int grid, cudaStream_t st) {
    static std::atomic<bool> done[64] = {};
    const cudaError_t e = allow_smem(norm_rows_kernel<X, VPT, H, N>, done);
    if (e != cudaSuccess) return e;
    return launch_k(kPdlTrain, norm_rows_kernel<X, VPT, H, N>, dim3(grid), dim3(s.threads), s.smem, st,
                    static_cast<const X*>(a.x), a.h, a.w_pre, a.w_post, a.gate, a.tgate, a.res, a.T, a.d, a.eps,
                    s.stages, static_cast<X*>(a.y), a.n);
}
template <typename X, int VPT>
cudaError_t forward_rows(const BlockNormArgs& a, const Shape& s, int grid, cudaStream_t st) {
    if (!a.h) return forward_as<X, VPT, false, true>(a, s, grid, st);
    return a.n ? forward_as<X, VPT, true, true>(a, s, grid, st) : forward_as<X, VPT, true, false>(a, s, grid, st);
}
template <typename X, int VPT>
cudaError_t forward_wide(const BlockNormArgs& a, const Shape& s, int grid, cudaStream_t st) {
    return launch_k(kPdlTrain, block_norm_kernel<X, VPT>, dim3(grid), dim3(s.threads), 0, st,
                    static_cast<const X*>(a.x), a.h, a.w_pre, a.w_post, a.gate, a.tgate, a.res, a.T, a.d, a.eps,
                    static_cast<X*>(a.y), a.n);
}
template <typename X, int VPT, bool H, bool N, bool SIDE>
cudaError_t backward_with(const BlockNormArgs& a, const Shape& s, int grid, cudaStream_t st) {
    static std::atomic<bool> done[64] = {};
    const cudaError_t e = allow_smem(norm_rows_backward_kernel<X, VPT, H, N, SIDE>, done);
    if (e != cudaSuccess) return e;
    return launch_k(kPdlTrain, norm_rows_backward_kernel<X, VPT, H, N, SIDE>, dim3(grid), dim3(s.threads, s.groups),
                    s.smem, st, static_cast<const X*>(a.x), a.h, static_cast<const X*>(a.dy), a.dn, a.w_pre, a.w_post,
                    a.gate, a.tgate, a.res, a.T, a.d, a.eps, s.stages, s.kept, static_cast<X*>(a.dx), a.dh, a.dtgate,
                    a.partial);
}
template <typename X, int VPT, bool H, bool N>
cudaError_t backward_as(const BlockNormArgs& a, const Shape& s, int grid, cudaStream_t st) {
    if constexpr (VPT == 1)
        if (s.groups > 1) return backward_with<X, VPT, H, N, true>(a, s, grid, st);
    return backward_with<X, VPT, H, N, false>(a, s, grid, st);
}
template <typename X, int VPT>
cudaError_t backward_rows(const BlockNormArgs& a, const Shape& s, int grid, cudaStream_t st) {
    if (a.h)
        return a.dn ? backward_as<X, VPT, true, true>(a, s, grid, st) : backward_as<X, VPT, true, false>(a, s, grid, st);
    return a.dn ? backward_as<X, VPT, false, true>(a, s, grid, st) : backward_as<X, VPT, false, false>(a, s, grid, st);
}
template <typename X, int VPT>
cudaError_t backward_wide(const BlockNormArgs& a, const Shape& s, int grid, cudaStream_t st) {
    return launch_k(kPdlTrain, block_norm_backward_kernel<X, VPT>, dim3(grid), dim3(s.threads), 0, st,
                    static_cast<const X*>(a.x), a.h, static_cast<const X*>(a.dy), a.dn, a.w_pre, a.w_post, a.gate,
                    a.tgate, a.res, a.T, a.d, a.eps, static_cast<X*>(a.dx), a.dh, a.dtgate, a.partial);
}

template <typename X>
cudaError_t launch_x(const BlockNormArgs& a, bool bwd, int num_sms, cudaStream_t st) {
    const Shape s = shape_of(a, bwd);
    const int grid = bwd ? block_norm_blocks(a.T, a.d) : std::min(a.T, num_sms * s.per_sm);
    if (!bwd) {
        if (s.vpt == 1) return forward_rows<X, 1>(a, s, grid, st);
        if (s.vpt == 2) return forward_rows<X, 2>(a, s, grid, st);
        return s.vpt == 4 ? forward_wide<X, 4>(a, s, grid, st) : forward_wide<X, 8>(a, s, grid, st);
    }
    const cudaError_t e = s.vpt == 1   ? backward_rows<X, 1>(a, s, grid, st)
                          : s.vpt == 2 ? backward_rows<X, 2>(a, s, grid, st)
                          : s.vpt == 4 ? backward_wide<X, 4>(a, s, grid, st)
                                       : backward_wide<X, 8>(a, s, grid, st);
    if (e != cudaSuccess || !(a.dw_pre || a.dw_post || a.dgate || a.dres)) return e;
    return launch_k(kPdlTrain, block_norm_join_kernel, dim3((3 * a.d + 31) / 32), dim3(512), 0, st,
                    static_cast<const float*>(a.partial), grid, a.d, a.w_post, a.gate, a.dw_pre, a.dw_post, a.dgate,
                    a.dres);
}

}  // namespace

// Blocks of the backward pass on GB300's 152 SMs (the workspace depends on the shape alone).
int block_norm_blocks(int T, int d) {
    BlockNormArgs a{};
    a.T = T, a.d = d;
    const Shape s = shape_of(a, true);
    return T == 0 ? 0 : std::min((T - 1) / s.groups + 1, kSms * s.per_sm);
}

cudaError_t launch_block_norm(const BlockNormArgs& a, bool backward_pass, int num_sms, cudaStream_t s) {
    return a.x_fp32 ? launch_x<float>(a, backward_pass, num_sms, s)
                    : launch_x<__nv_bfloat16>(a, backward_pass, num_sms, s);
}

}  // namespace moe
