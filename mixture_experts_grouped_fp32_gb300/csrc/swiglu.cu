// swiglu.cu — the activation of the training path, from the joined pre-activations gu [M, 2f] (gate
// columns first) and an optional weight per row (the routing weight of the row's token and slot):
//
//   forward    h = w silu(g) u,  silu(g) = g s,  s = 1 / (1 + exp(-g))
//   backward   dg = w dh u s (1 + g (1 - s)),  du = w dh g s,  dw = sum over the row of dh g s u,
//              and on request h again (for the down projection's weight gradient)
//
// The weight multiplies h rather than the layer's output rows: the down product is linear, so the
// combine becomes a plain sum, and the weight's gradient needs nothing of the down product.
//
// Arithmetic in fp32, one rounding at each store.  Both directions are one pass over memory and bound
// by it: forward 6 bytes per element of h, backward 10 (12 with h).  A thread owns 16-byte vectors of
// eight elements.  The backward pass gives a row to a warp (short rows) or to a 256-thread block (from
// 2048 columns), so that dw is one reduction without atomics.  Measured: gradient of 8192 x 14336 with h
// 213 us, 6.6 TB/s (97 % of the copy bandwidth), forward 115 us (6.1 TB/s); a call of 8 x 2048 1.5 us in a graph.
#include "train_util.cuh"

namespace moe {
namespace {

// 1 / (1 + exp(-g)).  The fast division gives 0 where its divisor is past 2^126 (g below -87.3), and a large u makes
// values of what should be left there: below -87 it is exp(g), to all of fp32's digits.  Once for a vector, so
// that others pay one comparison (each element by exp(-|g|) and a selection: 114 -> 119 us for 8192 x 14336).
__device__ __forceinline__ void sigmoid(const Vec8& g, float (&s)[8]) {
    float least = g.v[0];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        s[j] = __fdividef(1.0f, 1.0f + expf(-g.v[j]));
        least = fminf(least, g.v[j]);
    }
    if (least < -87.0f) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (g.v[j] < -87.0f) s[j] = expf(g.v[j]);
    }
}

__global__ void __launch_bounds__(256)
swiglu_kernel(const __nv_bfloat16* __restrict__ gu, const float* __restrict__ w, long long n8, int f8,
              __nv_bfloat16* __restrict__ h) {
    pdl_wait();
    pdl_trigger();
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n8;
         i += static_cast<long long>(gridDim.x) * 256) {
        const long long r = i / f8;
        const size_t base = static_cast<size_t>(i + r * f8);  // row r starts at vector 2 f8 r
        const Vec8 g = load8(gu, base), u = load8(gu, base + f8);
        const float wr = w ? __ldg(w + r) : 1.0f;
        Vec8 o;
        float s[8];
        sigmoid(g, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = wr * (g.v[j] * s[j] * u.v[j]);
        store8(h, static_cast<size_t>(i), o);
    }
}

// TPR threads per row, 256 / TPR rows per block.
template <int TPR>
__global__ void __launch_bounds__(256)
swiglu_backward_kernel(const __nv_bfloat16* __restrict__ gu, const __nv_bfloat16* __restrict__ dh,
                       const float* __restrict__ w, int M, int f8, __nv_bfloat16* __restrict__ dgu,
                       float* __restrict__ dw, __nv_bfloat16* __restrict__ h) {
    __shared__ float part[8];
    pdl_wait();
    pdl_trigger();
    const int sub = threadIdx.x / TPR, t = threadIdx.x % TPR;
    for (long long r = static_cast<long long>(blockIdx.x) * (256 / TPR) + sub; r < M;
         r += static_cast<long long>(gridDim.x) * (256 / TPR)) {
        const size_t gbase = static_cast<size_t>(r) * 2 * f8, hbase = static_cast<size_t>(r) * f8;
        const float wr = w ? __ldg(w + r) : 1.0f;
        float sum = 0.0f;
        for (int c = t; c < f8; c += TPR) {
            const Vec8 g = load8(gu, gbase + c), u = load8(gu, gbase + f8 + c), d = load8(dh, hbase + c);
            Vec8 og, ou, oh;
            float sg[8];
            sigmoid(g, sg);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float s = sg[j], silu = g.v[j] * s, a = silu * u.v[j];
                const float wd = wr * d.v[j];
                og.v[j] = wd * u.v[j] * s * (1.0f + g.v[j] * (1.0f - s));
                ou.v[j] = wd * silu;
                oh.v[j] = wr * a;
                sum += d.v[j] * a;
            }
            store8(dgu, gbase + c, og);
            store8(dgu, gbase + f8 + c, ou);
            if (h) store8(h, hbase + c, oh);
        }
        if (dw) {
            sum = warp_sum(sum);
            if (TPR == 32) {
                if (t == 0) dw[r] = sum;
            } else {
                if ((t & 31) == 0) part[t >> 5] = sum;
                __syncthreads();
                if (t == 0) {
                    float all = 0.0f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) all += part[k];
                    dw[r] = all;
                }
                __syncthreads();
            }
        }
    }
}

}  // namespace

cudaError_t launch_swiglu(const __nv_bfloat16* gu, const float* w, int M, int f, __nv_bfloat16* h, int num_sms,
                          cudaStream_t s) {
    const long long n8 = static_cast<long long>(M) * (f / 8), want = (n8 + 255) / 256, most = num_sms * 32ll;
    return launch_k(kPdlTrain, swiglu_kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(256), 0, s,
                    gu, w, n8, f / 8, h);
}

cudaError_t launch_swiglu_backward(const __nv_bfloat16* gu, const __nv_bfloat16* dh, const float* w, int M, int f,
                                   __nv_bfloat16* dgu, float* dw, __nv_bfloat16* h, int num_sms, cudaStream_t s) {
    const bool wide = f >= 2048;
    const long long want = wide ? M : (M + 7) / 8, most = num_sms * 64ll;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    return launch_k(kPdlTrain, wide ? swiglu_backward_kernel<256> : swiglu_backward_kernel<32>, grid, dim3(256), 0, s,
                    gu, dh, w, M, f / 8, dgu, dw, h);
}

}  // namespace moe
