// dropout.cu — out = residual + keep(i) x / (1 - p), the mask from a counter-based generator (stack_ops.cuh).
//
// Elements are taken in memory order, eight to a thread and step, the random block of an element its index / 8: the
// gradient is the same call on the gradient of the output.  One pass over memory, bound by it: the generator runs
// while the loads are under way.  8192 x 14336 bf16 74 us (6.3 TB/s, 94 % of the copy rate; 55 % of the issue slots, the
// generator's); 64 x 256 1.5 us in a graph, 4 us called from Python, which is the call.
#include <algorithm>

#include "stack_ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128, kPer = 2;  // vectors of eight of a thread

// WHOLE: all vectors are there and aligned; else `count` elements one by one.
template <typename X, typename R, bool RES, bool WHOLE>
__device__ __forceinline__ void drop_vectors(const X* x, const R* residual, size_t first, size_t n, const Drop& drop, R* out) {
    Raw8<X> xr[kPer];
    Raw8<R> rr[kPer];
    auto count = [&](int k) {
        const size_t at = 8 * (first + k * kThreads);
        return WHOLE ? 8 : at < n ? static_cast<int>(min(static_cast<size_t>(8), n - at)) : 0;
    };
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const size_t at = 8 * (first + k * kThreads);
        fetch_raw<WHOLE>(xr[k], x + at, count(k));
        if (RES) fetch_raw<WHOLE>(rr[k], residual + at, count(k));
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const size_t at = 8 * (first + k * kThreads);
        Vec8 v = values(xr[k]);
        if (drop.on()) drop.apply(v, at);
        if (RES) {
            const Vec8 r = values(rr[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) v.set(j, add2(v.pair(j), r.pair(j)));
        }
        put8<WHOLE>(out + at, v, count(k));
    }
}

template <typename X, typename R, bool RES, bool ALIGNED>
__global__ void __launch_bounds__(kThreads)
dropout_kernel(const X* x, const R* residual, size_t n, const __grid_constant__ DropArgs args, R* out) {
    pdl_wait();
    pdl_trigger();
    const Drop drop(args);
    const size_t begin = static_cast<size_t>(blockIdx.x) * (kThreads * kPer), first = begin + threadIdx.x;
    if (ALIGNED && 8 * (begin + kThreads * kPer) <= n) drop_vectors<X, R, RES, true>(x, residual, first, n, drop, out);
    else drop_vectors<X, R, RES, false>(x, residual, first, n, drop, out);
}

template <typename X, typename R, bool RES>
cudaError_t launch_as(const void* x, const void* residual, long long n, const DropArgs& a, void* out, cudaStream_t s) {
    const long long n8 = (n + 7) / 8, blocks = (n8 + kThreads * kPer - 1) / (kThreads * kPer);
    const auto words = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) | reinterpret_cast<uintptr_t>(out);
    const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
    const X* xp = static_cast<const X*>(x);
    const R* rp = static_cast<const R*>(residual);
    R* op = static_cast<R*>(out);
    if (words & 15) return launch_k(kPdlTrain, dropout_kernel<X, R, RES, false>, grid, block, 0, s, xp, rp, n, a, op);
    return launch_k(kPdlTrain, dropout_kernel<X, R, RES, true>, grid, block, 0, s, xp, rp, n, a, op);
}

}  // namespace

cudaError_t launch_dropout(const void* x, bool x_fp32, const void* residual, bool res_fp32, long long n,
                           const DropArgs& a, void* out, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (!residual) return x_fp32 ? launch_as<float, float, false>(x, nullptr, n, a, out, s) : launch_as<B, B, false>(x, nullptr, n, a, out, s);
    if (x_fp32) return res_fp32 ? launch_as<float, float, true>(x, residual, n, a, out, s) : launch_as<float, B, true>(x, residual, n, a, out, s);
    return res_fp32 ? launch_as<B, float, true>(x, residual, n, a, out, s) : launch_as<B, B, true>(x, residual, n, a, out, s);
}

}  // namespace moe
