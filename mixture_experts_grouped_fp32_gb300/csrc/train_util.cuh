// train_util.cuh — vectors of eight values and reductions, shared by the training kernels.
#pragma once

#include "common.cuh"

namespace moe {

// Eight consecutive values, loaded and stored as 16-byte words (bf16: one, fp32: two).
struct Vec8 {
    float v[8];
    __device__ __forceinline__ float2 pair(int j) const { return make_float2(v[2 * j], v[2 * j + 1]); }
    __device__ __forceinline__ void set(int j, float2 a) {
        v[2 * j] = a.x;
        v[2 * j + 1] = a.y;
    }
};
// Two fp32 operations in one instruction, each rounded as the single one.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float b) { return __fmul2_rn(a, make_float2(b, b)); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 fma2(float2 a, float b, float2 c) { return __ffma2_rn(a, make_float2(b, b), c); }
__device__ __forceinline__ void unpack_bf16x2(uint32_t u, float& lo, float& hi) {
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ Vec8 unpack8(const uint4& q) {
    Vec8 r;
    unpack_bf16x2(q.x, r.v[0], r.v[1]);
    unpack_bf16x2(q.y, r.v[2], r.v[3]);
    unpack_bf16x2(q.z, r.v[4], r.v[5]);
    unpack_bf16x2(q.w, r.v[6], r.v[7]);
    return r;
}
__device__ __forceinline__ uint4 pack8(const Vec8& a) {
    return make_uint4(pack_bf16x2(a.v[0], a.v[1]), pack_bf16x2(a.v[2], a.v[3]), pack_bf16x2(a.v[4], a.v[5]),
                      pack_bf16x2(a.v[6], a.v[7]));
}
// Vector i of an array of eights.  The data of these kernels is read once: no reuse in L1.
__device__ __forceinline__ Vec8 load8(const __nv_bfloat16* p, size_t i) {
    return unpack8(__ldcs(reinterpret_cast<const uint4*>(p) + i));
}
// Eight fp32 values are one 32-byte word where the array is aligned for it (a branch that is the same for
// all threads): two 16-byte words touch every 32-byte sector twice.
__device__ __forceinline__ Vec8 load8(const float* p, size_t i) {
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
        Vec8 r;
        asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(r.v[0]), "=f"(r.v[1]), "=f"(r.v[2]), "=f"(r.v[3]), "=f"(r.v[4]), "=f"(r.v[5]),
                       "=f"(r.v[6]), "=f"(r.v[7])
                     : "l"(p + 8 * i));
        return r;
    }
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p) + 2 * i);
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 2 * i + 1);
    return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
// The same for vectors that every row reads again (weights): cached.
__device__ __forceinline__ Vec8 load8_cached(const float* p, size_t i) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p) + 2 * i);
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 2 * i + 1);
    return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, size_t i, const Vec8& a) {
    reinterpret_cast<uint4*>(p)[i] = pack8(a);
}
__device__ __forceinline__ void store8(float* p, size_t i, const Vec8& a) {
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
        asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(a.v[0]), "f"(a.v[1]),
                     "f"(a.v[2]), "f"(a.v[3]), "f"(a.v[4]), "f"(a.v[5]), "f"(a.v[6]), "f"(a.v[7]), "l"(p + 8 * i)
                     : "memory");
        return;
    }
    float4* q = reinterpret_cast<float4*>(p) + 2 * i;
    q[0] = make_float4(a.v[0], a.v[1], a.v[2], a.v[3]);
    q[1] = make_float4(a.v[4], a.v[5], a.v[6], a.v[7]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace moe
