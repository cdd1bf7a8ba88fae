// stack_ops.cuh — dropout masks as a function of (seed, offset, element), so that none is stored.
//
// Philox4x32 with ten rounds (J. K. Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011): the counter of elements 8 b .. 8 b + 7 is (b, offset), 64 bits each, the key is the
// seed; the four words of the result are eight 16-bit numbers, the lower half of a word first.  An element stays if
// its number is at least `cut` = p 65536 (rounded); those that stay are multiplied by 65536 / (65536 - cut), the
// inverse of the probability itself, so that the expectation is exact for the p that is used.
//
// Sixteen bits an element: a block of ten rounds serves eight elements; with 32 bits it would be four, and a bf16 dropout
// (4 bytes an element) would wait for the arithmetic, not for the memory.  The rounds' keys come with the kernel's
// arguments, as operands of their instructions.
#pragma once

#include "train_util.cuh"

namespace moe {

constexpr int kRounds = 10;
struct DropArgs {
    uint32_t cut;  // 0: everything stays
    float up;
    uint32_t key[kRounds][2];  // of each round
    uint64_t offset;
    const int64_t* offset_dev;  // added to the offset, or null
};

// p in [0, 1) -> cut and factor; false for another p (or one that rounds to 1).
inline bool drop_args(double p, uint64_t seed, int64_t offset, const int64_t* offset_dev, DropArgs* a) {
    if (!(p >= 0.0 && p < 1.0)) return false;
    const long cut = static_cast<long>(p * 65536.0 + 0.5);
    if (cut > 65535) return false;
    a->cut = static_cast<uint32_t>(cut);
    a->up = static_cast<float>(65536.0 / (65536 - cut));
    for (uint32_t r = 0; r < kRounds; ++r) {
        a->key[r][0] = static_cast<uint32_t>(seed) + r * 0x9E3779B9u;
        a->key[r][1] = static_cast<uint32_t>(seed >> 32) + r * 0xBB67AE85u;
    }
    a->offset = static_cast<uint64_t>(offset);
    a->offset_dev = offset_dev;
    return true;
}

__device__ __forceinline__ uint4 philox(const DropArgs& a, uint64_t block, uint64_t offset) {
    uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
    uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint64_t m0 = static_cast<uint64_t>(c0) * 0xD2511F53u, m1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(m1 >> 32) ^ c1 ^ a.key[r][0];
        c1 = static_cast<uint32_t>(m1);
        c2 = static_cast<uint32_t>(m0 >> 32) ^ c3 ^ a.key[r][1];
        c3 = static_cast<uint32_t>(m0);
    }
    return make_uint4(c0, c1, c2, c3);
}

cudaError_t launch_dropout(const void* x, bool x_fp32, const void* residual, bool res_fp32, long long n,
                           const DropArgs& a, void* out, cudaStream_t s);

// Layer norm after a residual (layer_norm.cu); x, y, dy, dx fp32 with x_fp32, else bf16.
struct LayerNormArgs {
    bool x_fp32;
    const void* x;  // backward: the stream that was normed
    const __nv_bfloat16* h;
    const float *weight, *bias;
    int T, d;
    float eps;
    DropArgs drop;
    void* y;  // forward
    __nv_bfloat16* n;
    float* stats;             // [T, 2]: mean, 1 / standard deviation
    const __nv_bfloat16* dn;  // backward
    const void* dy;
    void* dx;
    __nv_bfloat16* dh;
    float *dweight, *dbias;
    float* partial;           // [layer_norm_blocks(T, d), 2, layer_norm_width(d)]
};
int layer_norm_blocks(int T, int d);
int layer_norm_width(int d);
cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm_backward(const LayerNormArgs& a, cudaStream_t s);

// A kernel's use of its arguments (which it must hold as a parameter: the keys are read from there).
struct Drop {
    const DropArgs& args;
    uint32_t cut16;  // cut << 16
    uint64_t offset;
    __device__ __forceinline__ explicit Drop(const DropArgs& a)
        : args(a), cut16(a.cut << 16),
          offset(a.offset + (a.offset_dev && a.cut ? static_cast<uint64_t>(__ldg(a.offset_dev)) : 0)) {}
    __device__ __forceinline__ bool on() const { return cut16 != 0; }
    // The eight elements from `first` on (a multiple of 8): zeroed or scaled.  What is dropped is 0 whatever it was,
    // an infinity or a NaN too.
    __device__ __forceinline__ void apply(Vec8& v, uint64_t first) const {
        const uint4 q = philox(args, first >> 3, offset);
        const float up = args.up;
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 s = mul2(v.pair(j), up);
            v.set(j, make_float2((w[j] << 16) >= cut16 ? s.x : 0.0f, w[j] >= cut16 ? s.y : 0.0f));
        }
    }
};

// ---------------------------------------------------------------------------------------------
// Eight values of a row whose width or alignment may be anything: as they are in memory (raw), so that loads can
// be under way while the last ones are worked on.  ALIGNED: width a multiple of 8, 16-byte aligned rows; else values
// one by one, `count` of them (the others are 0).
// ---------------------------------------------------------------------------------------------
template <typename X>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 q;
};
template <>
struct Raw8<float> {
    float4 a, b;
};

template <bool ALIGNED>
__device__ __forceinline__ void fetch_raw(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* p, int count) {
    if constexpr (ALIGNED) {
        r.q = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
        const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = j < count ? u[j] : 0u;
        r.q = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
}
template <bool ALIGNED>
__device__ __forceinline__ void fetch_raw(Raw8<float>& r, const float* p, int count) {
    if constexpr (ALIGNED) {
        const Vec8 v = load8(p, 0);
        r.a = make_float4(v.v[0], v.v[1], v.v[2], v.v[3]);
        r.b = make_float4(v.v[4], v.v[5], v.v[6], v.v[7]);
    } else {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = j < count ? p[j] : 0.0f;
        r.a = make_float4(f[0], f[1], f[2], f[3]);
        r.b = make_float4(f[4], f[5], f[6], f[7]);
    }
}
__device__ __forceinline__ Vec8 values(const Raw8<__nv_bfloat16>& r) { return unpack8(r.q); }
__device__ __forceinline__ Vec8 values(const Raw8<float>& r) {
    return Vec8{{r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w}};
}
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
// The values as they read after a store.
__device__ __forceinline__ Vec8 rounded(const Vec8& v, const __nv_bfloat16*) { return unpack8(pack8(v)); }
__device__ __forceinline__ Vec8 rounded(const Vec8& v, const float*) { return v; }

__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
template <bool ALIGNED, typename X>
__device__ __forceinline__ void put8(X* p, const Vec8& v, int count) {
    if constexpr (ALIGNED) {
        store8(p, 0, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < count) put(p + j, v.v[j]);
    }
}
}  // namespace moe
