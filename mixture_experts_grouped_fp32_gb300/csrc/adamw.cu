// adamw.cu — one AdamW step over many tensors in one launch.  Per element, with g' = c g:
//
//   m = b1 m + (1 - b1) g'          v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// in fp32.  In the moments every operation is rounded by itself (no contraction into fused multiply-adds),
// so that they do not depend on how a compiler pairs operations: with 8-bit moments a last-bit difference
// could move a code.  The step itself uses fused operations and a fast division (2 units in the last
// place of a term that is far smaller than the parameter).  The parameter is rounded once, when it is bf16; a bf16 copy of an
// fp32 parameter can be written along.
//
// 8-bit moments: blocks of 256 elements of a tensor share one fp32 scale.  The first moment is kept as
// E4M3 codes of m / scale, scale = max|m| / 448; of the second moment the root r = sqrt(v) is kept the
// same way (its range is half that of v in the exponent: E4M3's 2^18 then spans 2^36 of v).  A root that
// is not zero is coded at least as 2^-9 (the smallest code): rounded to zero it would divide the next
// step's m by eps alone.  A block whose maximum is below 2^-100 is zero with scale 1; one with a NaN or
// an infinity becomes NaN.  The step itself uses the new moments before their rounding to codes.
//
// Bound by memory, in bytes per element: with 32-bit moments 22 or 24 for bf16 parameters and 26 to 30 for fp32
// ones (gradient in bf16 or fp32, with a bf16 copy 2 more), with 8-bit moments 12 less and 1/16 for the scales.
// Measured: 93.5 M elements with 32-bit moments (fp32, bf16 gradients and copies: 28 bytes) 379 us (6.9 TB/s), 310 M
// with 8-bit moments (all fp32: 16 bytes) 802 us (6.2 TB/s, 64 % of the issue slots).  A
// warp handles one block of 256 elements, eight per lane in 16-byte words where the tensor's pieces are
// aligned for it, else element by element; chunks of 2048 elements over all tensors are dealt to the thread
// blocks in turn (neighbouring chunks run at the same time: contiguous runs of chunks measured 7 % slower,
// 420 against 390 us for 93.5 M elements with 32-bit moments); a thread block walks on in the table from its
// last chunk's tensor.  The table of tensors travels in the kernel's parameters (up to 32 KB): nothing is copied
// to the device before the launch and no memory is held.
#include <cuda_fp8.h>

#include "train_util.cuh"

namespace moe {
namespace {

constexpr int kBlock = 256;               // elements per scale
constexpr int kChunk = 8 * kBlock;        // elements of a thread block's step, one block per warp
constexpr unsigned kPerSm = 5;            // resident thread blocks per SM (48 registers a thread)
constexpr unsigned kGridPerSm = 80;       // launched ones: later ones even out what the first leave
constexpr int kSmallTable = 48, kLargeTable = 400;

struct Entry {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    void* copy;
    long long n;
    unsigned first;  // first chunk
    int vec;         // all pieces aligned for 16-byte words
};
template <int CAP>
struct Table {
    int count;
    unsigned chunks;
    Entry e[CAP];
};

struct Hyper {
    float b1, c1, b2, c2;     // beta, 1 - beta
    float step, inv_root, eps, decay;
    double lr, wd, db1, db2, corr1;  // where the step or the factors are read on the device
    const int32_t* step_dev;
    const float* factors;
};

__device__ __forceinline__ float mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }

__device__ __forceinline__ float load1(const float* p, long long i) { return p[i]; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p, long long i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void store1(float* p, long long i, float v) { p[i] = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, long long i, float v) { p[i] = __float2bfloat16_rn(v); }

// Eight codes and their values (E4M3 -> fp16 is exact), two at a time.
__device__ __forceinline__ void from_e4m3(uint2 c, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = j < 2 ? c.x : c.y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * (j & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}
__device__ __forceinline__ uint2 to_e4m3(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * j], v[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}
__device__ __forceinline__ uint8_t byte_of(uint2 c, int j) { return (j < 4 ? c.x : c.y) >> (8 * (j & 3)) & 255u; }

// Largest magnitude of the warp's values as fp32 bits: as unsigned integers NaN > infinity > numbers.
__device__ __forceinline__ float warp_absmax(const float (&v)[8]) {
    unsigned b = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) b = max(b, __float_as_uint(v[j]) & 0x7fffffffu);
    return __uint_as_float(__reduce_max_sync(0xffffffffu, b));
}

// One block of 256 elements by one warp.  Lane l holds elements 8 l + j (vector path) or l + 32 j.
template <typename P, typename G, bool EIGHT, bool VEC>
__device__ __forceinline__ void step_block(const Entry& t, long long block, const Hyper& h, float factor) {
    const int lane = threadIdx.x & 31;
    const long long first = block * kBlock;
    const long long i8 = first / 8 + lane;                     // vector index
    const long long left = t.n - first;
    auto at = [&](int j) { return first + (VEC ? 8 * lane + j : lane + 32 * j); };
    auto in = [&](int j) { return VEC || lane + 32 * j < left; };
    P* pp = static_cast<P*>(t.p);
    const G* gp = static_cast<const G*>(t.g);
    float p[8], g[8], m[8], r[8];
    if constexpr (VEC) {
        const Vec8 a = load8(pp, i8), b = load8(gp, i8);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = a.v[j], g[j] = b.v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = in(j) ? load1(pp, at(j)) : 0.0f, g[j] = in(j) ? load1(gp, at(j)) : 0.0f;
    }
    if constexpr (EIGHT) {
        uint8_t* mp = static_cast<uint8_t*>(t.m);
        uint8_t* vp = static_cast<uint8_t*>(t.v);
        const float ms = t.ms[block], vs = t.vs[block];
        uint2 mc, vc;
        if constexpr (VEC) {
            mc = __ldcs(reinterpret_cast<const uint2*>(mp) + i8);
            vc = __ldcs(reinterpret_cast<const uint2*>(vp) + i8);
        } else {
            mc = vc = make_uint2(0, 0);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (in(j)) {
                    (j < 4 ? mc.x : mc.y) |= static_cast<uint32_t>(mp[at(j)]) << (8 * (j & 3));
                    (j < 4 ? vc.x : vc.y) |= static_cast<uint32_t>(vp[at(j)]) << (8 * (j & 3));
                }
        }
        from_e4m3(mc, m);
        from_e4m3(vc, r);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 mj = mul2(make_float2(m[j], m[j + 1]), ms), root = mul2(make_float2(r[j], r[j + 1]), vs);
            const float2 vj = mul2(root, root);
            m[j] = mj.x, m[j + 1] = mj.y;
            r[j] = vj.x, r[j + 1] = vj.y;
        }
    } else {
        const float* mp = static_cast<const float*>(t.m);
        const float* vp = static_cast<const float*>(t.v);
        if constexpr (VEC) {
            const Vec8 a = load8(mp, i8), b = load8(vp, i8);
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = a.v[j], r[j] = b.v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = in(j) ? mp[at(j)] : 0.0f, r[j] = in(j) ? vp[at(j)] : 0.0f;
        }
    }
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        // The moments one by one: packed multiplications and additions are contracted.
#pragma unroll
        for (int k = j; k < j + 2; ++k) {
            const float gk = mul(g[k], factor);
            m[k] = add(mul(m[k], h.b1), mul(gk, h.c1));
            v[k] = add(mul(r[k], h.b2), mul(mul(gk, h.c2), gk));
            r[k] = __fsqrt_rn(v[k]);
        }
        const float2 num = mul2(make_float2(m[j], m[j + 1]), h.step);
        const float2 den = fma2(make_float2(r[j], r[j + 1]), h.inv_root, make_float2(h.eps, h.eps));
        const float2 up = make_float2(__fdividef(num.x, den.x), __fdividef(num.y, den.y));
        const float2 pj = fma2(make_float2(p[j], p[j + 1]), h.decay, make_float2(-up.x, -up.y));
        p[j] = pj.x, p[j + 1] = pj.y;
    }
    __nv_bfloat16* copy = static_cast<__nv_bfloat16*>(t.copy);
    if constexpr (VEC) {
        Vec8 o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = p[j];
        store8(pp, i8, o);
        if (copy) store8(copy, i8, o);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (in(j)) {
                store1(pp, at(j), p[j]);
                if (copy) store1(copy, at(j), p[j]);
            }
    }
    if constexpr (EIGHT) {
        // Lanes past the end hold zeros, which change no maximum.
        const float mmax = warp_absmax(m), rmax = warp_absmax(r);
        const bool msome = !(mmax < 0x1p-100f), rsome = !(rmax < 0x1p-100f);
        const float ms = msome ? mul(mmax, 1.0f / 448.0f) : 1.0f, rs = rsome ? mul(rmax, 1.0f / 448.0f) : 1.0f;
        const float mi = msome ? __frcp_rn(ms) : 0.0f, ri = rsome ? __frcp_rn(rs) : 0.0f;
        float qm[8], qr[8];
        const float least = rsome ? 0x1p-9f : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            qm[j] = mul(m[j], mi);
            const float q = mul(r[j], ri);
            qr[j] = (r[j] > 0.0f && q < least) ? least : q;
        }
        const uint2 mc = to_e4m3(qm), vc = to_e4m3(qr);
        uint8_t* mp = static_cast<uint8_t*>(t.m);
        uint8_t* vp = static_cast<uint8_t*>(t.v);
        if constexpr (VEC) {
            reinterpret_cast<uint2*>(mp)[i8] = mc;
            reinterpret_cast<uint2*>(vp)[i8] = vc;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (in(j)) mp[at(j)] = byte_of(mc, j), vp[at(j)] = byte_of(vc, j);
        }
        if (lane == 0) t.ms[block] = ms, t.vs[block] = rs;
    } else {
        float* mp = static_cast<float*>(t.m);
        float* vp = static_cast<float*>(t.v);
        if constexpr (VEC) {
            Vec8 a, b;
#pragma unroll
            for (int j = 0; j < 8; ++j) a.v[j] = m[j], b.v[j] = v[j];
            store8(mp, i8, a);
            store8(vp, i8, b);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (in(j)) mp[at(j)] = m[j], vp[at(j)] = v[j];
        }
    }
}

template <typename P, typename G, bool EIGHT, int CAP>
__global__ void __launch_bounds__(256, kPerSm)
adamw_kernel(const __grid_constant__ Table<CAP> tab, const __grid_constant__ Hyper given) {
    __shared__ Hyper sh;
    pdl_wait();
    pdl_trigger();
    float factor = 1.0f;
    Hyper h = given;
    if (given.step_dev || given.factors) {
        if (threadIdx.x == 0) {
            Hyper x = given;
            const double lr = given.lr * (given.factors ? static_cast<double>(given.factors[1]) : 1.0);
            x.decay = static_cast<float>(1.0 - lr * given.wd);
            double corr1 = given.corr1;
            if (given.step_dev) {
                const double t = static_cast<double>(*given.step_dev);
                corr1 = 1.0 - pow(given.db1, t);
                x.inv_root = static_cast<float>(1.0 / sqrt(1.0 - pow(given.db2, t)));
            }
            x.step = static_cast<float>(lr / corr1);
            sh = x;
        }
        __syncthreads();
        h = sh;
        if (given.factors) factor = given.factors[0];
    }
    const int warp = threadIdx.x >> 5;
    int i = 0;
    for (int hi = tab.count; hi - i > 1;) {  // the first chunk's tensor: e[i].first <= chunk < e[hi].first
        const int mid = (i + hi) >> 1;
        if (tab.e[mid].first <= blockIdx.x) i = mid; else hi = mid;
    }
    unsigned next = i + 1 < tab.count ? tab.e[i + 1].first : tab.chunks;
    for (unsigned c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
        while (c >= next) {
            ++i;
            next = i + 1 < tab.count ? tab.e[i + 1].first : tab.chunks;
        }
        const Entry& t = tab.e[i];
        const long long block = static_cast<long long>(c - t.first) * (kChunk / kBlock) + warp;
        if (block * kBlock >= t.n) continue;
        if (t.vec && (block + 1) * kBlock <= t.n)
            step_block<P, G, EIGHT, true>(t, block, h, factor);
        else
            step_block<P, G, EIGHT, false>(t, block, h, factor);
    }
}

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

template <typename P, typename G, bool EIGHT, int CAP>
cudaError_t launch_table(const moe_adamw_tensor* ts, int count, const Hyper& h, int num_sms, cudaStream_t s) {
    static thread_local Table<CAP> tab;  // up to 32 KB: not on the stack
    unsigned long long chunks = 0;
    int k = 0;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = ts[i];
        if (t.n == 0) continue;
        Entry& e = tab.e[k++];
        e = Entry{t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.copy, t.n, static_cast<unsigned>(chunks), 0};
        e.vec = aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.m, EIGHT ? 8 : 16) &&
                aligned(t.v, EIGHT ? 8 : 16) && aligned(t.copy, 16);
        chunks += static_cast<unsigned long long>((t.n + kChunk - 1) / kChunk);
    }
    if (k == 0) return cudaSuccess;
    if (chunks >= (1ull << 31)) return cudaErrorInvalidValue;
    tab.count = k;
    tab.chunks = static_cast<unsigned>(chunks);
    const unsigned most = num_sms * kGridPerSm;
    return launch_k(kPdlTrain, adamw_kernel<P, G, EIGHT, CAP>, dim3(tab.chunks < most ? tab.chunks : most), dim3(256),
                    0, s, tab, h);
}

template <typename P, typename G, bool EIGHT>
cudaError_t launch_types(const moe_adamw_tensor* ts, int count, const Hyper& h, int num_sms, cudaStream_t s) {
    for (int i = 0; i < count; i += kLargeTable) {
        const int n = count - i < kLargeTable ? count - i : kLargeTable;
        const cudaError_t e = n <= kSmallTable ? launch_table<P, G, EIGHT, kSmallTable>(ts + i, n, h, num_sms, s)
                                               : launch_table<P, G, EIGHT, kLargeTable>(ts + i, n, h, num_sms, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_adamw(const moe_adamw_tensor* ts, int count, bool p_bf16, bool g_bf16, bool eight, double lr,
                         double beta1, double beta2, double eps, double wd, double corr1, double corr2,
                         const int32_t* step_dev, const float* factors, int num_sms, cudaStream_t s) {
    Hyper h{};
    h.b1 = static_cast<float>(beta1);
    h.c1 = static_cast<float>(1.0 - beta1);
    h.b2 = static_cast<float>(beta2);
    h.c2 = static_cast<float>(1.0 - beta2);
    h.step = static_cast<float>(lr / corr1);
    h.inv_root = static_cast<float>(1.0 / corr2);
    h.eps = static_cast<float>(eps);
    h.decay = static_cast<float>(1.0 - lr * wd);
    h.lr = lr;
    h.wd = wd;
    h.corr1 = corr1;
    h.db1 = beta1;
    h.db2 = beta2;
    h.step_dev = step_dev;
    h.factors = factors;
    using B = __nv_bfloat16;
    if (eight) {
        if (p_bf16) return g_bf16 ? launch_types<B, B, true>(ts, count, h, num_sms, s) : launch_types<B, float, true>(ts, count, h, num_sms, s);
        return g_bf16 ? launch_types<float, B, true>(ts, count, h, num_sms, s) : launch_types<float, float, true>(ts, count, h, num_sms, s);
    }
    if (p_bf16) return g_bf16 ? launch_types<B, B, false>(ts, count, h, num_sms, s) : launch_types<B, float, false>(ts, count, h, num_sms, s);
    return g_bf16 ? launch_types<float, B, false>(ts, count, h, num_sms, s) : launch_types<float, float, false>(ts, count, h, num_sms, s);
}

}  // namespace moe
