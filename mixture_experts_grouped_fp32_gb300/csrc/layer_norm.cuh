// layer_norm.cuh — what the layer norm's two passes share: sums over a row, a thread's eights of it, launches.
//
// Rows of any width: the eights are those of the tensor in memory order, aligned whatever the row, so a row starts
// in the middle of one (at s = t d mod 8) and its first and last eights are shared with its neighbours: loaded whole,
// their other values masked, and stored value by value.  A block takes rows whose distance is a multiple of 8, which
// have the same s, so a thread's columns, its weights and its column sums stay the same from row to row.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "stack_ops.cuh"
#include "train_ptx.cuh"

namespace moe {
namespace {

constexpr int kSms = 152;  // of a GB300
constexpr int kMostBlocks = 16;  // of a cluster

// Two sums over a warp: lane l holds that of s[l / 16].
__device__ __forceinline__ float warp_sum2(const float (&s)[2]) {
    const bool up = threadIdx.x & 16;
    float v = (up ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, up ? s[0] : s[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
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

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// N = 1, 2 or 4 sums (MOST at the most) over the threads that hold a row.  One barrier each; the buffers alternate, so
// that none is needed behind it.
template <bool CLUSTER, int MOST>
struct RowSums {
    float* red;  // [2][blocks of the cluster x warps][MOST]
    int warps, barrier, blocks, rank, parity = 0;
    __device__ __forceinline__ RowSums(float* red_, int warps_, int barrier_, int blocks_)
        : red(red_), warps(warps_), barrier(barrier_), blocks(blocks_), rank(CLUSTER ? ptx::cluster_ctarank() : 0) {}
    template <int N>
    __device__ __forceinline__ void operator()(float (&s)[N]) {
        static_assert(N <= MOST);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, all = (CLUSTER ? blocks : 1) * warps;
        float mine;  // this lane's part of sum lane / (32 / N)
        if constexpr (N == 4) mine = warp_sum4(s);
        else if constexpr (N == 2) mine = warp_sum2(s);
        else mine = warp_sum(s[0]);
        if (CLUSTER || warps > 1) {
            float* buf = red + parity * all * MOST;
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
    // On their way to `word`, words nt apart.  Values that are not the row's may be any.  `end`: where the tensor ends if
    // that is inside this row's last eight, else 0 (the same for all threads of the row).
    template <typename X>
    __device__ __forceinline__ void copy(uint4* word, int nt, const X* p, long long base, long long end) const {
        const X* from = p + base + off;
        if (!EDGE || (vec && end == 0)) {
            if constexpr (sizeof(X) == 2) {
                copy_word(word, from, 16);
            } else {
                copy_word_l1(word, from, 16);
                copy_word_l1(word + nt, from + 4, 16);
            }
        } else if (vec) {  // (zeros behind the end)
            const long long left = min(8ll, end - base - off) * static_cast<long long>(sizeof(X));  // bytes
            if constexpr (sizeof(X) == 2) {
                copy_word(word, from, static_cast<int>(left));
            } else {
                copy_word_l1(word, from, static_cast<int>(min(left, 16ll)));
                copy_word_l1(word + nt, left > 16 ? from + 4 : from, static_cast<int>(max(0ll, left - 16)));
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
    // Of a vector over the columns (32-byte aligned unless EDGE), or `none` without it.  WIDE: as one word.  Two touch every
    // sector twice, and the L1 bounds what reads little else (8192 x 4096 bf16 without h 34 us, not 28).
    template <bool WIDE = true>
    __device__ __forceinline__ Vec8 column(const float* p, float none) const {
        Vec8 v;
        if (!EDGE && p) {
            if (!WIDE) return load8_cached(p + c, 0);
            asm volatile("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=f"(v.v[0]), "=f"(v.v[1]), "=f"(v.v[2]), "=f"(v.v[3]), "=f"(v.v[4]), "=f"(v.v[5]), "=f"(v.v[6]),
                           "=f"(v.v[7])
                         : "l"(p + c));
            return v;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v.v[j] = p && j >= lo && j < hi ? __ldg(p + c + j) : none;
        return v;
    }
};

inline bool aligned(std::initializer_list<const void*> ps, uintptr_t mask = 15) {
    uintptr_t all = 0;
    for (const void* p : ps) all |= reinterpret_cast<uintptr_t>(p);
    return (all & mask) == 0;
}

// How a pass is launched: blocks of a row's cluster, threads of a row in a block, rows side by side, clusters, eights of a
// thread.
struct Shape {
    int blocks, threads, groups, clusters, vpt;
};
// Eights that a row lies in, at most (one more where rows start inside one).
inline int eights_of(int d) { return (d + 7) / 8 + (d % 8 ? 1 : 0); }
inline int clusters_for(int rows, int per_sm, int blocks) {  // a multiple of 8, or one for each row
    return std::min(rows, std::max(8, kSms * per_sm / blocks / 8 * 8));
}
constexpr size_t kMostSmem = 216 * 1024;  // of a block

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
    cfg.attrs = attr;
    if (pdl_enabled(kPdlTrain)) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (f.blocks > 1) {
        cudaLaunchAttribute& c = attr[cfg.numAttrs++];
        c.id = cudaLaunchAttributeClusterDimension;
        c.val.clusterDim.x = f.blocks;
        c.val.clusterDim.y = c.val.clusterDim.z = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace
}  // namespace moe
