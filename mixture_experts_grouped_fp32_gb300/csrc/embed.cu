// embed.cu — rows of an embedding table by token ids, and the table's gradient.
//
//   forward    out[t] = scale table[ids[t]]
//   gradient   dtable[v] (+)= scale sum over the t with ids[t] = v of dy[t], in the order of t
//
// The gradient sorts the tokens by id (a stable counting sort) and adds up runs of equal ids: no atomic decides an
// order, the same result on every run.
//
//   sort   The vocabulary is cut into slices, one for a block.  Every block reads all ids (T values from the L2, which
//          costs less than a pass between blocks would), counts those below its slice and, warp by warp, those of each id
//          in it; sums over the warps and ids then give each warp and id the place of its next token, and a second
//          reading puts the tokens there.  Rows of the slice that no token has are zeroed in the same launch.
//   sum    A group of threads takes a piece of kPiece sorted tokens and the columns eight a thread: runs that begin and
//          end in it are written, the sums of those that go on beyond an end of it are left for
//   join   which adds the pieces' sums of such a run in order.
#include <algorithm>

#include "stack_ops.cuh"

namespace moe {
namespace {

template <typename I>
__device__ __forceinline__ int id_at(const I* ids, size_t t, int V) {  // -1: none of the table
    const long long v = static_cast<long long>(__ldg(ids + t));
    return v >= 0 && v < V ? static_cast<int>(v) : -1;
}

// blockDim.x threads to a row's vectors, blockDim.y rows side by side.
template <typename I, typename X, typename O, bool ALIGNED>
__global__ void __launch_bounds__(256)
embed_kernel(const I* __restrict__ ids, const X* __restrict__ table, int T, int V, int d, float scale,
             O* __restrict__ out, int32_t* status) {
    pdl_wait();
    pdl_trigger();
    const size_t t = static_cast<size_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (t >= static_cast<size_t>(T)) return;
    const int v = id_at(ids, t, V), d8 = (d + 7) / 8;
    if (v < 0 && threadIdx.x == 0 && blockIdx.y == 0) flag_status(status, MOE_STATUS_BAD_TOKEN);
    const int per = 2 * blockDim.x, c0 = blockIdx.y * per + threadIdx.x;
    Raw8<X> r[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int c = c0 + k * blockDim.x;
        r[k] = Raw8<X>{};
        if (c < d8 && v >= 0) fetch_raw<ALIGNED>(r[k], table + static_cast<size_t>(v) * d + 8 * c, min(8, d - 8 * c));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int c = c0 + k * blockDim.x;
        if (c >= d8) break;
        Vec8 o = values(r[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = v >= 0 ? o.v[j] * scale : 0.0f;
        put8<ALIGNED>(out + t * d + 8 * c, o, min(8, d - 8 * c));
    }
}

// ---------------------------------------------------------------------------------------------
// The gradient.
// ---------------------------------------------------------------------------------------------
constexpr int kPiece = 32;         // sorted tokens of a piece
constexpr int kSortWarps = 32;
constexpr int kMostSlice = 1600;   // ids of a slice: 32 warps' counts and the places fill 211 KB of shared memory
constexpr int kSms = 152;          // of a GB300

int slices_of(int V) { return std::max(std::min(V, kSms), (V - 1) / kMostSlice + 1); }

struct Workspace {
    int32_t* found;  // tokens with an id of the table
    int32_t* order;  // [T] tokens sorted by id, then by place
    int32_t* id;     // [T] their ids
    float* part;     // [pieces, 2, d] sums of the runs that begin before a piece, and that go on behind it
};

// Sum over the block's earlier threads and the block's total (1024 threads).
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int w = warp_sums[lane];
    const int own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w - own, warp);
    __syncthreads();
    return before + inc - v;
}

template <typename I, typename O, bool ALIGNED>
__global__ void __launch_bounds__(1024)
embed_sort_kernel(const I* __restrict__ ids, int T, int V, int d, int slice, bool zero, Workspace ws, O* __restrict__ out,
                  int32_t* status) {
    extern __shared__ int32_t counts[];  // [warps][slice], then [slice] tokens of an id
    __shared__ int32_t warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lo = static_cast<int>(min(static_cast<long long>(V), static_cast<long long>(blockIdx.x) * slice));
    const int n = min(slice, V - lo);
    int32_t* mine = counts + warp * slice;
    int32_t* totals = counts + kSortWarps * slice;
    for (int i = tid; i < kSortWarps * slice; i += 1024) counts[i] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    // A warp's tokens: a run of them, 32 at a time.
    const size_t per = (static_cast<size_t>(T) + kSortWarps * 32 - 1) / (kSortWarps * 32) * 32;
    const size_t t0 = warp * per, t1 = min(t0 + per, static_cast<size_t>(T));
    int below = 0;
    bool bad = false;
    for (size_t t = t0; t < t1; t += 32) {
        const bool there = t + lane < t1;
        const int v = there ? id_at(ids, t + lane, V) : V;
        bad |= v < 0;
        below += v >= 0 && v < lo;
        const int b = v - lo;
        const bool in = v >= 0 && b >= 0 && b < n;
        const unsigned hits = __ballot_sync(0xffffffffu, in);
        if (hits == 0) continue;
        const unsigned same = __match_any_sync(0xffffffffu, in ? b : -1);
        if (in && lane == __ffs(same) - 1) mine[b] += __popc(same);
        __syncwarp();
    }
    if (bad && blockIdx.x == 0) flag_status(status, MOE_STATUS_BAD_TOKEN);
    __syncthreads();
    int all_below, own;
    block_scan(below, warp_sums, &all_below);
    // Each id's places: those of the ids before it, then of the warps before one.
    const int ids_per = (n + 1023) / 1024, b0 = min(tid * ids_per, n), b1 = min(b0 + ids_per, n);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
        int c = 0;
        for (int w = 0; w < kSortWarps; ++w) c += counts[w * slice + b];
        totals[b] = c;
        sum += c;
    }
    int at = all_below + block_scan(sum, warp_sums, &own);
    for (int b = b0; b < b1; ++b)
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = counts[w * slice + b];
            counts[w * slice + b] = at;
            at += c;
        }
    if (blockIdx.x == gridDim.x - 1 && tid == 0) *ws.found = all_below + own;
    __syncthreads();
    if (own > 0)
        for (size_t t = t0; t < t1; t += 32) {
            const bool there = t + lane < t1;
            const int v = there ? id_at(ids, t + lane, V) : V;
            const int b = v - lo;
            const bool in = v >= 0 && b >= 0 && b < n;
            const unsigned hits = __ballot_sync(0xffffffffu, in);
            if (hits == 0) continue;
            const unsigned same = __match_any_sync(0xffffffffu, in ? b : -1);
            if (in) {
                const int place = mine[b] + __popc(same & ((1u << lane) - 1));
                ws.order[place] = static_cast<int32_t>(t + lane);
                ws.id[place] = v;
            }
            __syncwarp();
            if (in && lane == __ffs(same) - 1) mine[b] += __popc(same);
            __syncwarp();
        }
    if (!zero) return;
    const int d8 = (d + 7) / 8;
    for (int b = warp; b < n; b += kSortWarps) {  // a warp to a row
        if (totals[b]) continue;
        O* row = out + static_cast<size_t>(lo + b) * d;
        for (int c = lane; c < d8; c += 32) put8<ALIGNED>(row + 8 * c, Vec8{}, min(8, d - 8 * c));
    }
}

__device__ __forceinline__ void red_add4(float* p, float a, float b, float c, float e) {
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(e)
                 : "memory");
}

template <bool ALIGNED, typename O>
__device__ __forceinline__ void finish(O* p, const Vec8& v, float scale, int count, bool add) {
    Vec8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o.v[j] = v.v[j] * scale;
    if constexpr (sizeof(O) == 4) {
        if (add) {  // one addition to an element and call: no order matters
            if (ALIGNED) {
                red_add4(p, o.v[0], o.v[1], o.v[2], o.v[3]);
                red_add4(p + 4, o.v[4], o.v[5], o.v[6], o.v[7]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < count) atomicAdd(p + j, o.v[j]);
            }
            return;
        }
    }
    put8<ALIGNED>(p, o, count);
}

template <typename X, typename O, bool ALIGNED>
__global__ void __launch_bounds__(256)
embed_sum_kernel(const X* __restrict__ dy, int d, float scale, bool add, Workspace ws, O* __restrict__ out) {
    const int d8 = (d + 7) / 8, c = blockIdx.y * blockDim.x + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int found = __ldg(ws.found);
    const long long piece = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const long long p0 = piece * kPiece;
    if (p0 >= found || c >= d8) return;
    const int len = static_cast<int>(min(static_cast<long long>(kPiece), found - p0));
    const int count = min(8, d - 8 * c);
    const int32_t *order = ws.order + p0, *id = ws.id + p0;
    const int before = p0 > 0 ? __ldg(id - 1) : -1, behind = p0 + len < found ? __ldg(id + len) : -1;
    float* part = ws.part + static_cast<size_t>(piece) * 2 * d + 8 * c;
    Vec8 sum{};
    int begun = 0;  // where in the piece the run began
    constexpr int kAhead = 8;
    for (int i0 = 0; i0 < len; i0 += kAhead) {
        Raw8<X> r[kAhead];
        int v[kAhead + 1];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            v[u] = i0 + u < len ? __ldg(id + i0 + u) : -1;
            r[u] = Raw8<X>{};
            if (i0 + u < len)
                fetch_raw<ALIGNED>(r[u], dy + static_cast<size_t>(__ldg(order + i0 + u)) * d + 8 * c, count);
        }
        v[kAhead] = i0 + kAhead < len ? __ldg(id + i0 + kAhead) : -1;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u;
            if (i >= len) break;
            const Vec8 x = values(r[u]);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum.set(j, add2(sum.pair(j), x.pair(j)));
            const bool last = i + 1 == len;
            if (!last && v[u + 1] == v[u]) continue;
            if (begun == 0 && v[u] == before) put8<ALIGNED>(part, sum, count);
            else if (last && v[u] == behind) put8<ALIGNED>(part + d, sum, count);
            else finish<ALIGNED>(out + static_cast<size_t>(v[u]) * d + 8 * c, sum, scale, count, add);
            sum = Vec8{};
            begun = i + 1;
        }
    }
}

// Block (x, y): the run that goes on behind piece x; eight groups of 32 threads take a share of its pieces each.
template <typename O, bool ALIGNED>
__global__ void __launch_bounds__(256)
embed_join_kernel(int d, float scale, bool add, Workspace ws, O* __restrict__ out) {
    __shared__ float part[8][32][9];
    const int d8 = (d + 7) / 8, c = blockIdx.y * 32 + threadIdx.x, g = threadIdx.y;
    pdl_wait();
    pdl_trigger();
    const int found = __ldg(ws.found);
    const long long first = blockIdx.x, end = (first + 1) * kPiece;
    if (end >= found) return;  // (no token behind the piece)
    const int v = __ldg(ws.id + end);
    if (__ldg(ws.id + end - 1) != v) return;
    if (first > 0 && __ldg(ws.id + end - kPiece) == v && __ldg(ws.id + end - kPiece - 1) == v) return;  // begun before
    // The run's last token, by bisection in the sorted ids.
    long long a = end, b = found;
    while (b - a > 1) {
        const long long m = (a + b) / 2;
        if (__ldg(ws.id + m) == v) a = m;
        else b = m;
    }
    const long long pieces = a / kPiece - first;  // behind the first
    const int count = min(8, d - 8 * c);
    Vec8 sum{};
    if (c < d8) {
        const float* p = ws.part + static_cast<size_t>(first) * 2 * d + 8 * c;
        const long long per = (pieces + 8) / 8, k0 = g * per, k1 = min(k0 + per, pieces + 1);
#pragma unroll 4
        for (long long k = k0; k < k1; ++k) {
            Raw8<float> r;
            fetch_raw<ALIGNED>(r, k == 0 ? p + d : p + static_cast<size_t>(k) * 2 * d, count);
            const Vec8 x = values(r);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum.v[j] += x.v[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) part[g][threadIdx.x][j] = sum.v[j];
    __syncthreads();
    if (g != 0 || c >= d8) return;
    for (int k = 1; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum.v[j] += part[k][threadIdx.x][j];
    finish<ALIGNED>(out + static_cast<size_t>(v) * d + 8 * c, sum, scale, count, add);
}

bool vectors(int d, const void* a, const void* b) {
    return d % 8 == 0 && ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}
// Threads of a row's vectors (a power of two), so that 256 threads hold whole rows.
int across(int vectors_of_row) {
    int x = 8;
    while (x < vectors_of_row && x < 256) x *= 2;
    return x;
}
constexpr size_t kAlign = 256;
size_t up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

template <typename I, typename X, typename O, bool ALIGNED>
cudaError_t forward_as(const EmbedArgs& a, cudaStream_t s) {
    const int d8 = (a.d + 7) / 8, tx = across((d8 + 1) / 2), ty = 256 / tx;
    const dim3 grid((a.T - 1) / ty + 1, (d8 - 1) / (2 * tx) + 1);
    return launch_k(kPdlTrain, embed_kernel<I, X, O, ALIGNED>, grid, dim3(tx, ty), 0, s, static_cast<const I*>(a.ids),
                    static_cast<const X*>(a.rows), a.T, a.V, a.d, a.scale, static_cast<O*>(a.out), a.status);
}
template <typename I, typename X, typename O>
cudaError_t forward_io(const EmbedArgs& a, cudaStream_t s) {
    return vectors(a.d, a.rows, a.out) ? forward_as<I, X, O, true>(a, s) : forward_as<I, X, O, false>(a, s);
}
template <typename I>
cudaError_t forward_i(const EmbedArgs& a, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (a.rows_fp32) return a.out_fp32 ? forward_io<I, float, float>(a, s) : forward_io<I, float, B>(a, s);
    return a.out_fp32 ? forward_io<I, B, float>(a, s) : forward_io<I, B, B>(a, s);
}

template <typename I, typename O, bool ALIGNED>
cudaError_t sort_as(const EmbedArgs& a, const Workspace& ws, cudaStream_t s) {
    const int blocks = slices_of(a.V), slice = (a.V - 1) / blocks + 1;
    const size_t smem = sizeof(int32_t) * (kSortWarps + 1) * slice;
    const cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel<I, O, ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sizeof(int32_t) * (kSortWarps + 1) * kMostSlice));
    if (e != cudaSuccess) return e;
    return launch_k(kPdlTrain, embed_sort_kernel<I, O, ALIGNED>, dim3(blocks), dim3(1024), smem, s,
                    static_cast<const I*>(a.ids), a.T, a.V, a.d, slice, !a.accumulate, ws, static_cast<O*>(a.out), a.status);
}
template <typename X, typename O, bool ALIGNED>
cudaError_t sum_as(const EmbedArgs& a, const Workspace& ws, cudaStream_t s) {
    cudaError_t e = a.ids64 ? sort_as<long long, O, ALIGNED>(a, ws, s) : sort_as<int32_t, O, ALIGNED>(a, ws, s);
    if (e != cudaSuccess) return e;
    const int d8 = (a.d + 7) / 8, tx = across(d8), ty = 256 / tx, pieces = (a.T - 1) / kPiece + 1;
    e = launch_k(kPdlTrain, embed_sum_kernel<X, O, ALIGNED>, dim3((pieces - 1) / ty + 1, (d8 - 1) / tx + 1), dim3(tx, ty), 0, s,
                 static_cast<const X*>(a.rows), a.d, a.scale, a.accumulate, ws, static_cast<O*>(a.out));
    if (e != cudaSuccess || pieces == 1) return e;
    return launch_k(kPdlTrain, embed_join_kernel<O, ALIGNED>, dim3(pieces - 1, (d8 + 31) / 32), dim3(32, 8), 0, s, a.d,
                    a.scale, a.accumulate, ws, static_cast<O*>(a.out));
}

}  // namespace

size_t embed_backward_workspace(int T, int d) {
    const size_t pieces = (static_cast<size_t>(T) + kPiece - 1) / kPiece;
    return kAlign + 2 * up(sizeof(int32_t) * static_cast<size_t>(T)) + up(sizeof(float) * 2 * d * pieces);
}

cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t s) {
    return a.ids64 ? forward_i<long long>(a, s) : forward_i<int32_t>(a, s);
}

cudaError_t launch_embed_backward(const EmbedArgs& a, void* workspace, cudaStream_t s) {
    char* p = static_cast<char*>(workspace);
    Workspace ws;
    ws.found = reinterpret_cast<int32_t*>(p);
    ws.order = reinterpret_cast<int32_t*>(p += kAlign);
    ws.id = reinterpret_cast<int32_t*>(p += up(sizeof(int32_t) * static_cast<size_t>(a.T)));
    ws.part = reinterpret_cast<float*>(p + up(sizeof(int32_t) * static_cast<size_t>(a.T)));
    using B = __nv_bfloat16;
    const bool al = vectors(a.d, a.rows, a.out);
    if (a.rows_fp32) {
        if (a.out_fp32) return al ? sum_as<float, float, true>(a, ws, s) : sum_as<float, float, false>(a, ws, s);
        return al ? sum_as<float, B, true>(a, ws, s) : sum_as<float, B, false>(a, ws, s);
    }
    if (a.out_fp32) return al ? sum_as<B, float, true>(a, ws, s) : sum_as<B, float, false>(a, ws, s);
    return al ? sum_as<B, B, true>(a, ws, s) : sum_as<B, B, false>(a, ws, s);
}

}  // namespace moe
