// embed.cu — rows of an embedding table by token ids, and the table's gradient.
//
//   forward    out[t] = scale table[ids[t]]
//   gradient   dtable[v] (+)= scale sum over the t with ids[t] = v of dy[t], in the order of t
//
// The gradient sorts the tokens by id (a stable counting sort) and adds up runs of equal ids: no atomic decides an
// order, the same result on every run.
//
//   sort   The vocabulary is dealt out to the blocks.  Every block reads all ids (T values from the L2, which costs less
//          than a pass between blocks would), counts those of the blocks before it and lists its own tokens, warp by
//          warp, in shared memory.  Of these it counts each warp's of each id; sums over the warps and ids then give
//          each warp and id the place of its next token, and the lists are gone through again to put the tokens there.
//   sum    The sorted tokens are cut into pieces.  A group of threads takes a piece (and the columns eight a thread): it
//          adds up the runs that begin in it, and follows the last one beyond the piece's end.  A run that covers a
//          whole piece is long: its pieces' sums are left for the join.  Other blocks of the same launch zero the rows
//          that no token has.
//   join   adds the pieces' sums of a long run in order.
//
// What bounds it: the forward pass and the gradient of a whole table the memory (16384 tokens of 131072 x 4096, fp32 out:
// 325 us, 2.1 GB written at 7 TB/s).  An addition to the gradient moves little and waits for three kernels of one
// another (12001 tokens of 1028 columns, 50001 ids, Zipf 1.2: 24 us, about 8 the sort, 10 the sums, 6 the joins of the
// most frequent ids).  The sort's time is that of reading all ids in every block once (50000 tokens 24 us with 8 columns;
// with a second reading in place of the lists 37).  Zeroing in the sums' launch, in many small blocks, runs while the
// others wait for their rows (a launch of its own before it held the next kernel back: +115 us).
//
// Rows are taken in units of G = 8, 4, 2 or 1 elements, as width and addresses are aligned; neighbouring threads hold
// neighbouring units.
#include <algorithm>

#include "stack_ops.cuh"

namespace moe {
namespace {

// Where a thread's eight elements of a row lie: units of G, `step` elements apart, the first at `at`, `count` of them
// in the row (tx threads to a stretch of 8 tx columns).
template <int G>
struct Columns {
    int at, step, count;
    __device__ __forceinline__ Columns(int chunk, int tx, int x, int d) {
        at = chunk * 8 * tx + x * G;
        step = tx * G;
        count = min(8 / G, max(0, (d - at + step - 1) / step));
    }
};
// A thread's elements of a row as they were loaded: a register for each load's word, so that nothing waits for a load
// before the values are used.
template <typename X, int G>
struct Units;
template <int G>
struct Units<__nv_bfloat16, G> {
    uint32_t w[G == 1 ? 8 : 4];
    __device__ __forceinline__ void load(int j, const __nv_bfloat16* q) {
        if constexpr (G == 8) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(q));
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else if constexpr (G == 4) {
            const uint2 u = __ldcs(reinterpret_cast<const uint2*>(q));
            w[2 * j] = u.x, w[2 * j + 1] = u.y;
        } else if constexpr (G == 2) {
            w[j] = __ldcs(reinterpret_cast<const unsigned int*>(q));
        } else {
            w[j] = __ldcs(reinterpret_cast<const unsigned short*>(q));
        }
    }
    __device__ __forceinline__ Vec8 values() const {
        Vec8 v;
        if constexpr (G == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v.v[j] = __uint_as_float(w[j] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) unpack_bf16x2(w[j], v.v[2 * j], v.v[2 * j + 1]);
        }
        return v;
    }
};
template <int G>
struct Units<float, G> {
    Vec8 v;
    __device__ __forceinline__ void load(int j, const float* q) {
        if constexpr (G == 8) {
            v = load8(q, 0);
        } else if constexpr (G == 4) {
            const float4 u = __ldcs(reinterpret_cast<const float4*>(q));
            v.v[4 * j] = u.x, v.v[4 * j + 1] = u.y, v.v[4 * j + 2] = u.z, v.v[4 * j + 3] = u.w;
        } else if constexpr (G == 2) {
            const float2 u = __ldcs(reinterpret_cast<const float2*>(q));
            v.v[2 * j] = u.x, v.v[2 * j + 1] = u.y;
        } else {
            v.v[j] = __ldcs(q);
        }
    }
    __device__ __forceinline__ Vec8 values() const { return v; }
};
// Without a branch, so that the loads of several rows are under way together: in place of a unit behind the row the last
// one is loaded again (count >= 1), and not written anywhere.
template <int G, typename X>
__device__ __forceinline__ void fetch(Units<X, G>& r, const X* p, const Columns<G>& c) {
#pragma unroll
    for (int j = 0; j < 8 / G; ++j) r.load(j, p + min(j, c.count - 1) * c.step);
}
template <int G>
__device__ __forceinline__ void write(__nv_bfloat16* p, const Vec8& v, const Columns<G>& c) {
#pragma unroll
    for (int j = 0; j < 8 / G; ++j)
        if (j < c.count) {
            __nv_bfloat16* q = p + j * c.step;
            if constexpr (G == 8) store8(q, 0, v);
            else if constexpr (G == 4)
                *reinterpret_cast<uint2*>(q) = make_uint2(pack_bf16x2(v.v[4 * j], v.v[4 * j + 1]), pack_bf16x2(v.v[4 * j + 2], v.v[4 * j + 3]));
            else if constexpr (G == 2) *reinterpret_cast<uint32_t*>(q) = pack_bf16x2(v.v[2 * j], v.v[2 * j + 1]);
            else put(q, v.v[j]);
        }
}
template <int G>
__device__ __forceinline__ void write(float* p, const Vec8& v, const Columns<G>& c) {
#pragma unroll
    for (int j = 0; j < 8 / G; ++j)
        if (j < c.count) {
            float* q = p + j * c.step;
            if constexpr (G == 8) store8(q, 0, v);
            else if constexpr (G == 4)
                *reinterpret_cast<float4*>(q) = make_float4(v.v[4 * j], v.v[4 * j + 1], v.v[4 * j + 2], v.v[4 * j + 3]);
            else if constexpr (G == 2) *reinterpret_cast<float2*>(q) = make_float2(v.v[2 * j], v.v[2 * j + 1]);
            else *q = v.v[j];
        }
}

template <typename I>
__device__ __forceinline__ int id_of(I v, int V) {  // -1: none of the table
    return v >= 0 && v < V ? static_cast<int>(v) : -1;
}

// blockDim.x threads to a row's columns, blockDim.y rows side by side, two stretches of columns a thread.
template <typename I, typename X, typename O, int G>
__global__ void __launch_bounds__(256)
embed_kernel(const I* __restrict__ ids, const X* __restrict__ table, int T, int V, int d, float scale,
             O* __restrict__ out, int32_t* status) {
    pdl_wait();
    pdl_trigger();
    const size_t t = static_cast<size_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (t >= static_cast<size_t>(T)) return;
    const int v = id_of<I>(__ldg(ids + t), V);
    if (v < 0 && threadIdx.x == 0 && blockIdx.y == 0) flag_status(status, MOE_STATUS_BAD_TOKEN);
    const Columns<G> c[2] = {Columns<G>(2 * blockIdx.y, blockDim.x, threadIdx.x, d),
                             Columns<G>(2 * blockIdx.y + 1, blockDim.x, threadIdx.x, d)};
    Units<X, G> r[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (c[k].count > 0) fetch<G>(r[k], table + static_cast<size_t>(max(v, 0)) * d + c[k].at, c[k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (c[k].count == 0) break;
        Vec8 o = r[k].values();
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = v >= 0 ? o.v[j] * scale : 0.0f;
        write<G>(out + t * d + c[k].at, o, c[k]);
    }
}

// ---------------------------------------------------------------------------------------------
// The gradient.
// ---------------------------------------------------------------------------------------------
constexpr int kMostPiece = 32;
constexpr int kSortWarps = 32;
constexpr int kMostSlice = 1600;   // ids of a slice, whose counts of 32 warps take 205 KB of shared memory
constexpr int kSortSmem = 220 << 10;  // of a block of the sort: the counts, then the warps' lists
constexpr int kSms = 152;          // of a GB300
constexpr int kThreads = 256;      // of a block of the sums, at the most
constexpr int kZeroWords = 16;     // 16-byte words that a thread of the other blocks looks at

// log2 of the sort's blocks: 128 of them (the time is that of reading all ids, whatever their number), more for
// vocabularies whose slices would be too large, fewer where there are fewer ids.
int slice_bits(int V) {
    int bits = 7;
    while ((V - 1) >> bits >= kMostSlice) ++bits;
    while (bits > 0 && (1 << bits) > V) --bits;
    return bits;
}

struct Workspace {
    int32_t* found;    // tokens with an id of the table
    int32_t* order;    // [T] tokens sorted by id, then by place
    int32_t* id;       // [T] their ids
    float* part;       // [pieces, 2, d] sums of the long runs that begin before a piece, and that begin in it
    uint8_t* present;  // [V] whether a token has the id; null where that is not needed
    int32_t* more;     // [pieces] of the long run that begins in a piece: how many pieces it goes on for, else 0
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

// An id as 32 bits: one outside [0, 2^31) as 2^32 - 1.
__device__ __forceinline__ uint32_t word_of(int32_t v) { return static_cast<uint32_t>(v) | static_cast<uint32_t>(v >> 31); }
__device__ __forceinline__ uint32_t word_of(long long v) { return v >> 31 == 0 ? static_cast<uint32_t>(v) : ~0u; }

// Block r of 2^bits takes the ids with v mod 2^bits = r (a vocabulary's frequent tokens are often neighbours: like this
// they are spread), counted as v >> bits; the order of the ids is that of (v mod 2^bits, v >> bits).
template <typename I>
__global__ void __launch_bounds__(1024)
embed_sort_kernel(const I* __restrict__ ids, int T, int V, int slice, int list, int bits, int piece, Workspace ws, int32_t* status) {
    extern __shared__ int32_t counts[];  // [warps][slice], then the lists: [warps][list] {token, id}
    __shared__ int32_t warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t r = blockIdx.x, vocabulary = V, blocks = gridDim.x;
    const unsigned before = (1u << lane) - 1;
    const int n = r < vocabulary ? static_cast<int>((vocabulary - 1 - r) >> bits) + 1 : 0;
    int32_t* mine = counts + warp * slice;
    int2* own_list = reinterpret_cast<int2*>(counts + kSortWarps * slice) + warp * list;
    for (int i = tid; i < kSortWarps * slice; i += 1024) counts[i] = 0;
    pdl_wait();
    pdl_trigger();
    // A warp's tokens: a run of them, 32 at a time and the loads of eight times 32 together.
    const unsigned per = (static_cast<unsigned>(T) + kSortWarps * 32 - 1) / (kSortWarps * 32) * 32;
    const unsigned t0 = min(warp * per, static_cast<unsigned>(T)), t1 = min(t0 + per, static_cast<unsigned>(T));
    constexpr int kAhead = 8;
    auto each = [&](auto&& work) {  // work(token, its id as a word, the block that takes it)
        const I* p = ids + t0 + lane;
        for (unsigned t = t0; t < t1; t += 32 * kAhead, p += 32 * kAhead) {
            const int left = t1 - t;  // tokens
            uint32_t v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) v[u] = 32 * u + lane < left ? word_of(__ldg(p + 32 * u)) : vocabulary;
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (32 * u < left) work(t + 32 * u + lane, v[u], v[u] < vocabulary ? v[u] & (blocks - 1) : blocks);
        }
    };
    int below = 0, len = 0;
    bool bad = false;
    each([&](unsigned t, uint32_t v, uint32_t block) {
        if (r == 0) bad |= block == blocks && t < t1;
        below += block < r;
        const unsigned hits = __ballot_sync(0xffffffffu, block == r);
        if (hits) {
            const int at = len + __popc(hits & before);
            if (block == r && at < list) own_list[at] = make_int2(static_cast<int>(t), static_cast<int>(v));
            len += __popc(hits);
        }
    });
    if (bad) flag_status(status, MOE_STATUS_BAD_TOKEN);
    // The block's tokens from the lists, or from the ids once more where a list was too short.
    const bool listed = !__syncthreads_or(len > list);
    auto each_own = [&](auto&& work) {  // work(token, its id as a word, whether the lane has one)
        if (listed) {
            for (int i = lane; i - lane < len; i += 32) {
                const int2 e = i < len ? own_list[i] : make_int2(0, 0);
                work(static_cast<unsigned>(e.x), static_cast<uint32_t>(e.y), i < len);
            }
        } else {
            each([&](unsigned t, uint32_t v, uint32_t block) { work(t, v, block == r); });
        }
    };
    each_own([&](unsigned, uint32_t v, bool in) {
        if (in) atomicAdd(mine + (v >> bits), 1);
    });
    int all_below, own;
    block_scan(below, warp_sums, &all_below);  // (its barriers are behind the counts, too)
    // Each id's places: those of the ids before it, then of the warps before one.
    const int ids_per = (n + 1023) / 1024, b0 = min(tid * ids_per, n), b1 = min(b0 + ids_per, n);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
        int c = 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) c += counts[w * slice + b];
        if (ws.present) ws.present[(static_cast<size_t>(b) << bits) + r] = c != 0;
        sum += c;
    }
    int at = all_below + block_scan(sum, warp_sums, &own);
    if (blockIdx.x == gridDim.x - 1 && tid == 0) *ws.found = all_below + own;
    if (own == 0) return;
    // (a piece's word is that of the block that holds its last token: a run that goes on behind the piece holds it)
    for (int q = all_below / piece + tid; q < (all_below + own) / piece; q += 1024) ws.more[q] = 0;
    __syncthreads();
    if (sum > 0)
        for (int b = b0; b < b1; ++b) {
            const int start = at;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = counts[w * slice + b];
                counts[w * slice + b] = at;
                at += c;
            }
            const int first = start / piece;
            if (at - (start + piece - 1) / piece * piece >= piece && (at - 1) / piece > first)
                ws.more[first] = (at - 1) / piece - first;
        }
    __syncthreads();
    each_own([&](unsigned t, uint32_t v, bool in) {
        unsigned hits = __ballot_sync(0xffffffffu, in);
        if (hits == 0) return;
        const uint32_t q = v >> bits;
        unsigned same = 0;  // lanes with this lane's id: one distinct id after another
        while (hits) {
            const uint32_t one = __shfl_sync(0xffffffffu, v, __ffs(hits) - 1);
            const unsigned m = __ballot_sync(0xffffffffu, in && v == one);
            if (in && v == one) same = m;
            hits &= ~m;
        }
        if (in) {
            const int place = mine[q] + __popc(same & before);
            ws.order[place] = static_cast<int32_t>(t);
            ws.id[place] = static_cast<int32_t>(v);
        }
        __syncwarp();
        if (in && lane == __ffs(same) - 1) mine[q] += __popc(same);
        __syncwarp();
    });
}

// One addition to an element and call: no order matters.
template <int G>
__device__ __forceinline__ void add_to(float* p, const Vec8& v, const Columns<G>& c) {
    constexpr int W = G < 4 ? G : 4;  // elements of one instruction
#pragma unroll
    for (int j = 0; j < 8 / W; ++j)
        if (j * W / G < c.count) {
            float* q = p + (j * W / G) * c.step + (j * W) % G;
            const float* x = v.v + j * W;
            if constexpr (W == 4)
                asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(q), "f"(x[0]), "f"(x[1]),
                             "f"(x[2]), "f"(x[3])
                             : "memory");
            else if constexpr (W == 2)
                asm volatile("red.relaxed.gpu.global.add.v2.f32 [%0], {%1, %2};" ::"l"(q), "f"(x[0]), "f"(x[1]) : "memory");
            else
                asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(q), "f"(x[0]) : "memory");
        }
}
template <int G, typename O>
__device__ __forceinline__ void finish(O* p, const Vec8& v, float scale, const Columns<G>& c, bool add) {
    Vec8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o.v[j] = v.v[j] * scale;
    if constexpr (sizeof(O) == 4) {
        if (add) return add_to<G>(p, o, c);
    }
    write<G>(p, o, c);
}

struct SumArgs {
    int T, V, d, piece, pieces, chunks;  // tokens of a piece, pieces of the T tokens, stretches of columns
    int sum_blocks;                   // blocks that sum; the others zero
    float scale;
    bool add;
};

// AHEAD: the lines of what is added to are fetched ahead.
template <typename X, typename O, int G, bool AHEAD>
__global__ void __launch_bounds__(kThreads)
embed_sum_kernel(const X* __restrict__ dy, SumArgs a, Workspace ws, O* __restrict__ out) {
    __shared__ int32_t s_id[32 * (2 * kMostPiece + 1)], s_order[32 * 2 * kMostPiece];
    const int d = a.d, P = a.piece, tx = blockDim.x, x = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x >= static_cast<unsigned>(a.sum_blocks)) {
        // Rows without a token: the table's 16-byte words one after another, element by element where a word lies in
        // more than one row (or the table is not aligned for it).
        constexpr int E = 16 / sizeof(O);
        const int threads = tx * blockDim.y, tid = threadIdx.y * tx + x;
        const unsigned long long w0 = static_cast<unsigned long long>(blockIdx.x - a.sum_blocks) * (kZeroWords * threads) + tid;
        const unsigned long long e0 = w0 * E;
        long long row = static_cast<long long>(e0 / d);
        int col = static_cast<int>(e0 - static_cast<unsigned long long>(row) * d);
        const int step_rows = threads * E / d, step_cols = threads * E % d;
        const bool words = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        constexpr int kBatch = 8;  // words whose rows are looked up together
#pragma unroll 1
        for (int k = 0; k < kZeroWords; k += kBatch) {
            long long rows[kBatch];
            int cols[kBatch];
            bool zero[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                rows[u] = row;
                cols[u] = col;
                zero[u] = words && row < a.V && col + E <= d && !__ldg(ws.present + row);
                row += step_rows;
                col += step_cols;
                if (col >= d) col -= d, ++row;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                O* q = out + static_cast<size_t>(rows[u]) * d + cols[u];
                if (zero[u]) {
                    *reinterpret_cast<uint4*>(q) = make_uint4(0, 0, 0, 0);
                } else if (rows[u] < a.V && !(words && cols[u] + E <= d)) {
                    for (int i = 0; i < E && rows[u] < a.V; ++i) {
                        if (!__ldg(ws.present + rows[u])) put(q + i, 0.0f);
                        if (++cols[u] == d) cols[u] = 0, ++rows[u];
                    }
                }
            }
        }
        return;
    }
    const int chunk = blockIdx.x % a.chunks;
    const long long piece = static_cast<long long>(blockIdx.x / a.chunks) * blockDim.y + threadIdx.y, p0 = piece * P;
    const int found = __ldg(ws.found);
    int32_t *id = s_id + threadIdx.y * (2 * P + 1), *order = s_order + threadIdx.y * 2 * P;
    // Ids from the token before the piece to the end of the next piece (-1 before all and behind all).  All loads at
    // once: what lies behind the tokens found is read, and not used.
    for (int k = x; k <= 2 * P; k += tx) {
        const long long at = p0 - 1 + k;
        const int v = at >= 0 && at < a.T ? __ldg(ws.id + at) : -1, t = k < 2 * P && at + 1 < a.T ? __ldg(ws.order + at + 1) : 0;
        id[k] = at < found ? v : -1;
        if (k < 2 * P) order[k] = at + 1 < found ? t : 0;
    }
    const int first_back = p0 >= P && p0 < a.T ? __ldg(ws.id + p0 - P) : -1;  // the first of the piece before
    const int two_back = p0 < found ? first_back : -1;
    __syncthreads();
    const Columns<G> c(chunk, tx, x, d);
    if (p0 >= found || c.count == 0) return;
    const int len = static_cast<int>(min(static_cast<long long>(P), found - p0));
    ++id;  // id[-1]: before the piece
    auto end_of_run = [&](int v, int from, int to) {  // (tokens of an id are neighbours)
        while (from < to) {
            const int m = (from + to) / 2;
            if (id[m] == v) from = m + 1;
            else to = m;
        }
        return from;
    };
    // The run that comes from before: its share here if it is long, else the piece before has it all.
    const int head = id[0], tail = id[len - 1];
    const bool from_before = id[-1] == head;
    const bool head_long = from_before && (two_back == head || (len == P && tail == head));
    const int begin = from_before && !head_long ? end_of_run(head, 0, len) : 0;
    // The run that goes on behind the piece: all of it, unless it is long.
    int end = len;
    bool tail_long = false;
    if (len == P && id[P] == tail) {
        if (head == tail || id[2 * P - 1] == tail) tail_long = true;
        else end = end_of_run(tail, P, 2 * P);
    }
    float* part = ws.part + static_cast<size_t>(piece) * 2 * d + c.at;
    Vec8 sum{};
    constexpr int kAhead = sizeof(X) == 4 || G <= 2 ? 4 : 8;
    for (int i0 = begin; i0 < end; i0 += kAhead) {
        Units<X, G> r[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)  // (behind the end the last row again)
            fetch<G>(r[u], dy + static_cast<size_t>(order[min(i0 + u, end - 1)]) * d + c.at, c);
        // What is added to on its way into the L2 (a lane for 128 bytes).
        if (AHEAD && x % (32 / G) == 0)
            for (int i = i0; i < min(i0 + kAhead, end); ++i)
                if (i + 1 == end || id[i + 1] != id[i])
                    for (int j = 0; j < c.count; ++j)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(out + static_cast<size_t>(id[i]) * d + c.at + j * c.step));
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u;
            if (i >= end) break;
            const Vec8 row = r[u].values();
#pragma unroll
            for (int j = 0; j < 4; ++j) sum.set(j, add2(sum.pair(j), row.pair(j)));
            const int v = id[i];
            if (i + 1 < end && id[i + 1] == v) continue;
            if (head_long && v == head) write<G>(part, sum, c);
            else if (tail_long && v == tail) write<G>(part + d, sum, c);
            else finish<G>(out + static_cast<size_t>(v) * d + c.at, sum, a.scale, c, a.add);
            sum = Vec8{};
        }
    }
}

// Long runs: a block takes those that begin in its kWindow pieces, kShares groups of 32 threads a share of a run's pieces
// each.
constexpr int kWindow = 8, kShares = 16;
template <typename O, int G>
__global__ void __launch_bounds__(32 * kShares) embed_join_kernel(SumArgs a, Workspace ws, O* __restrict__ out) {
    __shared__ float share[kShares][32][9];
    const int P = a.piece, d = a.d, g = threadIdx.y, lane = threadIdx.x;
    const Columns<G> c(blockIdx.y, 32, lane, d);
    pdl_wait();
    pdl_trigger();
    const long long found = __ldg(ws.found);
    const long long piece = static_cast<long long>(blockIdx.x) * kWindow + lane;
    // (all loads at once: what lies behind the tokens found is read, and not used)
    const bool whole = lane < kWindow && (piece + 1) * P < a.T;
    const int pieces_more = whole ? __ldg(ws.more + piece) : 0, id = whole ? __ldg(ws.id + (piece + 1) * P) : 0;
    const int goes_on = (piece + 1) * P < found ? pieces_more : 0;
    unsigned todo = __ballot_sync(0xffffffffu, goes_on > 0);
    while (todo) {  // (the same in all warps)
        const int k = __ffs(todo) - 1, more = __shfl_sync(0xffffffffu, goes_on, k);
        todo &= todo - 1;
        const long long first = static_cast<long long>(blockIdx.x) * kWindow + k;
        const int value = __shfl_sync(0xffffffffu, id, k);
        Vec8 sum{};
        const float* p = ws.part + static_cast<size_t>(first) * 2 * d + c.at;
        const int per = more / kShares + 1, k0 = g * per, k1 = c.count > 0 ? min(k0 + per, more + 1) : k0;
#pragma unroll 8
        for (int q = k0; q < k1; ++q) {
            Units<float, G> r;
            fetch<G>(r, q == 0 ? p + d : p + static_cast<size_t>(q) * 2 * d, c);
            const Vec8 row = r.values();
#pragma unroll
            for (int j = 0; j < 8; ++j) sum.v[j] += row.v[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) share[g][lane][j] = sum.v[j];
        __syncthreads();
        if (g == 0) {
            for (int q = 1; q < kShares; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum.v[j] += share[q][lane][j];
            finish<G>(out + static_cast<size_t>(value) * d + c.at, sum, a.scale, c, a.add);
        }
        __syncthreads();
    }
}

// The largest unit that width and addresses allow: loads of up to 16 bytes.
int unit_of(int d, const void* a, size_t a_size, const void* b, size_t b_size) {
    for (int g = 8; g > 1; g /= 2)
        if (d % g == 0 && reinterpret_cast<uintptr_t>(a) % std::min<size_t>(16, g * a_size) == 0 &&
            reinterpret_cast<uintptr_t>(b) % std::min<size_t>(16, g * b_size) == 0)
            return g;
    return 1;
}
// Threads of a row, eight columns each: a power of two up to 32, then the multiple of 32 that leaves fewest idle.
int across(int eights) {
    if (eights <= 8) return 8;
    if (eights <= 16) return 16;
    const int stretches = (eights + kThreads - 1) / kThreads;
    return (eights + 32 * stretches - 1) / (32 * stretches) * 32;
}
constexpr size_t kAlign = 256;
size_t up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// Tokens of a piece: 32, fewer where that leaves less than three blocks of the sums to an SM (12001 tokens of 1028
// columns: 30 us with 16, 33 with 32 or 8).
int piece_of(int T, int d) {
    const int d8 = (d + 7) / 8, tx = across(d8), ty = kThreads / tx, stretches = (d8 - 1) / tx + 1;
    int piece = kMostPiece;
    while (piece > 8 && static_cast<long long>(T) / (piece * ty) * stretches < 3 * kSms) piece /= 2;
    return piece;
}

template <typename I, typename X, typename O, int G>
cudaError_t forward_as(const EmbedArgs& a, cudaStream_t s) {
    const int d8 = (a.d + 7) / 8, tx = across((d8 + 1) / 2), ty = kThreads / tx;
    const dim3 grid((a.T - 1) / ty + 1, (d8 - 1) / (2 * tx) + 1);
    return launch_k(kPdlTrain, embed_kernel<I, X, O, G>, grid, dim3(tx, ty), 0, s, static_cast<const I*>(a.ids),
                    static_cast<const X*>(a.rows), a.T, a.V, a.d, a.scale, static_cast<O*>(a.out), a.status);
}
template <typename I, typename X, typename O>
cudaError_t forward_io(const EmbedArgs& a, cudaStream_t s) {
    switch (unit_of(a.d, a.rows, sizeof(X), a.out, sizeof(O))) {
        case 8: return forward_as<I, X, O, 8>(a, s);
        case 4: return forward_as<I, X, O, 4>(a, s);
        case 2: return forward_as<I, X, O, 2>(a, s);
        default: return forward_as<I, X, O, 1>(a, s);
    }
}
template <typename I>
cudaError_t forward_i(const EmbedArgs& a, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (a.rows_fp32) return a.out_fp32 ? forward_io<I, float, float>(a, s) : forward_io<I, float, B>(a, s);
    return a.out_fp32 ? forward_io<I, B, float>(a, s) : forward_io<I, B, B>(a, s);
}

template <typename I>
cudaError_t sort(const EmbedArgs& a, const Workspace& ws, cudaStream_t s) {
    const int bits = slice_bits(a.V), slice = ((a.V - 1) >> bits) + 1;
    const int counts = kSortWarps * slice, per = (a.T - 1) / (kSortWarps * 32) * 32 + 32;
    const int list = std::min(per, (kSortSmem - 4 * counts) / (8 * kSortWarps));
    const int smem = 4 * counts + 8 * kSortWarps * list;
    const cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel<I>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
    if (e != cudaSuccess) return e;
    return launch_k(kPdlTrain, embed_sort_kernel<I>, dim3(1 << bits), dim3(1024), smem, s,
                    static_cast<const I*>(a.ids), a.T, a.V, slice, list, bits, piece_of(a.T, a.d), ws, a.status);
}
template <typename X, typename O, int G>
cudaError_t sum_as(const EmbedArgs& a, const Workspace& ws, cudaStream_t s) {
    const int d8 = (a.d + 7) / 8, tx = across(d8), ty = kThreads / tx;
    SumArgs g;
    g.T = a.T, g.V = a.V, g.d = a.d;
    g.piece = piece_of(a.T, a.d);
    g.pieces = (a.T - 1) / g.piece + 1;
    g.chunks = (d8 - 1) / tx + 1;
    g.sum_blocks = ((g.pieces - 1) / ty + 1) * g.chunks;
    g.scale = a.scale;
    g.add = a.accumulate;
    // An addition in the L2 waits for its line.  Fetched ahead where the rows are more than the 129 MB L2 holds: 16384
    // tokens of 128256 x 4096 140 -> 126 us; where they may be in it the requests cost (12001 of 50001 x 1028 24 -> 27 us).
    const bool ahead = a.accumulate && 4ll * std::min(a.T, a.V) * a.d > (129ll << 20);
    const long long words = (static_cast<long long>(a.V) * a.d * static_cast<long long>(sizeof(O)) + 15) / 16;
    const long long zero_blocks = a.accumulate ? 0 : (words - 1) / (kZeroWords * tx * ty) + 1;
    auto kernel = embed_sum_kernel<X, O, G, false>;
    if constexpr (sizeof(O) == 4) {
        if (ahead) kernel = embed_sum_kernel<X, O, G, true>;
    }
    cudaError_t e = launch_k(kPdlTrain, kernel, dim3(static_cast<unsigned>(g.sum_blocks + zero_blocks)), dim3(tx, ty), 0, s,
                             static_cast<const X*>(a.rows), g, ws, static_cast<O*>(a.out));
    if (e != cudaSuccess || g.pieces == 1) return e;
    return launch_k(kPdlTrain, embed_join_kernel<O, G>, dim3((g.pieces - 1) / kWindow + 1, (d8 + 31) / 32), dim3(32, kShares), 0, s,
                    g, ws, static_cast<O*>(a.out));
}
template <typename X, typename O>
cudaError_t sum_xo(const EmbedArgs& a, const Workspace& ws, cudaStream_t s) {
    const cudaError_t e = a.ids64 ? sort<long long>(a, ws, s) : sort<int32_t>(a, ws, s);
    if (e != cudaSuccess) return e;
    const int unit = unit_of(a.d, a.rows, sizeof(X), a.out, sizeof(O));
    if constexpr (sizeof(X) == 2) {
        if (unit == 8) return sum_as<X, O, 8>(a, ws, s);
    }
    switch (std::min(unit, 4)) {  // (fp32 rows: 15261 x 4864 65 us, 79 as eights)
        case 4: return sum_as<X, O, 4>(a, ws, s);
        case 2: return sum_as<X, O, 2>(a, ws, s);
        default: return sum_as<X, O, 1>(a, ws, s);
    }
}

}  // namespace

size_t embed_backward_workspace(int T, int V, int d) {
    const size_t piece = piece_of(T, d), pieces = (static_cast<size_t>(T) + piece - 1) / piece;
    return kAlign + 2 * up(sizeof(int32_t) * static_cast<size_t>(T)) + up(static_cast<size_t>(V)) +
           up(sizeof(int32_t) * pieces) + up(sizeof(float) * 2 * d * pieces);
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
    ws.present = reinterpret_cast<uint8_t*>(p += up(sizeof(int32_t) * static_cast<size_t>(a.T)));
    ws.more = reinterpret_cast<int32_t*>(p += up(static_cast<size_t>(a.V)));
    if (a.accumulate) ws.present = nullptr;  // no row is zeroed
    const int piece = piece_of(a.T, a.d);
    ws.part = reinterpret_cast<float*>(p + up(sizeof(int32_t) * ((static_cast<size_t>(a.T) + piece - 1) / piece)));
    using B = __nv_bfloat16;
    if (a.rows_fp32) return a.out_fp32 ? sum_xo<float, float>(a, ws, s) : sum_xo<float, B>(a, ws, s);
    return a.out_fp32 ? sum_xo<B, float>(a, ws, s) : sum_xo<B, B>(a, ws, s);
}

}  // namespace moe
