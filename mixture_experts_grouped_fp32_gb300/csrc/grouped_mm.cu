// grouped_mm.cu — the grouped products of the training path on SM pairs (tcgen05 cta_group::2):
//
//   kMmForward  C[r] = A[r] . B[e]      for the rows r of segment e   (B [E, K, N])
//   kMmTransB   C[r] = A[r] . B[e]^T                                  (B [E, N, K]: input gradient)
//   kMmWgrad    D[e] (+)= sum_{r in segment e} A[r]^T . G[r]          (weight gradient, D [E, K, N])
//
// bf16 operands, fp32 accumulation in tensor memory, one rounding at the store (or none: fp32 out).
//
// One orientation for all three: the output's contiguous index n is the UMMA M dimension (256 per CTA
// pair, 128 per CTA: "features") and the output's row index is the UMMA N dimension ("rows").
//   * A ragged segment then costs N = its rows rounded up to 32, not a 256-row tile: a segment of c
//     rows is cut into ceil(c / 256) tiles of equal size.
//   * In tensor memory a lane is a feature and a column is an output row, so for each output row the
//     32 lanes of a warp hold 32 consecutive outputs: the epilogue's plain stores are coalesced
//     (64 bytes of bf16 or 128 of fp32 per warp) without a pass through shared memory, and rows past
//     a segment's end are simply not stored.
// For the weight gradient the features are G's columns, the rows are A's columns and the reduction
// runs over the segment's rows.
//
// Shared-memory stage of each CTA (64 deep along the reduction, 128-byte swizzle as TMA writes it):
//   F (16 KB)  128 features.  kMmTransB: K-major, one box of 128 rows x 64 K.  Otherwise MN-major: two
//              boxes of 64 features x 64 deep, 8 KB apart.
//   R (16 KB)  this CTA's half of the tile's rows, at most 128.  Weight gradient: MN-major, two boxes
//              as for F.  Otherwise K-major: one box of 32, 64 or 128 rows.
// Each operand is one copy per stage (a view of the matrix as blocks of 64 columns makes two boxes one
// copy; a column count that is no multiple of 64 takes two): the copies' issue counts, four 32-row
// boxes instead of one of 128 rows cost 15 % of an 8192 x 4096 x 28672 product.
// Six stages; two 256-column accumulators, so that one tile's epilogue overlaps the next tile's
// products.
//
// The weight gradient's last block along a segment's rows holds rows of the next segment.  They are
// zeroed in shared memory in both operands (zeroing one would let an infinity in the other through as
// NaN): that block's copies complete on a barrier of the CTA's own, a warp zeroes the rows past the
// end up to the next multiple of 16 (one UMMA step; later steps are not issued) and then arrives on
// the stage's `full` barrier.  Every other block goes from the copy to the tensor cores directly.
//
// Work items (expert, group of up to 8 row tiles, feature tile, row tile, slice of the reduction) are
// numbered in this order and dealt round-robin to a persistent grid of CTA pairs: the row tiles of a
// group run together and share the feature operand through L2, and groups of 8 keep the rows
// re-read per feature tile few when a segment is long.
//
// Measured: 8192 rows, 4096 -> 28672 over 8 experts 1.19 to 1.29 ms (1.5 to 1.6 PFLOP/s; tensor pipe 82 %
// active at the power limit); two rows of 14336 -> 4096 45 us (5.2 TB/s); gradients of 256 experts,
// 2048 x 7168 from 16384 rows, 1.41 to 1.48 ms (5.5 TB/s of mostly writes); 32 experts' gradients of that size from as
// many rows 0.43 ms in bf16, 0.59 in fp32 (3.7 TB/s), 0.68 added to what was there (6.0 TB/s).
//
// Synchronisation across the pair is that of the layer's SM-pair kernel: full[s] lives in CTA 0 and
// counts both CTAs' copies, empty[s] and tfull[a] are arrived on in both CTAs by CTA 0's multicast
// commits, tempty[a] lives in CTA 0.  Every wait is bounded and reports MOE_STATUS_WAIT_TIMEOUT.
#include <atomic>

#include "common.cuh"
#include "train_ptx.cuh"

namespace moe {
namespace {

constexpr int BK = 64;
constexpr int UMMA_K = 16;
constexpr int TILE_F = 256;                      // features per pair
constexpr int TILE_R = 256;                      // output rows per tile, at most
constexpr int BOX_BYTES = 64 * BK * 2;           // 8 KB
constexpr int F_BYTES = 128 * BK * 2;            // 16 KB
constexpr int R_BYTES = 128 * BK * 2;            // 16 KB
constexpr int STAGE_BYTES = F_BYTES + R_BYTES;   // 32 KB per CTA
constexpr int STAGES = 6;
constexpr int ACC_COLS = 256;
constexpr int NUM_ACC = 2;
constexpr int TMEM_COLS = NUM_ACC * ACC_COLS;
constexpr int GROUP_R = 8;  // row tiles that run together
constexpr int MAX_E = 256;
constexpr int MAX_SPLIT = 16;
constexpr int kMaxCtas = kGroupedMmDone;  // of a launch; and threads of the join, one for each of them at least
constexpr uint16_t BOTH_CTAS = 0x3;
// Warps: 0 copies, 1 tensor memory and MMAs, then the epilogue's groups of eight, then (weight gradient)
// one that zeroes segment ends and one that stores the gradients of empty segments.
constexpr int kEpiWarps = 8;
// CHUNKED: long reductions, whose partial sums move from tensor memory to registers after every chunk_blocks
// blocks of 64, because an addition in tensor memory truncates: one epilogue group keeps the tile's sums across
// both accumulators.  Otherwise one group for each accumulator, so that short items (a few blocks of reduction)
// do not wait for one group to read, convert and store tile after tile; the whole reduction then runs in
// tensor memory.
//   fp32 outputs: chunks of 8 blocks, for reductions of more than one chunk.
//   bf16 outputs: unbroken up to UNBROKEN blocks (262144 rows; K ends at 65536), whose 4 truncations a block, of
//   2^-23 each, come to 2^-9 at the very most, half of a rounding to bf16.  Measured: of 8192 x 28672 outputs summed
//   over 4096 random products 0.23 % are the neighbour of what an fp32 sum is rounded to, and all are as far
//   from the sum in 64 bits.  Beyond, chunks of 64 blocks.
template <typename OUT>
constexpr int chunk_blocks() { return sizeof(OUT) == 4 ? 8 : 64; }
constexpr int UNBROKEN = 4096;
template <bool CHUNKED>
constexpr int epi_groups() { return CHUNKED ? 1 : 2; }
template <bool CHUNKED>
constexpr int fix_warp() { return 2 + kEpiWarps * epi_groups<CHUNKED>(); }
template <int MODE, bool CHUNKED>
constexpr int num_threads() { return 32 * (fix_warp<CHUNKED>() + (MODE == kMmWgrad ? 2 : 0)); }
constexpr int SMEM_BYTES = 232448;

struct Ctl {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tail[STAGES];  // weight gradient: copies of a segment's last block, per CTA
    uint64_t tfull[NUM_ACC];
    uint64_t tempty[NUM_ACC];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int bad_offsets;
    int total_items;
    int seg[MAX_E + 1];
    int item_start[MAX_E + 1];
};
static_assert(STAGES * STAGE_BYTES + 1024 + sizeof(Ctl) <= SMEM_BYTES, "shared memory budget");

// Tiles along the output rows of expert e, and rows per tile (a multiple of 32).
template <int MODE>
__device__ __forceinline__ int row_tiles(int cnt, int K) {
    return ((MODE == kMmWgrad ? K : cnt) + TILE_R - 1) / TILE_R;
}

struct Item {
    int e, f0;          // expert, first feature of the pair's tile
    int r0, rows;       // first output row (of the segment, or of the expert's [K, N]) and how many (> 0)
    int ntok;           // UMMA N: rows rounded up to 32
    int red0, red1;     // reduction range in blocks of 64
    int red_rows;       // weight gradient: rows of the segment
    int slice;
};

// A role's position in the items of its CTA pair, which it visits in ascending order: the expert is the last
// one, the next one or found by bisection of those after (walking over empty experts: 8 tokens in 256 experts
// 19.8 against 14.7 us), and what depends on the expert alone is kept.
template <int MODE>
struct Cursor {
    const Ctl& c;
    int K, E, f_tiles, ksplit;
    int e = -1, start = 0, next = 0;  // expert, its first item, the next expert's
    int cnt = 0, total = 0, rt = 1, per = 32, nkb = 0;

    __device__ __forceinline__ Cursor(const Ctl& ctl, int k, int experts, int ft, int ks)
        : c(ctl), K(k), E(experts), f_tiles(ft), ksplit(ks) {}

    __device__ __forceinline__ Item at(int i) {
        if (i >= next) {
            next = c.item_start[++e + 1];
            if (i >= next) {  // further on (i < item_start[E])
                int lo = e + 1, hi = E - 1;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (c.item_start[mid + 1] > i) hi = mid;
                    else lo = mid + 1;
                }
                e = lo;
                next = c.item_start[e + 1];
            }
            start = c.item_start[e];
            cnt = c.seg[e + 1] - c.seg[e];
            total = MODE == kMmWgrad ? K : cnt;
            rt = row_tiles<MODE>(cnt, K);
            // Equal tiles; the last one may be shorter.  (total + rt passes 2^31.)
            per = ((static_cast<int>((static_cast<unsigned>(total) + rt - 1u) / rt)) + 31) & ~31;
            nkb = ((MODE == kMmWgrad ? cnt : K) + BK - 1) / BK;
        }
        Item it;
        it.e = e;
        unsigned j = static_cast<unsigned>(i - start);
        it.slice = 0;
        if (ksplit > 1) {
            it.slice = static_cast<int>(j % static_cast<unsigned>(ksplit));
            j /= static_cast<unsigned>(ksplit);
        }
        unsigned g = 0, gr = static_cast<unsigned>(rt);
        if (rt > GROUP_R) {
            const unsigned per_group = static_cast<unsigned>(GROUP_R * f_tiles);
            g = j / per_group;
            j -= g * per_group;
            gr = min(static_cast<unsigned>(GROUP_R), gr - g * GROUP_R);
        }
        const unsigned ft = j / gr;
        it.f0 = static_cast<int>(ft) * TILE_F;
        it.r0 = static_cast<int>(g * GROUP_R + (j - ft * gr)) * per;
        it.rows = min(per, total - it.r0);
        it.ntok = (it.rows + 31) & ~31;
        it.red_rows = cnt;
        it.red0 = 0;
        it.red1 = nkb;
        if (ksplit > 1) {
            it.red0 = static_cast<int>(static_cast<long long>(nkb) * it.slice / ksplit);
            it.red1 = static_cast<int>(static_cast<long long>(nkb) * (it.slice + 1) / ksplit);
        }
        return it;
    }
};

__device__ __forceinline__ void raise_abort(Ctl& c, int32_t* status) {
    *reinterpret_cast<volatile int*>(&c.abort_flag) = 1;
    flag_status(status, MOE_STATUS_WAIT_TIMEOUT);
}

// Tensor maps.  f: the feature operand (weights [E, K, N] / [E, N, K], or G [M, N] as one matrix); r: the
// row operand A [M, K], for the products by rows with boxes of 128, 64 and 32 rows.  f_blocks / r_blocks:
// the map's box is both 64-column boxes of the operand.
struct Maps {
    CUtensorMap f, r, r64, r32;
    int f_blocks, r_blocks;
};

template <int MODE, typename OUT, bool CHUNKED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(num_threads<MODE, CHUNKED>(), 1)
grouped_mm_kernel(const __grid_constant__ Maps maps, const int32_t* __restrict__ offsets, int M, int K, int N, int E,
                  int ksplit, int accumulate, int inject_stall, OUT* __restrict__ out, int32_t* __restrict__ done,
                  int32_t* __restrict__ status) {
    constexpr bool WGRAD = MODE == kMmWgrad;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    uint8_t* tiles = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    Ctl& c = *reinterpret_cast<Ctl*>(tiles + STAGES * STAGE_BYTES);
    const volatile int* abort_flag = &c.abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    const bool leader = rank == 0;
    const int pair_id = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
    const int f_tiles = (N + TILE_F - 1) / TILE_F;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            // Weight gradient: two arrivals, of the leader's producer or of each CTA's zeroing warp.
            ptx::mbar_init(&c.full[s], WGRAD ? 2 : 1);
            ptx::mbar_init(&c.empty[s], 1);
            ptx::mbar_init(&c.tail[s], 1);
        }
        for (int a = 0; a < NUM_ACC; ++a) {
            ptx::mbar_init(&c.tfull[a], 1);
            ptx::mbar_init(&c.tempty[a], 2 * kEpiWarps);
        }
        ptx::mbar_init(&c.drain, 1);
        c.abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&maps.f);
        ptx::prefetch_tensormap(&maps.r);
        if (!WGRAD) {
            ptx::prefetch_tensormap(&maps.r64);
            ptx::prefetch_tensormap(&maps.r32);
        }
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(&c.tmem_base, TMEM_COLS);
        ptx::tmem_relinquish_pair();
    }
    __syncwarp();
    ptx::cluster_arrive();  // this CTA's barriers exist; the wait is after the offsets, whose latency covers it
    pdl_wait();
    pdl_trigger();
    if (warp == 2) {
        // Check the offsets and number the work items (8 experts per lane).
        for (int e = lane; e <= E; e += 32) c.seg[e] = __ldg(offsets + e);
        __syncwarp();
        bool ok = true;
        for (int e = lane; e < E; e += 32) ok = ok && c.seg[e] <= c.seg[e + 1];
        if (lane == 0) ok = ok && c.seg[0] >= 0 && c.seg[E] <= M;
        ok = __all_sync(0xffffffffu, ok);
        const int per = (E + 31) / 32;
        const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
        auto items = [&](int e) {
            const int cnt = c.seg[e + 1] - c.seg[e];
            // An empty segment's weight gradient is zero: written, or left as it is when added to.
            if (WGRAD && cnt == 0 && accumulate) return 0;
            return row_tiles<MODE>(cnt, K) * f_tiles * ksplit;
        };
        int sum = 0;
        if (ok)
            for (int e = e0; e < e1; ++e) sum += items(e);
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int run = incl - sum;
        for (int e = e0; e < e1; ++e) {
            c.item_start[e] = run;
            if (ok) run += items(e);
        }
        if (lane == 31) {
            c.item_start[E] = incl;
            c.total_items = incl;
            c.bad_offsets = !ok;
        }
        if (!ok && lane == 0 && leader) flag_status(status, MOE_STATUS_BAD_OFFSETS);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_wait();  // both CTAs' barriers exist before any cross-CTA arrive or copy
    ptx::tc_fence_after();

    const uint32_t tmem_base = c.tmem_base;
    const int total = c.total_items;
    uint32_t fill_parity[STAGES];
    int filled_mask = 0;
    Cursor<MODE> cur(c, K, E, f_tiles, ksplit);

    if (warp == 0 && lane == 0) {
        // ------------------------------ copies (both CTAs) ------------------------------
        const uint64_t pol_r = WGRAD ? ptx::policy_evict_normal() : ptx::policy_evict_last();
        const uint64_t pol_f = ptx::policy_evict_normal();
        int stage = 0;
        uint32_t phase = 0;
        uint32_t extra = inject_stall && blockIdx.x == 0 ? 16u : 0u;  // (test hook: the first stage waits in vain)
        bool aborted = false;
        for (int i = pair_id; i < total && !aborted; i += num_pairs) {
            const Item it = cur.at(i);
            const int half = it.ntok >> 1;
            const int f = it.f0 + 128 * rank;           // this CTA's features
            const int seg0 = c.seg[it.e];
            // The smallest row box that holds this CTA's rows (columns, for the weight gradient).
            const CUtensorMap* mr = WGRAD || half > 64 ? &maps.r : half > 32 ? &maps.r64 : &maps.r32;
            const uint32_t row_bytes = WGRAD || half > 64 ? R_BYTES : half > 32 ? R_BYTES / 2 : R_BYTES / 4;
            const uint32_t cta_bytes = F_BYTES + row_bytes;
            const int r = it.r0 + rank * half;  // this CTA's first output row
            for (int kb = it.red0; kb < it.red1; ++kb) {
                if (!ptx::mbar_wait(&c.empty[stage], phase ^ 1u, abort_flag)) {
                    raise_abort(c, status);
                    aborted = true;
                    break;
                }
                uint8_t* sf = tiles + stage * STAGE_BYTES;
                uint8_t* sr = sf + F_BYTES;
                const uint32_t full_leader = ptx::map_to_cta(ptx::smem_u32(&c.full[stage]), 0);
                if (WGRAD) {
                    const int row = seg0 + kb * BK;
                    if ((kb + 1) * BK > it.red_rows && (it.red_rows & 15)) {
                        // The segment's last block, with rows to be zeroed: its copies complete here.
                        ptx::mbar_arrive_expect_tx(&c.tail[stage], cta_bytes + extra);
                        if (maps.f_blocks) {
                            ptx::tma_load_4d(sf, &maps.f, &c.tail[stage], 0, row, f >> 6, 0, pol_f);
                        } else {
                            ptx::tma_load_2d(sf, &maps.f, &c.tail[stage], f, row, pol_f);
                            ptx::tma_load_2d(sf + BOX_BYTES, &maps.f, &c.tail[stage], f + 64, row, pol_f);
                        }
                        if (maps.r_blocks) {
                            ptx::tma_load_4d(sr, &maps.r, &c.tail[stage], 0, row, r >> 6, 0, pol_r);
                        } else {
                            ptx::tma_load_2d(sr, &maps.r, &c.tail[stage], r, row, pol_r);
                            ptx::tma_load_2d(sr + BOX_BYTES, &maps.r, &c.tail[stage], r + 64, row, pol_r);
                        }
                    } else {
                        if (leader) {  // both arrivals: a remote one for each block costs more (14 %)
                            ptx::mbar_arrive(&c.full[stage]);
                            ptx::mbar_arrive_expect_tx(&c.full[stage], 2u * cta_bytes + extra);
                        }
                        if (maps.f_blocks) {
                            ptx::tma_load_4d_pair(sf, &maps.f, full_leader, 0, row, f >> 6, 0, pol_f);
                        } else {
                            ptx::tma_load_2d_pair(sf, &maps.f, full_leader, f, row, pol_f);
                            ptx::tma_load_2d_pair(sf + BOX_BYTES, &maps.f, full_leader, f + 64, row, pol_f);
                        }
                        if (maps.r_blocks) {
                            ptx::tma_load_4d_pair(sr, &maps.r, full_leader, 0, row, r >> 6, 0, pol_r);
                        } else {
                            ptx::tma_load_2d_pair(sr, &maps.r, full_leader, r, row, pol_r);
                            ptx::tma_load_2d_pair(sr + BOX_BYTES, &maps.r, full_leader, r + 64, row, pol_r);
                        }
                    }
                } else {
                    if (leader) ptx::mbar_arrive_expect_tx(&c.full[stage], 2u * cta_bytes + extra);
                    ptx::tma_load_2d_pair(sr, mr, full_leader, kb * BK, seg0 + r, pol_r);
                    if (MODE == kMmTransB) {
                        ptx::tma_load_3d_pair(sf, &maps.f, full_leader, kb * BK, f, it.e, pol_f);
                    } else if (maps.f_blocks) {
                        ptx::tma_load_4d_pair(sf, &maps.f, full_leader, 0, kb * BK, f >> 6, it.e, pol_f);
                    } else {
                        ptx::tma_load_3d_pair(sf, &maps.f, full_leader, f, kb * BK, it.e, pol_f);
                        ptx::tma_load_3d_pair(sf + BOX_BYTES, &maps.f, full_leader, f + 64, kb * BK, it.e, pol_f);
                    }
                }
                extra = 0;
                fill_parity[stage] = phase;
                filled_mask |= 1 << stage;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1 && lane == 0 && leader) {
        // ------------------------------ pair MMAs (CTA 0) ------------------------------
        int stage = 0;
        uint32_t phase = 0, acc = 0, acc_phase = 0;
        bool aborted = false;
        for (int i = pair_id; i < total && !aborted; i += num_pairs) {
            const Item it = cur.at(i);
            if (it.red0 >= it.red1) continue;  // nothing to reduce: the epilogue stores zeros
            const uint32_t idesc = ptx::idesc_bf16_f32(TILE_F, static_cast<uint32_t>(it.ntok),
                                                       /*a_mn=*/MODE == kMmTransB ? 0 : 1, /*b_mn=*/WGRAD ? 1 : 0);
            const int depth = CHUNKED ? chunk_blocks<OUT>() : it.red1 - it.red0;
            for (int c0 = it.red0; c0 < it.red1 && !aborted; c0 += depth) {
                if (!ptx::mbar_wait(&c.tempty[acc], acc_phase ^ 1u, abort_flag)) {
                    raise_abort(c, status);
                    aborted = true;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * ACC_COLS;
                const int c1 = min(it.red1, c0 + depth);
                for (int kb = c0; kb < c1; ++kb) {
                    // (Weight gradient: the other CTA's zeroing warp arrives after its own writes.)
                    if (!(WGRAD ? ptx::mbar_wait_cluster(&c.full[stage], phase, abort_flag)
                                : ptx::mbar_wait(&c.full[stage], phase, abort_flag))) {
                        raise_abort(c, status);
                        aborted = true;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t sf = ptx::smem_u32(tiles + stage * STAGE_BYTES);
                    // MN-major: 64-wide boxes 8 KB apart, 16 deep = 2 KB.  K-major: 16 deep = 32 bytes.
                    const uint64_t f_desc = ptx::smem_desc_sw128(sf, MODE == kMmTransB ? 16 : BOX_BYTES, 1024);
                    const uint64_t r_desc = ptx::smem_desc_sw128(sf + F_BYTES, WGRAD ? BOX_BYTES : 16, 1024);
                    constexpr uint64_t f_step = (MODE == kMmTransB ? 32 : 2048) >> 4;
                    constexpr uint64_t r_step = (WGRAD ? 2048 : 32) >> 4;
                    const int steps =
                        WGRAD ? min(BK / UMMA_K, (it.red_rows - kb * BK + UMMA_K - 1) / UMMA_K) : BK / UMMA_K;
#pragma unroll
                    for (int kk = 0; kk < BK / UMMA_K; ++kk)
                        if (kk < steps)
                            ptx::mma_bf16_ss_pair(d_tmem, f_desc + kk * f_step, r_desc + kk * r_step, idesc,
                                                  (kb != c0 || kk != 0) ? 1u : 0u);
                    ptx::mma_commit_pair(&c.empty[stage], BOTH_CTAS);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (aborted) break;
                ptx::mma_commit_pair(&c.tfull[acc], BOTH_CTAS);
                if (++acc == NUM_ACC) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
        }
    } else if (WGRAD && warp == fix_warp<CHUNKED>()) {
        // ------------------- zero the rows past a segment's end (both CTAs) -------------------
        int stage = 0;
        uint32_t parity = 0;  // bit s: parity of tail[s]'s next phase
        long long before = 0;  // blocks that the copies go through before the next tail
        bool aborted = false;
        for (int i = pair_id; i < total && !aborted; i += num_pairs) {
            const Item it = cur.at(i);
            const int n = it.red1 - it.red0;
            before += n;
            if (n > 0 && it.red1 * BK > it.red_rows && (it.red_rows & 15)) {
                const int st = (stage + n - 1) % STAGES;
                // The one wait here that can be for a whole segment (or for those before it that have no tail): one
                // limit more for every 2^18 blocks, 3.8 us each (a block takes 0.2 to 0.8).
                bool ok = false;
                for (long long t = before >> 18; t >= 0 && !ok; --t) {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&c.tail[st], (parity >> st) & 1u, abort_flag));
                    if (__any_sync(0xffffffffu, *abort_flag)) break;
                }
                before = 0;
                if (!ok) {
                    if (lane == 0) raise_abort(c, status);
                    aborted = true;
                    break;
                }
                parity ^= 1u << st;
                const int z0 = it.red_rows - (it.red1 - 1) * BK;  // first row to zero, in [1, 63]
                const int z1 = (z0 + UMMA_K - 1) & ~(UMMA_K - 1);
                uint8_t* s0 = tiles + st * STAGE_BYTES;
                for (int b = 0; b < STAGE_BYTES / BOX_BYTES; ++b)
                    for (int o = z0 * 128 + lane * 16; o < z1 * 128; o += 512)
                        *reinterpret_cast<uint4*>(s0 + b * BOX_BYTES + o) = make_uint4(0, 0, 0, 0);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_cta(ptx::smem_u32(&c.full[st]), 0));
            }
            stage = (stage + n) % STAGES;
        }
    } else if (warp >= 2 && warp < fix_warp<CHUNKED>()) {
        // ------------------------------ epilogue (both CTAs) ------------------------------
        const int quarter = warp & 3;            // this warp's tensor-memory lanes: 32 quarter .. + 31
        const int col0 = 128 * (((warp - 2) >> 2) & 1);  // and its half of the tile's columns (output rows)
        const uint32_t group = (warp - 2) / kEpiWarps;   // bf16: the accumulator of this group
        uint32_t acc = 0, acc_phase = 0;
        const size_t slice_elems = WGRAD ? static_cast<size_t>(E) * K * N : static_cast<size_t>(M) * N;
        auto take = [&]() -> bool {  // the next accumulator is final
            if (!ptx::mbar_wait(&c.tfull[acc], acc_phase, abort_flag)) {
                raise_abort(c, status);
                return false;
            }
            ptx::tc_fence_after();
            return true;
        };
        auto give = [&]() {  // and may be overwritten
            ptx::tc_fence_before();
            __syncwarp();
            // Relaxed: what came before on this thread are reads of tensor memory, complete since wait::ld
            // (a releasing arrival would wait for the thread's stores to global memory too: 8 % of the
            // weight gradients' time).
            if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::map_to_cta(ptx::smem_u32(&c.tempty[acc]), 0));
        };
        auto pass = [&]() {  // on to the next accumulator
            if (++acc == NUM_ACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
        };
        // Stores 32 output rows of which a lane holds one column (column n, p its first row), up to `rows` of them.
        // bf16: neighbouring lanes exchange halves of their pairs of rows: an even lane then holds columns n and
        // n + 1 of the first row, an odd lane n - 1 and n of the second, one 4-byte store each.
        const uint32_t sel = lane & 1 ? 0x3276u : 0x5410u;
        auto put = [&](OUT* p, const uint32_t (&v)[32], int rows, bool mine) {
            if constexpr (sizeof(OUT) == 4) {
                if (!mine) return;
                if (rows >= 32) {
#pragma unroll
                    for (int j = 0; j < 32; ++j, p += N) *p = __uint_as_float(v[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j, p += N)
                        if (j < rows) *p = __uint_as_float(v[j]);
                }
            } else {
                p += static_cast<ptrdiff_t>(lane & 1) * (N - 1);
                const int nr = rows - (lane & 1);
#pragma unroll
                for (int j = 0; j < 16; ++j, p += 2 * static_cast<size_t>(N)) {
                    const uint32_t own = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
                    if (2 * j < nr && mine) *reinterpret_cast<uint32_t*>(p) = __byte_perm(own, other, sel);
                }
            }
        };
        // Adds to what is there, in the L2: each element is added to once in a launch, so that the result is
        // that of a load, an addition rounded to nearest and a store (where values under 2^-126 count as zero),
        // without waiting for the load (32 experts' 2048 x 7168 from 16384 rows: 1044 us with loads, 800 so, 691
        // with the lines fetched ahead; pairs of columns per addition took the same time).
        auto add = [&](OUT* p, const uint32_t (&v)[32], int rows, bool mine) {
            if constexpr (sizeof(OUT) == 4) {
#pragma unroll
                for (int j = 0; j < 32; ++j, p += N)
                    if (j < rows && mine) ptx::red_add_f32(p, __uint_as_float(v[j]));
            }
        };
        bool aborted = false;
        for (int i = pair_id; i < total && !aborted; i += num_pairs) {
            const Item it = cur.at(i);
            if (it.red0 >= it.red1) continue;  // nothing to add up
            const int n = it.f0 + 128 * rank + 32 * quarter + lane;
            const size_t row0 = WGRAD ? static_cast<size_t>(it.e) * K + it.r0 : static_cast<size_t>(c.seg[it.e]) + it.r0;
            OUT* dst = out + it.slice * slice_elems + (row0 + col0) * N + n;
            const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
            if (WGRAD && accumulate && i != pair_id) {
                // What will be added to, into the L2 while the products run (a pair's first item is short of
                // time itself: 10.5 against 11.1 us for 3 experts' 464 x 2688).
                const int n0 = n - lane;
                if (n0 < N)
                    for (int j = lane; j < 128 && col0 + j < it.rows; j += 32)
                        ptx::prefetch_l2(dst + static_cast<size_t>(j) * N - lane);
            }
            if constexpr (CHUNKED) {
                // The chunks' partial sums are added in registers, rounded to nearest.
                uint32_t sum[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[q][j] = 0u;
                for (int c0 = it.red0; c0 < it.red1; c0 += chunk_blocks<OUT>()) {
                    if (!take()) {
                        aborted = true;
                        break;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (col0 + 32 * q < it.rows) {
                            uint32_t v[32];
                            ptx::tmem_ld_32x32b_x32(lane_addr + acc * ACC_COLS + 32 * q, v);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                sum[q][j] = __float_as_uint(__uint_as_float(sum[q][j]) + __uint_as_float(v[j]));
                        }
                    }
                    give();
                    pass();
                }
                if (aborted) break;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int nr = it.rows - col0 - 32 * q;
                    if (nr > 0) {
                        OUT* p = dst + static_cast<size_t>(32 * q) * N;
                        if (WGRAD && accumulate) add(p, sum[q], nr, n < N);
                        else put(p, sum[q], nr, n < N);
                    }
                }
            } else {
                if (epi_groups<CHUNKED>() > 1 && acc != group) {  // the other group's
                    pass();
                    continue;
                }
                if (!take()) {
                    aborted = true;
                    break;
                }
#pragma unroll 1
                for (int j0 = 0; j0 < 128 && col0 + j0 < it.rows; j0 += 32) {
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(lane_addr + acc * ACC_COLS + j0, v);
                    ptx::tmem_ld_wait();
                    OUT* p = dst + static_cast<size_t>(j0) * N;
                    if (WGRAD && accumulate) add(p, v, it.rows - col0 - j0, n < N);
                    else put(p, v, it.rows - col0 - j0, n < N);
                }
                give();
                pass();
            }
        }
    } else if (WGRAD && warp == fix_warp<CHUNKED>() + 1) {
        // ------- zeros where there is nothing to add up (empty segments, slices past a short one) -------
        // A warp of its own: in the epilogue's loop this cost the other items registers (6 % of the gradients
        // of 256 experts).  An empty expert's tiles share its [K, N] as one run of memory, in equal parts: by
        // tiles, rows that do not start at whole 32-byte sectors took twice the time.
        const size_t slice_elems = static_cast<size_t>(E) * K * N;
        auto fill = [&](uint4* p, long long from, long long to, int stride) {
            long long w = from;
            for (; w + 7 * stride < to; w += 8 * stride)
#pragma unroll
                for (int k = 0; k < 8; ++k) p[w + k * stride] = make_uint4(0, 0, 0, 0);
            for (; w < to; w += stride) p[w] = make_uint4(0, 0, 0, 0);
        };
        for (int i = pair_id; i < total; i += num_pairs) {
            const Item it = cur.at(i);
            if (it.red0 < it.red1) continue;
            OUT* z = out + it.slice * slice_elems + static_cast<size_t>(it.e) * K * N;
            if (it.red_rows == 0) {
                const long long words = static_cast<long long>(K) * N * sizeof(OUT) / 16;
                const int tiles = (cur.next - cur.start) / ksplit, t = (i - cur.start) / ksplit;
                fill(reinterpret_cast<uint4*>(z), words * t / tiles + 32 * rank + lane, words * (t + 1) / tiles, 64);
            } else {
                constexpr int per_word = 16 / sizeof(OUT), lanes = 128 / per_word, step = 32 / lanes;
                const int col = it.f0 + 128 * rank + (lane % lanes) * per_word, r = lane / lanes;
                if (col < N)
                    for (int j = r; j < it.rows; j += step)
                        *reinterpret_cast<uint4*>(z + static_cast<size_t>(it.r0 + j) * N + col) = make_uint4(0, 0, 0, 0);
            }
        }
    }

    // ------------------------------ teardown ------------------------------
    ptx::tc_fence_before();
    __syncthreads();
    // A split reduction's slices are there (each CTA writes its word on every launch).
    if (done && tid == 0) done[blockIdx.x] = !c.bad_offsets && !c.abort_flag;
    if (warp == 0 && lane == 0 && c.abort_flag) {
        if (leader) {
            for (int s = 0; s < STAGES; ++s)
                if (filled_mask & (1 << s)) ptx::mbar_wait_ns(&c.full[s], fill_parity[s], 100000000ull);
        }
        const uint64_t t0 = ptx::globaltimer_ns();  // give this CTA's own copies time to land
        while (ptx::globaltimer_ns() - t0 < 1000000ull) {
        }
    }
    if (warp == 1 && lane == 0 && leader) {
        ptx::mma_commit_pair(&c.drain, 0x1);  // all pair MMAs issued by this thread have completed
        ptx::mbar_wait_ns(&c.drain, 0, 100000000ull);
    }
    __syncthreads();
    ptx::cluster_sync();  // neither CTA frees tensor memory or exits while the pair MMAs may run
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
    ptx::cluster_sync();
}

// Joins the slices of a split reduction: out = sum over s of partial[s], in slice order.  Rows outside
// [offsets[0], offsets[E]) are not touched (modes with row output).  Unless each of the product's `ctas` CTAs
// has left its word in `done` (a bad segmentation or an expired wait in one: its slices are not there), nothing is
// written; the first slices are loaded while the words are on their way.
template <typename OUT>
__global__ void __launch_bounds__(kMaxCtas)
grouped_mm_join_kernel(const float4* __restrict__ partial, const int32_t* __restrict__ done, int ctas,
                       const int32_t* __restrict__ offsets, int M, int N, int E, size_t n4, int ksplit, int by_row,
                       int accumulate, OUT* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int good = static_cast<int>(threadIdx.x) < ctas ? __ldcg(done + threadIdx.x) : 1;
    size_t lo = 0, hi = n4;
    if (by_row) {
        const int r0 = __ldg(offsets), r1 = __ldg(offsets + E);
        const bool inside = r0 >= 0 && r1 <= M && r0 <= r1;
        lo = inside ? static_cast<size_t>(r0) * N / 4 : 0;
        hi = inside ? static_cast<size_t>(r1) * N / 4 : 0;
    }
    auto sum = [&](size_t i) {
        float4 a = __ldcg(partial + i);
        for (int s = 1; s < ksplit; ++s) {
            const float4 b = __ldcg(partial + s * n4 + i);
            a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
        }
        return a;
    };
    const size_t step = static_cast<size_t>(gridDim.x) * kMaxCtas;
    size_t i = lo + static_cast<size_t>(blockIdx.x) * kMaxCtas + threadIdx.x;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < hi) a = sum(i);
    if (!__syncthreads_and(good)) return;
    while (i < hi) {
        if constexpr (sizeof(OUT) == 4) {
            float4* o = reinterpret_cast<float4*>(out) + i;
            if (accumulate) {
                const float4 b = *o;
                a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
            }
            *o = a;
        } else {
            reinterpret_cast<uint2*>(out)[i] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
        }
        i += step;
        if (i < hi) a = sum(i);
    }
}

int ctas_of(int num_sms) { return (num_sms < kMaxCtas ? num_sms : kMaxCtas) & ~1; }

template <int MODE, typename OUT, bool CHUNKED>
cudaError_t launch_as(const GroupedMmArgs& a, OUT* out, int ksplit, int accumulate, int num_sms, cudaStream_t s,
                        const char** why) {
    static std::atomic<bool> attr_set[64] = {};  // (set by whichever thread comes first, or by several)
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(grouped_mm_kernel<MODE, OUT, CHUNKED>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        if (e != cudaSuccess) {
            *why = "cudaFuncSetAttribute(max dynamic shared memory) failed";
            return e;
        }
        attr_set[dev] = true;
    }
    Maps m{};
    bool ok;
    if (MODE == kMmWgrad) {
        m.f_blocks = make_tensor_map_bf16_blocks(&m.f, a.B, a.N, a.M, 1, BK, 2);
        // A's tiles are 256 columns, each CTA's half 128: multiples of 64 when K has whole tiles.
        m.r_blocks = a.K % TILE_R == 0 && make_tensor_map_bf16_blocks(&m.r, a.A, a.K, a.M, 1, BK, 2);
        ok = (m.f_blocks || make_tensor_map_bf16(&m.f, a.B, a.N, a.M, BK)) &&
             (m.r_blocks || make_tensor_map_bf16(&m.r, a.A, a.K, a.M, BK));
    } else {
        ok = make_tensor_map_bf16(&m.r, a.A, a.K, a.M, 128) && make_tensor_map_bf16(&m.r64, a.A, a.K, a.M, 64) &&
             make_tensor_map_bf16(&m.r32, a.A, a.K, a.M, 32);
        if (MODE == kMmTransB) {
            ok = ok && make_tensor_map_bf16_3d(&m.f, a.B, a.K, a.N, a.E, 128);
        } else {
            m.f_blocks = make_tensor_map_bf16_blocks(&m.f, a.B, a.N, a.K, a.E, BK, 2);
            ok = ok && (m.f_blocks || make_tensor_map_bf16_3d(&m.f, a.B, a.N, a.K, a.E, BK));
        }
    }
    if (!ok) {
        *why = "cuTensorMapEncodeTiled failed (driver entry point missing or bad operand)";
        return cudaErrorInvalidValue;
    }
    return launch_k(kPdlTrain, grouped_mm_kernel<MODE, OUT, CHUNKED>, dim3(ctas_of(num_sms)), dim3(num_threads<MODE, CHUNKED>()),
                    SMEM_BYTES, s, m, a.offsets, a.M, a.K, a.N, a.E, ksplit, accumulate, a.inject_stall, out, ksplit > 1 ? a.done : nullptr,
                    a.status);
}

template <int MODE>
cudaError_t launch_mode(const GroupedMmArgs& a, float* out, int ksplit, int accumulate, int num_sms, cudaStream_t s,
                        const char** why) {
    // Blocks of the longest reduction, at most.
    const int blocks = ((MODE == kMmWgrad ? a.M : a.K) + BK - 1) / BK;
    return (blocks + ksplit - 1) / ksplit > chunk_blocks<float>() ? launch_as<MODE, float, true>(a, out, ksplit, accumulate, num_sms, s, why)
                                                  : launch_as<MODE, float, false>(a, out, ksplit, accumulate, num_sms, s, why);
}
template <int MODE>
cudaError_t launch_mode(const GroupedMmArgs& a, __nv_bfloat16* out, int ksplit, int accumulate, int num_sms,
                        cudaStream_t s, const char** why) {
    // A segment's rows are on the device: the rule goes by all of them (300000 rows, 2048 x 1408: 64 segments 1200 us
    // unbroken and 1228 in chunks, 256 segments 1355 and 1403; 256 of 512 x 512 150 and 155).
    if constexpr (MODE == kMmWgrad)
        if ((a.M + BK - 1) / BK > UNBROKEN) return launch_as<MODE, __nv_bfloat16, true>(a, out, ksplit, accumulate, num_sms, s, why);
    return launch_as<MODE, __nv_bfloat16, false>(a, out, ksplit, accumulate, num_sms, s, why);
}

template <int MODE>
cudaError_t launch_any(const GroupedMmArgs& a, int num_sms, cudaStream_t s, const char** why) {
    if (a.ksplit > 1) {
        cudaError_t e = launch_mode<MODE>(a, a.partial, a.ksplit, 0, num_sms, s, why);
        if (e != cudaSuccess) return e;
        const size_t n4 = (MODE == kMmWgrad ? static_cast<size_t>(a.E) * a.K : static_cast<size_t>(a.M)) * a.N / 4;
        const size_t want = (n4 + kMaxCtas - 1) / kMaxCtas, most = static_cast<size_t>(num_sms) * 8;
        const dim3 grid(static_cast<unsigned>(want < most ? want : most));
        const int by_row = MODE != kMmWgrad, acc = a.accumulate ? 1 : 0;
        *why = "slice join";
        const float4* p = reinterpret_cast<const float4*>(a.partial);
        if (a.out_f32)
            return launch_k(kPdlTrain, grouped_mm_join_kernel<float>, grid, dim3(kMaxCtas), 0, s, p, a.done,
                            ctas_of(num_sms), a.offsets, a.M, a.N, a.E, n4, a.ksplit, by_row, acc, static_cast<float*>(a.out));
        return launch_k(kPdlTrain, grouped_mm_join_kernel<__nv_bfloat16>, grid, dim3(kMaxCtas), 0, s, p, a.done,
                        ctas_of(num_sms), a.offsets, a.M, a.N, a.E, n4, a.ksplit, by_row, acc, static_cast<__nv_bfloat16*>(a.out));
    }
    const int acc = a.accumulate ? 1 : 0;
    return a.out_f32 ? launch_mode<MODE>(a, static_cast<float*>(a.out), 1, acc, num_sms, s, why)
                     : launch_mode<MODE>(a, static_cast<__nv_bfloat16*>(a.out), 1, acc, num_sms, s, why);
}

}  // namespace

// The reduction is split when its tiles would leave CTA pairs idle (serving a few tokens, few experts, the
// weight gradient of few experts over many rows).  The row counts are on the device, so the tiles
// are estimated from the shape, and the longest segment is taken as three times the average.  The slice count
// is the one with the least modelled time: rounds of CTA pairs x blocks per slice x 0.34 us (a block's
// products, or its share of the memory rate), not less than the bytes take; 1.5 us for each round's fill and
// drain; for slices the join's launch (3 us) and their way to the L2 and back.  Two rows of 14336 against
// 4096 columns (32 tiles): 45.9 us in 2 slices, 48.9 in 7, 73.7 unsplit; 1551 rows of 13136 against 344
// columns (14 tiles): 43 us in 2 slices, 30 in 5; 7 experts' gradients of 112 x 80 from 7597 rows: 27 us
// unsplit, 14 in 10.
int grouped_mm_ksplit(int mode, int M, int K, int N, int E, int num_sms) {
    const long long pairs = num_sms / 2;
    const long long f_tiles = (N + TILE_F - 1) / TILE_F;
    const long long active = M < E ? M : E;
    long long tiles, blocks;
    double out_elems, bytes;
    if (mode == kMmWgrad) {
        tiles = E * f_tiles * ((K + TILE_R - 1) / TILE_R);
        blocks = M / BK;
        if (blocks > 3 * blocks / E) blocks = 3 * blocks / E;
        out_elems = static_cast<double>(E) * K * N;
        bytes = 2.0 * M * (static_cast<double>(K) + N) + 4 * out_elems;
    } else {
        // Segments shorter than a tile take one each, longer ones half a tile more than their rows.
        tiles = f_tiles * (M < TILE_R * active ? active + M / (2 * TILE_R) : M / TILE_R + (active + 1) / 2);
        blocks = K / BK;
        out_elems = static_cast<double>(M) * N;
        bytes = 2.0 * M * K + 2.0 * active * K * N;
    }
    if (tiles == 0 || tiles > pairs) return 1;
    int best = 1;
    double best_us = 0.0;
    for (int n = 1; n <= MAX_SPLIT && (n == 1 || blocks / n >= 4); ++n) {
        const double rounds = static_cast<double>((tiles * n + pairs - 1) / pairs);
        const double work = rounds * static_cast<double>((blocks + n - 1) / n) * 0.34, memory = bytes / 6.5e6;
        const double us = (work > memory ? work : memory) + 1.5 * rounds + (n > 1 ? 3.0 + n * out_elems * 8 / 8e6 : 0.0);
        if (n == 1 || us < 0.97 * best_us) {
            best = n;
            best_us = us;
        }
    }
    return best;
}

cudaError_t launch_grouped_mm(int mode, const GroupedMmArgs& a, int num_sms, cudaStream_t s, const char** why) {
    if (mode == kMmForward) return launch_any<kMmForward>(a, num_sms, s, why);
    if (mode == kMmTransB) return launch_any<kMmTransB>(a, num_sms, s, why);
    return launch_any<kMmWgrad>(a, num_sms, s, why);
}

}  // namespace moe
