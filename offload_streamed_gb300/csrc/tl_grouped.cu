// tl_grouped.cu -- products whose weight depends on the row: out = x . w[group of
// the row], for experts and for adapters.
//
// The weight is the MMA's A side (128 of its own indices a CTA, either way it lies
// in memory) and the rows are its N side.  N is then chosen for each tile in steps
// of 16 or 32, so that a group's ragged end costs its rows and not a tile of 128 or
// 256, and a weight for few rows is read once and multiplied at the rate of its
// bytes.
// A result's columns are the tensor memory's lanes; it is turned on its way out
// through shared memory.
//
//  grouped_kernel    : a CTA pair (M = 256) and up to 256 rows a tile, persistent,
//                      two accumulators; for groups of many rows.  Indexed rows
//                      are sorted first, into a copy (see Picker in tl_grouped.cuh).
//  grouped_few_kernel: a CTA and up to 16 .. 128 rows a tile; the CTAs of a cluster
//                      share the reduction and add their parts in a fixed order.
//                      Indexed rows are picked up where they lie.
//
// What bounds them: the tensor cores for many rows (16384 rows of one
// group, 8192 x 4096: 677 us, 1.62 PFLOP/s; of eight groups through an index 806, 60 to
// 80 of it the copy), the weights' bytes for few (32 rows of 8 groups, 8192 x 4096:
// 86 us, 6.2 TB/s).
//
// Every wait on an mbarrier is bounded, as in tl_gemm.cu.
#include "tl_grouped.cuh"

#include <algorithm>

namespace tl {
namespace {

using namespace gr;

struct Params {
    int32_t rows, reduce, own, groups;
    int32_t num_k;     // K-blocks
    int32_t w_boxes;   // 64-wide boxes of the weight a CTA loads where own is contiguous
    uint32_t w_bytes;  // of the weight a stage and CTA
    int32_t num_m;
    const int32_t* offsets;
    const uint16_t* x;
    int64_t ldx;
    int32_t x_rows;
    const int32_t* x_index;
    const int32_t* out_index;
    int32_t out_rows;
    void* out;
    int64_t ldout;
    const float* scale;
    float scale_all;
    uint16_t* split_out;
    int32_t split_half;
    float* split_units;
    int32_t fp16;
    int32_t all_rows;
    uint32_t idesc;  // without N
    int32_t* err;
    uint64_t timeout_ns;
};

// The MMAs of one K-block.
template <bool W_MN, bool PAIR>
__device__ __forceinline__ void block_mmas(const Params& p, int kb, bool fresh, uint32_t d, uint32_t sa, uint32_t sb, uint32_t idesc) {
    const int steps = min(kBlockK / kUmmaK, (p.reduce - kb * kBlockK + kUmmaK - 1) / kUmmaK);
    for (int j = 0; j < steps; ++j)
        umma_16<PAIR>(d, operand_desc(W_MN, sa, j), operand_desc(false, sb, j), idesc, (!fresh || j != 0) ? 1u : 0u);
}

__device__ __forceinline__ int out_row(const Params& p, int place) { return p.out_index ? __ldg(p.out_index + place) : place; }

// Four results of a row at columns col .. col + 3: stored as `have` of them.
__device__ __forceinline__ void store_four(const Params& p, int64_t row, int col, int have, float4 f) {
    uint16_t* dst = static_cast<uint16_t*>(p.out) + row * p.ldout + col;
    const uint2 w = make_uint2(round16x2(f.x, f.y, p.fp16), round16x2(f.z, f.w, p.fp16));
    if (have == 4) {  // (rows start on 16 bytes, so col does on 8)
        *reinterpret_cast<uint2*>(dst) = w;
    } else {
        const uint32_t h[4] = {w.x, w.x >> 16, w.y, w.y >> 16};
        for (int j = 0; j < have; ++j) dst[j] = uint16_t(h[j]);
    }
}

// The unrounded result of a place, of which each lane of a warp has four columns, as two
// parts: what rounding keeps and what it takes off, rounded in its turn (an infinity leaves
// nothing).  Rounded to the type at once it would err as much as the rounding of what is
// made of it; two parts keep 16 (bf16) or 22 digits of fp32's 24, for half the bytes and
// none of the instructions of a third.
__device__ __forceinline__ void store_split(const Params& p, int64_t place, int col, const float (&f)[4]) {
    float to_units = 1.0f;
    if (p.split_units) {
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t size = __float_as_uint(f[j]) & 0x7fffffffu;
            if (col + j < p.own && size < 0x7f800000u) most = max(most, size);
        }
        const float unit = unit_of(__reduce_max_sync(0xffffffffu, most));
        if (col == 0) p.split_units[place] = unit;
        to_units = reciprocal_of_unit(unit);
    }
    if (col >= p.split_half) return;
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float v = col + j < p.own ? f[j] * to_units : 0.0f;
        hi[j] = round16(v, p.fp16);
        if (!p.fp16 && isfinite(v) && (hi[j] & 0x7fffu) == 0x7f80u) --hi[j];  // (past bf16's largest number: that one, and the rest)
        const float rest = v - value16(hi[j], p.fp16);
        lo[j] = round16(isfinite(rest) ? rest : 0.0f, p.fp16);
    }
    uint16_t* dst = p.split_out + place * 2 * p.split_half + col;
    *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | uint32_t(hi[1]) << 16, hi[2] | uint32_t(hi[3]) << 16);
    *reinterpret_cast<uint2*>(dst + p.split_half) = make_uint2(lo[0] | uint32_t(lo[1]) << 16, lo[2] | uint32_t(lo[3]) << 16);
}

// ---- groups of many rows ---------------------------------------------------------

constexpr int kPairStages = 6;
constexpr uint32_t kPairStage = 2 * kStageA;       // 128 own indices and 128 rows of a K-block
constexpr int kTurnPitch = 36;                     // floats: 16-byte rows, and no two lanes in one bank
constexpr uint32_t kTurnBytes = 32 * kTurnPitch * 4;  // of an epilogue warp: 32 rows x 32 columns
constexpr int kTable = kMaxGroupsSeen + 1;
constexpr uint32_t kTableBytes = (3 * kTable + 15) / 16 * 64;  // for each group: its first tile, its first place and its end
constexpr size_t kPairSmem = size_t(kPairStages) * kPairStage + 4 * kTurnBytes + kTableBytes + kBarBytes + 1024;
static_assert(kPairSmem + 64 <= 232448, "shared memory budget");

struct Tile {
    int g, p0, count, n, m;  // group, first place, places, N (a multiple of 32), block of 256 own indices
};

// Tiles of a group: blocks of at most 256 rows, of equal sizes, by blocks of own
// indices; eight blocks of rows go through all own indices together, so that the
// tiles in flight share both operands in L2.
__device__ __forceinline__ Tile find_tile(const Params& p, const int* first, int seen, int tile) {
    int lo = 0, hi = seen;  // first[lo] <= tile < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first[mid] <= tile) lo = mid;
        else hi = mid;
    }
    constexpr int kTogether = 8;
    const int local = tile - first[lo], blocks = (first[lo + 1] - first[lo]) / p.num_m;
    const int q = local / (kTogether * p.num_m), r = local - q * kTogether * p.num_m;
    const int width = min(kTogether, blocks - q * kTogether);
    Tile t;
    t.g = lo;
    t.m = r / width;
    const int begin = first[kTable + lo], rows = first[2 * kTable + lo] - begin;
    const int size = ((rows + blocks - 1) / blocks + 31) & ~31, at = (q * kTogether + r % width) * size;
    t.p0 = begin + at;
    t.count = min(size, rows - at);
    t.n = (t.count + 31) & ~31;
    return t;
}

constexpr int kBoxRows = 32;  // of x, in boxes for few rows (with one box of 128 for more: each load costs the issuing thread)

template <bool W_MN>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_x_few,
                   const Params p) {
    const SharedWaitCtx wc{p.err, p.timeout_ns};
    constexpr int S = kPairStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* turn = reinterpret_cast<float*>(smem + S * kPairStage);
    int* first = reinterpret_cast<int*>(smem + S * kPairStage + 4 * kTurnBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * kPairStage + 4 * kTurnBytes + kTableBytes);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
    static_assert((2 * S + 5) * 8 + 4 <= int(kBarBytes), "barrier area");
    __shared__ int sums[kThreads / 32];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint32_t bar0 = smem_addr(bars), smem0 = smem_addr(smem);
    // full[] and tmem_empty[] are used in the first CTA only
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (S + s); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * S + a); };
    auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * S + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);

    if (threadIdx.x == 0) {
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_x);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 8);
        }
        mbar_init(drain_bar, 1);
        mbar_init_fence();
    }
    if (warp == 2) {
        tmem_alloc<true>(smem_addr(tmem_slot), kTmemCols);
        tmem_relinquish<true>();
    }
    // every group's tiles, counted by each CTA for itself
    const int seen = p.groups;
    {
        const int per = (seen + kThreads - 1) / kThreads, g0 = min(seen, int(threadIdx.x) * per), g1 = min(seen, g0 + per);
        int mine = 0;
        for (int g = g0; g < g1; ++g) {
            int b, e;
            group_span(p.offsets, p.groups, p.rows, g, b, e);
            first[kTable + g] = b;
            first[2 * kTable + g] = e;
            mine += (e - b + kBlockN - 1) / kBlockN * p.num_m;
        }
        int s = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += u;
        }
        if (lane == 31) sums[warp] = s;
        __syncthreads();
        int at = s - mine;
        for (int w = 0; w < warp; ++w) at += sums[w];
        for (int g = g0; g < g1; ++g) {
            first[g] = at;
            at += (first[2 * kTable + g] - first[kTable + g] + kBlockN - 1) / kBlockN * p.num_m;
        }
        if (threadIdx.x == kThreads - 1) first[seen] = at;
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int tiles = first[seen], step = int(cluster_count_x());
    auto tile_at = [&](int tile) { return find_tile(p, first, seen, tile); };

    if (warp == 0) {
        // ---------------- loads: each CTA its own indices and half of the rows ----------------
        uint32_t fills = 0;
        bool ok = true;
        if (lane == 0) {
            for (int tile = int(cluster_id_x()); ok && tile < tiles; tile += step) {
                const Tile t = tile_at(tile);
                const int m0 = t.m * 256 + int(rank) * kBlockM, half_n = t.n / 2, row0 = t.p0 + int(rank) * half_n;
                const int boxes = half_n > kBlockM / 2 ? 0 : (half_n + kBoxRows - 1) / kBoxRows;
                const uint32_t bytes = 2u * (p.w_bytes + uint32_t(boxes ? boxes * kBoxRows : kBlockM) * 128u);
                for (int kb = 0; kb < p.num_k; ++kb, ++fills) {
                    const uint32_t s = fills % S;
                    if (!wait_bounded(empty_bar(s), ((fills / S) & 1u) ^ 1u, wc, kErrProducerWait)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = smem0 + s * kPairStage, sb = sa + kStageA;
                    const uint32_t fb = map_to_rank(full_bar(s), 0);
                    if (leader) mbar_arrive_expect_tx(full_bar(s), bytes);
                    const int k0 = kb * kBlockK;
                    if (W_MN) {
                        for (int c = 0; c < p.w_boxes; ++c) tma_load_box_pair(sa + c * kMnChunk, &map_w, fb, m0 + 64 * c, k0, t.g);
                    } else {
                        tma_load_box_pair(sa, &map_w, fb, k0, m0, t.g);
                    }
                    // (rows past the tile's last are others or zeros: their results are not stored)
                    if (boxes == 0) tma_load_2d_pair(sb, &map_x, fb, kb * kBlockK, row0);
                    for (int c = 0; c < boxes; ++c) tma_load_2d_pair(sb + c * kBoxRows * 128, &map_x_few, fb, kb * kBlockK, row0 + c * kBoxRows);
                }
            }
        }
        if (leader && lane == 0) {  // loads land before the CTA may exit
            const uint32_t outstanding = fills < uint32_t(S) ? fills : uint32_t(S);
            for (uint32_t j = 0; j < outstanding; ++j) {
                const uint32_t f = fills - 1 - j;
                wait_bounded(full_bar(f % S), (f / S) & 1u, wc, kErrDrainWait, false);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            uint32_t fills = 0;
            bool ok = true;
            int it = 0;
            for (int tile = int(cluster_id_x()); ok && tile < tiles; tile += step, ++it) {
                const Tile t = tile_at(tile);
                const uint32_t acc = it & 1;
                if (!wait_bounded(tempty_bar(acc), ((uint32_t(it) >> 1) & 1u) ^ 1u, wc, kErrMmaWaitTmem)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + acc * kBlockN, idesc = with_n(p.idesc, t.n);
                for (int kb = 0; kb < p.num_k; ++kb, ++fills) {
                    const uint32_t s = fills % S;
                    if (!wait_bounded(full_bar(s), (fills / S) & 1u, wc, kErrMmaWaitFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem0 + s * kPairStage;
                    block_mmas<W_MN, true>(p, kb, kb == 0, d, sa, sa + kStageA, idesc);
                    umma_commit_pair(empty_bar(s), 0x3);
                }
                if (ok) umma_commit_pair(tfull_bar(acc), 0x3);
            }
            umma_commit_pair(drain_bar, 0x3);
            wait_bounded(drain_bar, 0, wc, kErrDrainWait, false);
        }
    } else if (warp >= kFirstEpilogueWarp) {
        // ---------------- results: 32 rows at a time, turned in shared memory ----------------
        const int q = warp & 3;
        float* box = turn + q * (kTurnBytes / 4);
        const int sub = lane >> 2, c8 = 8 * (lane & 3);  // of a row's 32 columns, this lane's 8
        int it = 0;
        for (int tile = int(cluster_id_x()); tile < tiles; tile += step, ++it) {
            const Tile t = tile_at(tile);
            const uint32_t acc = it & 1;
            const int col = t.m * 256 + int(rank) * kBlockM + q * 32 + c8;  // this lane's first
            const int have = min(8, p.own - col);
            if (!warp_wait(tfull_bar(acc), (uint32_t(it) >> 1) & 1u, wc, kErrEpilogueWait, lane)) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + (uint32_t(q * 32) << 16) + acc * kBlockN;
            for (int c = 0; c < t.count; c += 32) {
                uint32_t v[32];
                tmem_ld_32cols(t_row + uint32_t(c), v);
                tmem_ld_wait();
                if (c + 32 >= t.count) {  // the accumulator has been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader) mbar_arrive(tempty_bar(acc));
                        else mbar_arrive_cluster(map_to_rank(tempty_bar(acc), 0));
                    }
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) box[j * kTurnPitch + lane] = __uint_as_float(v[j]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = t.p0 + c + i * 8 + sub;
                    if (c + i * 8 + sub >= t.count || have <= 0) continue;
                    const float4* src = reinterpret_cast<const float4*>(box + (i * 8 + sub) * kTurnPitch + c8);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int n = min(4, have - 4 * h);
                        if (n <= 0) break;
                        store_four(p, row, col + 4 * h, n, src[h]);
                    }
                }
                __syncwarp();
            }
        }
    }

    tc_fence_before();
    cluster_sync();
    if (warp == 2) {
        tc_fence_after();
        if (!leader) wait_bounded(drain_bar, 0, wc, kErrDrainWait, false);
        tmem_dealloc<true>(tmem_base, kTmemCols);
    }
}

// ---- groups of few rows ----------------------------------------------------------

// A ninth warp: when the others have read the parts of the sums, it arrives with
// release semantics at the barrier past which the cluster's CTAs may leave.
constexpr int kFewThreads = kThreads + 32;
constexpr size_t kFewSmem = 112 * 1024;  // of a CTA: two share an SM

// A stage is N rows of x and what there is of the weight: where own is small, less
// than the 16 KiB that the MMA reads (what it finds past them makes rows of the
// result that are not stored), which therefore have to be there after the last stage.
constexpr int kFewMostStages = 8;
template <int N>
struct Few {
    static constexpr uint32_t kRowBytes = uint32_t(N) * 128;
    static constexpr uint32_t kFixed = kBarBytes + 1024;
    static constexpr uint32_t kCols = N <= 32 ? 32 : N;
    static constexpr uint32_t stage(uint32_t w_bytes) { return kRowBytes + (w_bytes + 1023) / 1024 * 1024; }
    static constexpr int stages(uint32_t w_bytes) {
        const int s = int((kFewSmem - kFixed - (kStageA - (w_bytes + 1023) / 1024 * 1024)) / stage(w_bytes));
        return s < kFewMostStages ? s : kFewMostStages;
    }
    static_assert(stages(kStageA) >= 3 && size_t(N) * 128 * 4 + kFixed <= kFewSmem, "the parts fit the stages");
};

template <bool W_MN, int N>
__global__ void __launch_bounds__(kFewThreads, 2)
    grouped_few_kernel(const __grid_constant__ CUtensorMap map_w, const Params p, int splits, int per, uint32_t S, uint32_t stage) {
    using F = Few<N>;
    const SharedWaitCtx wc{p.err, p.timeout_ns};
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kFewSmem - F::kFixed);
    const uint32_t bar0 = smem_addr(bars), smem0 = smem_addr(smem);
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (kFewMostStages + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * kFewMostStages);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kFewMostStages + 1);
    static_assert((2 * kFewMostStages + 1) * 8 + 4 <= int(kBarBytes), "barrier area");
    __shared__ int found[3];  // group, first place, places
    __shared__ int sums[kFewThreads / 32];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = splits > 1 ? cluster_ctarank() : 0;
    const uint32_t unit = blockIdx.x / uint32_t(splits);
    const int m0 = int(unit % uint32_t(p.num_m)) * 128, wanted = int(unit / uint32_t(p.num_m));  // block of rows

    find_block(p.offsets, p.groups, p.rows, p.all_rows != 0, N, wanted, found, sums);
    const int group = found[0], p0 = found[1], count = found[2];
    if (group < 0) return;  // (every CTA of the cluster: the grid is made for the most blocks there can be)
    const bool none = group == p.groups;
    const int kb0 = none ? 0 : min(p.num_k, int(rank) * per), kb1 = none ? 0 : min(p.num_k, kb0 + per);

    if (threadIdx.x == 0) {
        tma_prefetch_map(&map_w);
        for (uint32_t s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1 + kPickWarps);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        mbar_init_fence();
    }
    if (warp == 2) {
        tmem_alloc<false>(smem_addr(tmem_slot), F::kCols);
        tmem_relinquish<false>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        auto load_w = [&](int kb, uint32_t s) {
            const uint32_t sa = smem0 + s * stage + F::kRowBytes;
            const int k0 = kb * kBlockK;
            if (W_MN) {
                for (int c = 0; c < p.w_boxes; ++c) tma_load_box(sa + c * kMnChunk, &map_w, full_bar(s), m0 + 64 * c, k0, group);
            } else {
                tma_load_box(sa, &map_w, full_bar(s), k0, m0, group);
            }
        };
        uint32_t fills = 0;
        if (lane == 0) {
            for (int kb = kb0; kb < kb1; ++kb, ++fills) {
                const uint32_t s = fills % S;
                if (!wait_bounded(empty_bar(s), ((fills / S) & 1u) ^ 1u, wc, kErrProducerWait)) break;
                mbar_arrive_expect_tx(full_bar(s), p.w_bytes);
                load_w(kb, s);
            }
            const uint32_t outstanding = fills < S ? fills : S;
            for (uint32_t j = 0; j < outstanding; ++j) {
                const uint32_t f = fills - 1 - j;
                wait_bounded(full_bar(f % S), (f / S) & 1u, wc, kErrDrainWait, false);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t fills = 0;
            const uint32_t idesc = with_n(p.idesc, N);
            for (int kb = kb0; kb < kb1; ++kb, ++fills) {
                const uint32_t s = fills % S;
                if (!wait_bounded(full_bar(s), (fills / S) & 1u, wc, kErrMmaWaitFull)) break;
                tc_fence_after();
                const uint32_t sa = smem0 + s * stage + F::kRowBytes;
                block_mmas<W_MN, false>(p, kb, kb == kb0, tmem_base, sa, sa - F::kRowBytes, idesc);
                umma_commit(empty_bar(s));
            }
            umma_commit(done_bar);
            wait_bounded(done_bar, 0, wc, kErrDrainWait, false);
        }
    } else if (warp >= kFirstEpilogueWarp && warp < kThreads / 32) {
        // these warps pick up the rows first
        {
            const Picker pick(int(threadIdx.x) - 32 * kFirstEpilogueWarp);
            constexpr int kRows = (N + kPickRows - 1) / kPickRows, kUnderWay = 2;  // (fewer than the stages)
            const uint16_t* src[kRows];
            bool there[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int place = p0 + min(pick.row + kPickRows * r, count - 1), row = p.x_index ? __ldg(p.x_index + place) : place;
                there[r] = unsigned(row) < unsigned(p.x_rows);
                src[r] = p.x + (there[r] ? row * p.ldx : 0);
            }
            uint32_t fills = 0, handed = 0;
            auto hand_over = [&] {
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(full_bar(handed % S));
                ++handed;
            };
            bool go = true;
            for (int kb = kb0; kb < kb1; ++kb, ++fills) {
                const uint32_t s = fills % S;
                if (!warp_test(empty_bar(s), ((fills / S) & 1u) ^ 1u)) {
                    cp_async_wait<0>();
                    while (handed < fills) hand_over();
                }
                if (!warp_wait(empty_bar(s), ((fills / S) & 1u) ^ 1u, wc, kErrProducerWait, lane)) {
                    go = false;
                    break;
                }
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    // (past the last row: what the stage held before, whose results are not stored)
                    if (kPickRows * r < count) pick.copy(smem0 + s * stage, r, src[r] + kb * kBlockK, there[r] ? p.reduce - kb * kBlockK : 0);
                cp_async_commit();
                if (fills - handed == kUnderWay) {
                    cp_async_wait<kUnderWay>();
                    hand_over();
                }
            }
            cp_async_wait<0>();
            if (go)
                while (handed < fills) hand_over();
        }
        const int q = warp & 3, i = q * 32 + lane;
        const bool ok = warp_wait(done_bar, 0, wc, kErrEpilogueWait, lane);
        tc_fence_after();
        const uint32_t t_row = tmem_base + (uint32_t(q * 32) << 16);
        float* part = reinterpret_cast<float*>(smem);  // [row][128], once the stages are done with
        constexpr int kStep = N < 32 ? N : 32;
        if (ok)
#pragma unroll 1
            for (int c = 0; c < count; c += kStep) {
                uint32_t v[kStep];
                if constexpr (kStep == 32) tmem_ld_32cols(t_row + uint32_t(c), v);
                else tmem_ld_16cols(t_row + uint32_t(c), v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < kStep; ++j)
                    if (c + j < count) part[(c + j) * 128 + i] = kb1 > kb0 ? __uint_as_float(v[j]) : 0.0f;
            }
        tc_fence_before();
    }
    if (splits > 1) cluster_sync();  // every part stands
    else __syncthreads();
    const float scale = none ? 0.0f : p.scale ? __ldg(p.scale + group) : p.scale_all;
    if (warp == kThreads / 32) {
        if (splits > 1) {
            cta_barrier_sync(1, kFewThreads);  // the others' reads are done
            cluster_arrive();
        }
    } else {
        // Four outputs of a row at a time; at most this many of a thread, with one
        // CTA or two.  All are read and summed before one is written: nobody waits
        // for the writes.
        constexpr int kMine = N * 32 / kThreads;
        float4 sum[kMine];
        const int e0 = int(rank) * kThreads + int(threadIdx.x), step = splits * kThreads;
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int e = e0 + u * step;
            if (e >= count * 32) break;
            const uint32_t at = smem0 + uint32_t(e / 32 * 128 + e % 32 * 4) * 4u;
            if (splits == 1) {
                uint32_t a, b, c, d;
                ld_shared_v4(at, a, b, c, d);
                sum[u] = make_float4(__uint_as_float(a), __uint_as_float(b), __uint_as_float(c), __uint_as_float(d));
                continue;
            }
            float4 v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < splits) v[r] = ld_cluster_f32x4(at, uint32_t(r));
            sum[u] = v[0];
#pragma unroll
            for (int r = 1; r < 8; ++r)
                if (r < splits) sum[u] = make_float4(sum[u].x + v[r].x, sum[u].y + v[r].y, sum[u].z + v[r].z, sum[u].w + v[r].w);
        }
        if (splits > 1) {
            cta_barrier_arrive(1, kFewThreads);
            cluster_arrive_relaxed();  // (the ninth warp's arrival orders the reads)
        }
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int e = e0 + u * step, col = m0 + e % 32 * 4;
            if (e >= count * 32) break;
            const int row = out_row(p, p0 + e / 32);
            if (unsigned(row) >= unsigned(p.out_rows)) continue;
            const int have = min(4, p.own - col);
            const float4 f = make_float4(sum[u].x * scale, sum[u].y * scale, sum[u].z * scale, sum[u].w * scale);
            if (have > 0 && p.out) store_four(p, row, col, have, f);
            if (p.split_out) {  // (a warp has a row: all of its 128 columns, m0 being 0)
                const float w[4] = {f.x, f.y, f.z, f.w};
                store_split(p, p0 + e / 32, col, w);
            }
        }
    }
    if (splits > 1) cluster_wait();  // nobody leaves while its part is read
    else __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc<false>(tmem_base, F::kCols);
    }
}

// Asked about, never launched (see tl_fp8.cu): how many clusters of
// grouped_few_kernel's threads and shared memory run at a time.
__global__ void __launch_bounds__(kFewThreads, 2) grouped_few_shape_kernel() {}

bool off(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// Rows of a group in the mean decide.  Forward, 2048 x 2048, us, few / many: 64 groups of
// 32 rows 124 / 107, of 64 rows 179 / 119; 8192 x 4096, 8 groups of 32 117 / 123, of 17
// - / 116 and of 16 105 / -.
int64_t mean_rows(const GroupedDesc& d) { return (d.rows + d.groups - 1) / d.groups; }
bool by_pairs(const GroupedDesc& d) { return d.own > kBlockM && !d.split_out && !d.all_rows && !d.out.index && mean_rows(d) > 16; }
// Rows of a block of few: room for half as many again as the mean, since groups differ, and a
// second block reads the weight again.
int few_size(const GroupedDesc& d) {
    const int64_t want = mean_rows(d) + mean_rows(d) / 2;
    return want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : 128;
}
// The most blocks of rows there can be: whole ones, and one of each group that has a row.
int64_t few_blocks(const GroupedDesc& d) { return d.rows / few_size(d) + std::min(d.groups + (d.all_rows ? 1 : 0), d.rows); }

template <bool W_MN, int N>
cudaError_t launch_few(const CUtensorMap& mw, Params p, const GroupedDesc& d, int num_sms, cudaStream_t stream) {
    const int64_t seen = d.groups + (d.all_rows ? 1 : 0);
    const int64_t blocks = few_blocks(d), units = blocks * p.num_m;
    const int64_t likely = std::max<int64_t>(1, std::min(blocks, (d.rows + N - 1) / N + std::min(seen, d.rows) / 2)) * p.num_m;
    int splits = 1, per_sm = 0, clusters = 0;
    const void* shape = reinterpret_cast<const void*>(grouped_few_shape_kernel);
    cudaError_t e = ctas_per_sm(shape, kFewThreads, kFewSmem, &per_sm);
    // CTAs of a cluster: as many as two an SM allow, with four K-blocks each
    while (e == cudaSuccess && splits < 8 && likely * splits * 2 <= 2 * num_sms && p.num_k >= 8 * splits) {
        e = clusters_at_a_time(shape, kFewThreads, kFewSmem, 2 * splits, &clusters);
        if (e != cudaSuccess || likely > clusters) break;
        splits *= 2;
    }
    if (e != cudaSuccess) return e;
    const int per = (p.num_k + splits - 1) / splits;
    return launch_in_clusters(grouped_few_kernel<W_MN, N>, dim3(unsigned(units * splits)), kFewThreads, splits, kFewSmem, false, stream, mw,
                              p, splits, per, uint32_t(Few<N>::stages(p.w_bytes)), Few<N>::stage(p.w_bytes));
}

// A sorted copy of indexed rows: rows outside the matrix as zeros.
constexpr int kPickCopyThreads = 256;
__global__ void __launch_bounds__(kPickCopyThreads) pick_rows_kernel(const uint16_t* x, int64_t ldx, int x_rows, const int32_t* index, int rows,
                                                                     int cols, int lanes, uint16_t* out, int64_t ldo) {
    // `lanes` threads (a power of two) walk a row; four vectors of each under way
    const int64_t p = int64_t(blockIdx.x) * (kPickCopyThreads / lanes) + threadIdx.x / lanes;
    if (p >= rows) return;
    const int row = __ldg(index + p);
    const bool there = unsigned(row) < unsigned(x_rows);
    const uint4* src = reinterpret_cast<const uint4*>(x + (there ? row * ldx : 0));
    uint4* dst = reinterpret_cast<uint4*>(out + p * ldo);
    const int whole = cols / 8, first = int(threadIdx.x % lanes);
#pragma unroll 4
    for (int v = first; v < whole; v += lanes) dst[v] = there ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
    if (first == whole % lanes && cols % 8)  // (behind a row's end is not the row's)
        dst[whole] = there ? load_eight(reinterpret_cast<const uint16_t*>(src + whole), cols % 8) : make_uint4(0, 0, 0, 0);
}

}  // namespace

int64_t picked_ld(int64_t cols) { return (cols + 7) / 8 * 8; }

cudaError_t pick_rows_launch(const RowsOperand& x, int64_t rows, int64_t cols, void* out, cudaStream_t stream) {
    const int64_t vectors = picked_ld(cols) / 8;
    int lanes = 32;
    while (lanes < kPickCopyThreads && lanes * 4 < vectors) lanes *= 2;
    const int per = kPickCopyThreads / lanes;
    pick_rows_kernel<<<unsigned((rows + per - 1) / per), kPickCopyThreads, 0, stream>>>(static_cast<const uint16_t*>(x.at), x.ld, int(x.count), x.index,
                                                                                     int(rows), int(cols), lanes, static_cast<uint16_t*>(out), picked_ld(cols));
    return cudaGetLastError();
}

std::string grouped_check(const GroupedDesc& d) {
    constexpr int64_t kMost = INT32_MAX / 2;
    if (d.rows < 0 || d.rows > kMost || d.x.count < 0 || d.x.count > kMost || d.out.count < 0 || d.out.count > kMost)
        return "rows must be >= 0 and below 2^30";
    if (d.reduce < 1 || d.own < 1 || d.reduce > kMost || d.own > kMost) return "the weight's sizes must be >= 1 and below 2^30";
    if (d.groups < 1 || d.groups > kMaxGroupsSeen - 1) return "groups must be 1..1024";
    if (d.type != TL_TYPE_BF16 && d.type != TL_TYPE_F16) return "the product takes bf16 or fp16 (tl_type)";
    if (!d.offsets || !d.err || off(d.offsets, 4) || off(d.err, 4)) return "offsets or err is null or not 4-byte aligned";
    if (d.rows == 0) return {};
    if (!d.x.at || !d.w || (!d.out.at && !d.split_out)) return "null pointer";
    if (off(d.x.at, 16) || off(d.w, 16) || off(d.out.at, 16) || off(d.split_out, 16)) return "operand pointers must be 16-byte aligned";
    if (d.x.ld % 8 || d.ldw % 8 || d.w_apart % 8 || d.out.ld % 8) return "leading dimensions must be multiples of 8 elements";
    const int64_t inner = d.own_contiguous ? d.own : d.reduce, outer = d.own_contiguous ? d.reduce : d.own;
    if (d.x.ld < d.reduce || d.ldw < inner || (d.out.at && d.out.ld < d.own)) return "a leading dimension is smaller than a row";
    if (d.groups > 1 && d.w_apart < (outer - 1) * d.ldw + inner) return "the groups' weights overlap";
    if (d.x.ld >= (int64_t(1) << 38) || d.ldw >= (int64_t(1) << 38) || d.w_apart >= (int64_t(1) << 38)) return "a leading dimension is too large";
    if (d.x.count < 1 || (!d.x.index && d.x.count < d.rows)) return "x has too few rows";
    if (!d.out.index && d.out.count < d.rows) return "the result has too few rows";
    if (off(d.gathered, 16)) return "the workspace is not 16-byte aligned";
    if (off(d.x.index, 4) || off(d.out.index, 4) || off(d.scale, 4) || off(d.split_units, 4)) return "indexes and scales must be 4-byte aligned";
    if (d.split_out && (d.own > d.split_half || d.split_half > kBlockM)) return "a result in two parts has 128 columns at most";
    // (of pairs: whatever the offsets hold, a CTA's count of the tiles stays in 32 bits)
    const int64_t tiles = by_pairs(d) ? d.groups * ((d.rows + kBlockN - 1) / kBlockN) * ((d.own + 255) / 256) : few_blocks(d) * ((d.own + kBlockM - 1) / kBlockM);
    if (tiles > INT32_MAX) return "too many tiles";
    return {};
}

cudaError_t grouped_launch(const GroupedDesc& d, int num_sms, cudaStream_t stream, std::string* why) {
    if (d.rows == 0) return cudaSuccess;
    Params p{};
    p.rows = int32_t(d.rows);
    p.reduce = int32_t(d.reduce);
    p.own = int32_t(d.own);
    p.groups = int32_t(d.groups);
    p.num_k = int32_t((d.reduce + kBlockK - 1) / kBlockK);
    p.offsets = d.offsets;
    p.x = static_cast<const uint16_t*>(d.x.at);
    p.ldx = d.x.ld;
    p.x_rows = int32_t(d.x.count);
    p.x_index = d.x.index;
    p.out_index = d.out.index;
    p.out_rows = int32_t(d.out.count);
    p.out = const_cast<void*>(d.out.at);
    p.ldout = d.out.ld;
    p.scale = d.scale;
    p.scale_all = d.scale_all;
    p.split_out = static_cast<uint16_t*>(d.split_out);
    p.split_half = d.split_half;
    p.split_units = d.split_units;
    p.fp16 = d.type == TL_TYPE_F16 ? 1 : 0;
    p.all_rows = d.all_rows ? 1 : 0;
    p.err = d.err;
    p.timeout_ns = 2000000000ull;
    CUtensorMap mx, mw;
    const int64_t inner = d.own_contiguous ? d.own : d.reduce, outer = d.own_contiguous ? d.reduce : d.own;
    const int64_t apart = d.groups > 1 ? d.w_apart : (outer * d.ldw);
    const uint32_t box_rows = d.own_contiguous ? uint32_t(kBlockK) : uint32_t(std::min<int64_t>(kBlockM, (d.own + 7) / 8 * 8));
    if (!swizzled_map(&mw, map_type16(d.type), 2, d.w, uint64_t(inner), uint64_t(outer), uint64_t(d.ldw), box_rows, why, uint64_t(d.groups), uint64_t(apart)))
        return cudaErrorInvalidValue;
    p.w_boxes = d.own <= 64 ? 1 : 2;
    p.w_bytes = d.own_contiguous ? uint32_t(p.w_boxes) * kMnChunk : box_rows * 128u;

    cudaError_t e;
    if (by_pairs(d)) {
        p.num_m = int32_t((d.own + 255) / 256);
        p.idesc = idesc_16(256, d.own_contiguous, false, p.fp16 != 0);
        const int64_t tiles = (d.rows / kBlockN + std::min(d.groups, d.rows)) * p.num_m;
        const unsigned grid = 2 * unsigned(std::min<int64_t>(tiles, std::max(1, num_sms / 2)));
        RowsOperand x = d.x;
        if (x.index) {
            if (!d.gathered) return cudaErrorInvalidValue;
            const cudaError_t g = pick_rows_launch(d.x, d.rows, d.reduce, d.gathered, stream);
            if (g != cudaSuccess) return g;
            x = {d.gathered, picked_ld(d.reduce), d.rows, nullptr};
        }
        CUtensorMap few;
        if (!rows_map(&mx, d.type, x, d.reduce, kBlockM, why) || !rows_map(&few, d.type, x, d.reduce, kBoxRows, why)) return cudaErrorInvalidValue;
        auto run = [&](auto kern) { return launch_in_clusters(kern, dim3(grid), kThreads, 2, kPairSmem, false, stream, mw, mx, few, p); };
        e = d.own_contiguous ? run(grouped_kernel<true>) : run(grouped_kernel<false>);
    } else {
        p.num_m = int32_t((d.own + kBlockM - 1) / kBlockM);
        p.idesc = idesc_16(128, d.own_contiguous, false, p.fp16 != 0);
        auto run = [&](auto mn) {
            constexpr bool MN = decltype(mn)::value;
            switch (few_size(d)) {
                case 16: return launch_few<MN, 16>(mw, p, d, num_sms, stream);
                case 32: return launch_few<MN, 32>(mw, p, d, num_sms, stream);
                case 64: return launch_few<MN, 64>(mw, p, d, num_sms, stream);
                default: return launch_few<MN, 128>(mw, p, d, num_sms, stream);
            }
        };
        e = d.own_contiguous ? run(std::true_type{}) : run(std::false_type{});
    }
    if (e != cudaSuccess && why && why->empty()) *why = std::string("kernel launch: ") + cudaGetErrorString(e);
    return e;
}

}  // namespace tl
