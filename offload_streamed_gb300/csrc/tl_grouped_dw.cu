// tl_grouped_dw.cu -- the weights' gradients of products whose weight depends on
// the row: dw[g] = sum over g's rows of x[row]^T dy[row].
//
// The reduction runs over a group's rows, 64 a block.  Rows past the group's end
// are zeros in its last block, so that the next group's rows (which may hold
// infinities) add nothing.
//
//  grouped_dw_kernel       : a CTA pair and 256 x 256 of a dw, persistent, as the
//                            dW product in tl_gemm.cu; a group without rows gets zeros.
//                            Blocks come by TMA; in a group's last one, gathers of
//                            four rows ask for rows past the matrix where the group
//                            has none, which arrive as zeros.  Indexed rows are sorted
//                            first, into a copy.
//  grouped_dw_narrow_kernel: 128 of x's columns and all (at most 128) of dy's, for
//                            adapters; the CTAs of a cluster share a group's rows and
//                            add their parts in a fixed order.  It takes a dy in two
//                            parts (twice the type's digits) as twice the columns,
//                            which are added out of tensor memory.
//
// What bounds them: the tensor cores (16384 rows of one group, 8192 x 4096: 662 us, 1.66
// PFLOP/s), with few rows the writing of dw (512 rows, 64 groups, 2048 x 2048: 163 us for
// 537 MB, which a memset takes 138 for; eight storing warps instead of four: the same).  The
// narrow one has 48 KB a CTA of x under way: 8192 x 16 of four adapters from 8192 rows, 68 us for
// 134 MB, a quarter of memory's rate (92 while the next block's rows were not on their way).
#include "tl_grouped.cuh"

#include <algorithm>

namespace tl {
namespace {

using namespace gr;

struct DwParams {
    int32_t rows, m_dim, n_dim, groups;
    int32_t num_m, num_n;
    const int32_t* offsets;
    const int32_t* x_index;
    const int32_t* dy_index;
    const uint16_t* x;
    const uint16_t* dy;
    int64_t ldx, lddy;
    int32_t x_rows, dy_rows, dy_cols;
    const float* scale;
    float scale_all;
    int32_t fp16;
    uint32_t idesc;
    // narrow only
    int32_t half, n;  // dy_cols rounded up: dy's columns in the product (twice `half` with two parts)
    const float* dy_units;
    uint16_t* dw;
    int64_t lddw, dw_apart;
    int32_t transposed;
    int32_t* err;
    uint64_t timeout_ns;
};

constexpr int kStages = 6;
constexpr uint32_t kStage = 2 * kStageA;
constexpr uint32_t kEpiBytes = 4 * 2 * kEpiBuf;
constexpr size_t kSmem = size_t(kStages) * kStage + kEpiBytes + kBarBytes + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

struct DwMaps {
    CUtensorMap x, dy, x_rows, dy_rows, dw;  // boxes of 64 rows, and rows one by one
};

__global__ void __launch_bounds__(kThreads, 1) grouped_dw_kernel(const __grid_constant__ DwMaps maps, const DwParams p) {
    const SharedWaitCtx wc{p.err, p.timeout_ns};
    constexpr int S = kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * kStage + kEpiBytes);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint32_t bar0 = smem_addr(bars), smem0 = smem_addr(smem);
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (S + s); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * S + a); };
    auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * S + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);

    if (threadIdx.x == 0) {
        tma_prefetch_map(&maps.x);
        tma_prefetch_map(&maps.dy);
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
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int of_group = p.num_m * p.num_n, step = int(cluster_count_x());
    const int64_t tiles = int64_t(of_group) * p.groups;

    if (warp == 0) {
        uint32_t fills = 0;
        bool ok = true;
        for (int64_t tile = cluster_id_x(); ok && tile < tiles; tile += step) {
            const int g = int(tile / of_group), local = int(tile % of_group);
            int begin, end;
            group_span(p.offsets, p.groups, p.rows, g, begin, end);
            const int cx = local % p.num_m * 256 + int(rank) * 128, cy = local / p.num_m * 256 + int(rank) * 128;
            for (int p0 = begin; p0 < end; p0 += kBlockK, ++fills) {
                const uint32_t s = fills % S;
                const uint32_t sa = smem0 + s * kStage, sb = sa + kStageA, fb = map_to_rank(full_bar(s), 0);
                int go = 1;
                if (lane == 0) {
                    go = wait_bounded(empty_bar(s), ((fills / S) & 1u) ^ 1u, wc, kErrProducerWait) ? 1 : 0;
                    if (go && leader) mbar_arrive_expect_tx(full_bar(s), 2u * kStage);
                    if (go && p0 + kBlockK <= end)
                        for (int c = 0; c < 2; ++c) {
                            tma_load_2d_pair(sa + c * kMnChunk, &maps.x, fb, cx + 64 * c, p0);
                            tma_load_2d_pair(sb + c * kMnChunk, &maps.dy, fb, cy + 64 * c, p0);
                        }
                }
                go = __shfl_sync(0xffffffffu, go, 0);
                if (!go) {
                    ok = false;
                    break;
                }
                if (p0 + kBlockK > end) {  // a lane's four rows, in one of the two 64-wide boxes
                    const int quad = 4 * (lane & 15), chunk = lane >> 4;
                    const uint32_t at = uint32_t(chunk) * kMnChunk + uint32_t(lane & 15) * 512u;
                    int r[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) r[j] = p0 + quad + j < end ? p0 + quad + j : p.rows;  // (a row past both matrices)
                    tma_gather4_pair(sa + at, &maps.x_rows, fb, cx + 64 * chunk, r);
                    tma_gather4_pair(sb + at, &maps.dy_rows, fb, cy + 64 * chunk, r);
                    __syncwarp();
                }
            }
        }
        if (leader && lane == 0) {
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
            const uint32_t idesc = with_n(p.idesc, kBlockN);
            for (int64_t tile = cluster_id_x(); ok && tile < tiles; tile += step, ++it) {
                int begin, end;
                group_span(p.offsets, p.groups, p.rows, int(tile / of_group), begin, end);
                const uint32_t acc = it & 1;
                if (!wait_bounded(tempty_bar(acc), ((uint32_t(it) >> 1) & 1u) ^ 1u, wc, kErrMmaWaitTmem)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + acc * kBlockN;
                for (int p0 = begin; p0 < end; p0 += kBlockK, ++fills) {
                    const uint32_t s = fills % S;
                    if (!wait_bounded(full_bar(s), (fills / S) & 1u, wc, kErrMmaWaitFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem0 + s * kStage, sb = sa + kStageA;
                    const int steps = min(kBlockK / kUmmaK, (end - p0 + kUmmaK - 1) / kUmmaK);
                    for (int j = 0; j < steps; ++j)
                        umma_16<true>(d, operand_desc(true, sa, j), operand_desc(true, sb, j), idesc, (p0 != begin || j) ? 1u : 0u);
                    umma_commit_pair(empty_bar(s), 0x3);
                }
                if (ok) umma_commit_pair(tfull_bar(acc), 0x3);
            }
            umma_commit_pair(drain_bar, 0x3);
            wait_bounded(drain_bar, 0, wc, kErrDrainWait, false);
        }
    } else if (warp >= kFirstEpilogueWarp) {
        const int q = warp & 3;
        const uint32_t epi0 = smem0 + S * kStage + uint32_t(q) * 2u * kEpiBuf;
        uint32_t buf = 0;
        int it = 0;
        for (int64_t tile = cluster_id_x(); tile < tiles; tile += step, ++it) {
            const int g = int(tile / of_group), local = int(tile % of_group);
            int begin, end;
            group_span(p.offsets, p.groups, p.rows, g, begin, end);
            const uint32_t acc = it & 1;
            const int row0 = local % p.num_m * 256 + int(rank) * 128 + q * 32, n0 = local / p.num_m * 256;
            const int chunks = row0 < p.m_dim ? min(kBlockN / 64, (p.n_dim - n0 + 63) / 64) : 0;
            const float scale = p.scale ? __ldg(p.scale + g) : p.scale_all;
            if (!warp_wait(tfull_bar(acc), (uint32_t(it) >> 1) & 1u, wc, kErrEpilogueWait, lane)) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + (uint32_t(q * 32) << 16) + acc * kBlockN;
            for (int c = 0; c < chunks; ++c) {
                uint32_t w[32], v[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tmem_ld_32cols(t_row + uint32_t(c) * 64u + 32u * uint32_t(h), v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        w[16 * h + j] = begin < end ? round16x2(__uint_as_float(v[2 * j]) * scale, __uint_as_float(v[2 * j + 1]) * scale, p.fp16) : 0u;
                }
                const uint32_t box = epi0 + buf * kEpiBuf;
                if (lane == 0) bulk_wait_group_read<1>();  // the store that last used this box has read it
                __syncwarp();
                const uint32_t at = box + uint32_t(lane) * 128u;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st_shared_v4(at + ((uint32_t(j) ^ (uint32_t(lane) & 7u)) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    tma_store_box(&maps.dw, box, n0 + c * 64, row0, g);
                    bulk_commit_group();
                }
                buf ^= 1u;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(tempty_bar(acc));
                else mbar_arrive_cluster(map_to_rank(tempty_bar(acc), 0));
            }
        }
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
    }

    tc_fence_before();
    cluster_sync();
    if (warp == 2) {
        tc_fence_after();
        if (!leader) wait_bounded(drain_bar, 0, wc, kErrDrainWait, false);
        tmem_dealloc<true>(tmem_base, kTmemCols);
    }
}

// ---- narrow gradients --------------------------------------------------------

// The rows of a block that a picking thread copies, of one operand: numbers, so that
// the next block's can be on their way.
struct BlockRows {
    int row[kBlockK / kPickRows];
    __device__ __forceinline__ void find(const int32_t* index, int p, int end) {
#pragma unroll
        for (int i = 0; i < kBlockK / kPickRows; ++i) {
            const int place = p + kPickRows * i;
            row[i] = place < end ? (index ? __ldg(index + place) : place) : -1;
        }
    }
    // columns col .. col + 63 of `cols`, to the box at `box`; a row outside the matrix as zeros
    __device__ __forceinline__ void copy(const Picker& pick, uint32_t box, const uint16_t* at, int64_t ld, int rows, int col, int cols) const {
#pragma unroll
        for (int i = 0; i < kBlockK / kPickRows; ++i) {
            const int have = unsigned(row[i]) < unsigned(rows) ? cols - col : 0;
            pick.copy(box, i, at + (have > 0 ? row[i] * ld + col : 0), have);
        }
    }
};

// What a picking thread has copied of a box, in fp16, each row times its factor.
template <int R>
__device__ __forceinline__ void scale_rows(const Picker& pick, uint32_t box, const float (&to)[R]) {
    uint32_t w[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i) ld_shared_v4(pick.at(box, i), w[i][0], w[i][1], w[i][2], w[i][3]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i][j]));
            w[i][j] = round16x2(v.x * to[i], v.y * to[i], true);
        }
        st_shared_v4(pick.at(box, i), w[i][0], w[i][1], w[i][2], w[i][3]);
    }
}

constexpr int kNarrowThreads = kThreads + 32;  // the ninth warp as in tl_grouped.cu
constexpr size_t kNarrowSmem = 112 * 1024;     // of a CTA: two share an SM
constexpr int kNarrowMostStages = 8;
// Blocks that a picking thread has under way behind the one handed over: fewer than the stages.
constexpr int kNarrowUnderWay = 2;
constexpr uint32_t kNarrowFixed = kBarBytes + 1024;
__host__ __device__ constexpr uint32_t narrow_stage(int n) { return kStageA + uint32_t((n + 63) / 64) * kMnChunk; }
constexpr int narrow_stages(int n) {
    const int s = int((kNarrowSmem - kNarrowFixed) / narrow_stage(n));
    return s < kNarrowMostStages ? s : kNarrowMostStages;
}
// the parts: [128 columns of dy or fewer][128] floats, or [128][as many + 4]
constexpr size_t part_floats(int cols, bool transposed) { return transposed ? size_t(cols) * 128 : size_t(128) * (cols + 4); }
static_assert(part_floats(128, false) * 4 <= size_t(narrow_stages(256)) * narrow_stage(256), "the parts fit the stages");
static_assert(part_floats(128, false) * 4 <= size_t(narrow_stages(128)) * narrow_stage(128), "the parts fit the stages");
static_assert(part_floats(64, false) * 4 <= size_t(narrow_stages(16)) * narrow_stage(16) && narrow_stages(256) >= 2, "the parts fit the stages");

// UNITS: dy's parts are in units of their places (fp16), and are put into the largest of the
// CTA's places by the threads that copied them, before they hand them over.  (Their loads are issued
// together, and the units' a block ahead: of an adapters' backward of 8192 rows, 8192 x
// 4096, rank 64 of 8, 231 us instead of 256; without units, in bf16, 215.)
template <bool UNITS>
__global__ void __launch_bounds__(kNarrowThreads, 2)
    grouped_dw_narrow_kernel(const DwParams p, int splits, int stages) {
    const SharedWaitCtx wc{p.err, p.timeout_ns};
    const int S = stages;
    const uint32_t stage = narrow_stage(p.n);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * stage);
    const uint32_t bar0 = smem_addr(bars), smem0 = smem_addr(smem);
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (kNarrowMostStages + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * kNarrowMostStages);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kNarrowMostStages + 1);
    __shared__ uint32_t largest[kNarrowThreads / 32];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = splits > 1 ? cluster_ctarank() : 0;
    const int block = int(blockIdx.x / uint32_t(splits)), g = block / p.num_m, m0 = block % p.num_m * 128;
    int begin, end;
    group_span(p.offsets, p.groups, p.rows, g, begin, end);
    // this CTA's blocks of the group's rows, perhaps none
    const int blocks = (end - begin + kBlockK - 1) / kBlockK, per = (blocks + splits - 1) / splits;
    const int kb0 = min(blocks, int(rank) * per), kb1 = min(blocks, kb0 + per);
    uint32_t cols = 32;  // of tensor memory
    while (cols < uint32_t(p.n)) cols *= 2;
    if constexpr (UNITS) {  // the largest unit of this CTA's places, in which it sums them (positive floats compare as their bits)
        uint32_t most = 0;
        const int last = min(end, begin + kb1 * kBlockK);
#pragma unroll 4
        for (int place = begin + kb0 * kBlockK + int(threadIdx.x); place < last; place += kNarrowThreads)
            most = max(most, __float_as_uint(__ldg(p.dy_units + place)));
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) largest[warp] = most;
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), kPickWarps);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        mbar_init_fence();
    }
    if (warp == 2) {
        tmem_alloc<false>(smem_addr(tmem_slot), cols);
        tmem_relinquish<false>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    float unit = 1.0f;
    if (UNITS && kb1 > kb0) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < kNarrowThreads / 32; ++i) most = max(most, largest[i]);
        unit = __uint_as_float(most);
    }

    if (warp == 1) {
        if (lane == 0) {
            uint32_t fills = 0;
            const uint32_t idesc = with_n(p.idesc, p.n);
            for (int kb = kb0; kb < kb1; ++kb, ++fills) {
                const uint32_t s = fills % uint32_t(S);
                if (!wait_bounded(full_bar(s), (fills / uint32_t(S)) & 1u, wc, kErrMmaWaitFull)) break;
                tc_fence_after();
                const uint32_t sa = smem0 + s * stage, sb = sa + kStageA;
                const int steps = min(kBlockK / kUmmaK, (end - begin - kb * kBlockK + kUmmaK - 1) / kUmmaK);
                for (int j = 0; j < steps; ++j)
                    umma_16<false>(tmem_base, operand_desc(true, sa, j), operand_desc(true, sb, j), idesc, (kb != kb0 || j) ? 1u : 0u);
                umma_commit(empty_bar(s));
            }
            umma_commit(done_bar);
            wait_bounded(done_bar, 0, wc, kErrDrainWait, false);
        }
    }
    // The parts, so that four neighbours of the result are four neighbours there.
    float* part = reinterpret_cast<float*>(smem);
    const int width = p.half ? p.half : p.n, pitch = p.transposed ? 128 : width + 4;
    if (warp >= kFirstEpilogueWarp && warp < kThreads / 32) {
        {  // these warps pick up the rows of both operands first
            const Picker pick(int(threadIdx.x) - 32 * kFirstEpilogueWarp);
            const int boxes = (p.n + 63) / 64;
            BlockRows x, dy, nx, ny;
            x.find(p.x_index, begin + kb0 * kBlockK + pick.row, end);
            dy.find(p.dy_index, begin + kb0 * kBlockK + pick.row, end);
            uint32_t fills = 0, handed = 0;
            constexpr int kRows = kBlockK / kPickRows;
            const float reciprocal = reciprocal_of_unit(unit);
            float units[kRows];  // of the rows to be handed over next
            auto ask_units = [&] {
                const int place = begin + (kb0 + int(handed)) * kBlockK + pick.row;
#pragma unroll
                for (int i = 0; i < kRows; ++i) units[i] = place + kPickRows * i < end ? __ldg(p.dy_units + place + kPickRows * i) : unit;
            };
            if constexpr (UNITS) ask_units();
            auto hand_over = [&] {
                if constexpr (UNITS) {
                    const uint32_t box = smem0 + handed % uint32_t(S) * stage + kStageA;
                    float to[kRows];
                    bool all_ones = true;
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        to[i] = between_units(units[i], reciprocal);
                        all_ones = all_ones && to[i] == 1.0f;
                    }
                    if (!all_ones && 8 * pick.chunk < p.n)
                        for (int c = 0; c < boxes; ++c) scale_rows(pick, box + c * kMnChunk, to);
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(full_bar(handed % uint32_t(S)));
                ++handed;
                if constexpr (UNITS) ask_units();
            };
            bool go = true;
            for (int kb = kb0; kb < kb1; ++kb, ++fills) {
                const uint32_t s = fills % uint32_t(S);
                nx.find(p.x_index, begin + (kb + 1) * kBlockK + pick.row, end);
                ny.find(p.dy_index, begin + (kb + 1) * kBlockK + pick.row, end);
                if (!warp_test(empty_bar(s), ((fills / uint32_t(S)) & 1u) ^ 1u)) {
                    cp_async_wait<0>();
                    while (handed < fills) hand_over();
                }
                if (!warp_wait(empty_bar(s), ((fills / uint32_t(S)) & 1u) ^ 1u, wc, kErrProducerWait, lane)) {
                    go = false;
                    break;
                }
                const uint32_t sa = smem0 + s * stage, sb = sa + kStageA;
                for (int c = 0; c < 2; ++c) x.copy(pick, sa + c * kMnChunk, p.x, p.ldx, p.x_rows, m0 + 64 * c, p.m_dim);
                for (int c = 0; c < boxes; ++c) dy.copy(pick, sb + c * kMnChunk, p.dy, p.lddy, p.dy_rows, 64 * c, p.dy_cols);
                cp_async_commit();
                if (S > kNarrowUnderWay && fills - handed == kNarrowUnderWay) {  // (else before the next wait)
                    cp_async_wait<kNarrowUnderWay>();
                    hand_over();
                }
                x = nx;
                dy = ny;
            }
            cp_async_wait<0>();
            if (go)
                while (handed < fills) hand_over();
        }
        const int q = warp & 3, i = q * 32 + lane;
        const bool ok = warp_wait(done_bar, 0, wc, kErrEpilogueWait, lane);
        tc_fence_after();
        const uint32_t t_row = tmem_base + (uint32_t(q * 32) << 16);
        if (ok)
#pragma unroll 1
            for (int c = 0; c < width; c += 16) {
                uint32_t v[16], u[16];
                tmem_ld_16cols(t_row + uint32_t(c), v);
                if (p.half) tmem_ld_16cols(t_row + uint32_t(p.half + c), u);
                tmem_ld_wait();
                float f[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    f[j] = kb1 > kb0 ? __uint_as_float(v[j]) : 0.0f;
                    if (p.half && kb1 > kb0) f[j] += __uint_as_float(u[j]);
                    if constexpr (UNITS) f[j] *= unit;
                }
                if (p.transposed) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c + j) * 128 + i] = f[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4*>(part + i * pitch + c + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
                }
            }
        tc_fence_before();
    }
    if (splits > 1) cluster_sync();  // every part stands
    else __syncthreads();
    if (warp == kThreads / 32) {
        if (splits > 1) {
            cta_barrier_sync(1, kNarrowThreads);  // the others' reads are done
            cluster_arrive();
        }
    } else {
        // quads of neighbours: rows of the result of 128 or `width` elements
        const int of_row = p.transposed ? 32 : width / 4, quads = (p.transposed ? width : 128) * of_row;
        const float scale = begin == end ? 0.0f : p.scale ? __ldg(p.scale + g) : p.scale_all;  // (nothing's sum is zero, scaled by whatever)
        const int out_rows = p.transposed ? p.n_dim : p.m_dim - m0, out_cols = p.transposed ? p.m_dim - m0 : p.n_dim;
        uint16_t* out = p.dw + int64_t(g) * p.dw_apart + (p.transposed ? int64_t(m0) : int64_t(m0) * p.lddw);
        for (int e = int(rank) * kThreads + int(threadIdx.x); e < quads; e += splits * kThreads) {
            const int row = e / of_row, col = e % of_row * 4;
            const uint32_t at = smem0 + uint32_t(row * pitch + col) * 4u;
            float4 sum;
            if (splits == 1) {
                uint32_t a, b, c, d;
                ld_shared_v4(at, a, b, c, d);
                sum = make_float4(__uint_as_float(a), __uint_as_float(b), __uint_as_float(c), __uint_as_float(d));
            } else {
                float4 v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < splits) v[r] = ld_cluster_f32x4(at, uint32_t(r));
                sum = v[0];
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < splits) sum = make_float4(sum.x + v[r].x, sum.y + v[r].y, sum.z + v[r].z, sum.w + v[r].w);
            }
            const int have = row < out_rows ? min(4, out_cols - col) : 0;
            const uint2 w = make_uint2(round16x2(sum.x * scale, sum.y * scale, p.fp16), round16x2(sum.z * scale, sum.w * scale, p.fp16));
            uint16_t* dst = out + int64_t(row) * p.lddw + col;
            if (have == 4) {
                *reinterpret_cast<uint2*>(dst) = w;
            } else {
                const uint32_t h[4] = {w.x, w.x >> 16, w.y, w.y >> 16};
                for (int j = 0; j < have; ++j) dst[j] = uint16_t(h[j]);
            }
        }
        if (splits > 1) {
            cta_barrier_arrive(1, kNarrowThreads);
            cluster_arrive_relaxed();  // (the ninth warp's arrival orders the reads)
        }
    }
    if (splits > 1) cluster_wait();  // nobody leaves while its part is read
    else __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc<false>(tmem_base, cols);
    }
}

// Asked about, never launched (see tl_fp8.cu).
__global__ void __launch_bounds__(kNarrowThreads, 2) narrow_shape_kernel() {}

bool narrow(const GroupedDwDesc& d) { return d.half || d.n_dim <= 128; }

bool off(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

}  // namespace

std::string grouped_dw_check(const GroupedDwDesc& d) {
    constexpr int64_t kMost = INT32_MAX / 2;
    if (d.rows < 0 || d.rows > kMost || d.x.count < 0 || d.x.count > kMost || d.dy.count < 0 || d.dy.count > kMost)
        return "rows must be >= 0 and below 2^30";
    if (d.m_dim < 1 || d.n_dim < 1 || d.m_dim > kMost || d.n_dim > kMost) return "the weight's sizes must be >= 1 and below 2^30";
    if (d.groups < 1 || d.groups > kMaxGroupsSeen - 1) return "groups must be 1..1024";
    if (d.type != TL_TYPE_BF16 && d.type != TL_TYPE_F16) return "the product takes bf16 or fp16 (tl_type)";
    if (!d.offsets || !d.err || off(d.offsets, 4) || off(d.err, 4)) return "offsets or err is null or not 4-byte aligned";
    const int64_t inner = d.transposed ? d.m_dim : d.n_dim, outer = d.transposed ? d.n_dim : d.m_dim;
    if (!d.dw || off(d.dw, 16)) return "dw is null or not 16-byte aligned";
    if (d.lddw % 8 || d.dw_apart % 8) return "leading dimensions must be multiples of 8 elements";
    if (d.lddw < inner || (d.groups > 1 && d.dw_apart < (outer - 1) * d.lddw + inner)) return "dw's leading dimension or distance is smaller than a row or matrix";
    if (d.lddw >= (int64_t(1) << 38) || d.dw_apart >= (int64_t(1) << 38)) return "a leading dimension is too large";
    if (d.rows == 0) return {};
    if (!d.x.at || !d.dy.at) return "null pointer";
    if (off(d.x.at, 16) || off(d.dy.at, 16)) return "operand pointers must be 16-byte aligned";
    if (d.x.ld % 8 || d.dy.ld % 8) return "leading dimensions must be multiples of 8 elements";
    if (d.x.ld < d.m_dim || d.dy.ld < (d.half ? 2 * d.half : d.n_dim)) return "a leading dimension is smaller than a row";
    if (d.x.ld >= (int64_t(1) << 38) || d.dy.ld >= (int64_t(1) << 38)) return "a leading dimension is too large";
    if (d.x.count < 1 || d.dy.count < 1 || (!d.x.index && d.x.count < d.rows) || (!d.dy.index && d.dy.count < d.rows)) return "x or dy has too few rows";
    if (off(d.gathered, 16)) return "the workspace is not 16-byte aligned";
    if (off(d.x.index, 4) || off(d.dy.index, 4) || off(d.scale, 4) || off(d.dy_units, 4)) return "indexes and scales must be 4-byte aligned";
    const int64_t tiles = narrow(d) ? (d.m_dim + 127) / 128 * d.groups : (d.m_dim + 255) / 256 * ((d.n_dim + 255) / 256);  // of all groups, or of one
    if (tiles > INT32_MAX) return "too many tiles";
    return {};
}

cudaError_t grouped_dw_launch(const GroupedDwDesc& d, int num_sms, cudaStream_t stream, std::string* why) {
    const int64_t outer = d.transposed ? d.n_dim : d.m_dim;
    if (d.rows == 0) {  // sums of nothing
        for (int64_t g = 0; g < d.groups; ++g) {
            const cudaError_t e = cudaMemset2DAsync(static_cast<uint16_t*>(d.dw) + g * d.dw_apart, size_t(d.lddw) * 2, 0,
                                                    size_t(d.transposed ? d.m_dim : d.n_dim) * 2, size_t(outer), stream);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    DwParams p{};
    p.rows = int32_t(d.rows);
    p.m_dim = int32_t(d.m_dim);
    p.n_dim = int32_t(d.n_dim);
    p.groups = int32_t(d.groups);
    p.offsets = d.offsets;
    p.x_index = d.x.index;
    p.dy_index = d.dy.index;
    p.x = static_cast<const uint16_t*>(d.x.at);
    p.dy = static_cast<const uint16_t*>(d.dy.at);
    p.ldx = d.x.ld;
    p.lddy = d.dy.ld;
    p.x_rows = int32_t(d.x.count);
    p.dy_rows = int32_t(d.dy.count);
    p.dy_cols = d.half ? 2 * d.half : int32_t(d.n_dim);
    p.scale = d.scale;
    p.scale_all = d.scale_all;
    p.fp16 = d.type == TL_TYPE_F16 ? 1 : 0;
    p.half = d.half;
    p.dy_units = d.dy_units;
    p.dw = static_cast<uint16_t*>(d.dw);
    p.lddw = d.lddw;
    p.dw_apart = d.dw_apart;
    p.transposed = d.transposed ? 1 : 0;
    p.err = d.err;
    p.timeout_ns = 2000000000ull;
    cudaError_t e;
    if (narrow(d)) {
        p.num_m = int32_t((d.m_dim + 127) / 128);
        p.n = d.half ? 2 * d.half : int32_t((d.n_dim + 15) / 16 * 16);
        p.idesc = idesc_16(128, true, true, p.fp16 != 0);
        const int stages = narrow_stages(p.n);
        const size_t smem = size_t(stages) * narrow_stage(p.n) + kNarrowFixed;
        const int64_t units = int64_t(p.num_m) * d.groups, blocks = (d.rows / d.groups + kBlockK - 1) / kBlockK;
        int splits = 1, per_sm = 0, clusters = 0;
        const void* shape = reinterpret_cast<const void*>(narrow_shape_kernel);
        e = ctas_per_sm(shape, kNarrowThreads, smem, &per_sm);
        while (e == cudaSuccess && splits < 8 && units * splits * 2 <= 2 * num_sms && blocks >= 4 * splits) {
            e = clusters_at_a_time(shape, kNarrowThreads, smem, 2 * splits, &clusters);
            if (e != cudaSuccess || units > clusters) break;
            splits *= 2;
        }
        if (e != cudaSuccess) return e;
        e = launch_in_clusters(d.dy_units ? grouped_dw_narrow_kernel<true> : grouped_dw_narrow_kernel<false>, dim3(unsigned(units * splits)), kNarrowThreads,
                               splits, smem, false, stream, p, splits, stages);
    } else {
        if (d.transposed) return cudaErrorInvalidValue;
        const int64_t apart = d.groups > 1 ? d.dw_apart : outer * d.lddw;
        if (d.dy.index) return cudaErrorInvalidValue;
        RowsOperand x = d.x, dy = d.dy;
        if (x.index) {
            if (!d.gathered) return cudaErrorInvalidValue;
            e = pick_rows_launch(d.x, d.rows, d.m_dim, d.gathered, stream);
            if (e != cudaSuccess) return e;
            x = {d.gathered, picked_ld(d.m_dim), d.rows, nullptr};
        }
        x.count = dy.count = d.rows;  // no row past the last place is there
        DwMaps maps;
        if (!rows_map(&maps.x, d.type, x, d.m_dim, kBlockK, why) || !rows_map(&maps.dy, d.type, dy, d.n_dim, kBlockK, why) ||
            !rows_map(&maps.x_rows, d.type, x, d.m_dim, 1, why) || !rows_map(&maps.dy_rows, d.type, dy, d.n_dim, 1, why) ||
            !swizzled_map(&maps.dw, map_type16(d.type), 2, d.dw, uint64_t(d.n_dim), uint64_t(d.m_dim), uint64_t(d.lddw), 32, why, uint64_t(d.groups), uint64_t(apart)))
            return cudaErrorInvalidValue;
        p.num_m = int32_t((d.m_dim + 255) / 256);
        p.num_n = int32_t((d.n_dim + 255) / 256);
        p.idesc = idesc_16(256, true, true, p.fp16 != 0);
        const int64_t tiles = int64_t(p.num_m) * p.num_n * d.groups;
        const unsigned grid = 2 * unsigned(std::min<int64_t>(tiles, std::max(1, num_sms / 2)));
        e = launch_in_clusters(grouped_dw_kernel, dim3(grid), kThreads, 2, kSmem, false, stream, maps, p);
    }
    if (e != cudaSuccess && why && why->empty()) *why = std::string("kernel launch: ") + cudaGetErrorString(e);
    return e;
}

}  // namespace tl
