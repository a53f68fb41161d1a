// tl_fp8.cu -- the three products of a linear layer on 8-bit operands with a
// power-of-two scale for each block of 128 along the reduction:
//
//   D[i, j] = bf16( sum_b 2^(sa[i, b] + sb[j, b] - 254) sum_{k in block b} A[i, k] B[j, k] )
//
// The scales go to the tensor core with the operands: tcgen05.mma's
// block-scaled form multiplies each 32 products by the two scales' powers of
// two and adds them in fp32, so there is nothing to do between the blocks and
// the accumulator stays in tensor memory for the whole reduction.  (A scale of
// 128 elements is the same byte in four consecutive MMAs.)
//
// gemm (many rows): CTA pairs, 256 x 256 output tiles, K-blocks of 128 bytes:
//   warp 0      TMA producer: 128-row slices of A and B into a shared ring of
//               three stages of two K-blocks
//   warp 1      MMA issuer (first CTA): scales shared -> tensor memory once in
//               four K-blocks, then four MMAs of K = 32 a K-block.  At this
//               rate the issuing thread's own time counts: a commit takes it
//               about 150 ns, half of a K-block's MMAs, so a stage holds two
//   warp 2      allocates the tensor memory
//   warp 3      gathers the scales of four K-blocks (a 32-bit word for each
//               row) into the layout that the copy to tensor memory takes
//   warps 4..7  epilogue: fp32 accumulator -> bf16 -> TMA store
// Two 256-column accumulators and the scales need more than the 512 columns of
// tensor memory, so the accumulators share 48: the epilogue reads those first,
// and the next tile's MMAs wait for no more than that.
//
// few (up to 128 tokens): the weight's bytes are the work, so the weight is the
// MMA's A side, 128 of its rows (columns) a CTA, and the tokens are N = 16 to
// 128 columns.  The CTAs of a cluster share a reduction: each sums its part in
// its tensor memory, and they add the parts up through distributed shared
// memory in a fixed order.
//
// Every wait is bounded; see tl_gemm.cu, whose error protocol this shares but for
// one thing: the error word is many launches', so its bits end no wait here.
#include "tl_fp8.h"
#include "tl_gemm.h"
#include "tl_kernel_common.cuh"
#include "tl_launch.h"
#include "tl_tmap.h"

#include "tiled_linear.h"

#include <algorithm>
#include <climits>
#include <type_traits>

namespace tl {
namespace {

using namespace kc;

constexpr int kFp8BlockK = 128;     // one K-block: one scale block, one 128-byte swizzle row
constexpr int kChunkBlocks = 4;     // K-blocks whose scales share a 32-bit word
constexpr int kStageBlocks = 2;      // K-blocks of a stage
constexpr int kStagesPair = 3;
constexpr uint32_t kStageHalf = 128 * 128;  // one operand's K-block of a CTA: 128 rows (or reduction indices) of 128 bytes
constexpr int kBatch = 4;           // chunks whose scales are handed over at once,
constexpr int kSfSlots = 2;         // and how many batches shared memory holds
constexpr uint32_t kSfA = 512, kSfB = 1024, kSfChunk = kSfA + kSfB, kSfSlot = kBatch * kSfChunk;
constexpr uint32_t kAcc1 = 208;     // columns: accumulators at 0 and 208, 256 each,
constexpr uint32_t kSfCols = 464;   // then four sets of 4 + 8 scale columns
constexpr uint32_t kSfSet = 12, kSfSets = 4;

// tcgen05.mma, 8-bit operands with one scale byte per 32 reduction elements.
template <bool PAIR>
__device__ __forceinline__ void umma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}
// 32 lanes x 16 bytes of shared memory to 4 tensor-memory columns, the same in
// all four quarters of the lanes.
template <bool PAIR>
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint32_t saddr) {
    // no swizzle: 8-row groups of 16-byte rows, 128 bytes apart
    const uint64_t desc = uint64_t((saddr >> 4) & 0x3fffu) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Instruction descriptor of kind::mxf8f6f4: scale id of B (bits 4-5), formats
// of A (7-9) and B (10-12; 0 = e4m3, 1 = e5m2), majors (15, 16; 1 = MN),
// N >> 3 (17-22), scale type (23; 1 = a power of two in 8 bits), M >> 4 at
// 24-28, scale id of A (29-30).
__host__ __device__ constexpr uint32_t idesc_fp8(int m, int n, bool a_mn, bool b_mn, int fa, int fb) {
    return (uint32_t(fa) << 7) | (uint32_t(fb) << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (uint32_t(n >> 3) << 17) | (1u << 23) | (uint32_t(m >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_scale_id(uint32_t idesc, uint32_t id) { return idesc | (id << 4) | (id << 29); }

__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Wait until the kernel before this one has completed and its writes are
// visible (at once, unless the launch allowed this one to begin early).
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// wait_bounded_cluster, without its reading of the clock where the phase is
// over already: that takes longer than four K-blocks' MMAs.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, const SharedWaitCtx& w, int32_t code) {
    return mbar_try_wait_cluster(bar, parity) || wait_bounded_cluster(bar, parity, w, code);
}

// Step j (32 reduction elements) of a 128 x 128-byte operand.
__device__ __forceinline__ uint64_t fp8_desc(bool mn, uint32_t base, int j) {
    return mn ? smem_desc_sw128(base + uint32_t(j) * 4096u, 16384, 1024) : smem_desc_sw128(base + uint32_t(j) * 32u, 16, 1024);
}

// Scales of an operand, as words of four K-blocks' bytes: [chunk][dim] words
// for vectors, bytes at (i / 128) * i_step + (k / 128) * k_step for tiles.
struct Scales {
    const void* p;
    int64_t i_step, k_step;
    int32_t dim, tiles;
};

struct Fp8Params {
    int32_t m_dim, n_dim, k_dim;
    int32_t num_m, num_n, num_k, num_tiles;
    int32_t raster, group, stream_shared;
    uint32_t idesc;
    Scales a, b;
    int32_t* err;
    uint64_t timeout_ns;
};

// A word that a kernel which may still run when this one begins has written, read
// after the wait for it: __ldg is for what no one writes while this kernel runs.
__device__ __forceinline__ uint32_t ld_written_u32(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// The words of ROWS indices from i0 on, 32 apart (lane l has i0 + l, i0 + 32 + l,
// ...), for chunk c: 1.0 (127) outside the matrix.  EARLY: the vectors' words may
// be what the kernel ahead writes (the tiles' bytes never are: Fp8GemmDesc::early).
template <int ROWS, bool EARLY>
__device__ __forceinline__ void scale_words(const Scales& s, int i0, int c, int num_k, int lane, uint32_t* w) {
    if (s.tiles) {  // one word for 128 indices, the same in all lanes
#pragma unroll
        for (int t = 0; t < ROWS / 4; ++t) {
            uint32_t v = 0x7f7f7f7fu;
            if (i0 + 128 * t < s.dim) {
                const uint8_t* at = static_cast<const uint8_t*>(s.p) + int64_t(i0 / 128 + t) * s.i_step + int64_t(c) * kChunkBlocks * s.k_step;
                const int have = num_k - c * kChunkBlocks;
                v = 0;
#pragma unroll
                for (int j = 0; j < kChunkBlocks; ++j) v |= (j < have ? uint32_t(__ldg(at + j * s.k_step)) : 127u) << (8 * j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * t + j] = v;
        }
    } else {
        const uint32_t* at = static_cast<const uint32_t*>(s.p) + int64_t(c) * s.dim + i0 + lane;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            w[j] = 0x7f7f7f7fu;
            if (i0 + 32 * j + lane < s.dim) w[j] = EARLY ? ld_written_u32(at + 32 * j) : __ldg(at + 32 * j);
        }
    }
}

constexpr size_t kSmemPair = size_t(kStagesPair) * 2 * kStageBlocks * kStageHalf + 4 * kEpiBuf + kSfSlots * kSfSlot + kBarBytes + 1024;
static_assert(kSmemPair <= 232448, "shared memory budget");

// The lane's row of 64 accumulator columns, as bf16 pairs.
__device__ __forceinline__ void read_bf16(uint32_t taddr, uint32_t (&w)[32]) {
    uint32_t v[2][32];
    tmem_ld_32cols(taddr, v[0]);
    tmem_ld_32cols(taddr + 32u, v[1]);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) w[j] = pack_bf16x2(__uint_as_float(v[j / 16][2 * j % 32]), __uint_as_float(v[j / 16][2 * j % 32 + 1]));
}
// The warp's 32 rows of them through its staging box (128B-swizzled) to the result.
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t box, const uint32_t (&w)[32], int col, int row, int lane) {
    if (lane == 0) bulk_wait_group_read<0>();  // the box's last store has read it
    __syncwarp();
    const uint32_t row_addr = box + uint32_t(lane) * 128u;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        st_shared_v4(row_addr + ((uint32_t(j) ^ (uint32_t(lane) & 7u)) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(map, box, col, row);
        bulk_commit_group();
    }
}

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_d, const Fp8Params p) {
    const SharedWaitCtx wc{p.err, p.timeout_ns};
    constexpr int S = kStagesPair;
    constexpr uint32_t kStage = 2 * kStageBlocks * kStageHalf;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem0 = smem_addr(smem);
    const uint32_t epi_base = smem0 + S * kStage, sf0 = epi_base + 4 * kEpiBuf;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * kStage + 4 * kEpiBuf + kSfSlots * kSfSlot);
    const uint32_t bar0 = smem_addr(bars);
    // full[s], empty[s], sf_full[q], sf_empty[q], tmem_full[a], shared columns
    // read, drain.  full, sf_full and the shared columns' barrier are used in
    // the first CTA only.
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (S + s); };
    auto sf_full_bar = [&](uint32_t q) { return bar0 + 8u * (2 * S + q); };
    auto sf_empty_bar = [&](uint32_t q) { return bar0 + 8u * (2 * S + kSfSlots + q); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * S + 2 * kSfSlots + a); };
    const uint32_t tread_bar = bar0 + 8u * (2 * S + 2 * kSfSlots + 2);
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 2 * kSfSlots + 3);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 2 * kSfSlots + 4);
    static_assert((2 * S + 2 * kSfSlots + 4) * 8 + 4 <= int(kBarBytes), "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int first_tile = int(cluster_id_x()), tile_step = int(cluster_count_x());
    const int chunks = (p.num_k + kChunkBlocks - 1) / kChunkBlocks;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int q = 0; q < kSfSlots; ++q) {
            mbar_init(sf_full_bar(q), 2);  // the scale warps of both CTAs
            mbar_init(sf_empty_bar(q), 1);
        }
        for (int a = 0; a < 2; ++a) mbar_init(tfull_bar(a), 1);
        mbar_init(tread_bar, 8);  // the epilogue warps of both CTAs
        mbar_init(drain_bar, 1);
        mbar_init_fence();
    }
    if (warp == 2) {
        tmem_alloc<true>(smem_addr(tmem_slot), 512);
        tmem_relinquish<true>();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_map(&map_a);
            tma_prefetch_map(&map_b);
            const uint64_t pol_s = p.stream_shared ? l2_policy_evict_normal() : l2_policy_evict_first();
            const uint64_t pol_a = p.raster == 0 ? l2_policy_evict_last() : pol_s;
            const uint64_t pol_b = p.raster == 0 ? pol_s : l2_policy_evict_last();
            uint32_t fills = 0;
            bool ok = true;
            for (int tile = first_tile; ok && tile < p.num_tiles; tile += tile_step) {
                int mb, nb;
                tile_coords(tile, p.num_m, p.num_n, p.raster, p.group, mb, nb);
                const int m0 = mb * 256 + int(rank) * 128, n0 = nb * 256 + int(rank) * 128;
                for (int kb = 0; kb < p.num_k; kb += kStageBlocks, ++fills) {
                    const uint32_t s = fills % S;
                    if (!wait_bounded(empty_bar(s), ((fills / S) & 1u) ^ 1u, wc, kErrProducerWait)) {
                        ok = false;
                        break;
                    }
                    if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * kStage);
                    const uint32_t fb = map_to_rank(full_bar(s), 0);
#pragma unroll
                    for (int j = 0; j < kStageBlocks; ++j) {  // a K-block past the end loads zeros
                        const uint32_t sa = smem0 + s * kStage + uint32_t(2 * j) * kStageHalf, sb = sa + kStageHalf;
                        const int k0 = (kb + j) * kFp8BlockK;
                        if (A_MN) tma_load_2d_pair_hint(sa, &map_a, fb, m0, k0, pol_a);
                        else tma_load_2d_pair_hint(sa, &map_a, fb, k0, m0, pol_a);
                        if (B_MN) tma_load_2d_pair_hint(sb, &map_b, fb, n0, k0, pol_b);
                        else tma_load_2d_pair_hint(sb, &map_b, fb, k0, n0, pol_b);
                    }
                }
            }
            if (leader) {  // loads must land before the CTAs may exit
                const uint32_t outstanding = fills < uint32_t(S) ? fills : uint32_t(S);
                for (uint32_t j = 0; j < outstanding; ++j) {
                    const uint32_t f = fills - 1 - j;
                    wait_bounded(full_bar(f % S), (f / S) & 1u, wc, kErrDrainWait, false);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            uint32_t fills = 0, chunk = 0;
            const int tiles = first_tile < p.num_tiles ? (p.num_tiles - 1 - first_tile) / tile_step + 1 : 0;
            const uint32_t all_chunks = uint32_t(tiles) * uint32_t(chunks);
            // The next chunk's scales to their columns, in the middle of the
            // MMAs of the chunk before it: the copy runs in the tensor pipe's
            // order, and placed directly before its own MMAs it holds them up.
            uint32_t copied = 0, batch = 0;
            int c = 0;  // the chunk's place in its tile
            auto copy_scales = [&] {
                if (copied >= all_chunks) return true;
                // The MMAs that last read this set of columns are done: they
                // are three chunks and more back, so at least three stages,
                // and this thread has just seen the stage full that those
                // three stages' ring slot was given back for.
                static_assert(kSfSets >= S + 1, "a set outlives the stages in flight");
                const uint32_t set = copied % kSfSets;
                if (c % kBatch == 0 && !wait_cluster(sf_full_bar(batch % kSfSlots), (batch / kSfSlots) & 1u, wc, kErrMmaWaitFull))
                    return false;
                tc_fence_after();
                const uint32_t to = tmem_base + kSfCols + set * kSfSet;
                const uint32_t src = sf0 + (batch % kSfSlots) * kSfSlot + uint32_t(c % kBatch) * kSfChunk;
                tmem_copy_scales<true>(to, src);
                tmem_copy_scales<true>(to + 4, src + kSfA);
                tmem_copy_scales<true>(to + 8, src + kSfA + 512);
                ++copied;
                if (++c == chunks || c % kBatch == 0) {
                    umma_commit_pair(sf_empty_bar(batch % kSfSlots), 0x3);
                    ++batch;
                    if (c == chunks) c = 0;
                }
                return true;
            };
            bool ok = copy_scales();
            int it = 0;
            for (int tile = first_tile; ok && tile < p.num_tiles; tile += tile_step, ++it) {
                // the other accumulator's tile has left the shared columns
                // (and the tile before that, all of this accumulator)
                if (it > 0 && !wait_bounded(tread_bar, uint32_t(it - 1) & 1u, wc, kErrMmaWaitTmem)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (it & 1 ? kAcc1 : 0u);
                for (int kb = 0; kb < p.num_k; kb += kStageBlocks, ++fills) {
                    const uint32_t set = tmem_base + kSfCols + (chunk % kSfSets) * kSfSet;
                    const uint32_t s = fills % S;
                    if (!wait_bounded(full_bar(s), (fills / S) & 1u, wc, kErrMmaWaitFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const bool first = kb % kChunkBlocks == 0;  // stage of its chunk
#pragma unroll
                    for (int i = 0; i < kStageBlocks; ++i) {
                        const uint32_t sa = smem0 + s * kStage + uint32_t(2 * i) * kStageHalf, sb = sa + kStageHalf;
                        const uint32_t idesc = with_scale_id(p.idesc, uint32_t(i) + (first ? 0u : uint32_t(kStageBlocks)));
#pragma unroll
                        for (int j = 0; j < kFp8BlockK / 32; ++j)
                            umma_fp8<true>(d_tmem, fp8_desc(A_MN, sa, j), fp8_desc(B_MN, sb, j), idesc, set, set + 4,
                                           (kb | i | j) != 0 ? 1u : 0u);
                    }
                    umma_commit_pair(empty_bar(s), 0x3);
                    if (first && !copy_scales()) {
                        ok = false;
                        break;
                    }
                    if (!first || kb + kStageBlocks >= p.num_k) ++chunk;
                }
                if (ok) umma_commit_pair(tfull_bar(it & 1), 0x3);
            }
            umma_commit_pair(drain_bar, 0x3);
            wait_bounded(drain_bar, 0, wc, kErrDrainWait, false);
        }
    } else if (warp == 3) {
        // ---------------- scales: this CTA's 128 rows of A, all 256 of B ----------------
        // A batch at a time: the loads of four chunks are in flight together,
        // and one proxy fence and one arrival hand all of them over.
        uint32_t batch = 0;
        bool ok = true;
        for (int tile = first_tile; ok && tile < p.num_tiles; tile += tile_step) {
            int mb, nb;
            tile_coords(tile, p.num_m, p.num_n, p.raster, p.group, mb, nb);
            const int m0 = mb * 256 + int(rank) * 128, n0 = nb * 256;
            for (int c0 = 0; c0 < chunks; c0 += kBatch, ++batch) {
                uint32_t w[kBatch][12];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (c0 + i >= chunks) break;
                    scale_words<4, false>(p.a, m0, c0 + i, p.num_k, lane, w[i]);
                    scale_words<8, false>(p.b, n0, c0 + i, p.num_k, lane, w[i] + 4);
                }
                const uint32_t q = batch % kSfSlots;
                if (!warp_wait(sf_empty_bar(q), ((batch / kSfSlots) & 1u) ^ 1u, wc, kErrProducerWait, lane)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (c0 + i >= chunks) break;
                    const uint32_t dst = sf0 + q * kSfSlot + uint32_t(i) * kSfChunk + uint32_t(lane) * 16;
                    st_shared_v4(dst, w[i][0], w[i][1], w[i][2], w[i][3]);
                    st_shared_v4(dst + kSfA, w[i][4], w[i][5], w[i][6], w[i][7]);
                    st_shared_v4(dst + kSfA + 512, w[i][8], w[i][9], w[i][10], w[i][11]);
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(sf_full_bar(q), 0));
            }
        }
    } else if (warp >= kFirstEpilogueWarp) {
        const int q = warp & 3;
        const uint32_t box = epi_base + uint32_t(q) * kEpiBuf;
        if (lane == 0) tma_prefetch_map(&map_d);
        int it = 0;
        for (int tile = first_tile; tile < p.num_tiles; tile += tile_step, ++it) {
            const uint32_t acc = it & 1;
            int mb, nb;
            tile_coords(tile, p.num_m, p.num_n, p.raster, p.group, mb, nb);
            const int row0 = mb * 256 + int(rank) * 128 + q * 32, n0 = nb * 256;
            const int have = row0 < p.m_dim ? min(4, (p.n_dim - n0 + 63) / 64) : 0;
            if (!warp_wait(tfull_bar(acc), uint32_t(it >> 1) & 1u, wc, kErrEpilogueWait, lane)) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + (uint32_t(q * 32) << 16) + (acc ? kAcc1 : 0u);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int c = acc ? i : 3 - i;  // the shared columns first
                uint32_t w[32];
                if (c < have) read_bf16(t_row + uint32_t(c) * 64u, w);
                if (i == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader) mbar_arrive(tread_bar);
                        else mbar_arrive_cluster(map_to_rank(tread_bar, 0));
                    }
                }
                if (c < have) store_box(&map_d, box, w, n0 + c * 64, row0, lane);
            }
            tc_fence_before();
            __syncwarp();
        }
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
    }

    tc_fence_before();
    cluster_sync();
    if (warp == 2) {
        tc_fence_after();
        if (!leader) wait_bounded(drain_bar, 0, wc, kErrDrainWait, false);
        tmem_dealloc<true>(tmem_base, 512);
    }
}

// ---- few tokens --------------------------------------------------------------

constexpr int kFewTokens = 128;
// A ninth warp: when the others have read the parts of the sums, it arrives with
// release semantics at the barrier past which the cluster's CTAs may leave.
constexpr int kFewThreads = kThreads + 32;
constexpr size_t kFewSmem = 112 * 1024;  // of a CTA: two share an SM
constexpr uint32_t kFewSfSlots = 4, kFewSfSlot = 1024;

template <int N>
struct Few {
    static constexpr uint32_t kStageBytes = kStageHalf + uint32_t(N) * 128;
    static constexpr uint32_t kFixed = kFewSfSlots * kFewSfSlot + kBarBytes + 1024;
    static constexpr int kStages = int((kFewSmem - kFixed) / kStageBytes);
    static constexpr size_t kSmem = size_t(kStages) * kStageBytes + kFixed;
    static constexpr uint32_t kCols = N <= 16 ? 32 : N <= 32 ? 64 : N <= 64 ? 128 : 256;  // accumulator, then two sets of 4 + 4 scales
    static_assert(N + 16 <= int(kCols) && kStages >= 3, "tensor memory, shared memory");
    static_assert(size_t(N) * 128 * 4 <= size_t(kStages) * kStageBytes, "the partial sums fit the stages");
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t local, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(local), "r"(rank)
        : "memory");
    return v;
}

// map_w: the weight, 128 of its own indices a box; map_t: the tokens, N a box.
// w: m_dim = own indices of the weight, n_dim = tokens.  out[token][index].
template <bool W_MN, int N>
__global__ void __launch_bounds__(kFewThreads, 2)
    fp8_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_t, const Fp8Params p,
                   __nv_bfloat16* out, int64_t ldo, int splits, int per) {
    using F = Few<N>;
    const SharedWaitCtx wc{p.err, p.timeout_ns};
    constexpr int S = F::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem0 = smem_addr(smem), sf0 = smem0 + S * F::kStageBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * F::kStageBytes + kFewSfSlots * kFewSfSlot);
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (S + s); };
    auto sf_full_bar = [&](uint32_t q) { return bar0 + 8u * (2 * S + q); };
    auto sf_empty_bar = [&](uint32_t q) { return bar0 + 8u * (2 * S + kFewSfSlots + q); };
    const uint32_t done_bar = bar0 + 8u * (2 * S + 2 * kFewSfSlots);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 2 * kFewSfSlots + 1);
    static_assert((2 * S + 2 * int(kFewSfSlots) + 1) * 8 + 4 <= int(kBarBytes), "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = splits > 1 ? cluster_ctarank() : 0;
    const int m0 = int(blockIdx.x / uint32_t(splits)) * 128;
    const int t0 = int(blockIdx.y) * N, tokens = min(N, p.n_dim - t0);  // this CTA's block of tokens
    const int kb0 = int(rank) * per, kb1 = min(p.num_k, kb0 + per);  // this CTA's K-blocks, perhaps none

    if (threadIdx.x == 0) {
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_t);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (uint32_t q = 0; q < kFewSfSlots; ++q) {
            mbar_init(sf_full_bar(q), 1);
            mbar_init(sf_empty_bar(q), 1);
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
        if (lane == 0) {
            // The weight is there before the kernel ahead of this one began
            // (Fp8GemmDesc::early); the tokens may be what that one makes.
            auto load_w = [&](int kb, uint32_t s) {
                const int k0 = kb * kFp8BlockK;
                if (W_MN) tma_load_2d(smem0 + s * F::kStageBytes, &map_w, full_bar(s), m0, k0);
                else tma_load_2d(smem0 + s * F::kStageBytes, &map_w, full_bar(s), k0, m0);
            };
            const int ahead = min(S, kb1 - kb0);
            for (int i = 0; i < ahead; ++i) {
                mbar_arrive_expect_tx(full_bar(i), F::kStageBytes);
                load_w(kb0 + i, i);
            }
            grid_dependency_wait();
            uint32_t fills = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++fills) {
                const uint32_t s = fills % S;
                if (int(fills) >= ahead) {
                    if (!wait_bounded(empty_bar(s), ((fills / S) & 1u) ^ 1u, wc, kErrProducerWait)) break;
                    mbar_arrive_expect_tx(full_bar(s), F::kStageBytes);
                    load_w(kb, s);
                }
                tma_load_2d(smem0 + s * F::kStageBytes + kStageHalf, &map_t, full_bar(s), kb * kFp8BlockK, t0);
            }
            const uint32_t outstanding = fills < uint32_t(S) ? fills : uint32_t(S);
            for (uint32_t j = 0; j < outstanding; ++j) {
                const uint32_t f = fills - 1 - j;
                wait_bounded(full_bar(f % S), (f / S) & 1u, wc, kErrDrainWait, false);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t fills = 0, chunk = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++fills) {
                const uint32_t id = uint32_t(kb) % kChunkBlocks, q = chunk % kFewSfSlots;
                const uint32_t set = tmem_base + N + (chunk & 1u) * 8u;
                if (id == 0 || kb == kb0) {
                    // the MMAs that last read this set are done
                    if (chunk >= 2 && !wait_bounded(sf_empty_bar((chunk - 2) % kFewSfSlots), ((chunk - 2) / kFewSfSlots) & 1u, wc, kErrMmaWaitTmem))
                        break;
                    if (!wait_bounded(sf_full_bar(q), (chunk / kFewSfSlots) & 1u, wc, kErrMmaWaitFull)) break;
                    tc_fence_after();
                    tmem_copy_scales<false>(set, sf0 + q * kFewSfSlot);
                    tmem_copy_scales<false>(set + 4, sf0 + q * kFewSfSlot + 512);
                }
                const uint32_t s = fills % S;
                if (!wait_bounded(full_bar(s), (fills / S) & 1u, wc, kErrMmaWaitFull)) break;
                tc_fence_after();
                const uint32_t sa = smem0 + s * F::kStageBytes, sb = sa + kStageHalf;
                const uint32_t idesc = with_scale_id(p.idesc, id);
#pragma unroll
                for (int j = 0; j < kFp8BlockK / 32; ++j)
                    umma_fp8<false>(tmem_base, fp8_desc(W_MN, sa, j), fp8_desc(false, sb, j), idesc, set, set + 4,
                                    (kb != kb0 || j) ? 1u : 0u);
                umma_commit(empty_bar(s));
                if (id == kChunkBlocks - 1 || kb == kb1 - 1) {
                    umma_commit(sf_empty_bar(q));
                    ++chunk;
                }
            }
            umma_commit(done_bar);
            wait_bounded(done_bar, 0, wc, kErrDrainWait, false);
        }
    } else if (warp == 3) {
        grid_dependency_wait();
        uint32_t chunk = 0;
        if (kb1 > kb0)
            for (int c = kb0 / kChunkBlocks; c <= (kb1 - 1) / kChunkBlocks; ++c, ++chunk) {
                uint32_t w[8];
                scale_words<4, true>(p.a, m0, c, p.num_k, lane, w);
                scale_words<4, true>(p.b, t0, c, p.num_k, lane, w + 4);
                const uint32_t q = chunk % kFewSfSlots, dst = sf0 + q * kFewSfSlot + uint32_t(lane) * 16;
                if (!warp_wait(sf_empty_bar(q), ((chunk / kFewSfSlots) & 1u) ^ 1u, wc, kErrProducerWait, lane)) break;
                st_shared_v4(dst, w[0], w[1], w[2], w[3]);
                st_shared_v4(dst + 512, w[4], w[5], w[6], w[7]);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(sf_full_bar(q));
            }
    } else if (warp >= kFirstEpilogueWarp && warp < kThreads / 32) {
        grid_dependency_wait();  // (the result may be what the kernel before this one reads)
        const int q = warp & 3, i = q * 32 + lane;
        const bool ok = warp_wait(done_bar, 0, wc, kErrEpilogueWait, lane);
        tc_fence_after();
        const uint32_t t_row = tmem_base + (uint32_t(q * 32) << 16);
        float* part = reinterpret_cast<float*>(smem);  // [token][128], once the stages are done with
        constexpr int kStep = N < 32 ? N : 32;
        if (ok)
#pragma unroll 1
            for (int c = 0; c < tokens; c += kStep) {
                uint32_t v[kStep];
                if constexpr (kStep == 32) tmem_ld_32cols(t_row + uint32_t(c), v);
                else tmem_ld_16cols(t_row + uint32_t(c), v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < kStep; ++j)
                    if (c + j < tokens) {
                        const float f = kb1 > kb0 ? __uint_as_float(v[j]) : 0.0f;
                        if (splits > 1) part[(c + j) * 128 + i] = f;
                        else if (m0 + i < p.m_dim) out[int64_t(t0 + c + j) * ldo + m0 + i] = __float2bfloat16_rn(f);
                    }
            }
        tc_fence_before();
    }
    if (splits > 1) {
        cluster_sync();  // every part stands
        if (warp == kThreads / 32) {
            cta_barrier_sync(1, kFewThreads);  // the others' reads are done
            cluster_arrive();
        } else {
            // Four outputs of a token at a time; at most this many of a thread,
            // with two CTAs.  All are read and summed before one is written:
            // nobody waits for the writes.
            constexpr int kMine = N * 32 / (2 * kThreads);
            uint2 w[kMine];
            const int e0 = int(rank) * kThreads + int(threadIdx.x), step = splits * kThreads;
#pragma unroll
            for (int u = 0; u < kMine; ++u) {
                const int e = e0 + u * step;
                if (e >= tokens * 32) break;
                float4 v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < splits) v[r] = ld_cluster_f32x4(smem0 + uint32_t(e / 32 * 128 + e % 32 * 4) * 4u, uint32_t(r));
                float4 sum = v[0];
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < splits) sum = make_float4(sum.x + v[r].x, sum.y + v[r].y, sum.z + v[r].z, sum.w + v[r].w);
                w[u] = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
            }
            cta_barrier_arrive(1, kFewThreads);
            cluster_arrive_relaxed();  // (the ninth warp's arrival orders the reads)
#pragma unroll
            for (int u = 0; u < kMine; ++u) {
                const int e = e0 + u * step, i = e % 32 * 4;
                if (e >= tokens * 32) break;
                __nv_bfloat16* dst = out + int64_t(t0 + e / 32) * ldo + m0 + i;
                if (m0 + i + 4 <= p.m_dim) {  // (rows of the result start on 16 bytes, so i does on 8)
                    *reinterpret_cast<uint2*>(dst) = w[u];
                } else {
                    const uint32_t h[4] = {w[u].x, w[u].x >> 16, w[u].y, w[u].y >> 16};
                    for (int j = 0; j < 4; ++j)
                        if (m0 + i + j < p.m_dim) dst[j] = __ushort_as_bfloat16(uint16_t(h[j]));
                }
            }
        }
        cluster_wait();  // nobody leaves while its part is read
    } else {
        __syncthreads();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc<false>(tmem_base, F::kCols);
    }
}

bool map_operand(CUtensorMap* map, const Fp8Operand& o, int64_t dim, int64_t k, uint32_t box_rows, std::string* why) {
    return o.mn_major ? swizzled_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.q, uint64_t(dim), uint64_t(k), uint64_t(o.ld), 128, why)
                      : swizzled_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.q, uint64_t(k), uint64_t(dim), uint64_t(o.ld), box_rows, why);
}

Scales scales_of(const Fp8Operand& o, int64_t dim) {
    return Scales{o.scale, o.mn_major ? 1 : o.tile_cols, o.mn_major ? o.tile_cols : 1, int32_t(dim), o.tiles ? 1 : 0};
}

template <typename T>
struct Same {
    using type = T;
};
// early: the kernel may begin before the one ahead of it in the stream has
// completed (it waits for that where it has to).
template <typename... A>
cudaError_t launch_clusters(void (*kern)(A...), dim3 grid, int threads, int cluster, size_t smem, bool early, cudaStream_t stream,
                            typename Same<A>::type... args) {
    int per_sm = 0;
    const cudaError_t e = ctas_per_sm(reinterpret_cast<const void*>(kern), threads, smem, &per_sm);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Asked about, never launched: how many clusters of fp8_few_kernel's threads and
// shared memory run at a time.  For a kernel that uses tensor memory the runtime
// answers for one CTA an SM, whatever it allocates; two of fp8_few_kernel fit
// (twice its kCols are at most 512 columns, and its launch bounds keep its
// registers to what two allow) and are seen to run.
__global__ void __launch_bounds__(kFewThreads, 2) few_shape_kernel() {}

template <bool W_MN, int N>
cudaError_t launch_few(const CUtensorMap& mw, const CUtensorMap& mt, Fp8Params p, const Fp8GemmDesc& g, int num_sms, cudaStream_t stream) {
    p.idesc = idesc_fp8(128, N, W_MN, false, g.b.format, g.a.format);
    const int tiles = (p.m_dim + 127) / 128;
    const int blocks = (p.n_dim + N - 1) / N;
    // CTAs of a cluster: as many as two an SM allow, with two K-blocks each and
    // all clusters at a time.  One token, us, with 2 / 4 / 8: 8192 x 1024 (8
    // tiles) 15.5 / 10.0 / 7.7, 16384 x 4736 (37) 27.6 / 17.5 / 23.1, 25600 x 6400
    // (50) 40.9 / 29.1 / 34.5, 8192 x 8192 (64) 16.8 / 14.9 / 18.6, 8192 x 9728
    // (76) 17.5 / 23.1 / 23.9.
    int splits = 1, per_sm = 0, clusters = 0;
    const void* shape = reinterpret_cast<const void*>(few_shape_kernel);
    cudaError_t e = ctas_per_sm(shape, kFewThreads, Few<N>::kSmem, &per_sm);
    while (e == cudaSuccess && splits < 8 && int64_t(tiles) * blocks * splits * 2 <= 2 * num_sms && p.num_k >= 4 * splits) {
        e = clusters_at_a_time(shape, kFewThreads, Few<N>::kSmem, 2 * splits, &clusters);
        if (e != cudaSuccess || int64_t(tiles) * blocks > clusters) break;
        splits *= 2;
    }
    if (e != cudaSuccess) return e;
    const int per = (p.num_k + splits - 1) / splits;
    return launch_clusters(fp8_few_kernel<W_MN, N>, dim3(unsigned(tiles * splits), unsigned(blocks)), kFewThreads, splits, Few<N>::kSmem, g.early,
                           stream, mw, mt, p, static_cast<__nv_bfloat16*>(g.d), g.ldd, splits, per);
}

// The few-token kernel with the operands' sides exchanged: g.b is the weight.
cudaError_t few_launch(const Fp8GemmDesc& g, int num_sms, cudaStream_t stream, std::string* why) {
    const int n = g.m_dim <= 16 ? 16 : g.m_dim <= 32 ? 32 : g.m_dim <= 64 ? 64 : 128;
    CUtensorMap mw, mt;
    if (!map_operand(&mw, g.b, g.n_dim, g.k_dim, 128, why) || !map_operand(&mt, g.a, g.m_dim, g.k_dim, uint32_t(n), why))
        return cudaErrorInvalidValue;
    Fp8Params p{};
    p.m_dim = int32_t(g.n_dim);
    p.n_dim = int32_t(g.m_dim);
    p.k_dim = int32_t(g.k_dim);
    p.num_k = int32_t((g.k_dim + kFp8BlockK - 1) / kFp8BlockK);
    p.a = scales_of(g.b, g.n_dim);
    p.b = scales_of(g.a, g.m_dim);
    p.err = g.err;
    p.timeout_ns = 2000000000ull;
    auto run = [&](auto mn) {
        constexpr bool MN = decltype(mn)::value;
        switch (n) {
            case 16: return launch_few<MN, 16>(mw, mt, p, g, num_sms, stream);
            case 32: return launch_few<MN, 32>(mw, mt, p, g, num_sms, stream);
            case 64: return launch_few<MN, 64>(mw, mt, p, g, num_sms, stream);
            default: return launch_few<MN, 128>(mw, mt, p, g, num_sms, stream);
        }
    };
    return g.b.mn_major ? run(std::true_type{}) : run(std::false_type{});
}

}  // namespace

std::string fp8_gemm_check(const Fp8GemmDesc& g) {
    if (g.m_dim < 1 || g.n_dim < 1 || g.k_dim < 1) return "sizes must be >= 1";
    if (g.m_dim > INT32_MAX / 2 || g.n_dim > INT32_MAX / 2 || g.k_dim > INT32_MAX / 2) return "size too large";
    if (!g.a.q || !g.b.q || !g.a.scale || !g.b.scale || !g.d || !g.err) return "null pointer";
    auto off = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (off(g.a.q, 16) || off(g.b.q, 16) || off(g.d, 16)) return "operand pointers must be 16-byte aligned";
    if (off(g.err, 4)) return "err must be 4-byte aligned";
    if (g.a.ld % 16 || g.b.ld % 16) return "leading dimensions of 8-bit matrices must be multiples of 16";
    if (g.ldd % 8) return "the result's leading dimension must be a multiple of 8";
    if (g.a.ld < (g.a.mn_major ? g.m_dim : g.k_dim) || g.b.ld < (g.b.mn_major ? g.n_dim : g.k_dim) || g.ldd < g.n_dim)
        return "a leading dimension is smaller than a row";
    for (const auto* o : {&g.a, &g.b})
        if (!o->tiles && off(o->scale, 4)) return "scales of the row and col forms must be 4-byte aligned";
    for (const auto* o : {&g.a, &g.b})
        if (o->format != TL_FP8_E4M3 && o->format != TL_FP8_E5M2) return "unknown tl_fp8_format";
    if (((g.m_dim + 255) / 256) * ((g.n_dim + 255) / 256) > INT32_MAX) return "too many output tiles";
    return {};
}

cudaError_t fp8_gemm_launch(const Fp8GemmDesc& g, int num_sms, cudaStream_t stream, std::string* why) {
    const int64_t pair_tiles = ((g.m_dim + 255) / 256) * ((g.n_dim + 255) / 256);
    // Few tokens, or fewer tiles than half the CTA pairs and a reduction long
    // enough to share: the kernel whose clusters split the reduction.  Other
    // kernel against this one, us, at K x n of the weight and T tokens: 8192 x
    // 8192, T = 256 (32 tiles) 30.3 / 25.1, T = 512 (64 tiles) 31.8 / 38.5;
    // 25600 x 6400, T = 256 (25 tiles) 72.9 / 55.4; 8192 x 1024, T = 1024 (16
    // tiles) 27.7 / 17.3; 1024 x 4096, T = 256 (16 tiles, short) 10.5 / 10.3.
    constexpr int kLongBlocks = 32;
    if (!g.a.mn_major && (g.m_dim <= kFewTokens ||
                          (pair_tiles <= num_sms / 4 && g.k_dim >= int64_t(kLongBlocks) * kFp8BlockK))) {
        const cudaError_t e = few_launch(g, num_sms, stream, why);
        if (e != cudaSuccess && why && why->empty()) *why = std::string("kernel launch: ") + cudaGetErrorString(e);
        return e;
    }
    CUtensorMap ma, mb, md;
    if (!map_operand(&ma, g.a, g.m_dim, g.k_dim, 128, why) || !map_operand(&mb, g.b, g.n_dim, g.k_dim, 128, why) ||
        !swizzled_map(&md, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.d, uint64_t(g.n_dim), uint64_t(g.m_dim), uint64_t(g.ldd), 32, why))
        return cudaErrorInvalidValue;
    Fp8Params p{};
    p.m_dim = int32_t(g.m_dim);
    p.n_dim = int32_t(g.n_dim);
    p.k_dim = int32_t(g.k_dim);
    p.num_m = int32_t((g.m_dim + 255) / 256);
    p.num_n = int32_t((g.n_dim + 255) / 256);
    p.num_k = int32_t((g.k_dim + kFp8BlockK - 1) / kFp8BlockK);
    p.num_tiles = p.num_m * p.num_n;
    const int slots = std::max(1, num_sms / 2);
    // the order is chosen by the blocks' bytes: an 8-bit reduction of k counts as a bf16 one of k / 2
    choose_tile_order(std::max<int64_t>(1, g.k_dim / 2), 256, p.num_m, p.num_n, slots, &p.raster, &p.group, &p.stream_shared);
    p.a = scales_of(g.a, g.m_dim);
    p.b = scales_of(g.b, g.n_dim);
    p.err = g.err;
    p.timeout_ns = 2000000000ull;
    p.idesc = idesc_fp8(256, 256, g.a.mn_major, g.b.mn_major, g.a.format, g.b.format);
    const int grid = 2 * std::min(p.num_tiles, slots);
    auto run = [&](auto kern) { return launch_clusters(kern, dim3(unsigned(grid)), kThreads, 2, kSmemPair, false, stream, ma, mb, md, p); };
    cudaError_t e;
    if (g.a.mn_major) e = g.b.mn_major ? run(fp8_gemm_kernel<true, true>) : cudaErrorInvalidValue;
    else e = g.b.mn_major ? run(fp8_gemm_kernel<false, true>) : run(fp8_gemm_kernel<false, false>);
    if (e != cudaSuccess && why) *why = std::string("kernel launch: ") + cudaGetErrorString(e);
    return e;
}

}  // namespace tl
