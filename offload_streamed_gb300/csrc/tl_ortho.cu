// tl_ortho.cu -- orthogonalising matrices by Newton-Schulz products, as an
// optimizer's update of a weight: for each matrix G of a stack
//
//   X = G / (|G|_F + eps);  steps times:  P = X X^T,  X = a X + (b P + c P^2) X
//
// which drives the singular values of G towards one and leaves its singular
// vectors alone.  A matrix with more rows than columns uses P = X^T X and
// X = a X + X (b P + c P^2), so P always has the short side.
//
// Bound by the tensor cores: per step 2 R^2 C flops for P (R the short side, C
// the long one), 2 R^3 for P^2 and 2 R^2 C for the update.  P and its square
// are symmetric, so only the tiles on and above the diagonal are computed and
// each is written twice, once mirrored.
//
// Two kernels share the work: large products go through CTA pairs with 256 x 256
// tiles, products of few such tiles through single CTAs with 128 x 128 tiles, a
// cluster of them sharing a reduction.  The launches follow each other closely:
// each may begin while the one before it ends, and waits for that one's results
// before it reads any.
//
// Numbers.  The iterate X is held in fp32; the products take it in fp16, whose
// 11 bits keep the result's error under that of its own rounding to bf16 (in
// bf16 operands it would be several times larger).  Once the singular values are
// near one, P is near the identity, and what is held and multiplied is
// E = P - s 1 with s = 1:
//   a X + (b P + c P^2) X = (a + b s + c s^2) X + Q X,  Q = (b + 2 c s) E + c E^2.
// With the usual coefficients both factors are small there, and so is the effect
// of rounding E and Q to fp16.  While the singular values are small a X is most of
// the result, and s = 0 leaves that part to the fp32 iterate.  So s follows the
// square of one representative singular value, 1 / sqrt(R) at first, until that
// is about one, and is 1 from there on (shift_of_step).  What the roundings but
// the last to bf16 make of the result's norm, emulated, with this s / with s = 1 /
// with s = 0 throughout: 256 x 256 0.7 / 1.1 / 1.5e-3, 512 x 512 with strong
// directions 0.6 / 2.8 / 0.5e-3, 512 x 2048 0.4 / 0.9 / 1.4e-3.  X, E and Q are
// scaled by 2^8 in fp16, far from its subnormals; |X| <= 255 is needed, which
// singular values below 255 ensure.
// Sums are fp32 in tensor memory.
#include "tl_ortho.h"
#include "tl_gemm.h"
#include "tl_kernel_common.cuh"
#include "tl_launch.h"
#include "tl_tmap.h"
#include "tl_types.cuh"

#include "tiled_linear.h"

#include <algorithm>
#include <climits>
#include <cmath>

namespace tl {
namespace {

using namespace kc;

constexpr float kUp = 256.0f, kDown = 1.0f / 256.0f;  // the fp16 operands' scale
enum Mode { GRAM = 0, SQUARE = 1, UPDATE = 2, LAST = 3 };

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void tma_load_3d_pair_hint(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int32_t x,
                                                      int32_t y, int32_t z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
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
// The launch before this one is complete and its results visible; and the next
// one may begin.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// kind::f16 with fp16 operands (formats 0) and fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

struct OrthoParams {
    int32_t m_dim, n_dim, num_k;
    int32_t num_m, num_n, per_matrix, num_tiles;  // tiles of a matrix and of all
    int32_t raster, group, stream_shared;
    float shift, k0, k1, k2, scale;
    const __half* e;  // SQUARE: E, ld and distance of a matrix
    float* x;         // UPDATE, LAST: the iterate
    int64_t ld, apart;
    void* out;        // small products: E, Q, X in fp16 or the bf16 result
    int64_t ldo, o_apart;
    int32_t splits, per;
    int32_t* err;
    uint64_t timeout_ns;
};

// Tile t of the upper triangle of an n x n grid of tiles, row by row.
__device__ __forceinline__ void triangle_coords(int t, int n, int& r, int& c) {
    // rows 0..r-1 hold r n - r (r - 1) / 2 tiles
    const float f = float(2 * n + 1);
    r = int((f - sqrtf(f * f - 8.0f * float(t))) * 0.5f);
    auto before = [n](int r) { return r * n - r * (r - 1) / 2; };
    while (r > 0 && before(r) > t) --r;
    while (before(r + 1) <= t) ++r;
    c = r + t - before(r);
}

// The maps of what a launch writes.
struct OutMaps {
    CUtensorMap half;    // fp16 (E, Q, X) or, in LAST, the bf16 result: boxes of 64 x 32 rows, swizzled
    CUtensorMap mirror;  // GRAM, SQUARE: boxes of 32 x 64 rows, not swizzled
    CUtensorMap wide;    // UPDATE: the fp32 iterate, boxes of 32 x 32 rows, swizzled
};

constexpr int kOrthoStages = 6;
constexpr uint32_t kHalfStage = 16384;  // one operand's K-block of a CTA
constexpr size_t kOrthoSmem = size_t(kOrthoStages) * 2 * kHalfStage + 8 * kEpiBuf + kBarBytes + 1024;
static_assert(kOrthoSmem <= 232448, "shared memory budget");

// What 32 columns of lane l's row (row0 + l) need from global memory.
template <int MODE>
__device__ __forceinline__ void ortho_fetch(const OrthoParams& p, int col, int row, int b, uint4 (&mem)[8]) {
    if constexpr (MODE != GRAM) {
        constexpr int kVecs = MODE == SQUARE ? 4 : 8, kPer = MODE == SQUARE ? 8 : 4;
        const int64_t at = int64_t(b) * p.apart + int64_t(row) * p.ld + col;
        const uint4* src = MODE == SQUARE ? reinterpret_cast<const uint4*>(p.e + at) : reinterpret_cast<const uint4*>(p.x + at);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {  // (rows are padded to 8 elements: whole vectors stay inside them)
            mem[j] = make_uint4(0, 0, 0, 0);
            if (row < p.m_dim && col + kPer * j < p.n_dim) mem[j] = src[j];
        }
    }
}

// The epilogue of 64 columns of a warp's 32 rows: lane l has row row0 + l, what
// its first 32 columns need is in mem[0], and what the next 64 columns' first 32
// need is there afterwards (`more`).
template <int MODE>
__device__ __forceinline__ void ortho_columns(const OrthoParams& p, const OutMaps& maps, uint32_t taddr, uint32_t box_half,
                                              uint32_t box_wide, int col, int row0, int b, bool mirrored, bool more, int lane,
                                              uint4 (&mem)[2][8]) {
    const int row = row0 + lane;
    uint32_t w[32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
        const int c0 = col + 32 * h;
        if (h == 0 || more) ortho_fetch<MODE>(p, c0 + 32, row, b, mem[h ^ 1]);
        tmem_ld_32cols(taddr + 32u * uint32_t(h), v);
        float f[32];
        if constexpr (MODE == SQUARE) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2* e2 = reinterpret_cast<const __half2*>(&mem[h][j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 e = __half22float2(e2[i]);
                    f[8 * j + 2 * i] = e.x;
                    f[8 * j + 2 * i + 1] = e.y;
                }
            }
        } else if constexpr (MODE == UPDATE || MODE == LAST) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[4 * j] = __uint_as_float(mem[h][j].x);
                f[4 * j + 1] = __uint_as_float(mem[h][j].y);
                f[4 * j + 2] = __uint_as_float(mem[h][j].z);
                f[4 * j + 3] = __uint_as_float(mem[h][j].w);
            }
        }
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float acc = __uint_as_float(v[j]) * (kDown * kDown);  // the product itself
            if constexpr (MODE == GRAM) f[j] = (row == c0 + j ? acc - p.shift : acc) * kUp;
            else if constexpr (MODE == SQUARE) f[j] = p.k1 * f[j] + p.k2 * (acc * kUp);
            else f[j] = p.k0 * f[j] + acc;
        }
        if constexpr (MODE == UPDATE) {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                st_shared_v4(box_wide + uint32_t(lane) * 128u + ((uint32_t(j) ^ (uint32_t(lane) & 7u)) << 4), __float_as_uint(f[4 * j]),
                             __float_as_uint(f[4 * j + 1]), __float_as_uint(f[4 * j + 2]), __float_as_uint(f[4 * j + 3]));
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0 && c0 < p.n_dim) {
                tma_store_3d(&maps.wide, box_wide, c0, row0, b);
                bulk_commit_group();
            }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if constexpr (MODE == LAST) w[16 * h + j] = pack_bf16x2(f[2 * j] * p.scale, f[2 * j + 1] * p.scale);
            else if constexpr (MODE == UPDATE) w[16 * h + j] = pack_f16x2(f[2 * j] * kUp, f[2 * j + 1] * kUp);
            else w[16 * h + j] = pack_f16x2(f[2 * j], f[2 * j + 1]);
        }
    }
    if (lane == 0) bulk_wait_group_read<0>();  // the boxes' last stores have read them
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        st_shared_v4(box_half + uint32_t(lane) * 128u + ((uint32_t(j) ^ (uint32_t(lane) & 7u)) << 4), w[4 * j], w[4 * j + 1],
                     w[4 * j + 2], w[4 * j + 3]);
    if ((MODE == GRAM || MODE == SQUARE) && mirrored) {  // column j of the 64 is row j of the mirrored box
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const uint32_t at = box_wide + uint32_t(2 * j) * 64u + uint32_t(lane) * 2u;
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(uint16_t(w[j] & 0xffffu)) : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 64u), "h"(uint16_t(w[j] >> 16)) : "memory");
        }
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
        tma_store_3d(&maps.half, box_half, col, row0, b);
        if ((MODE == GRAM || MODE == SQUARE) && mirrored) tma_store_3d(&maps.mirror, box_wide, row0, col, b);
        bulk_commit_group();
    }
}

// D = A B for every matrix of the stack, 256 x 256 tiles of CTA pairs; the
// pipeline is that of tl_gemm.cu's kernel with its static schedule.
template <bool A_MN, bool B_MN, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    ortho_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ OutMaps maps, const OrthoParams p) {
    const SharedWaitCtx wc{p.err, p.timeout_ns};
    constexpr int S = kOrthoStages;
    constexpr uint32_t kStage = 2 * kHalfStage;
    constexpr bool SYM = MODE == GRAM || MODE == SQUARE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem0 = smem_addr(smem), epi_base = smem0 + S * kStage;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * kStage + 8 * kEpiBuf);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (S + s); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * S + a); };
    auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * S + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int first_tile = int(cluster_id_x()), tile_step = int(cluster_count_x());
    auto place = [&](int tile, int& b, int& mb, int& nb) {
        b = tile / p.per_matrix;
        const int t = tile - b * p.per_matrix;
        if constexpr (SYM) triangle_coords(t, p.num_n, mb, nb);
        else tile_coords(t, p.num_m, p.num_n, p.raster, p.group, mb, nb);
    };

    if (threadIdx.x == 0) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
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
        tmem_alloc<true>(smem_addr(tmem_slot), 512);
        tmem_relinquish<true>();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dependents_go();
    grid_dependency_wait();

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_n = l2_policy_evict_normal(), pol_s = p.stream_shared ? pol_n : l2_policy_evict_first();
            const uint64_t pol_a = SYM ? pol_n : p.raster == 0 ? l2_policy_evict_last() : pol_s;
            const uint64_t pol_b = SYM ? pol_n : p.raster == 0 ? pol_s : l2_policy_evict_last();
            uint32_t fills = 0;
            bool ok = true;
            for (int tile = first_tile; ok && tile < p.num_tiles; tile += tile_step) {
                int b, mb, nb;
                place(tile, b, mb, nb);
                const int m0 = mb * 256 + int(rank) * 128, n0 = nb * 256 + int(rank) * 128;
                for (int kb = 0; kb < p.num_k; ++kb, ++fills) {
                    const uint32_t s = fills % S;
                    if (!wait_bounded(empty_bar(s), ((fills / S) & 1u) ^ 1u, wc, kErrProducerWait)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = smem0 + s * kStage, sb = sa + kHalfStage;
                    const int k0 = kb * kBlockK;
                    if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * kStage);
                    const uint32_t fb = map_to_rank(full_bar(s), 0);
                    if (A_MN) {
                        tma_load_3d_pair_hint(sa, &map_a, fb, m0, k0, b, pol_a);
                        tma_load_3d_pair_hint(sa + kMnChunk, &map_a, fb, m0 + 64, k0, b, pol_a);
                    } else {
                        tma_load_3d_pair_hint(sa, &map_a, fb, k0, m0, b, pol_a);
                    }
                    if (B_MN) {
                        tma_load_3d_pair_hint(sb, &map_b, fb, n0, k0, b, pol_b);
                        tma_load_3d_pair_hint(sb + kMnChunk, &map_b, fb, n0 + 64, k0, b, pol_b);
                    } else {
                        tma_load_3d_pair_hint(sb, &map_b, fb, k0, n0, b, pol_b);
                    }
                }
            }
            if (leader) {
                const uint32_t outstanding = fills < uint32_t(S) ? fills : uint32_t(S);
                for (uint32_t j = 0; j < outstanding; ++j) {
                    const uint32_t f = fills - 1 - j;
                    wait_bounded(full_bar(f % S), (f / S) & 1u, wc, kErrDrainWait, false);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            constexpr uint32_t idesc = idesc_f16_f32(256, 256, A_MN, B_MN);
            uint32_t fills = 0;
            bool ok = true;
            int it = 0;
            for (int tile = first_tile; ok && tile < p.num_tiles; tile += tile_step, ++it) {
                const uint32_t acc = it & 1;
                if (!wait_bounded(tempty_bar(acc), (uint32_t(it >> 1) & 1u) ^ 1u, wc, kErrMmaWaitTmem)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * 256;
                for (int kb = 0; kb < p.num_k; ++kb, ++fills) {
                    const uint32_t s = fills % S;
                    if (!wait_bounded(full_bar(s), (fills / S) & 1u, wc, kErrMmaWaitFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem0 + s * kStage, sb = sa + kHalfStage;
#pragma unroll
                    for (int j = 0; j < kBlockK / kUmmaK; ++j)
                        umma_bf16_pair(d_tmem, operand_desc(A_MN, sa, j), operand_desc(B_MN, sb, j), idesc, (kb | j) != 0 ? 1u : 0u);
                    umma_commit_pair(empty_bar(s), 0x3);
                }
                if (ok) umma_commit_pair(tfull_bar(acc), 0x3);
            }
            umma_commit_pair(drain_bar, 0x3);
            wait_bounded(drain_bar, 0, wc, kErrDrainWait, false);
        }
    } else if (warp >= kFirstEpilogueWarp) {
        const int q = warp & 3;
        const uint32_t box_half = epi_base + uint32_t(q) * 2u * kEpiBuf, box_wide = box_half + kEpiBuf;
        int it = 0;
        for (int tile = first_tile; tile < p.num_tiles; tile += tile_step, ++it) {
            const uint32_t acc = it & 1;
            int b, mb, nb;
            place(tile, b, mb, nb);
            const int row0 = mb * 256 + int(rank) * 128 + q * 32, n0 = nb * 256;
            const int chunks = row0 < p.m_dim ? min(4, (p.n_dim - n0 + 63) / 64) : 0;
            uint4 mem[2][8];
            if (chunks > 0) ortho_fetch<MODE>(p, n0, row0 + lane, b, mem[0]);
            if (!warp_wait(tfull_bar(acc), uint32_t(it >> 1) & 1u, wc, kErrEpilogueWait, lane)) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + (uint32_t(q * 32) << 16) + acc * 256;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c)
                ortho_columns<MODE>(p, maps, t_row + uint32_t(c) * 64u, box_half, box_wide, n0 + c * 64, row0, b, mb != nb,
                                    c + 1 < chunks, lane, mem);
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
        tmem_dealloc<true>(tmem_base, 512);
    }
}

// ---- small products ----------------------------------------------------------------
// One 128 x 128 tile a cluster; its CTAs have a part of the reduction each, leave
// their sums in shared memory, and each finishes some of the tile's rows from all
// of them, in a fixed order.
constexpr int kSmallStages = 6;
constexpr int kPartLd = 132;  // floats of a row of sums: 16-byte accesses of a column of lanes meet no bank twice
// Halves of a row of the turned tile: a warp's 4-byte writes, four rows apart, meet
// each bank four times.  (136, which allows 16-byte reads, with 2-byte writes: 16
// times.  The whole update, us, with this / with that, both before the ninth warp
// (kSmallThreads): 4 x 200 x 520 102 / 111, 512 x 512 98 / 104, 3 x 777 x 130 110 /
// 126, 1024 x 4096 187 / 192.)
constexpr int kTurnLd = 130;
constexpr uint32_t kTurn = 128 * kPartLd * 4;  // where the turned tile is, after the sums
constexpr size_t kSmallSmem = size_t(kSmallStages) * 2 * kHalfStage + kBarBytes + 1024;
static_assert(size_t(kTurn) + 128 * kTurnLd * 2 <= size_t(kSmallStages) * 2 * kHalfStage, "sums and turned tile fit the stages");

__device__ __forceinline__ float4 ld_shared_f32x4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

// The warps that finish rows go on as soon as they have read the others' sums.  A
// ninth waits for their reads and arrives with release semantics at the barrier
// past which the others may leave: a relaxed arrival is not ordered after the
// reads, and a releasing one holds its warp up.  The whole update, us, with this /
// with a releasing arrival of every warp: 4 x 200 x 520 107 / 125, 512 x 512 103 /
// 118, 1024 x 4096 189 / 198, 3 x 777 x 130 114 / 116.
constexpr int kSmallThreads = kThreads + 32;

template <bool A_MN, bool B_MN, int MODE>
__global__ void __launch_bounds__(kSmallThreads, 1)
    ortho_small_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const OrthoParams p) {
    const SharedWaitCtx wc{p.err, p.timeout_ns};
    constexpr int S = kSmallStages;
    constexpr uint32_t kStage = 2 * kHalfStage;
    constexpr bool SYM = MODE == GRAM || MODE == SQUARE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem0 = smem_addr(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * kStage);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 1);
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (S + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * S);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = p.splits > 1 ? cluster_ctarank() : 0;
    const int tile = int(blockIdx.x / uint32_t(p.splits));
    const int b = tile / p.per_matrix;
    int mb, nb;
    if constexpr (SYM) {
        triangle_coords(tile - b * p.per_matrix, p.num_n, mb, nb);
    } else {
        mb = (tile - b * p.per_matrix) / p.num_n;
        nb = tile - b * p.per_matrix - mb * p.num_n;
    }
    const int m0 = mb * 128, n0 = nb * 128;
    const int kb0 = int(rank) * p.per, kb1 = min(p.num_k, kb0 + p.per);

    if (threadIdx.x == 0) {
        tma_prefetch_map(&map_a);  // while the launch before this one ends
        tma_prefetch_map(&map_b);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        mbar_init_fence();
    }
    if (warp == 2) {
        tmem_alloc<false>(smem_addr(tmem_slot), 128);
        tmem_relinquish<false>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dependents_go();
    grid_dependency_wait();

    // This CTA finishes rows [r0, r0 + rows) of the tile, a warp an eighth of
    // them, a lane four columns: 16 / splits rows a warp, with `splits` sums each.
    // What the rows need from global memory is asked for first of all, and
    // all sixteen reads of sums are under way before one is used.
    const int rows = 128 / p.splits, r0 = int(rank) * rows, log = 31 - __clz(p.splits);
    const int c = lane * 4, col = n0 + c;
    uint4 mem[16];
    auto row_of = [&](int u) { return r0 + (warp << (4 - log)) + u; };
    auto in = [&](int u) { return u < 16 >> log && m0 + row_of(u) < p.m_dim && col < p.n_dim; };
    if (MODE != GRAM && warp < kThreads / 32) {
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            mem[u] = make_uint4(0, 0, 0, 0);
            if (!in(u)) continue;
            const int64_t at = int64_t(b) * p.apart + int64_t(m0 + row_of(u)) * p.ld + col;
            if constexpr (MODE == SQUARE) {
                const uint2 e = *reinterpret_cast<const uint2*>(p.e + at);
                mem[u].x = e.x;
                mem[u].y = e.y;
            } else {
                mem[u] = *reinterpret_cast<const uint4*>(p.x + at);
            }
        }
    }
    if (warp == 0) {
        if (lane == 0) {
            uint32_t fills = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++fills) {
                const uint32_t s = fills % S;
                if (!wait_bounded(empty_bar(s), ((fills / S) & 1u) ^ 1u, wc, kErrProducerWait)) break;
                const uint32_t sa = smem0 + s * kStage, sb = sa + kHalfStage, fb = full_bar(s);
                const int k0 = kb * kBlockK;
                mbar_arrive_expect_tx(fb, kStage);
                if (A_MN) {
                    tma_load_3d(sa, &map_a, fb, m0, k0, b);
                    tma_load_3d(sa + kMnChunk, &map_a, fb, m0 + 64, k0, b);
                } else {
                    tma_load_3d(sa, &map_a, fb, k0, m0, b);
                }
                if (B_MN) {
                    tma_load_3d(sb, &map_b, fb, n0, k0, b);
                    tma_load_3d(sb + kMnChunk, &map_b, fb, n0 + 64, k0, b);
                } else {
                    tma_load_3d(sb, &map_b, fb, k0, n0, b);
                }
            }
            const uint32_t outstanding = fills < uint32_t(S) ? fills : uint32_t(S);
            for (uint32_t j = 0; j < outstanding; ++j) {
                const uint32_t f = fills - 1 - j;
                wait_bounded(full_bar(f % S), (f / S) & 1u, wc, kErrDrainWait, false);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_f16_f32(128, 128, A_MN, B_MN);
            uint32_t fills = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++fills) {
                const uint32_t s = fills % S;
                if (!wait_bounded(full_bar(s), (fills / S) & 1u, wc, kErrMmaWaitFull)) break;
                tc_fence_after();
                const uint32_t sa = smem0 + s * kStage, sb = sa + kHalfStage;
#pragma unroll
                for (int j = 0; j < kBlockK / kUmmaK; ++j)
                    umma_bf16(tmem_base, operand_desc(A_MN, sa, j), operand_desc(B_MN, sb, j), idesc, (kb != kb0 || j) ? 1u : 0u);
                umma_commit(empty_bar(s));
            }
            umma_commit(done_bar);
            wait_bounded(done_bar, 0, wc, kErrDrainWait, false);
        }
    } else if (warp >= kFirstEpilogueWarp && warp < kThreads / 32) {
        const int q = warp & 3, i = q * 32 + lane;
        const bool ok = warp_wait(done_bar, 0, wc, kErrEpilogueWait, lane);
        tc_fence_after();
        if (ok)
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                uint32_t v[32];
                tmem_ld_32cols(tmem_base + (uint32_t(q * 32) << 16) + uint32_t(c), v);
                tmem_ld_wait();
                const bool any = kb1 > kb0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st_shared_v4(smem0 + uint32_t(i * kPartLd + c + 4 * j) * 4u, any ? v[4 * j] : 0u, any ? v[4 * j + 1] : 0u,
                                 any ? v[4 * j + 2] : 0u, any ? v[4 * j + 3] : 0u);
            }
        tc_fence_before();
    }
    if (p.splits > 1) cluster_sync(); else __syncthreads();

    if (warp == kThreads / 32) {
        if (p.splits > 1) {
            cta_barrier_sync(1, kSmallThreads);  // the others' reads are done
            cluster_arrive();
            cluster_wait();
        }
        return;
    }
    float4 acc[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const uint32_t at = smem0 + uint32_t(row_of(q >> log) * kPartLd + c) * 4u;
        const uint32_t from = uint32_t(q & (p.splits - 1));
        acc[q] = from == rank ? ld_shared_f32x4(at) : ld_cluster_f32x4(at, from);
    }
    // the sums of a row, neighbours first: row u's end up in acc[u]
#pragma unroll
    for (int level = 0; level < 3; ++level)
        if (level < log)
#pragma unroll
            for (int i = 0; i < 8 >> level; ++i)
                acc[i] = make_float4(acc[2 * i].x + acc[2 * i + 1].x, acc[2 * i].y + acc[2 * i + 1].y, acc[2 * i].z + acc[2 * i + 1].z,
                                     acc[2 * i].w + acc[2 * i + 1].w);

    if (p.splits > 1) {
        cta_barrier_arrive(1, kSmallThreads);
        cluster_arrive_relaxed();  // (the ninth warp's arrival orders the reads)
    }

    uint16_t* turn = reinterpret_cast<uint16_t*>(smem + kTurn);
    const bool mirrored = SYM && mb != nb;
    uint2 above = make_uint2(0, 0);  // the halves of the row before
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        if (u >= 16 >> log) break;
        const int r = row_of(u), row = m0 + r;
        float f[4] = {acc[u].x, acc[u].y, acc[u].z, acc[u].w};
        if constexpr (MODE == GRAM) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = (f[j] * (kDown * kDown) - (row == col + j ? p.shift : 0.0f)) * kUp;
        } else if constexpr (MODE == SQUARE) {
            const float2 e0 = __half22float2(*reinterpret_cast<const __half2*>(&mem[u].x));
            const float2 e1 = __half22float2(*reinterpret_cast<const __half2*>(&mem[u].y));
            const float e[4] = {e0.x, e0.y, e1.x, e1.y};
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = p.k1 * e[j] + p.k2 * (f[j] * kDown);
        } else {
            const float x[4] = {__uint_as_float(mem[u].x), __uint_as_float(mem[u].y), __uint_as_float(mem[u].z), __uint_as_float(mem[u].w)};
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = p.k0 * x[j] + f[j] * (kDown * kDown);
        }
        uint2 w;
        if constexpr (MODE == LAST)
            w = make_uint2(pack_bf16x2(f[0] * p.scale, f[1] * p.scale), pack_bf16x2(f[2] * p.scale, f[3] * p.scale));
        else if constexpr (MODE == UPDATE)
            w = make_uint2(pack_f16x2(f[0] * kUp, f[1] * kUp), pack_f16x2(f[2] * kUp, f[3] * kUp));
        else
            w = make_uint2(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]));
        const uint16_t h[4] = {uint16_t(w.x & 0xffffu), uint16_t(w.x >> 16), uint16_t(w.y & 0xffffu), uint16_t(w.y >> 16)};
        // (rows of E, Q and X are padded to 8 elements: four at a time stay
        // inside them; the padding of the result's rows is the caller's)
        if (in(u)) {
            if constexpr (MODE == UPDATE)
                *reinterpret_cast<float4*>(p.x + int64_t(b) * p.apart + int64_t(row) * p.ld + col) = make_float4(f[0], f[1], f[2], f[3]);
            uint16_t* dst = static_cast<uint16_t*>(p.out) + int64_t(b) * p.o_apart + int64_t(row) * p.ldo + col;
            if (MODE != LAST || col + 4 <= p.n_dim) *reinterpret_cast<uint2*>(dst) = w;
            else
                for (int j = 0; col + j < p.n_dim; ++j) dst[j] = h[j];
        }
        if (mirrored) {  // a column's halves of two rows at a time (a warp has at least two)
            if (u & 1) {
                const uint32_t two[4] = {__byte_perm(above.x, w.x, 0x5410), __byte_perm(above.x, w.x, 0x7632),
                                         __byte_perm(above.y, w.y, 0x5410), __byte_perm(above.y, w.y, 0x7632)};
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(turn + (c + j) * kTurnLd + (r - r0 - 1)) = two[j];
            }
            above = w;
        }
    }
    if (mirrored) {
        cta_barrier_sync(2, kThreads);
        // column i of these rows is row n0 + i of the result, from column m0 + r0 on
        const int groups = rows / 8;
        for (int idx = int(threadIdx.x); idx < 128 * groups; idx += kThreads) {
            const int i = idx / groups, g = idx % groups * 8;
            const int row = n0 + i, at = m0 + r0 + g;
            const uint32_t* from = reinterpret_cast<const uint32_t*>(turn + i * kTurnLd + g);
            if (row < p.n_dim && at < p.m_dim)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + int64_t(b) * p.o_apart + int64_t(row) * p.ldo + at) =
                    make_uint4(from[0], from[1], from[2], from[3]);
        }
    }
    if (p.splits > 1) cluster_wait();  // nobody leaves while its sums are read
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc<false>(tmem_base, 128);
    }
}

// ---- the norm and the first iterate ----------------------------------------------
constexpr int kNormThreads = 256;
constexpr int kNormParts = 1024;  // partial sums of squares a matrix, at most

struct StartArgs {
    const void* g;
    int64_t ldg, g_apart;
    int64_t rows, cols;
    float* parts;  // [batch][kNormParts]
    float* x;
    __half* h;
    int64_t ld, apart;
    float eps;
    int32_t vec;  // rows of g start on 16-byte boundaries and hold whole vectors
};

__device__ __forceinline__ float block_sum(float v) {
    __shared__ float part[kNormThreads / 32];
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(~0u, v, s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float sum = 0;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; ++w) sum += part[w];
    return sum;
}

// Walk over the vectors of a matrix that this CTA (of `parts`) has, four loads
// at a time: f(row, col, vector).
template <typename T, int VEC, typename F>
__device__ __forceinline__ void each_vector(const StartArgs& p, int part, int parts, F&& f) {
    const T* g = static_cast<const T*>(p.g) + int64_t(blockIdx.y) * p.g_apart;
    const uint32_t per_row = uint32_t(p.cols / VEC);
    const uint64_t n = uint64_t(p.rows) * per_row, step = uint64_t(parts) * kNormThreads;
    for (uint64_t i0 = uint64_t(part) * kNormThreads + threadIdx.x; i0 < n; i0 += 4 * step) {
        Vec<T, VEC> v[4];
        uint32_t r[4], c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t i = i0 + k * step;
            if (i >= n) continue;
            // (a 32-bit division where the index allows it)
            r[k] = n <= 0xffffffffull ? uint32_t(i) / per_row : uint32_t(i / per_row);
            c[k] = uint32_t(i - uint64_t(r[k]) * per_row) * VEC;
            v[k] = *reinterpret_cast<const Vec<T, VEC>*>(g + int64_t(r[k]) * p.ldg + c[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * step < n) f(int64_t(r[k]), int64_t(c[k]), v[k]);
    }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kNormThreads) ortho_squares_kernel(const StartArgs p) {
    float s = 0;
    each_vector<T, VEC>(p, blockIdx.x, gridDim.x, [&](int64_t, int64_t, const Vec<T, VEC>& v) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += to_f32(v.v[e]) * to_f32(v.v[e]);
    });
    s = block_sum(s);
    if (threadIdx.x == 0) p.parts[int64_t(blockIdx.y) * kNormParts + blockIdx.x] = s;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kNormThreads) ortho_start_kernel(const StartArgs p, int parts) {
    const float* all = p.parts + int64_t(blockIdx.y) * kNormParts;
    float mine = 0;
    for (int i = int(threadIdx.x); i < parts; i += kNormThreads) mine += all[i];
    const float sum = block_sum(mine);
    const float inv = 1.0f / (sqrtf(sum) + p.eps);
    float* x = p.x + int64_t(blockIdx.y) * p.apart;
    __half* h = p.h + int64_t(blockIdx.y) * p.apart;
    each_vector<T, VEC>(p, blockIdx.x, gridDim.x, [&](int64_t r, int64_t c, const Vec<T, VEC>& v) {
        Vec<float, VEC> f;
        Vec<__half, VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            f.v[e] = to_f32(v.v[e]) * inv;
            o.v[e] = __float2half_rn(f.v[e] * kUp);
        }
        if constexpr (VEC == 8) {
            Vec<float, 4>* dst = reinterpret_cast<Vec<float, 4>*>(x + r * p.ld + c);
            dst[0] = Vec<float, 4>{{f.v[0], f.v[1], f.v[2], f.v[3]}};
            dst[1] = Vec<float, 4>{{f.v[4], f.v[5], f.v[6], f.v[7]}};
        } else {
            *reinterpret_cast<Vec<float, VEC>*>(x + r * p.ld + c) = f;
        }
        *reinterpret_cast<Vec<__half, VEC>*>(h + r * p.ld + c) = o;
    });
}

template <typename T>
cudaError_t start_launch(const StartArgs& a, int64_t batch, int num_sms, cudaStream_t stream) {
    constexpr int V = 16 / int(sizeof(T));
    const int64_t vectors = a.rows * a.cols / (a.vec ? V : 1);
    const int64_t want = (vectors + 4 * kNormThreads - 1) / (4 * kNormThreads);
    const int64_t room = std::max<int64_t>(1, 8 * num_sms / batch);
    const int parts = int(std::max<int64_t>(1, std::min({want, room, int64_t(kNormParts)})));
    const dim3 g1{unsigned(parts), unsigned(batch)}, g2{unsigned(std::max<int64_t>(1, std::min(want, room))), unsigned(batch)};
    if (a.vec) {
        ortho_squares_kernel<T, V><<<g1, kNormThreads, 0, stream>>>(a);
        ortho_start_kernel<T, V><<<g2, kNormThreads, 0, stream>>>(a, parts);
    } else {
        ortho_squares_kernel<T, 1><<<g1, kNormThreads, 0, stream>>>(a);
        ortho_start_kernel<T, 1><<<g2, kNormThreads, 0, stream>>>(a, parts);
    }
    return cudaGetLastError();
}

// ---- host --------------------------------------------------------------------------
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

struct Work {
    int64_t r, c, ldx, ldp, x_apart, p_apart;
    size_t parts, x, h0, h1, e, q, bytes;
};
Work layout(int64_t batch, int64_t rows, int64_t cols) {
    Work w{};
    w.r = std::min(rows, cols);
    w.c = std::max(rows, cols);
    w.ldx = up8(cols);
    w.ldp = up8(w.r);
    w.x_apart = rows * w.ldx;
    w.p_apart = w.r * w.ldp;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t p = at;
        at += up256(n);
        return p;
    };
    w.parts = take(size_t(batch) * kNormParts * 4);
    w.x = take(size_t(batch) * size_t(w.x_apart) * 4);
    w.h0 = take(size_t(batch) * size_t(w.x_apart) * 2);
    w.h1 = take(size_t(batch) * size_t(w.x_apart) * 2);
    w.e = take(size_t(batch) * size_t(w.p_apart) * 2);
    w.q = take(size_t(batch) * size_t(w.p_apart) * 2);
    w.bytes = at;
    return w;
}

constexpr auto kF16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;

// Boxes of 32 elements x 64 rows, as they lie in shared memory (no swizzle).
bool mirror_map(CUtensorMap* map, const void* base, uint64_t n, uint64_t ld, uint64_t count, uint64_t apart, std::string* why) {
    auto fn = tensor_map_encoder();
    cuuint64_t dims[3] = {n, n, count};
    cuuint64_t strides[2] = {ld * 2, apart * 2};
    cuuint32_t box[3] = {32, 64, 1}, estr[3] = {1, 1, 1};
    const CUresult r = fn ? fn(map, kF16, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE)
                          : CUDA_ERROR_NOT_SUPPORTED;
    if (r != CUDA_SUCCESS && why) *why = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string(int(r));
    return r == CUDA_SUCCESS;
}

// s of each step: see the top of this file.
struct Shift {
    double sigma;
    bool near = false;
    explicit Shift(int64_t r) : sigma(1.0 / std::sqrt(double(r))) {}
    float next(const OrthoDesc& d) {
        const double v = std::min(1.0, sigma * sigma);
        near = near || !(v < 0.8);
        sigma = std::fabs(sigma * (d.a + sigma * sigma * (d.b + sigma * sigma * d.c)));
        return near ? 1.0f : float(v);
    }
};

// An operand of a product: `outer` rows of `inner` halves.
struct Half {
    const void* p;
    int64_t inner, outer, ld, apart;
};

cudaError_t launch(const void* kern, int threads, int grid, int cluster, size_t smem, cudaStream_t stream, void** args) {
    int per_sm = 0;
    const cudaError_t e = ctas_per_sm(kern, threads, smem, &per_sm);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(threads));
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
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

// Products of up to a quarter as many 256 x 256 tiles as there are CTA pairs go
// through the small kernel.  The whole update, us, by pairs alone / with this
// rule / with one three times as wide: 512 x 512 164 / 103 / 103, 128 x 512 112 /
// 98 / 99, 1024 x 4096 277 / 190 / 190, 2048 x 2048 290 / 289 / 261.  (When the rule
// was chosen, before kTurnLd and kSmallThreads, the last two of the wider one
// were 203 and 315: what it costs elsewhere now is not measured.)
bool small_product(int64_t pair_tiles, int num_sms) { return pair_tiles <= num_sms / 8; }

template <bool A_MN, bool B_MN, int MODE>
cudaError_t product(const Half& a, const Half& b, int64_t m, int64_t n, int64_t k, const OutMaps& maps, OrthoParams p, int64_t batch,
                    int num_sms, cudaStream_t stream, std::string* why) {
    CUtensorMap ma, mb;
    if (!swizzled_map(&ma, kF16, 2, a.p, uint64_t(a.inner), uint64_t(a.outer), uint64_t(a.ld), A_MN ? 64 : 128, why, uint64_t(batch), uint64_t(a.apart)) ||
        !swizzled_map(&mb, kF16, 2, b.p, uint64_t(b.inner), uint64_t(b.outer), uint64_t(b.ld), B_MN ? 64 : 128, why, uint64_t(batch), uint64_t(b.apart)))
        return cudaErrorInvalidValue;
    const bool sym = MODE == GRAM || MODE == SQUARE;
    auto tiles = [&](int64_t side) {
        p.num_m = int32_t((m + side - 1) / side);
        p.num_n = int32_t((n + side - 1) / side);
        return sym ? int64_t(p.num_n) * (p.num_n + 1) / 2 : int64_t(p.num_m) * p.num_n;
    };
    p.m_dim = int32_t(m);
    p.n_dim = int32_t(n);
    p.num_k = int32_t((k + kBlockK - 1) / kBlockK);
    const bool small = small_product(tiles(256) * batch, num_sms);
    const int64_t per = tiles(small ? 128 : 256);
    if (per * batch > INT32_MAX / 8) {
        if (why) *why = "too many output tiles";
        return cudaErrorInvalidValue;
    }
    p.per_matrix = int32_t(per);
    p.num_tiles = int32_t(per * batch);
    OutMaps to = maps;
    void* args[] = {&ma, &mb, &to, &p};
    if (small) {
        // CTAs of a cluster: as many as there are SMs for, with two K-blocks each,
        // and as many clusters as run at a time.  512 x 512 (8 K-blocks), us: one
        // CTA 131, two 114, four 103 (chosen), eight 139.  With / without that last
        // bound: 6 x 200 x 4096 192 / 222, 6 x 256 x 2048 143 / 174.
        p.splits = 1;
        const void* kern = reinterpret_cast<const void*>(ortho_small_kernel<A_MN, B_MN, MODE>);
        int per_sm = 0, clusters = 0;
        cudaError_t e = ctas_per_sm(kern, kSmallThreads, kSmallSmem, &per_sm);
        while (e == cudaSuccess && p.splits < 8 && int64_t(p.num_tiles) * p.splits * 2 <= num_sms && p.num_k >= 4 * p.splits) {
            e = clusters_at_a_time(kern, kSmallThreads, kSmallSmem, 2 * p.splits, &clusters);
            if (e != cudaSuccess || p.num_tiles > clusters) break;
            p.splits *= 2;
        }
        if (e != cudaSuccess) return e;
        p.per = (p.num_k + p.splits - 1) / p.splits;
        void* few[] = {&ma, &mb, &p};
        return launch(kern, kSmallThreads, p.num_tiles * p.splits, p.splits, kSmallSmem, stream, few);
    }
    const int slots = std::max(1, num_sms / 2);
    choose_tile_order(k, 256, p.num_m, p.num_n, slots, &p.raster, &p.group, &p.stream_shared);
    return launch(reinterpret_cast<const void*>(ortho_kernel<A_MN, B_MN, MODE>), kThreads, 2 * std::min(p.num_tiles, slots), 2,
                  kOrthoSmem, stream, args);
}

}  // namespace

std::string ortho_check(const OrthoDesc& d) {
    if (d.batch < 0 || d.batch > 65535) return "batch must be in 0..65535";
    if (d.rows < 1 || d.cols < 1 || d.rows > (1 << 20) || d.cols > (1 << 20)) return "rows and cols must be in 1..2^20";
    if (d.steps < 1 || d.steps > 100) return "steps must be in 1..100";
    if (!type_known(d.type)) return "unknown tl_type";
    if (!(d.eps >= 0)) return "eps must be >= 0";
    if (d.batch == 0) return {};
    if (!d.g || !d.out || !d.err) return "null pointer";
    auto off = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (off(d.g, type_bytes(d.type)) || off(d.err, 4)) return "g or err is not aligned to its type";
    if (off(d.out, 16) || d.ldo % 8 || d.o_apart % 8) return "out must be 16-byte aligned, its strides multiples of 8";
    if (d.ldg < d.cols || d.ldo < d.cols) return "a leading dimension is smaller than cols";
    if (d.batch > 1 && (d.g_apart < 0 || d.o_apart < (d.rows - 1) * d.ldo + d.cols)) return "the matrices of out overlap";
    return {};
}

size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols) {
    if (batch < 0 || batch > 65535 || rows < 1 || cols < 1 || rows > (1 << 20) || cols > (1 << 20)) return 0;
    return std::max<size_t>(256, layout(batch, rows, cols).bytes);
}

cudaError_t ortho_launch(const OrthoDesc& d, int num_sms, cudaStream_t stream, std::string* why) {
    if (d.batch == 0) return cudaSuccess;
    const Work w = layout(d.batch, d.rows, d.cols);
    uint8_t* base = static_cast<uint8_t*>(d.workspace);
    StartArgs s{};
    s.g = d.g;
    s.ldg = d.ldg;
    s.g_apart = d.g_apart;
    s.rows = d.rows;
    s.cols = d.cols;
    s.parts = reinterpret_cast<float*>(base + w.parts);
    s.x = reinterpret_cast<float*>(base + w.x);
    s.h = reinterpret_cast<__half*>(base + w.h0);
    s.ld = w.ldx;
    s.apart = w.x_apart;
    s.eps = d.eps;
    const int64_t vec = int64_t(16 / type_bytes(d.type));
    s.vec = d.cols % vec == 0 && d.ldg % vec == 0 && d.g_apart % vec == 0 && (reinterpret_cast<uintptr_t>(d.g) & 15) == 0;
    cudaError_t e = d.type == TL_TYPE_BF16  ? start_launch<__nv_bfloat16>(s, d.batch, num_sms, stream)
                    : d.type == TL_TYPE_F16 ? start_launch<__half>(s, d.batch, num_sms, stream)
                                            : start_launch<float>(s, d.batch, num_sms, stream);
    if (e != cudaSuccess) return e;

    const bool tall = d.rows > d.cols;
    OrthoParams p{};
    p.scale = d.scale;
    p.err = d.err;
    p.timeout_ns = 2000000000ull;
    const uint64_t count = uint64_t(d.batch);
    auto half_map = [&](CUtensorMap* m, size_t at, int64_t rows, int64_t cols, int64_t ld, int64_t apart) {
        return swizzled_map(m, kF16, 2, base + at, uint64_t(cols), uint64_t(rows), uint64_t(ld), 32, why, count, uint64_t(apart));
    };
    OutMaps gram{}, square{}, update[2] = {}, last{};
    if (!half_map(&gram.half, w.e, w.r, w.r, w.ldp, w.p_apart) || !half_map(&square.half, w.q, w.r, w.r, w.ldp, w.p_apart) ||
        !mirror_map(&gram.mirror, base + w.e, uint64_t(w.r), uint64_t(w.ldp), count, uint64_t(w.p_apart), why) ||
        !mirror_map(&square.mirror, base + w.q, uint64_t(w.r), uint64_t(w.ldp), count, uint64_t(w.p_apart), why) ||
        !half_map(&update[0].half, w.h1, d.rows, d.cols, w.ldx, w.x_apart) || !half_map(&update[1].half, w.h0, d.rows, d.cols, w.ldx, w.x_apart) ||
        !swizzled_map(&update[0].wide, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base + w.x, uint64_t(d.cols), uint64_t(d.rows), uint64_t(w.ldx), 32, why, count, uint64_t(w.x_apart)) ||
        !swizzled_map(&last.half, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d.out, uint64_t(d.cols), uint64_t(d.rows), uint64_t(d.ldo), 32, why, count,
                      uint64_t(d.batch > 1 ? d.o_apart : up8(d.rows * d.ldo))))
        return cudaErrorInvalidValue;
    update[1].wide = update[0].wide;
    gram.wide = square.wide = last.wide = update[0].wide;  // not used there
    update[0].mirror = update[1].mirror = last.mirror = gram.mirror;

    Shift shift(w.r);
    for (int step = 0; step < d.steps && e == cudaSuccess; ++step) {
        p.shift = shift.next(d);
        p.k0 = d.a + p.shift * (d.b + p.shift * d.c);
        p.k1 = d.b + 2.0f * d.c * p.shift;
        p.k2 = d.c;
        const Half x{base + (step & 1 ? w.h1 : w.h0), d.cols, d.rows, w.ldx, w.x_apart};
        p.out = base + w.e;
        p.ldo = w.ldp;
        p.o_apart = w.p_apart;
        const Half pe{base + w.e, w.r, w.r, w.ldp, w.p_apart}, pq{base + w.q, w.r, w.r, w.ldp, w.p_apart};
        e = tall ? product<true, true, GRAM>(x, x, w.r, w.r, w.c, gram, p, d.batch, num_sms, stream, why)
                 : product<false, false, GRAM>(x, x, w.r, w.r, w.c, gram, p, d.batch, num_sms, stream, why);
        if (e != cudaSuccess) break;
        p.e = static_cast<const __half*>(pe.p);
        p.ld = w.ldp;
        p.apart = w.p_apart;
        p.out = base + w.q;
        e = product<false, false, SQUARE>(pe, pe, w.r, w.r, w.r, square, p, d.batch, num_sms, stream, why);
        if (e != cudaSuccess) break;
        p.x = reinterpret_cast<float*>(base + w.x);
        p.ld = w.ldx;
        p.apart = w.x_apart;
        const bool end = step == d.steps - 1;
        const OutMaps& to = end ? last : update[step & 1];
        p.out = end ? d.out : base + (step & 1 ? w.h0 : w.h1);
        p.ldo = end ? d.ldo : w.ldx;
        p.o_apart = end ? d.o_apart : w.x_apart;
        if (tall)
            e = end ? product<false, false, LAST>(x, pq, d.rows, d.cols, w.r, to, p, d.batch, num_sms, stream, why)
                    : product<false, false, UPDATE>(x, pq, d.rows, d.cols, w.r, to, p, d.batch, num_sms, stream, why);
        else
            e = end ? product<false, true, LAST>(pq, x, d.rows, d.cols, w.r, to, p, d.batch, num_sms, stream, why)
                    : product<false, true, UPDATE>(pq, x, d.rows, d.cols, w.r, to, p, d.batch, num_sms, stream, why);
    }
    return e;
}

}  // namespace tl
