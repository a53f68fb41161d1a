// tl_grouped.cuh -- device building blocks of the products whose weight depends
// on the row: loads of indexed rows, where a group's rows are, the joining of
// sums that a cluster's CTAs share.
#pragma once
#include "tl_grouped.h"
#include "tl_kernel_common.cuh"
#include "tl_launch.h"
#include "tl_tmap.h"
#include "tl_types.cuh"

#include <climits>

namespace tl {
namespace gr {

using namespace kc;

constexpr int kMaxGroupsSeen = 1025;  // the groups and the rows behind them

// ---- PTX ---------------------------------------------------------------------

// Four rows of a matrix, 128 bytes of each from column x on, one after another in
// shared memory (128B-swizzled by address, so 512 bytes from one to the next make
// the image of one box), for a CTA pair, whose barrier may be in the other CTA.
// Rows past the matrix arrive as zeros.
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int32_t x, const int (&r)[4]) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
        : "memory");
}
// 16 bytes of global memory to shared memory, the last 16 - bytes of them as zeros.
// (What follows in the row is wanted next: 256 bytes of it go to L2.)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's groups are under way.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_box_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_store_box(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
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

// Instruction descriptor of kind::f16: as idesc_bf16_f32, with A and B both fp16
// (format 0) where asked, N left out.
__host__ __device__ constexpr uint32_t idesc_16(int m, bool a_mn, bool b_mn, bool fp16) {
    return idesc_bf16_f32(m, 0, a_mn, b_mn) & (fp16 ? ~((1u << 7) | (1u << 10)) : ~0u);
}
__device__ __forceinline__ uint32_t with_n(uint32_t idesc, int n) { return idesc | (uint32_t(n >> 3) << 17); }

template <bool PAIR>
__device__ __forceinline__ void umma_16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR) umma_bf16_pair(d, a, b, idesc, accumulate);
    else umma_bf16(d, a, b, idesc, accumulate);
}

// Whether a phase has completed, as every lane of the warp sees it.
__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, ok) != 0;
}

// ---- where the rows are ------------------------------------------------------------

// Offsets come from the caller's memory: whatever they hold, a group's rows are some of 0 .. rows - 1.
__device__ __forceinline__ void group_span(const int32_t* offsets, int groups, int rows, int g, int& begin, int& end) {
    // (g == groups: the rows behind the last group)
    begin = min(max(offsets[g], 0), rows);
    end = g == groups ? rows : min(max(offsets[g + 1], begin), rows);
}

// The block of at most `size` rows of one group that is the `wanted`-th of all
// groups' (with all_rows, of the rows behind them, too): found = group, first place
// and places; the group is -1 if there are fewer.  Every thread of the CTA takes
// part; sums holds an int for each warp.
__device__ __forceinline__ void find_block(const int32_t* offsets, int groups, int rows, bool all_rows, int size, int wanted, int* found, int* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, seen = groups + (all_rows ? 1 : 0);
    if (threadIdx.x == 0) found[0] = -1;
    __syncthreads();
    int before = 0;
    for (int g0 = 0; g0 < seen && before <= wanted; g0 += blockDim.x) {
        const int g = g0 + int(threadIdx.x);
        int b = 0, e = 0;
        if (g < seen) group_span(offsets, groups, rows, g, b, e);
        const int blocks = (e - b + size - 1) / size;
        int s = blocks;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += u;
        }
        if (lane == 31) sums[warp] = s;
        __syncthreads();
        int at = before + s - blocks, all = 0;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) at += sums[w];
            all += sums[w];
        }
        if (blocks > 0 && at <= wanted && wanted < at + blocks) {
            found[0] = g;
            found[1] = b + (wanted - at) * size;
            found[2] = min(size, e - found[1]);
        }
        before += all;
        __syncthreads();
    }
    __syncthreads();
}

// ---- rows picked up ------------------------------------------------------------------

// 128 threads pick up rows 16 bytes at a time by cp.async (TMA's gathers of four rows
// take some 36 clocks each, whoever issues them: 14 bytes a clock and SM): eight threads for 128 bytes of a row, sixteen rows at
// a time, into the image that a TMA load of a box with 128-byte swizzle leaves.
// What they wrote is handed to the tensor cores by a proxy fence of each thread
// after its copies have landed and an arrival of each warp: a stage when two
// further ones are under way (the widest shapes have two or three stages in all), or all
// of them before a wait for a free stage, which would otherwise keep from the tensor
// cores what that wait depends on.
// For single CTAs alone: the arrival at the other CTA of a pair would need release
// semantics in the cluster for each stage, which took longer than the stage's MMAs
// (8192 x 8192 x 4096 in eight groups, 2 rows a token: 3.0 ms, against 1.2 with
// gathers and 0.8 with a sorted copy made first).
constexpr int kPickThreads = 128, kPickWarps = kPickThreads / 32, kPickRows = kPickThreads / 8;
struct Picker {
    int row, chunk;     // of the first sixteen rows; 16 bytes of the row's 128
    uint32_t dst;       // in a box, from its start on
    __device__ __forceinline__ explicit Picker(int thread) : row(thread >> 3), chunk(thread & 7) {
        dst = uint32_t(row) * 128u + (uint32_t(chunk ^ (row & 7)) << 4);
    }
    // Row row + 16 i of a box at `box`: from `src` on (the row's first element of the
    // box's columns), `cols` of which are there (none: zeros).
    __device__ __forceinline__ uint32_t at(uint32_t box, int i) const { return box + dst + uint32_t(i) * (kPickRows * 128u); }
    __device__ __forceinline__ void copy(uint32_t box, int i, const uint16_t* src, int cols) const {
        const int have = min(max(cols - 8 * chunk, 0), 8);
        cp_async16(at(box, i), src + (have ? 8 * chunk : 0), uint32_t(have) * 2u);
    }
};

// Eight elements, of which `have` are there.
__device__ __forceinline__ uint4 load_eight(const uint16_t* p, int have) {
    if (have >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < have) w[j / 2] |= uint32_t(p[j]) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint16_t round16(float v, bool fp16) {
    return fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ float value16(uint16_t v, bool fp16) {
    return fp16 ? __half2float(__ushort_as_half(v)) : __bfloat162float(__ushort_as_bfloat16(v));
}
__device__ __forceinline__ uint32_t round16x2(float lo, float hi, bool fp16) {
    if (!fp16) return pack_bf16x2(lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- fp16's units --------------------------------------------------------------------

// Two parts hold twice fp16's digits only well within its range, so they are those of a
// number in units of a power of two of the place, which puts the largest of its finite
// numbers (`most`, the bits of its magnitude) into [2^14, 2^15): 2^-22 of a number and 2^-39 of
// the place's largest are lost, whatever their sizes.  (bf16 has fp32's range and needs none.)  A unit is at
// least 2^-126, so that its reciprocal is a normal number; a place without a number but
// 0 has that one, and so does not count where units are compared.
__device__ __forceinline__ float unit_of(uint32_t most) { return __uint_as_float(uint32_t(max(int(most >> 23) - 14, 1)) << 23); }
__device__ __forceinline__ float reciprocal_of_unit(float unit) { return __uint_as_float((254u << 23) - __float_as_uint(unit)); }
// Part of a place from its unit to a larger one.  (Below 2^-60 no finite part is left of
// any; an infinite one stays infinite.)
__device__ __forceinline__ float between_units(float unit, float reciprocal) { return fmaxf(unit * reciprocal, 0x1p-60f); }

}  // namespace gr

// ---- host side ---------------------------------------------------------------------

template <typename T>
struct SameType {
    using type = T;
};
// early: the kernel may begin before the one ahead of it in the stream has completed.
template <typename... A>
cudaError_t launch_in_clusters(void (*kern)(A...), dim3 grid, int threads, int cluster, size_t smem, bool early, cudaStream_t stream,
                               typename SameType<A>::type... args) {
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

inline CUtensorMapDataType map_type16(int32_t type) {
    return type == TL_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// The map of an operand's rows where they follow each other.
inline bool rows_map(CUtensorMap* map, int32_t type, const RowsOperand& o, int64_t cols, uint32_t box_rows, std::string* why) {
    return swizzled_map(map, map_type16(type), 2, o.at, uint64_t(cols), uint64_t(o.count), uint64_t(o.ld), box_rows, why);
}

}  // namespace tl
