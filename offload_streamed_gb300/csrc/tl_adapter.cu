// tl_adapter.cu -- low-rank adapters of many requests beside a shared projection.
//
// Many rows: the rows are sorted by adapter (tl_route.cu); h = x . a, bound by the
// bytes of x, is a product whose weight depends on the row (tl_grouped.cu), and
// y = base + s h . b, bound by those of base and y, a kernel of its own
// (expand_kernel).  h goes from one to the other in two parts of the type's digits, whose sum is the unrounded h to
// twice those digits: rounding it to one would err as much as rounding y does.  fp16's
// are scaled by a power of two for each place (unit_of in tl_grouped.cuh), so that an h outside fp16's
// range passes like any other.  The same holds for dh = s dy . b^T in the backward pass.
//
// Few rows, in the forward: nothing is sorted; a CTA takes a row and a share of the reduction
// (first launch) or of the columns (second), on the CUDA cores, since each weight
// is met by about one row and bytes bound it.  The second launch asks for its
// weights while the first still runs.  (The backward sorts any number of rows: da and db
// are sums over an adapter's.)
#include "tl_adapter.h"
#include "tl_route.h"

#include "tl_grouped.cuh"

#include <algorithm>
#include <type_traits>

namespace tl {
namespace {

using gr::grid_dependency_wait;
using gr::grid_dependents_go;
using gr::load_eight;
using gr::round16;
using gr::value16;

constexpr int kFewThreads = 256;
constexpr int64_t kFewRows = 256, kFewWork = 4096;
// Rows too few to sort: each reads an adapter's weights for itself.  8192 x 8192, us in
// a graph, this way against sorted: rank 16 of 64, 65 rows 19 / 69, 256 rows 36 / 72;
// of 2, 256 rows 33 / 44; rank 64, 64 rows 56 / 109; rank 128, 32 rows 89 / 115.  The
// limit is below the crossover, which has not been measured.
bool few_rows(int64_t tokens, int64_t rank) { return tokens <= kFewRows && tokens * rank <= kFewWork; }

struct FewArgs {
    int32_t tokens, K, n, rank, adapters, fp16;
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* a;
    int64_t lda, a_apart;
    const uint16_t* b;
    int64_t ldb, b_apart;
    const int32_t* ids;
    const float* scale;
    float scale_all;
    const void* base;
    int64_t ldbase;
    int32_t base_f32, base_vectors;
    uint16_t* h;
    int64_t ldh;
    uint16_t* y;
    int64_t ldy;
    float* parts;  // [tokens][splits][padded rank]
    int32_t padded, splits, per;
};

__device__ __forceinline__ void eight_values(const uint4& u, bool fp16, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (fp16) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            f[2 * j] = v.x;
            f[2 * j + 1] = v.y;
        } else {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}

// Grid (splits, tokens): a share of x[t] . a[id].  Eight ranks a thread.
__global__ void __launch_bounds__(kFewThreads) shrink_few_kernel(const FewArgs p) {
    __shared__ float sums[kFewThreads][9];
    grid_dependents_go();
    const int t = blockIdx.y, id = p.ids[t];
    if (unsigned(id) >= unsigned(p.adapters)) return;
    const int vectors = p.padded / 8, together = kFewThreads / vectors;  // rows of a at a time
    const int v = int(threadIdx.x) % vectors, first = int(threadIdx.x) / vectors;
    const int k0 = int(blockIdx.x) * p.per, k1 = min(p.K, k0 + p.per);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (first < together) {
        const uint16_t* x = p.x + int64_t(t) * p.ldx;
        const uint16_t* a = p.a + int64_t(id) * p.a_apart + 8 * v;
        const int have = p.rank - 8 * v;
        constexpr int kAhead = 8;  // loads under way
        for (int k = k0 + first; k < k1; k += kAhead * together) {
            uint4 u[kAhead];
            uint16_t w[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const bool there = k + q * together < k1;
                u[q] = there ? load_eight(a + int64_t(k + q * together) * p.lda, have) : make_uint4(0, 0, 0, 0);
                w[q] = there ? x[k + q * together] : uint16_t(0);
            }
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                float f[8];
                eight_values(u[q], p.fp16, f);
                const float v = value16(w[q], p.fp16);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = fmaf(v, f[j], acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[threadIdx.x][j] = acc[j];
    // halves of the threads with the same ranks are added until one is left
    int n = together;
    while (n > 1) {
        __syncthreads();
        const int upper = (n + 1) / 2;
        if (first + upper < n) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[threadIdx.x][j] += sums[threadIdx.x + upper * vectors][j];
        }
        n = upper;
    }
    __syncthreads();
    if (int(threadIdx.x) < p.padded)
        p.parts[(int64_t(t) * p.splits + blockIdx.x) * p.padded + threadIdx.x] = sums[threadIdx.x / 8][threadIdx.x % 8];
}

// Grid (columns / 2048, tokens): y[t] = base[t] + s h[t] . b[id], eight columns a thread.
__global__ void __launch_bounds__(kFewThreads) expand_few_kernel(const FewArgs p) {
    __shared__ float h[kAdapterMaxRank];
    const int t = blockIdx.y, id = p.ids[t];
    const bool some = unsigned(id) < unsigned(p.adapters);
    const int col = (int(blockIdx.x) * kFewThreads + int(threadIdx.x)) * 8, have = p.n - col;
    const uint16_t* b = p.b + (some ? int64_t(id) * p.b_apart : 0) + col;
    constexpr int kAhead = 16;
    uint4 w[kAhead];
    if (some && have > 0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (j < p.rank) w[j] = load_eight(b + int64_t(j) * p.ldb, have);
    }
    grid_dependency_wait();
    if (int(threadIdx.x) < p.rank) {
        float s = 0;
        if (some)
            for (int i = 0; i < p.splits; ++i) s += __ldcg(p.parts + (int64_t(t) * p.splits + i) * p.padded + threadIdx.x);
        h[threadIdx.x] = s;
        if (blockIdx.x == 0) p.h[int64_t(t) * p.ldh + threadIdx.x] = round16(s, p.fp16);
    }
    __syncthreads();
    if (have <= 0) return;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (some) {
        for (int j0 = 0; j0 < p.rank; j0 += kAhead) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (j0 + j < p.rank) {
                    float f[8];
                    eight_values(j0 ? load_eight(b + int64_t(j0 + j) * p.ldb, have) : w[j], p.fp16, f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] = fmaf(h[j0 + j], f[i], acc[i]);
                }
        }
    }
    const float scale = !some ? 0.0f : p.scale ? p.scale[id] : p.scale_all;
    float base[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (p.base) {
        const int64_t at = int64_t(t) * p.ldbase + col;
        if (p.base_vectors && have >= 8 && !p.base_f32) {
            eight_values(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.base) + at), p.fp16, base);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < have) base[i] = p.base_f32 ? static_cast<const float*>(p.base)[at + i] : value16(static_cast<const uint16_t*>(p.base)[at + i], p.fp16);
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = gr::round16x2(fmaf(acc[2 * i], scale, base[2 * i]), fmaf(acc[2 * i + 1], scale, base[2 * i + 1]), p.fp16);
    uint16_t* y = p.y + int64_t(t) * p.ldy + col;
    if (have >= 8) {
        *reinterpret_cast<uint4*>(y) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
        for (int i = 0; i < have; ++i) y[i] = uint16_t(o[i / 2] >> (16 * (i & 1)));
    }
}

// ---- base + s h . b for many rows ------------------------------------------------

// A CTA takes 128 rows of one adapter and, one after another, some tiles of 128
// columns; bytes bound it, so what counts is how many of base are asked for at a
// time: all of a thread's before the product, and by as many CTAs as fit.  The product is short (2 x 16 .. 128) and its
// operands are in shared memory; mma.sync leaves its sums in registers, in which a
// row's 16-byte vector is one thread's: column 8 c + 2 j + e of each 32 is
// column 2 c + e of the j-th MMA's eight.  8192 rows, us: 4096 columns, rank 16, 37 (3.6
// TB/s), rank 64 about 55; 8192 columns, rank 16, 67 (4.0 TB/s).  The grouped product's
// kernel with base added in its epilogue took 228 and 456; CTAs of 64 rows and 128
// threads, four an SM, 40 and 69.
constexpr int kExpandThreads = 256, kExpandRows = 128, kExpandCols = 128;

struct ExpandArgs {
    int32_t rows, own, groups, rank;
    const int32_t* offsets;
    const int32_t* index;  // the row of each place
    const uint16_t* h;     // [rows, 2 half], by place
    const float* units;    // of h's rows (fp16)
    const uint16_t* w;
    int64_t ldw, w_apart;
    const float* scale;
    float scale_all;
    const void* base;
    int64_t ldbase;
    int32_t base_f32, base_vectors;
    uint16_t* out;
    int64_t ldout;
    int32_t tiles, per, shares;  // tiles of columns, those of a CTA, CTAs for a block of rows
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <bool FP16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FP16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// HALF: the padded rank.  Shared memory: h's rows, then the weight as [HALF][128]
// (own contiguous; columns in the order above) or [128][HALF].
template <bool CONTIG, int HALF>
struct Expand {
    static constexpr int kPitchH = 4 * HALF + 16;                          // bytes; 16 more, so that eight rows are in different banks
    static constexpr int kPitchW = CONTIG ? 2 * kExpandCols + 16 : 2 * HALF + 16;
    static constexpr size_t kSmem = size_t(kExpandRows) * kPitchH + size_t(CONTIG ? HALF : kExpandCols) * kPitchW;
};

template <bool CONTIG, int HALF, bool FP16>
__global__ void __launch_bounds__(kExpandThreads, 2) expand_kernel(const ExpandArgs p) {
    using E = Expand<CONTIG, HALF>;
    extern __shared__ __align__(16) uint8_t expand_smem[];
    __shared__ int found[3], sums[kExpandThreads / 32];
    const int first = int(blockIdx.x % unsigned(p.shares)) * p.per, wanted = int(blockIdx.x / unsigned(p.shares));
    gr::find_block(p.offsets, p.groups, p.rows, true, kExpandRows, wanted, found, sums);
    const int group = found[0], p0 = found[1], count = found[2];
    if (group < 0) return;
    const bool none = group == p.groups;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int row0 = (warp & 3) * 32, col0 = (warp >> 2) * 64;  // of the warp: 32 x 64

    // what this thread adds to: rows g and g + 8 of two blocks of 16, a vector of each 32 columns
    int rows[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = row0 + i * 8 + g;
        rows[i] = r < count ? __ldg(p.index + p0 + r) : -1;
        if (unsigned(rows[i]) >= unsigned(p.rows)) rows[i] = -1;
    }
    const float scale = none ? 0.0f : p.scale ? __ldg(p.scale + group) : p.scale_all;
    const uint32_t sh = smem_addr(expand_smem), sw = sh + kExpandRows * E::kPitchH;
    __shared__ float unit[kExpandRows];
    if constexpr (FP16) {
        if (int(threadIdx.x) < kExpandRows) unit[threadIdx.x] = int(threadIdx.x) < count ? __ldg(p.units + p0 + int(threadIdx.x)) : 0.0f;
        __syncthreads();
    }
    if (!none) {
        constexpr int kVecH = HALF / 4;  // 16-byte vectors of h's row
        for (int v = threadIdx.x; v < kExpandRows * kVecH; v += kExpandThreads) {
            const int r = v / kVecH, k = v % kVecH;
            gr::cp_async16(sh + uint32_t(r) * E::kPitchH + uint32_t(k) * 16u, p.h + int64_t(p0 + min(r, count - 1)) * (2 * HALF) + k * 8, 16);
        }
        gr::cp_async_commit();
    }
#pragma unroll 1
    for (int tile = first; tile < min(p.tiles, first + p.per); ++tile) {
        const int n0 = tile * kExpandCols;
        uint4 base[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = n0 + col0 + j * 32 + c * 8;
                base[i][j] = make_uint4(0, 0, 0, 0);
                if (p.base_vectors && rows[i] >= 0 && col + 8 <= p.own)
                    base[i][j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.base) + int64_t(rows[i]) * p.ldbase + col);
            }

        float acc[2][8][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][j][k] = 0;
        if (!none) {
            if (tile != first) __syncthreads();  // (the tile before has been multiplied)
            const uint16_t* w = p.w + int64_t(group) * p.w_apart;
            if constexpr (CONTIG) {
                for (int v = threadIdx.x; v < HALF * 16; v += kExpandThreads) {
                    const int k = v / 16, q = v % 16, col = n0 + q * 8;
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (k < p.rank && col < p.own) u = load_eight(w + int64_t(k) * p.ldw + col, p.own - col);
                    uint8_t* at = expand_smem + kExpandRows * E::kPitchH + k * E::kPitchW + (q / 4 * 32 + q % 4 * 2) * 2;
                    *reinterpret_cast<uint32_t*>(at) = u.x;
                    *reinterpret_cast<uint32_t*>(at + 16) = u.y;
                    *reinterpret_cast<uint32_t*>(at + 32) = u.z;
                    *reinterpret_cast<uint32_t*>(at + 48) = u.w;
                }
            } else {
                constexpr int kVecW = HALF / 8;
                for (int v = threadIdx.x; v < kExpandCols * kVecW; v += kExpandThreads) {
                    const int col = v / kVecW, k = v % kVecW * 8;
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (n0 + col < p.own && k < p.rank) u = load_eight(w + int64_t(n0 + col) * p.ldw + k, p.rank - k);
                    *reinterpret_cast<uint4*>(expand_smem + kExpandRows * E::kPitchH + col * E::kPitchW + k * 2) = u;
                }
            }
            gr::cp_async_wait<0>();
            __syncthreads();
            // (a lane's row of the four 8 x 8 parts that an ldmatrix takes)
            const int part = lane >> 3, in = lane & 7;
#pragma unroll 1
            for (int ks = 0; ks < HALF / 16; ++ks) {
                uint32_t a[2][2][4];  // [part of h][block of 16 rows]
#pragma unroll
                for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        ldmatrix4(sh + uint32_t(row0 + i * 16 + (part & 1) * 8 + in) * E::kPitchH + uint32_t(hl * HALF + ks * 16 + (part >> 1) * 8) * 2u, a[hl][i]);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {  // MMAs' columns j * 8 .., j of each four in one 32
                    uint32_t b[4];
                    const int q = j / 4 * 32, t = j % 4 + (part >> 1);
                    if constexpr (CONTIG)
                        ldmatrix4_trans(sw + uint32_t(ks * 16 + (part & 1) * 8 + in) * E::kPitchW + uint32_t(col0 + q + t * 8) * 2u, b);
                    else
                        ldmatrix4(sw + uint32_t(col0 + q + 8 * (in >> 1) + 2 * t + (in & 1)) * E::kPitchW + uint32_t(ks * 16 + (part & 1) * 8) * 2u, b);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int hl = 0; hl < 2; ++hl) {
                            mma16816<FP16>(acc[i][j], a[hl][i], b[0], b[1]);
                            mma16816<FP16>(acc[i][j + 1], a[hl][i], b[2], b[3]);
                        }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = n0 + col0 + j * 32 + c * 8, have = p.own - col;
                if (rows[i] < 0 || have <= 0) continue;
                float b[8];
                eight_values(base[i][j], FP16, b);
                if (p.base && (!p.base_vectors || have < 8)) {
                    const int64_t at = int64_t(rows[i]) * p.ldbase + col;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < have) b[k] = p.base_f32 ? static_cast<const float*>(p.base)[at + k] : value16(static_cast<const uint16_t*>(p.base)[at + k], FP16);
                }
                uint32_t o[4];
                const float u = FP16 ? unit[row0 + i * 8 + g] : 1.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float* f = acc[i >> 1][j * 4 + k] + (i & 1) * 2;
                    o[k] = gr::round16x2(fmaf(f[0] * u, scale, b[2 * k]), fmaf(f[1] * u, scale, b[2 * k + 1]), FP16);
                }
                uint16_t* dst = p.out + int64_t(rows[i]) * p.ldout + col;
                if (have >= 8) {
                    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
                    for (int k = 0; k < have; ++k) dst[k] = uint16_t(o[k / 2] >> (16 * (k & 1)));
                }
            }
    }
}

bool off(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int32_t half_of(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

constexpr int kFewSplits = 16;

struct Workspace {
    int32_t *slots, *rows, *offsets, *counts;
    uint16_t* split;  // [tokens, 2 half], by place
    float* units;     // fp16: of the split's rows
    size_t bytes;
    Workspace(void* base, int64_t tokens, int64_t rank, int64_t adapters) {
        uintptr_t at = reinterpret_cast<uintptr_t>(base);
        const auto take = [&](size_t n) {
            void* p = reinterpret_cast<void*>(at);
            at += up256(n);
            return p;
        };
        slots = static_cast<int32_t*>(take(size_t(tokens) * 4));
        rows = static_cast<int32_t*>(take(size_t(tokens) * 4));
        offsets = static_cast<int32_t*>(take(size_t(adapters + 1) * 4));
        counts = static_cast<int32_t*>(take(route_workspace(tokens, 1, adapters)));
        units = reinterpret_cast<float*>(slots);  // (the sort's slots are nobody's; its launches have ended by then)
        split = static_cast<uint16_t*>(take(size_t(tokens) * 4 * size_t(half_of(rank))));
        bytes = size_t(at - reinterpret_cast<uintptr_t>(base));
    }
};

cudaError_t sort_rows(const AdapterDesc& d, const Workspace& w, cudaStream_t stream) {
    RouteDesc r;
    r.tokens = d.tokens;
    r.k = 1;
    r.groups = d.adapters;
    r.ids = const_cast<int32_t*>(d.ids);
    r.slots = w.slots;
    r.rows = w.rows;
    r.offsets = w.offsets;
    r.counts = w.counts;
    return group_rows_launch(r, stream);
}

GroupedDesc product(const AdapterDesc& d, const Workspace& w) {
    GroupedDesc g;
    g.rows = d.tokens;
    g.groups = d.adapters;
    g.type = d.type;
    g.offsets = w.offsets;
    g.x.count = g.out.count = d.tokens;
    g.x.index = g.out.index = w.rows;
    g.all_rows = true;
    g.err = d.err;
    return g;
}

// h (or dh) of all rows: x . a, or s dy . b^T.
GroupedDesc shrink(const AdapterDesc& d, const Workspace& w, bool backward) {
    GroupedDesc g = product(d, w);
    g.x.at = backward ? d.dy : d.x;
    g.x.ld = backward ? d.lddy : d.ldx;
    g.w = backward ? d.b : d.a;
    g.ldw = backward ? d.ldb : d.lda;
    g.w_apart = backward ? d.b_apart : d.a_apart;
    g.own_contiguous = !backward;
    g.reduce = backward ? d.n : d.K;
    g.own = d.rank;
    if (!backward) {
        g.out.at = d.h;
        g.out.ld = d.ldh;
    } else {
        g.scale = d.scale;
        g.scale_all = d.scale_all;
    }
    g.split_out = w.split;
    g.split_half = half_of(d.rank);
    if (d.type == TL_TYPE_F16) g.split_units = w.units;
    return g;
}

// Whole blocks of rows, and one of each adapter (and of the rows behind them) that has a row.
int64_t expand_blocks(const AdapterDesc& d) { return d.tokens / kExpandRows + std::min(d.adapters + 1, d.tokens); }
int64_t expand_tiles(int64_t cols) { return (cols + kExpandCols - 1) / kExpandCols; }
constexpr int64_t kExpandMost = 8;  // tiles of a CTA

// y (or dx) of all rows: base + s h . b, or base + dh . a^T.
cudaError_t expand(const AdapterDesc& d, const Workspace& w, bool backward, int num_sms, cudaStream_t stream) {
    ExpandArgs p{};
    p.rows = int32_t(d.tokens);
    p.own = int32_t(backward ? d.K : d.n);
    p.groups = int32_t(d.adapters);
    p.rank = int32_t(d.rank);
    p.offsets = w.offsets;
    p.index = w.rows;
    p.h = w.split;
    p.units = w.units;
    p.w = static_cast<const uint16_t*>(backward ? d.a : d.b);
    p.ldw = backward ? d.lda : d.ldb;
    p.w_apart = backward ? d.a_apart : d.b_apart;
    p.scale = backward ? nullptr : d.scale;  // (dh has it already)
    p.scale_all = backward ? 1.0f : d.scale_all;
    p.base = d.base;
    p.ldbase = d.ldbase;
    p.base_f32 = d.base_type == TL_TYPE_F32 ? 1 : 0;
    p.base_vectors = d.base && !p.base_f32 && !off(d.base, 16) && d.ldbase % 8 == 0 ? 1 : 0;
    p.out = static_cast<uint16_t*>(backward ? d.dx : d.y);
    p.ldout = backward ? d.lddx : d.ldy;
    p.tiles = int32_t(expand_tiles(p.own));
    const int64_t blocks = expand_blocks(d);
    // tiles of a CTA: what it finds and loads once counts less with more of them, as
    // long as there are four CTAs for an SM (8192 x 8192, rank 16, us with 1 / 7: 74 / 67)
    p.per = int32_t(std::max<int64_t>(1, std::min<int64_t>(kExpandMost, blocks * p.tiles / (4 * std::max(1, num_sms)))));
    p.shares = (p.tiles + p.per - 1) / p.per;
    const int64_t ctas = blocks * p.shares;
    auto run = [&](auto contig, auto half) {
        constexpr bool CONTIG = decltype(contig)::value;
        constexpr int HALF = decltype(half)::value;
        constexpr size_t smem = Expand<CONTIG, HALF>::kSmem;
        return d.type == TL_TYPE_F16 ? launch_in_clusters(expand_kernel<CONTIG, HALF, true>, dim3(unsigned(ctas)), kExpandThreads, 1, smem, false, stream, p)
                                     : launch_in_clusters(expand_kernel<CONTIG, HALF, false>, dim3(unsigned(ctas)), kExpandThreads, 1, smem, false, stream, p);
    };
    auto by_half = [&](auto contig) {
        switch (half_of(d.rank)) {
            case 16: return run(contig, std::integral_constant<int, 16>{});
            case 32: return run(contig, std::integral_constant<int, 32>{});
            case 64: return run(contig, std::integral_constant<int, 64>{});
            default: return run(contig, std::integral_constant<int, 128>{});
        }
    };
    return backward ? by_half(std::false_type{}) : by_half(std::true_type{});
}

GroupedDwDesc gradient(const AdapterDesc& d, const Workspace& w, bool of_b) {
    GroupedDwDesc g;
    g.rows = d.tokens;
    g.groups = d.adapters;
    g.type = d.type;
    g.offsets = w.offsets;
    g.x.count = g.dy.count = d.tokens;
    g.x.index = g.dy.index = w.rows;
    g.n_dim = d.rank;
    g.err = d.err;
    if (!of_b) {
        g.m_dim = d.K;
        g.x.at = d.x;
        g.x.ld = d.ldx;
        g.half = half_of(d.rank);
        if (d.type == TL_TYPE_F16) g.dy_units = w.units;
        g.dy = {w.split, 2 * g.half, d.tokens, nullptr};  // by place
        g.dw = d.da;
        g.lddw = d.ldda;
        g.dw_apart = d.da_apart;
    } else {
        g.m_dim = d.n;
        g.x.at = d.dy;
        g.x.ld = d.lddy;
        g.dy.at = d.h;
        g.dy.ld = d.ldh;
        g.dw = d.db;
        g.lddw = d.lddb;
        g.dw_apart = d.db_apart;
        g.transposed = true;
        g.scale = d.scale;
        g.scale_all = d.scale_all;
    }
    return g;
}

cudaError_t few_forward(const AdapterDesc& d, int num_sms, cudaStream_t stream) {
    FewArgs p{};
    p.tokens = int32_t(d.tokens);
    p.K = int32_t(d.K);
    p.n = int32_t(d.n);
    p.rank = int32_t(d.rank);
    p.adapters = int32_t(d.adapters);
    p.fp16 = d.type == TL_TYPE_F16 ? 1 : 0;
    p.x = static_cast<const uint16_t*>(d.x);
    p.ldx = d.ldx;
    p.a = static_cast<const uint16_t*>(d.a);
    p.lda = d.lda;
    p.a_apart = d.a_apart;
    p.b = static_cast<const uint16_t*>(d.b);
    p.ldb = d.ldb;
    p.b_apart = d.b_apart;
    p.ids = d.ids;
    p.scale = d.scale;
    p.scale_all = d.scale_all;
    p.base = d.base;
    p.ldbase = d.ldbase;
    p.base_f32 = d.base_type == TL_TYPE_F32 ? 1 : 0;
    p.base_vectors = d.base && !off(d.base, 16) && d.ldbase % 8 == 0 ? 1 : 0;
    p.h = static_cast<uint16_t*>(d.h);
    p.ldh = d.ldh;
    p.y = static_cast<uint16_t*>(d.y);
    p.ldy = d.ldy;
    p.parts = static_cast<float*>(d.workspace);
    p.padded = int32_t((d.rank + 7) / 8 * 8);
    // shares of the reduction: about two CTAs an SM, of 256 elements at least
    int64_t splits = std::max<int64_t>(1, std::min<int64_t>(kFewSplits, 2 * num_sms / d.tokens));
    splits = std::min(splits, (d.K + 255) / 256);
    p.per = int32_t((d.K + splits - 1) / splits);
    p.splits = int32_t((d.K + p.per - 1) / p.per);
    shrink_few_kernel<<<dim3(unsigned(p.splits), unsigned(d.tokens)), kFewThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((d.n + 8 * kFewThreads - 1) / (8 * kFewThreads)), unsigned(d.tokens));
    cfg.blockDim = dim3(kFewThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, expand_few_kernel, p);
}

}  // namespace

size_t adapter_workspace(int64_t tokens, int64_t rank, int64_t adapters) {
    if (tokens < 0 || tokens > INT32_MAX / 2 || rank < 1 || rank > kAdapterMaxRank || adapters < 1 || adapters > kMaxGroups) return 0;
    const size_t few = few_rows(tokens, rank) ? size_t(tokens) * kFewSplits * size_t((rank + 7) / 8 * 8) * 4 : 0;
    return std::max<size_t>(256, std::max(few, Workspace(nullptr, tokens, rank, adapters).bytes));
}

std::string adapter_check(const AdapterDesc& d, bool backward) {
    constexpr int64_t kMost = INT32_MAX / 2;
    if (d.tokens < 0 || d.K < 1 || d.n < 1 || d.tokens > kMost || d.K > kMost || d.n > kMost) return "T must be >= 0, K and n >= 1, all below 2^30";
    if (d.rank < 1 || d.rank > kAdapterMaxRank) return "the rank must be 1..128";
    if (d.adapters < 1 || d.adapters > kMaxGroups) return "adapters must be 1..1024";
    if (d.tokens > 0 && (!d.ids || off(d.ids, 4))) return "ids is null or not 4-byte aligned";
    const Workspace w(reinterpret_cast<void*>(uintptr_t(256)), d.tokens, d.rank, d.adapters);
    std::string bad = grouped_check(shrink(d, w, backward));
    if (!bad.empty()) return bad;
    if (d.tokens > 0) {
        if (backward ? !d.dx && !d.da : !d.h || !d.y) return "null pointer";
        if (!d.x || !d.a || !d.b || off(d.x, 16) || off(d.a, 16) || off(d.b, 16)) return "x, a or b is null or not 16-byte aligned";
        if (d.lda % 8 || d.ldb % 8 || d.a_apart % 8 || d.b_apart % 8 || d.ldx % 8) return "leading dimensions must be multiples of 8 elements";
        if (d.ldx < d.K || d.lda < d.rank || d.ldb < d.n) return "a leading dimension is smaller than a row";
        if (d.adapters > 1 && (d.a_apart < (d.K - 1) * d.lda + d.rank || d.b_apart < (d.rank - 1) * d.ldb + d.n)) return "the adapters' weights overlap";
        const void* out = backward ? d.dx : d.y;
        const int64_t ldout = backward ? d.lddx : d.ldy, cols = backward ? d.K : d.n;
        if (out && (off(out, 16) || ldout % 8 || ldout < cols)) return "the result is not 16-byte aligned, or its leading dimension no multiple of 8 or too small";
        if (off(d.scale, 4)) return "scales must be 4-byte aligned";
        if (d.base && d.base == out && (d.base_type != d.type || (d.tokens > 1 && d.ldbase != ldout)))
            return "base lies where the result does, but is of another type or leading dimension";
        if (out && expand_blocks(d) * ((expand_tiles(cols) + kExpandMost - 1) / kExpandMost) > INT32_MAX) return "too many tiles";
        if (d.base && d.base_type != d.type && d.base_type != TL_TYPE_F32) return "base must be of x's type or fp32";
        if (d.base && (off(d.base, type_bytes(d.base_type)) || d.ldbase < cols)) return "base is not aligned to its elements, or its leading dimension too small";
    }
    if (backward && !d.da != !d.db) return "one of da and db is null, the other not";
    if (backward && d.da) {
        bad = grouped_dw_check(gradient(d, w, false));
        if (bad.empty()) bad = grouped_dw_check(gradient(d, w, true));
    }
    return bad;
}

cudaError_t adapter_forward_launch(const AdapterDesc& d, int num_sms, cudaStream_t stream, std::string* why) {
    if (d.tokens == 0) return cudaSuccess;
    if (few_rows(d.tokens, d.rank)) return few_forward(d, num_sms, stream);
    const Workspace w(d.workspace, d.tokens, d.rank, d.adapters);
    cudaError_t e = sort_rows(d, w, stream);
    if (e == cudaSuccess) e = grouped_launch(shrink(d, w, false), num_sms, stream, why);
    if (e == cudaSuccess) e = expand(d, w, false, num_sms, stream);
    return e;
}

cudaError_t adapter_backward_launch(const AdapterDesc& d, int num_sms, cudaStream_t stream, std::string* why) {
    const Workspace w(d.workspace, d.tokens, d.rank, d.adapters);
    cudaError_t e = cudaSuccess;
    if (d.tokens > 0) {
        e = sort_rows(d, w, stream);
        if (e == cudaSuccess) e = grouped_launch(shrink(d, w, true), num_sms, stream, why);
        if (e == cudaSuccess && d.dx) e = expand(d, w, true, num_sms, stream);
    }
    if (e == cudaSuccess && d.da) e = grouped_dw_launch(gradient(d, w, false), num_sms, stream, why);
    if (e == cudaSuccess && d.da) e = grouped_dw_launch(gradient(d, w, true), num_sms, stream, why);
    return e;
}

}  // namespace tl
