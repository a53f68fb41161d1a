// tl_adapter.cu -- low-rank adapters of many requests beside a shared projection.
//
// Many rows: the rows are sorted by adapter (tl_route.cu) and both products are
// products whose weight depends on the row (tl_grouped.cu): h = x . a, bound by the
// bytes of x, and y = base + s h . b, bound by those of base and y.  h goes from one
// to the other in two parts of the type's digits, whose sum is the unrounded h to
// twice those digits: rounding it to one would err as much as rounding y does.  The
// same holds for dh = s dy . b^T in the backward pass.
//
// Few rows: nothing is sorted; a CTA takes a row and a share of the reduction
// (first launch) or of the columns (second), on the CUDA cores, since each weight
// is met by about one row and bytes bound it.  The second launch asks for its
// weights while the first still runs.
#include "tl_adapter.h"
#include "tl_route.h"

#include "tl_grouped.cuh"

#include <algorithm>

namespace tl {
namespace {

using gr::grid_dependency_wait;
using gr::grid_dependents_go;
using gr::round16;
using gr::value16;

constexpr int kFewThreads = 256;
constexpr int64_t kFewRows = 64;

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

// Eight elements, of which `have` are there.
__device__ __forceinline__ uint4 load_eight(const uint16_t* p, int have) {
    if (have >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < have) w[j / 2] |= uint32_t(p[j]) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
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
#pragma unroll 8
        for (int k = k0 + first; k < k1; k += together) {
            float f[8];
            eight_values(load_eight(a + int64_t(k) * p.lda, have), p.fp16, f);
            const float w = value16(x[k], p.fp16);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = fmaf(w, f[j], acc[j]);
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

bool off(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int32_t half_of(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

constexpr int kFewSplits = 16;

struct Workspace {
    int32_t *slots, *rows, *offsets, *counts;
    uint16_t* split;  // [tokens, 2 half], by place
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
    return g;
}

// y (or dx) of all rows: base + s h . b, or base + dh . a^T.
GroupedDesc expand(const AdapterDesc& d, const Workspace& w, bool backward) {
    GroupedDesc g = product(d, w);
    g.half = half_of(d.rank);
    g.x = {w.split, 2 * g.half, d.tokens, nullptr};  // by place
    g.w = backward ? d.a : d.b;
    g.ldw = backward ? d.lda : d.ldb;
    g.w_apart = backward ? d.a_apart : d.b_apart;
    g.own_contiguous = !backward;
    g.reduce = d.rank;
    g.own = backward ? d.K : d.n;
    g.out.at = backward ? d.dx : d.y;
    g.out.ld = backward ? d.lddx : d.ldy;
    if (!backward) {
        g.scale = d.scale;
        g.scale_all = d.scale_all;
    }
    g.base = d.base;
    g.base_type = d.base_type;
    g.ldbase = d.ldbase;
    return g;
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
    const size_t few = size_t(std::min(tokens, kFewRows)) * kFewSplits * size_t(kAdapterMaxRank) * 4;
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
    if (bad.empty() && (!backward || d.dx)) bad = grouped_check(expand(d, w, backward));
    if (bad.empty() && d.tokens > 0 && (backward ? !d.dx && !d.da : !d.h || !d.y)) bad = "null pointer";
    if (bad.empty() && backward && !d.da != !d.db) bad = "one of da and db is null, the other not";
    if (bad.empty() && backward && d.da) {
        bad = grouped_dw_check(gradient(d, w, false));
        if (bad.empty()) bad = grouped_dw_check(gradient(d, w, true));
    }
    return bad;
}

cudaError_t adapter_forward_launch(const AdapterDesc& d, int num_sms, cudaStream_t stream, std::string* why) {
    if (d.tokens == 0) return cudaSuccess;
    if (d.tokens <= kFewRows) return few_forward(d, num_sms, stream);
    const Workspace w(d.workspace, d.tokens, d.rank, d.adapters);
    cudaError_t e = sort_rows(d, w, stream);
    if (e == cudaSuccess) e = grouped_launch(shrink(d, w, false), num_sms, stream, why);
    if (e == cudaSuccess) e = grouped_launch(expand(d, w, false), num_sms, stream, why);
    return e;
}

cudaError_t adapter_backward_launch(const AdapterDesc& d, int num_sms, cudaStream_t stream, std::string* why) {
    const Workspace w(d.workspace, d.tokens, d.rank, d.adapters);
    cudaError_t e = cudaSuccess;
    if (d.tokens > 0) {
        e = sort_rows(d, w, stream);
        if (e == cudaSuccess) e = grouped_launch(shrink(d, w, true), num_sms, stream, why);
        if (e == cudaSuccess && d.dx) e = grouped_launch(expand(d, w, true), num_sms, stream, why);
    }
    if (e == cudaSuccess && d.da) e = grouped_dw_launch(gradient(d, w, false), num_sms, stream, why);
    if (e == cudaSuccess && d.da) e = grouped_dw_launch(gradient(d, w, true), num_sms, stream, why);
    return e;
}

}  // namespace tl
