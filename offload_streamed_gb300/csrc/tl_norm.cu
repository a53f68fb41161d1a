// tl_norm.cu -- layer norm over the rows of a [rows, cols] matrix, forward and
// backward, for bf16, fp16 and fp32.
//
//   forward   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps)
//             y = (x - m) r w + b
//   backward  xh = (x - m) r, g = dy w
//             dx = r (g - mean(g) - xh mean(g xh))
//             dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both are bound by memory: the forward reads and writes each element once,
// the backward reads two and writes one.  So a row is read from global memory
// once, and the rest of its work is done on the copy in shared memory:
//  - Every CTA (or cluster, or warp) walks over many rows.  A thread owns the
//    same columns of all of them, so the weight stays with it, and the sums
//    of the weight's gradient grow in its registers; only one partial sum per
//    CTA and column goes through memory.
//  - A thread copies its own columns of the next rows into its own shared
//    memory (cp.async, several rows ahead) and is the only reader of them:
//    the copies need no barrier, only the thread's own wait.
//  - A row's statistics need all its threads.  Rows of up to 1024 columns
//    belong to one warp (shuffles alone); longer ones to a CTA, or to a
//    cluster of up to eight when a CTA cannot hold them.  There every
//    warp leaves its sums for all others, and one barrier a row is all there is.
// Measured: 8192 x 8192 bf16 forward 57 us (4.7 TB/s), backward 81 us (5.0 TB/s,
// its reduction included); 2048 x 65536, clusters of eight, 133 and 183 us (4.0
// and 4.4 TB/s).  DRAM is about half busy at 8192 x 8192, with 15 warps an SM;
// what their counted stalls wait for most is shared memory.
// All statistics and sums are fp32.  A row's variance is joined from the
// warps' sums of squares about their own means, which loses nothing to
// cancellation, whatever the row's mean.  Every order of summation is fixed by
// the sizes, the type, the alignment (which picks the vectors) and the device's
// SMs and clusters (which pick the grid).
#include "tl_norm.h"
#include "tl_launch.h"
#include "tl_types.cuh"

#include <algorithm>

namespace tl {
namespace {

constexpr int kMaxRing = 4;         // rows in flight per thread
constexpr int kWarpRowWarps = 8;    // rows of a CTA at a time where a warp has a row
constexpr int kMaxWarps = 16;       // of a CTA that shares a row
constexpr int kMaxCluster = 8;
constexpr size_t kSmemBudget = 220 * 1024;  // of an SM, for its CTAs
constexpr uint32_t kMaxPolls = 200000;  // of an mbarrier, up to 10 us each
constexpr int kMaxSms = 152, kCtasPerSm = 4;  // bound the grid, and with it the partial sums

struct NormArgs {
    const void* x;
    int64_t ldx;
    const void* dy;
    int64_t lddy;
    void* out;
    int64_t ldout;
    const void* weight;
    const void* bias;
    float* mean;
    float* rstd;
    float* dweight;
    float* dbias;
    float* partials;
    int64_t rows;
    int32_t cols, seg;  // seg: columns of each CTA of a cluster
    int32_t param_type, ring, cluster;
    float eps;
    int32_t* err;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// At most `pending` of the thread's newest groups may be unfinished.
__device__ __forceinline__ void cp_async_wait(int pending) {
    switch (pending) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}
__device__ __forceinline__ uint32_t saddr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The exchange of a row's sums among the warps of a cluster.  Every warp sends
// its entry to every CTA; the stores carry their own completion to the
// receiving CTA's mbarrier, so that no fence waits for the row's other writes
// (a cluster barrier's release does: 2048 x 65536 bf16 forward 258 us with it,
// 214 us with this, both measured with a grid of more clusters than run at a time).
// Two mbarriers and two buffers in turn: a CTA sends for the row after next
// only once it has had the next row's entries from all, and each of those was
// sent by a warp that was done with this row.
template <int WORDS>
struct Exchange {
    uint32_t bar, buf;  // shared addresses: mbarrier b at bar + 8 b, buffer b at buf + b * kBuf
    uint32_t bytes, entry, phase = 0;
    int32_t* err;
    bool ok = true;
    static constexpr uint32_t kBuf = kMaxCluster * kMaxWarps * WORDS * 4;
    // Entry of this warp: `entry`, of `n` in all.
    __device__ __forceinline__ void send(int b, int lane, int cluster, const float (&v)[WORDS]) {
        if (threadIdx.x == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar + 8 * b), "r"(bytes) : "memory");
        if (lane < cluster) {
            const uint32_t dst = buf + b * kBuf + entry * (WORDS * 4);
#pragma unroll
            for (int i = 0; i < WORDS; i += 2)
                asm volatile(
                    "{\n\t.reg .b32 a, m;\n\t"
                    "mapa.shared::cluster.u32 a, %0, %2;\n\t"
                    "mapa.shared::cluster.u32 m, %1, %2;\n\t"
                    "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [a], {%3, %4}, [m];\n\t}" ::"r"(dst + 4 * i),
                    "r"(bar + 8 * b), "r"(lane), "r"(__float_as_uint(v[i])), "r"(__float_as_uint(v[i + 1]))
                    : "memory");
        }
    }
    // Wait (bounded) for all entries of buffer b.
    __device__ __forceinline__ void wait(int b) {
        const uint32_t parity = (phase >> 1) & 1;
        ++phase;
        for (uint32_t n = 0; ok; ++n) {
            uint32_t done;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 10000;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(done)
                : "r"(bar + 8 * b), "r"(parity)
                : "memory");
            if (done) return;
            if (n > kMaxPolls) {
                atomicOr(err, 1);
                ok = false;  // the rows that follow are not waited for: the caller reads the error word
            }
        }
    }
};

// Count, mean and sum of squares about the mean of a set of values.
struct Moments {
    float n, mean, m2, none;
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(~0u, v, s);
    return v;
}

// Sums over the n entries that a row's warps left: up to 16 are had by both
// halves of the warp, which saves a step.
template <typename F>
__device__ __forceinline__ void for_entries(int lane, int n, F&& f) {
    if (n <= 16) {
        if ((lane & 15) < n) f(lane & 15);
    } else {
        for (int i = lane; i < n; i += 32) f(i);
    }
}
__device__ __forceinline__ float set_sum(float v, int n) {
    if (n > 16) v += __shfl_xor_sync(~0u, v, 16);
#pragma unroll
    for (int s = 8; s; s >>= 1) v += __shfl_xor_sync(~0u, v, s);
    return v;
}
__device__ __forceinline__ float lane_of(const float (&v)[1], int) { return v[0]; }
template <int N>
__device__ __forceinline__ float lane_of(const float2 (&v)[N], int e) {
    return e & 1 ? v[e / 2].y : v[e / 2].x;
}

// A vector in shared memory, by its 32-bit address.
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> lds(uint32_t a) {
    Vec<T, VEC> u;
    if constexpr (VEC * sizeof(T) == 16) {
        uint32_t* w = reinterpret_cast<uint32_t*>(u.v);
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
    } else if constexpr (sizeof(T) == 4) {
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(*reinterpret_cast<float*>(u.v)) : "r"(a) : "memory");
    } else {
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(*reinterpret_cast<uint16_t*>(u.v)) : "r"(a) : "memory");
    }
    return u;
}
template <typename T, int VEC>
__device__ __forceinline__ void sts(uint32_t a, const Vec<T, VEC>& u) {
    if constexpr (VEC * sizeof(T) == 16) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(u.v);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    } else if constexpr (sizeof(T) == 4) {
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(*reinterpret_cast<const float*>(u.v)) : "memory");
    } else {
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(*reinterpret_cast<const uint16_t*>(u.v)) : "memory");
    }
}

// The columns of one thread: ITEMS vectors of VEC elements.  A warp's columns
// are adjacent, and so are its lanes' k-th vectors: its accesses are
// contiguous, and the distances between a thread's vectors are constants.
// FULL: the row has all of the warp's columns, and nothing is asked.
template <typename T, int VEC, int ITEMS, bool FULL>
struct Cols {
    static constexpr int kStep = 32 * VEC;               // columns between its vectors
    static constexpr uint32_t kSlot = kStep * sizeof(T);  // bytes between them in a ring slot
    int first;  // column of its first vector, in the row
    int end;    // columns of the CTA end here
    __device__ __forceinline__ int col(int k) const { return first + k * kStep; }
    __device__ __forceinline__ bool has(int k) const { return FULL || col(k) < end; }
};

// Copy the thread's columns of a row to its part of a ring slot.  `row` points
// at the thread's first column.
template <typename T, int VEC, int ITEMS, bool FULL>
__device__ __forceinline__ void fetch(const Cols<T, VEC, ITEMS, FULL>& c, const T* row, uint32_t slot) {
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (c.has(k)) cp_async16(slot + k * c.kSlot, row + k * c.kStep);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (c.has(k)) cp_async4(slot + k * c.kSlot, row + k * c.kStep);
    } else {
        Vec<T, 1> v[ITEMS];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (c.has(k)) v[k].v[0] = row[k * c.kStep];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (c.has(k)) sts(slot + k * c.kSlot, v[k]);
    }
}

// A parameter (weight or bias) at the thread's columns, as fp32 in the thread's
// own shared memory, in chunks of up to 16 bytes.
template <int VEC>
struct Param {
    static constexpr int kChunk = VEC > 1 ? 4 : 1;
    static constexpr uint32_t kStep = 32 * kChunk * 4;  // bytes between a thread's chunks
    uint32_t at;
    template <typename T, int ITEMS, bool FULL>
    __device__ __forceinline__ Param(uint32_t base, const Cols<T, VEC, ITEMS, FULL>& c, const void* p, int32_t type, float none) {
        at = base + (threadIdx.x / 32) * (ITEMS * VEC / kChunk) * kStep + (threadIdx.x % 32) * (kChunk * 4);
        if (VEC > 1 && p && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {  // (a thread's columns start on VEC)
            Vec<float, 4> u[ITEMS * VEC / kChunk];
#pragma unroll
            for (int k = 0; k < ITEMS * VEC / kChunk; ++k)
                if (c.has(k * kChunk / VEC)) u[k] = load4_as_f32(p, type, c.col(k * kChunk / VEC) + k * kChunk % VEC);
#pragma unroll
            for (int k = 0; k < ITEMS * VEC / kChunk; ++k)
                if (c.has(k * kChunk / VEC)) sts(at + k * kStep, u[k]);
            return;
        }
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (c.has(k))
#pragma unroll
                for (int q = 0; q < VEC / kChunk; ++q) {
                    Vec<float, kChunk> u;
#pragma unroll
                    for (int e = 0; e < kChunk; ++e) u.v[e] = p ? load_as_f32(p, type, c.col(k) + q * kChunk + e) : none;
                    sts(at + (k * (VEC / kChunk) + q) * kStep, u);
                }
    }
    __device__ __forceinline__ void get(int k, float (&v)[1]) const { v[0] = lds<float, 1>(at + k * kStep).v[0]; }
    template <int N>
    __device__ __forceinline__ void get(int k, float2 (&v)[N]) const {
#pragma unroll
        for (int q = 0; q < N / 2; ++q) {
            const Vec<float, 4> u = lds<float, 4>(at + (k * (VEC / kChunk) + q) * kStep);
            v[2 * q] = make_float2(u.v[0], u.v[1]);
            v[2 * q + 1] = make_float2(u.v[2], u.v[3]);
        }
    }
};

// Which rows and columns a thread works on, and where its part of the CTA's
// ring begins.
template <typename T, int VEC, int ITEMS, bool WARP_ROW, bool FULL>
struct Place {
    Cols<T, VEC, ITEMS, FULL> c;
    int64_t row, stride;  // first row and the distance to the next
    uint32_t rank, ring, slot_bytes;
    __device__ __forceinline__ Place(const NormArgs& p, const void* smem) {
        const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        slot_bytes = blockDim.x * (VEC * ITEMS * sizeof(T));
        ring = saddr(smem) + warp * (ITEMS * c.kSlot) + lane * (VEC * sizeof(T));
        if constexpr (WARP_ROW) {
            const int warps = blockDim.x / 32;
            rank = 0;
            c.first = lane * VEC;
            c.end = p.cols;
            row = int64_t(blockIdx.x) * warps + warp;
            stride = int64_t(gridDim.x) * warps;
        } else {
            rank = p.cluster > 1 ? cluster_rank() : 0;
            const int c0 = int(rank) * p.seg;
            c.first = c0 + warp * ITEMS * c.kStep + lane * VEC;
            c.end = min(p.cols, c0 + p.seg);
            row = blockIdx.x / uint32_t(p.cluster);
            stride = gridDim.x / uint32_t(p.cluster);
        }
    }
};

// Whether the row has all of this warp's columns.
template <int E, bool WARP_ROW>
__device__ __forceinline__ bool full_warp(const NormArgs& p) {
    if (WARP_ROW) return p.cols == 32 * E;
    const int c0 = (p.cluster > 1 ? int(cluster_rank()) : 0) * p.seg;
    return c0 + int(threadIdx.x / 32 + 1) * 32 * E <= min(p.cols, c0 + p.seg);
}

// The CTA's barrier, from either of the two copies of a kernel's body (a
// barrier counts warps, whatever instruction they arrive by).
__device__ __forceinline__ void row_barrier() { asm volatile("barrier.sync 0;" ::: "memory"); }

// Threads of a CTA that shares a row, at most, and the columns that each has:
// 32, or 16 where rows are read element by element (32 in rows over 65536).
constexpr int kRowThreads = 512;
constexpr int row_items(int vec, int64_t cols) { return vec > 1 || cols > 65536 ? 32 : 16; }

// ---- forward -----------------------------------------------------------------
template <typename T, int VEC, int ITEMS, bool WARP_ROW, bool FULL>
__device__ __forceinline__ void norm_forward_rows(const NormArgs& p, uint8_t* smem, Moments (*red)[kMaxCluster * kMaxWarps],
                                               Exchange<4>& ex) {
    constexpr int E = VEC * ITEMS, NL = VEC > 1 ? VEC / 2 : 1;
    using V = Vec<T, VEC>;
    using L = Lanes<VEC>;
    const Place<T, VEC, ITEMS, WARP_ROW, FULL> at(p, smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = int(blockDim.x) / 32;
    const T* x = static_cast<const T*>(p.x) + at.c.first;
    T* y = static_cast<T*>(p.out) + at.c.first;

    int64_t next = at.row;  // the next row to fetch, and where it is
    const T* next_x = x + next * p.ldx;
    const int64_t step_x = at.stride * p.ldx;
    auto refill = [&](int slot) {
        if (next < p.rows) fetch(at.c, next_x, at.ring + slot * at.slot_bytes);
        next += at.stride;
        next_x += step_x;
        cp_async_commit();
    };
    for (int s = 0; s < p.ring; ++s) refill(s);
    const uint32_t params = saddr(smem) + p.ring * at.slot_bytes;
    const Param<VEC> weight(params, at.c, p.weight, p.param_type, 1.0f);
    const Param<VEC> bias(params + E * blockDim.x * 4, at.c, p.bias, p.param_type, 0.0f);
    const float inv_c = 1.0f / float(p.cols);
    float n_warp = 0;  // columns of the warp
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) n_warp += at.c.has(k) ? VEC : 0;
    n_warp = warp_sum(n_warp);
    const float inv_n = n_warp > 0 ? 1.0f / n_warp : 0.0f;

    // Moments of the warp's columns of the row in ring slot `slot`.
    auto own = [&](int slot) {
        const uint32_t src = at.ring + slot * at.slot_bytes;
        L v[ITEMS][NL], sum = splat<L>(0), m2 = splat<L>(0);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                unpack(lds<T, VEC>(src + k * at.c.kSlot), v[k]);
#pragma unroll
                for (int i = 0; i < NL; ++i) sum = add(sum, v[k][i]);
            }
        const float m = warp_sum(total(sum)) * inv_n;
        const L minus_m = splat<L>(-m);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k))
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const L d = add(v[k][i], minus_m);
                    m2 = fma(d, d, m2);
                }
        return Moments{n_warp, m, warp_sum(total(m2)), 0.0f};
    };
    auto apply = [&](int64_t row, int slot, const Moments& s) {
        const float mean = s.mean;
        const float rstd = rsqrtf(s.m2 * inv_c + p.eps);
        const uint32_t src = at.ring + slot * at.slot_bytes;
        T* dst = y + row * p.ldout;
        const L minus_m = splat<L>(-mean), r = splat<L>(rstd);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                L v[NL], w[NL], b[NL];
                unpack(lds<T, VEC>(src + k * at.c.kSlot), v);
                weight.get(k, w);
                bias.get(k, b);
#pragma unroll
                for (int i = 0; i < NL; ++i) v[i] = fma(mul(add(v[i], minus_m), r), w[i], b[i]);
                V o;
                pack(v, o);
                *reinterpret_cast<V*>(dst + k * at.c.kStep) = o;
            }
        const bool writes = WARP_ROW ? lane == 0 : threadIdx.x == 0 && at.rank == 0;
        if (writes) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
    };

    if constexpr (WARP_ROW) {
        int slot = 0;
        for (int64_t row = at.row; row < p.rows; row += at.stride) {
            cp_async_wait(p.ring - 1);
            apply(row, slot, own(slot));
            refill(slot);
            slot = slot + 1 == p.ring ? 0 : slot + 1;
        }
    } else {
        // The moments of a row's warps.  Two buffers: whoever writes to one for
        // the row after next has passed the next row's barrier, before which
        // all had read it.
        auto send = [&](int buf, const Moments& s) {
            if (p.cluster == 1) {
                if (lane == 0) red[buf][warp] = s;
                row_barrier();
            } else {
                const float v[4] = {s.n, s.mean, s.m2, 0.0f};
                ex.send(buf, lane, p.cluster, v);
                ex.wait(buf);
            }
        };
        auto receive = [&](int buf) {
            // The union of the warps' sets, in one pass about the first set's
            // mean.  That mean is off the row's by no more than the first
            // set's share of the squares lets it be, so that little cancels.
            const float first = red[buf][0].mean, pivot = isfinite(first) ? first : 0.0f;
            float sum = 0, sq = 0;
            auto take = [&](const Moments& w) {
                const float d = w.mean - pivot, nd = w.n * d;
                if (w.n > 0) {
                    sum += nd;
                    sq += w.m2 + nd * d;
                }
            };
            for_entries(lane, p.cluster * warps, [&](int i) { take(red[buf][i]); });
            sum = set_sum(sum, p.cluster * warps);
            sq = set_sum(sq, p.cluster * warps);
            const float off = sum * inv_c;
            const float m2 = sq - sum * off;
            return Moments{float(p.cols), pivot + off, m2 < 0.0f ? 0.0f : m2, 0.0f};  // (a NaN stays one)
        };
        int slot = 0, buf = 0;
        for (int64_t row = at.row; row < p.rows; row += at.stride) {
            cp_async_wait(p.ring - 1);
            send(buf, own(slot));
            apply(row, slot, receive(buf));
            refill(slot);
            slot = slot + 1 == p.ring ? 0 : slot + 1;
            buf ^= 1;
        }
    }
    cp_async_wait(0);
}

template <typename T, int VEC, int ITEMS, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowWarps * 32 : kRowThreads, 1)
    norm_forward_kernel(const NormArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) Moments red[2][kMaxCluster * kMaxWarps];  // by CTA of the cluster, then by warp
    __shared__ uint64_t bars[2];
    Exchange<4> ex;
    if (!WARP_ROW && p.cluster > 1) {
        const uint32_t warps = blockDim.x / 32;
        ex.bar = saddr(bars);
        ex.buf = saddr(&red[0][0]);
        ex.bytes = uint32_t(p.cluster) * warps * 16;
        ex.entry = cluster_rank() * warps + threadIdx.x / 32;
        ex.err = p.err;
        if (threadIdx.x == 0) {
            for (int b = 0; b < 2; ++b) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(ex.bar + 8 * b) : "memory");
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        cluster_barrier();  // every CTA's mbarriers stand before anyone sends
    }
    if (full_warp<VEC * ITEMS, WARP_ROW>(p)) norm_forward_rows<T, VEC, ITEMS, WARP_ROW, true>(p, smem, red, ex);
    else norm_forward_rows<T, VEC, ITEMS, WARP_ROW, false>(p, smem, red, ex);
    if (!WARP_ROW && p.cluster > 1) cluster_barrier();  // nobody sends to a CTA that has gone
}

// ---- backward ----------------------------------------------------------------
template <typename T, int VEC, int ITEMS, bool WARP_ROW, bool FULL>
__device__ __forceinline__ void norm_backward_rows(const NormArgs& p, uint8_t* smem, float2 (*red)[kMaxCluster * kMaxWarps],
                                               Exchange<2>& ex) {
    constexpr int NL = VEC > 1 ? VEC / 2 : 1;
    using V = Vec<T, VEC>;
    using L = Lanes<VEC>;
    const Place<T, VEC, ITEMS, WARP_ROW, FULL> at(p, smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = int(blockDim.x) / 32;
    const uint32_t ring_dy = at.ring + p.ring * at.slot_bytes;
    const T* x = static_cast<const T*>(p.x) + at.c.first;
    const T* dy = static_cast<const T*>(p.dy) + at.c.first;
    T* dx = static_cast<T*>(p.out) + at.c.first;
    const float inv_c = 1.0f / float(p.cols);

    int64_t next = at.row;
    const T *next_x = x + next * p.ldx, *next_dy = dy + next * p.lddy;
    const int64_t step_x = at.stride * p.ldx, step_dy = at.stride * p.lddy;
    auto refill = [&](int slot) {
        if (next < p.rows) {
            fetch(at.c, next_x, at.ring + slot * at.slot_bytes);
            fetch(at.c, next_dy, ring_dy + slot * at.slot_bytes);
        }
        next += at.stride;
        next_x += step_x;
        next_dy += step_dy;
        cp_async_commit();
    };
    for (int s = 0; s < p.ring; ++s) refill(s);
    // the weight goes to shared memory: registers go to the two sums
    const Param<VEC> weight(saddr(smem) + 2 * p.ring * at.slot_bytes, at.c, p.weight, p.param_type, 1.0f);
    L aw[ITEMS][NL], ab[ITEMS][NL];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int i = 0; i < NL; ++i) aw[k][i] = ab[k][i] = splat<L>(0);

    struct Stat {
        float mean, rstd;
    };
    auto stat = [&](int64_t row) {
        return row < p.rows ? Stat{__ldg(p.mean + row), __ldg(p.rstd + row)} : Stat{0.0f, 0.0f};
    };
    // sums of g and of g xh over the thread's columns, over its warp
    auto own = [&](int slot, const Stat& st) {
        const uint32_t sx = at.ring + slot * at.slot_bytes, sd = ring_dy + slot * at.slot_bytes;
        L s1 = splat<L>(0), s2 = splat<L>(0);
        const L minus_m = splat<L>(-st.mean), r = splat<L>(st.rstd);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                L v[NL], d[NL], w[NL];
                unpack(lds<T, VEC>(sx + k * at.c.kSlot), v);
                unpack(lds<T, VEC>(sd + k * at.c.kSlot), d);
                weight.get(k, w);
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const L g = mul(d[i], w[i]);
                    s1 = add(s1, g);
                    s2 = fma(g, mul(add(v[i], minus_m), r), s2);
                }
            }
        return make_float2(warp_sum(total(s1)), warp_sum(total(s2)));
    };
    auto apply = [&](int64_t row, int slot, const Stat& st, float2 s) {
        const uint32_t sx = at.ring + slot * at.slot_bytes, sd = ring_dy + slot * at.slot_bytes;
        T* dst = dx + row * p.ldout;
        const L minus_m = splat<L>(-st.mean), r = splat<L>(st.rstd);
        const L minus_c1 = splat<L>(-s.x * inv_c), minus_c2 = splat<L>(-s.y * inv_c);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                L v[NL], d[NL], w[NL];
                unpack(lds<T, VEC>(sx + k * at.c.kSlot), v);
                unpack(lds<T, VEC>(sd + k * at.c.kSlot), d);
                weight.get(k, w);
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const L xh = mul(add(v[i], minus_m), r);
                    aw[k][i] = fma(d[i], xh, aw[k][i]);
                    ab[k][i] = add(ab[k][i], d[i]);
                    v[i] = mul(r, fma(xh, minus_c2, fma(d[i], w[i], minus_c1)));
                }
                V o;
                pack(v, o);
                *reinterpret_cast<V*>(dst + k * at.c.kStep) = o;
            }
    };

    Stat st = stat(at.row);
    if constexpr (WARP_ROW) {
        int slot = 0;
        for (int64_t row = at.row; row < p.rows; row += at.stride) {
            const Stat st1 = stat(row + at.stride);
            cp_async_wait(p.ring - 1);
            apply(row, slot, st, own(slot, st));
            refill(slot);
            slot = slot + 1 == p.ring ? 0 : slot + 1;
            st = st1;
        }
    } else {
        auto send = [&](int buf, float2 s) {  // as in the forward
            if (p.cluster == 1) {
                if (lane == 0) red[buf][warp] = s;
                row_barrier();
            } else {
                const float v[2] = {s.x, s.y};
                ex.send(buf, lane, p.cluster, v);
                ex.wait(buf);
            }
        };
        auto receive = [&](int buf) {
            float2 s = make_float2(0.0f, 0.0f);
            for_entries(lane, p.cluster * warps, [&](int i) { s = add(s, red[buf][i]); });
            return make_float2(set_sum(s.x, p.cluster * warps), set_sum(s.y, p.cluster * warps));
        };
        int slot = 0, buf = 0;
        for (int64_t row = at.row; row < p.rows; row += at.stride) {
            const Stat st1 = stat(row + at.stride);
            cp_async_wait(p.ring - 1);
            send(buf, own(slot, st));
            apply(row, slot, st, receive(buf));
            refill(slot);
            slot = slot + 1 == p.ring ? 0 : slot + 1;
            buf ^= 1;
            st = st1;
        }
    }
    cp_async_wait(0);
    if (!p.dweight && !p.dbias) return;

    if constexpr (WARP_ROW) {
        // every warp leaves its sums where the ring was; a thread then has
        // columns of all warps, in their order
        float* acc = reinterpret_cast<float*>(smem);
        __syncthreads();
        float* mine = acc + warp * 2 * p.cols;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k))
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    mine[at.c.col(k) + e] = lane_of(aw[k], e);
                    mine[p.cols + at.c.col(k) + e] = lane_of(ab[k], e);
                }
        __syncthreads();
        for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
            float sw = 0, sb = 0;
            for (int w = 0; w < warps; ++w) {
                sw += acc[w * 2 * p.cols + c];
                sb += acc[(w * 2 + 1) * p.cols + c];
            }
            if (gridDim.x == 1) {
                if (p.dweight) p.dweight[c] = sw;
                if (p.dbias) p.dbias[c] = sb;
            } else {
                p.partials[int64_t(blockIdx.x) * 2 * p.cols + c] = sw;
                p.partials[(int64_t(blockIdx.x) * 2 + 1) * p.cols + c] = sb;
            }
        }
    } else {
        const bool whole = gridDim.x == uint32_t(p.cluster);
        float* to_w = whole ? p.dweight : p.partials + at.row * 2 * p.cols;
        float* to_b = whole ? p.dbias : p.partials + (at.row * 2 + 1) * p.cols;
        // (rows of vectors have a multiple of four columns; the caller's arrays
        // may start anywhere)
        const bool wide = VEC > 1 && ((reinterpret_cast<uintptr_t>(to_w) | reinterpret_cast<uintptr_t>(to_b)) & 15) == 0;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                if (wide) {
                    if constexpr (VEC > 1)
#pragma unroll
                        for (int q = 0; q < VEC / 4; ++q) {
                            const int c = at.c.col(k) + 4 * q;
                            if (to_w) *reinterpret_cast<float4*>(to_w + c) = make_float4(aw[k][2 * q].x, aw[k][2 * q].y, aw[k][2 * q + 1].x, aw[k][2 * q + 1].y);
                            if (to_b) *reinterpret_cast<float4*>(to_b + c) = make_float4(ab[k][2 * q].x, ab[k][2 * q].y, ab[k][2 * q + 1].x, ab[k][2 * q + 1].y);
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int c = at.c.col(k) + e;
                        if (to_w) to_w[c] = lane_of(aw[k], e);
                        if (to_b) to_b[c] = lane_of(ab[k], e);
                    }
                }
            }
    }
}

template <typename T, int VEC, int ITEMS, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowWarps * 32 : kRowThreads, 1)
    norm_backward_kernel(const NormArgs p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // norm_reduce_kernel, which waits for this one
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float2 red[2][kMaxCluster * kMaxWarps];  // by CTA of the cluster, then by warp
    __shared__ uint64_t bars[2];
    Exchange<2> ex;
    if (!WARP_ROW && p.cluster > 1) {
        const uint32_t warps = blockDim.x / 32;
        ex.bar = saddr(bars);
        ex.buf = saddr(&red[0][0]);
        ex.bytes = uint32_t(p.cluster) * warps * 8;
        ex.entry = cluster_rank() * warps + threadIdx.x / 32;
        ex.err = p.err;
        if (threadIdx.x == 0) {
            for (int b = 0; b < 2; ++b) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(ex.bar + 8 * b) : "memory");
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        cluster_barrier();  // every CTA's mbarriers stand before anyone sends
    }
    if (full_warp<VEC * ITEMS, WARP_ROW>(p)) norm_backward_rows<T, VEC, ITEMS, WARP_ROW, true>(p, smem, red, ex);
    else norm_backward_rows<T, VEC, ITEMS, WARP_ROW, false>(p, smem, red, ex);
    if (!WARP_ROW && p.cluster > 1) cluster_barrier();  // nobody sends to a CTA that has gone
}

// Sums of the partial weight and bias gradients: 32 columns a CTA, the
// partials shared among its warps and joined in a fixed order.
constexpr int kReduceWarps = 16;
__global__ void __launch_bounds__(kReduceWarps * 32)
    norm_reduce_kernel(const float* partials, int32_t n, int32_t cols, float* dweight, float* dbias) {
    __shared__ float acc[kReduceWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float* out = blockIdx.y == 0 ? dweight : dbias;
    if (!out) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are there
    float s = 0;
    if (c < cols)
#pragma unroll 8
        for (int i = warp; i < n; i += kReduceWarps) s += partials[(int64_t(i) * 2 + blockIdx.y) * cols + c];
    acc[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
        s = 0;
#pragma unroll
        for (int w = 0; w < kReduceWarps; ++w) s += acc[w][lane];
        out[c] = s;
    }
}

// ---- host --------------------------------------------------------------------
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

using NormKernel = void (*)(NormArgs);

// Elements a thread has of each row: 8 or 32 where a warp has the row, 16 or 32
// where a CTA or cluster does.
template <typename T, int VEC>
NormKernel pick(bool backward, bool warp_row, int e) {
    if (!warp_row && e == 32) return backward ? norm_backward_kernel<T, VEC, 32 / VEC, false> : norm_forward_kernel<T, VEC, 32 / VEC, false>;
    if constexpr (VEC == 1)
        if (!warp_row) return backward ? norm_backward_kernel<T, 1, 16, false> : norm_forward_kernel<T, 1, 16, false>;
    if (backward) return e == 8 ? norm_backward_kernel<T, VEC, 8 / VEC, true> : norm_backward_kernel<T, VEC, 32 / VEC, true>;
    return e == 8 ? norm_forward_kernel<T, VEC, 8 / VEC, true> : norm_forward_kernel<T, VEC, 32 / VEC, true>;
}

// CTAs that share a row: one for each 8192 columns, up to eight, and more
// columns each in the longest rows.  Two CTAs of 256 threads, an SM's, work
// on different rows, and one moves data while the other waits for its row's
// sums.  Measured, forward / backward, us, with 8192 / with 16384 columns a CTA:
// 2048 x 65536 bf16 133 / 183 and 139 / 182, 4096 x 32768 123 / 171 and 136 / 170,
// 8192 x 16384 112 / 150 and 120 / 152.
int cluster_size(int64_t cols) {
    int c = 1;
    while (c < kMaxCluster && cols > int64_t(c) * 8192) c *= 2;
    return c;
}
static_assert(kNormMaxCols == int64_t(kMaxCluster) * kRowThreads * 32 && 8192 == kRowThreads * 16, "the rows fit their clusters");

struct Plan {
    NormKernel kernel;
    int threads, cluster, grid, seg, ring;
    size_t smem;
    bool warp_row;
};

cudaError_t make_plan(const NormDesc& d, bool backward, int num_sms, Plan* out) {
    const int esize = int(type_bytes(d.type));
    int vec = 16 / esize;
    const bool whole = d.cols % vec == 0 && d.ldx % vec == 0 && d.ldout % vec == 0 && aligned16(d.x) &&
                       aligned16(d.out) && (!backward || (d.lddy % vec == 0 && aligned16(d.dy)));
    if (!whole) vec = 1;
    Plan p{};
    p.warp_row = d.cols <= 1024;
    int e;
    if (p.warp_row) {
        e = d.cols <= 256 ? 8 : 32;
        p.cluster = 1;
        p.threads = kWarpRowWarps * 32;
        p.seg = int(d.cols);
    } else {
        p.cluster = cluster_size(d.cols);
        e = row_items(vec, d.cols);
        const int64_t per = (d.cols + p.cluster - 1) / p.cluster;
        p.seg = int((per + vec - 1) / vec * vec);
        p.threads = int(((p.seg + e - 1) / e + 31) / 32 * 32);
    }
    const size_t row_bytes = size_t(p.threads) * e * esize * (backward ? 2 : 1);
    const size_t fixed = size_t(p.threads) * e * 4 * (backward ? 1 : 2);
    // single 2-byte elements cannot be copied asynchronously: a longer ring
    // would hide nothing
    auto fits = [&](size_t budget) { return budget < fixed ? 0 : int(std::min<size_t>(kMaxRing, (budget - fixed) / row_bytes)); };
    p.ring = vec == 1 && esize == 2 ? 1 : fits(kSmemBudget / 2) >= 2 ? fits(kSmemBudget / 2) : std::max(1, fits(kSmemBudget));
    p.smem = p.ring * row_bytes + fixed;
    if (backward && p.warp_row) p.smem = std::max(p.smem, size_t(kWarpRowWarps) * size_t(d.cols) * 8);
    if (d.type == TL_TYPE_BF16)
        p.kernel = vec > 1 ? pick<__nv_bfloat16, 8>(backward, p.warp_row, e) : pick<__nv_bfloat16, 1>(backward, p.warp_row, e);
    else if (d.type == TL_TYPE_F16)
        p.kernel = vec > 1 ? pick<__half, 8>(backward, p.warp_row, e) : pick<__half, 1>(backward, p.warp_row, e);
    else
        p.kernel = vec > 1 ? pick<float, 4>(backward, p.warp_row, e) : pick<float, 1>(backward, p.warp_row, e);
    int per_sm = 1;
    const cudaError_t err = ctas_per_sm(reinterpret_cast<const void*>(p.kernel), p.threads, p.smem, &per_sm);
    if (err != cudaSuccess) return err;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    per_sm = std::min(per_sm, kCtasPerSm);
    const int64_t units = p.warp_row ? (d.rows + kWarpRowWarps - 1) / kWarpRowWarps : d.rows;
    const int64_t sms = std::min(num_sms, kMaxSms);
    int64_t room = std::max<int64_t>(1, sms * per_sm / p.cluster);
    // More clusters than run at a time would begin their rows when the others had
    // done theirs.  Forward / backward, us, with as many as run / with as many as
    // the SMs' CTAs would make: 2048 x 65536 bf16 133 / 183 and 205 / 253, 4096 x
    // 32768 124 / 171 and 201 / 244.
    if (p.cluster > 1) {
        int clusters = 0;
        const cudaError_t c = clusters_at_a_time(reinterpret_cast<const void*>(p.kernel), p.threads, p.smem, p.cluster, &clusters);
        if (c != cudaSuccess) return c;
        if (clusters < 1) return cudaErrorInvalidConfiguration;
        room = std::min<int64_t>(room, clusters);
    }
    // Each CTA of the backward also writes a sum for every column, which the
    // reduction reads: with few rows, fewer CTAs that walk over several of them
    // do less in all, as long as their rows come ahead of them.  Backward, us,
    // with this / with a row a CTA: 512 x 8192 bf16 22 / 33, 256 x 4096 12 / 18,
    // 300 x 30000 44 / 54.  (Two an SM where elements come one by one: 517 x
    // 5003 fp32 24 / 33, with one 30.)
    if (backward && p.ring > 1 && units < 8 * room)
        room = std::min(room, std::max({int64_t(1), sms / p.cluster * (vec > 1 ? 1 : 2), units / 8}));
    p.grid = int(std::min(units, std::min(room, norm_partials(d.rows, d.cols)))) * p.cluster;
    *out = p;
    return cudaSuccess;
}

cudaError_t launch(const Plan& pl, const NormDesc& d, cudaStream_t stream) {
    NormArgs a{};
    a.x = d.x;
    a.ldx = d.ldx;
    a.dy = d.dy;
    a.lddy = d.lddy;
    a.out = d.out;
    a.ldout = d.ldout;
    a.weight = d.weight;
    a.bias = d.bias;
    a.mean = d.mean;
    a.rstd = d.rstd;
    a.dweight = d.dweight;
    a.dbias = d.dbias;
    a.partials = d.partials;
    a.rows = d.rows;
    a.cols = int32_t(d.cols);
    a.seg = pl.seg;
    a.param_type = d.param_type;
    a.ring = pl.ring;
    a.cluster = pl.cluster;
    a.eps = d.eps;
    a.err = d.err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(pl.grid));
    cfg.blockDim = dim3(unsigned(pl.threads));
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(pl.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pl.kernel, a);
}

}  // namespace

int64_t norm_partials(int64_t rows, int64_t cols) {
    const int64_t ctas = int64_t(kMaxSms) * kCtasPerSm / cluster_size(cols);
    return std::max<int64_t>(1, std::min(rows, ctas));
}

std::string norm_check(const NormDesc& d, bool backward) {
    if (d.rows < 0 || d.cols < 1 || d.cols > kNormMaxCols) return "rows must be >= 0 and cols in 1..131072";
    if (d.rows > (int64_t(1) << 40)) return "too many rows";
    if (!type_known(d.type) || !type_known(d.param_type)) return "unknown tl_type";
    const size_t es = type_bytes(d.type), ps = type_bytes(d.param_type);
    auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (off(d.weight, ps) || off(d.bias, ps)) return "weight or bias is not aligned to its type";
    if (off(d.dweight, 4) || off(d.dbias, 4)) return "dweight or dbias is not aligned to fp32";
    if (!d.err || off(d.err, 4)) return "err is null or not aligned to int32";
    if (!(d.eps >= 0)) return "eps must be >= 0";
    if (d.rows == 0) return {};
    if (!d.x || !d.out || !d.mean || !d.rstd || (backward && !d.dy)) return "null pointer";
    if (off(d.x, es) || off(d.out, es) || off(d.dy, es)) return "a matrix is not aligned to its type";
    if (off(d.mean, 4) || off(d.rstd, 4)) return "mean or rstd is not aligned to fp32";
    if (d.ldx < d.cols || d.ldout < d.cols || (backward && d.lddy < d.cols)) return "a leading dimension is smaller than cols";
    return {};
}

cudaError_t norm_forward_launch(const NormDesc& d, int num_sms, cudaStream_t stream) {
    Plan p;
    const cudaError_t e = make_plan(d, false, num_sms, &p);
    return e == cudaSuccess ? launch(p, d, stream) : e;
}

cudaError_t norm_backward_launch(const NormDesc& d, int num_sms, cudaStream_t stream) {
    cudaError_t e;
    if (d.rows == 0) {
        for (float* g : {d.dweight, d.dbias})
            if (g && (e = cudaMemsetAsync(g, 0, size_t(d.cols) * 4, stream)) != cudaSuccess) return e;
        return cudaSuccess;
    }
    Plan p;
    e = make_plan(d, true, num_sms, &p);
    if (e == cudaSuccess) e = launch(p, d, stream);
    const int n = p.grid / p.cluster;
    if (e != cudaSuccess || n == 1 || (!d.dweight && !d.dbias)) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((d.cols + 31) / 32), 2);
    cfg.blockDim = dim3(kReduceWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];  // its launch may overlap the end of the kernel before it
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_reduce_kernel, static_cast<const float*>(d.partials), int32_t(n), int32_t(d.cols), d.dweight,
                              d.dbias);
}

}  // namespace tl
