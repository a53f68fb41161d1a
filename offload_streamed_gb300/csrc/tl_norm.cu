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
//    cluster of up to eight when a CTA cannot hold them.  There the exchange
//    of row i + 1's sums is under way while row i is written, so one barrier
//    a row is all there is, and its wait is mostly hidden.
// All statistics and sums are fp32.  A row's variance is joined from the
// warps' sums of squares about their own means, which loses nothing to
// cancellation, whatever the row's mean.  Every order of summation is fixed by
// the sizes alone.
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
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ void st_cluster_f32(uint32_t local, uint32_t rank, float v) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, %1;\n\t"
        "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(local), "r"(rank), "f"(v)
        : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Count, mean and sum of squares about the mean of a set of values.
struct Moments {
    float n, mean, m2;
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
    if (n <= kMaxWarps) {
        if ((lane & 15) < n) f(lane & 15);
    } else {
        for (int i = lane; i < n; i += 32) f(i);
    }
}
__device__ __forceinline__ float set_sum(float v, int n) {
    if (n > kMaxWarps) v += __shfl_xor_sync(~0u, v, 16);
#pragma unroll
    for (int s = 8; s; s >>= 1) v += __shfl_xor_sync(~0u, v, s);
    return v;
}
__device__ __forceinline__ float lane_of(const float (&v)[1], int) { return v[0]; }
template <int N>
__device__ __forceinline__ float lane_of(const float2 (&v)[N], int e) {
    return e & 1 ? v[e / 2].y : v[e / 2].x;
}

// The columns of one thread: ITEMS vectors of VEC elements, `step` vectors
// apart, so that a warp's accesses are contiguous.
template <typename T, int VEC, int ITEMS>
struct Cols {
    using V = Vec<T, VEC>;
    int first;  // column of the thread's first vector, in the row
    int step;   // columns between its vectors
    int end;    // columns of the CTA end here
    __device__ __forceinline__ int col(int k) const { return first + k * step; }
    __device__ __forceinline__ bool has(int k) const { return col(k) < end; }
};

// Copy the thread's columns of a row into its part of a ring slot: vector k at
// slot[k * threads + thread].
template <typename T, int VEC, int ITEMS>
__device__ __forceinline__ void fetch(const Cols<T, VEC, ITEMS>& c, const T* row, Vec<T, VEC>* slot, int threads) {
    if constexpr (VEC > 1) {
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (c.has(k)) cp_async16(saddr(slot + k * threads), row + c.col(k));
    } else {
        T v[ITEMS];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (c.has(k)) v[k] = row[c.col(k)];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (c.has(k)) slot[k * threads].v[0] = v[k];
    }
}

// A parameter (weight or bias) at the thread's columns, as fp32 in the thread's
// own shared memory, in 16-byte chunks a thread apart.
template <int VEC>
struct Param {
    static constexpr int kChunk = VEC > 1 ? 4 : 1;
    using C = Vec<float, kChunk>;
    C* at;
    int threads;
    __device__ __forceinline__ Param(float* base, int threads_) : at(reinterpret_cast<C*>(base) + threadIdx.x), threads(threads_) {}
    template <typename T, int ITEMS>
    __device__ __forceinline__ void fill(const Cols<T, VEC, ITEMS>& c, const void* p, int32_t type, float none) {
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (c.has(k))
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    at[(k * (VEC / kChunk) + e / kChunk) * threads].v[e % kChunk] =
                        p ? load_as_f32(p, type, c.col(k) + e) : none;
    }
    __device__ __forceinline__ void get(int k, float (&v)[1]) const { v[0] = at[k * threads].v[0]; }
    template <int N>
    __device__ __forceinline__ void get(int k, float2 (&v)[N]) const {
#pragma unroll
        for (int q = 0; q < N / 2; ++q) {
            const C u = at[(k * (VEC / kChunk) + q) * threads];
            v[2 * q] = make_float2(u.v[0], u.v[1]);
            v[2 * q + 1] = make_float2(u.v[2], u.v[3]);
        }
    }
};

// Which rows and columns a thread works on.
template <typename T, int VEC, int ITEMS, bool WARP_ROW>
struct Place {
    Cols<T, VEC, ITEMS> c;
    int64_t row, stride;  // first row and the distance to the next
    int threads;          // threads of the CTA
    uint32_t rank;
    __device__ __forceinline__ explicit Place(const NormArgs& p) {
        threads = int(blockDim.x);
        const int tid = int(threadIdx.x);
        if constexpr (WARP_ROW) {
            rank = 0;
            c.first = (tid & 31) * VEC;
            c.step = 32 * VEC;
            c.end = p.cols;
            row = int64_t(blockIdx.x) * (threads / 32) + tid / 32;
            stride = int64_t(gridDim.x) * (threads / 32);
        } else {
            rank = p.cluster > 1 ? cluster_rank() : 0;
            const int c0 = int(rank) * p.seg;
            c.first = c0 + tid * VEC;
            c.step = threads * VEC;
            c.end = min(p.cols, c0 + p.seg);
            row = blockIdx.x / uint32_t(p.cluster);
            stride = gridDim.x / uint32_t(p.cluster);
        }
    }
};

// ---- forward -----------------------------------------------------------------
template <typename T, int VEC, int ITEMS, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowWarps * 32 : kMaxWarps * 32, WARP_ROW || VEC * ITEMS > 16 ? 1 : 2)
    norm_forward_kernel(const NormArgs p) {
    constexpr int E = VEC * ITEMS, NL = VEC > 1 ? VEC / 2 : 1;
    using V = Vec<T, VEC>;
    using L = Lanes<VEC>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Moments red[3][kMaxCluster * kMaxWarps];  // by CTA of the cluster, then by warp
    const Place<T, VEC, ITEMS, WARP_ROW> at(p);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = at.threads / 32;
    V* ring = reinterpret_cast<V*>(smem) + threadIdx.x;
    const int slot_vecs = ITEMS * at.threads;
    const T* x = static_cast<const T*>(p.x);
    T* y = static_cast<T*>(p.out);

    int64_t next = at.row;  // the next row to fetch, and where it is
    const T* next_x = x + next * p.ldx;
    const int64_t step_x = at.stride * p.ldx;
    auto refill = [&](int slot) {
        if (next < p.rows) fetch(at.c, next_x, ring + slot * slot_vecs, at.threads);
        next += at.stride;
        next_x += step_x;
        cp_async_commit();
    };
    for (int s = 0; s < p.ring; ++s) refill(s);
    float* params = reinterpret_cast<float*>(smem + size_t(p.ring) * slot_vecs * sizeof(V));
    Param<VEC> weight(params, at.threads), bias(params + E * at.threads, at.threads);
    weight.fill(at.c, p.weight, p.param_type, 1.0f);
    bias.fill(at.c, p.bias, p.param_type, 0.0f);
    const float inv_c = 1.0f / float(p.cols);
    float n_warp = 0;  // columns of the warp
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) n_warp += at.c.has(k) ? VEC : 0;
    n_warp = warp_sum(n_warp);
    const float inv_n = n_warp > 0 ? 1.0f / n_warp : 0.0f;

    // Moments of the warp's columns of the row in ring slot `slot`.
    auto own = [&](int slot) {
        const V* src = ring + slot * slot_vecs;
        L v[ITEMS][NL], sum = splat<L>(0), m2 = splat<L>(0);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                unpack(src[k * at.threads], v[k]);
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
        return Moments{n_warp, m, warp_sum(total(m2))};
    };
    auto apply = [&](int64_t row, int slot, const Moments& s) {
        const float mean = s.mean;
        const float rstd = rsqrtf(s.m2 * inv_c + p.eps);
        const V* src = ring + slot * slot_vecs;
        T* dst = y + row * p.ldout;
        const L minus_m = splat<L>(-mean), r = splat<L>(rstd);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                L v[NL], w[NL], b[NL];
                unpack(src[k * at.threads], v);
                weight.get(k, w);
                bias.get(k, b);
#pragma unroll
                for (int i = 0; i < NL; ++i) v[i] = fma(mul(add(v[i], minus_m), r), w[i], b[i]);
                V o;
                pack(v, o);
                *reinterpret_cast<V*>(dst + at.c.col(k)) = o;
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
        // The moments of a row's warps: every warp writes its own to each CTA
        // of the cluster; three buffers, since a CTA may be one row ahead of
        // another's last read.
        auto send = [&](int buf, const Moments& s) {
            if (p.cluster == 1) {
                if (lane == 0) red[buf][warp] = s;
            } else {
                if (lane < p.cluster) {
                    const uint32_t a = saddr(&red[buf][int(at.rank) * warps + warp]);
                    st_cluster_f32(a, uint32_t(lane), s.n);
                    st_cluster_f32(a + 4, uint32_t(lane), s.mean);
                    st_cluster_f32(a + 8, uint32_t(lane), s.m2);
                }
                cluster_arrive();
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
            return Moments{float(p.cols), pivot + off, m2 < 0.0f ? 0.0f : m2};  // (a NaN stays one)
        };
        if (p.cluster > 1) {  // every CTA of the cluster runs before its memory is written
            cluster_arrive();
            cluster_wait();
        }
        int slot = 0, buf = 0;
        if (at.row < p.rows) {
            cp_async_wait(p.ring - 1);
            send(0, own(0));
        }
        for (int64_t row = at.row; row < p.rows; row += at.stride) {
            const int slot1 = slot + 1 == p.ring ? 0 : slot + 1, buf1 = buf == 2 ? 0 : buf + 1;
            const bool more = row + at.stride < p.rows;
            Moments ahead{};
            if (more && p.ring > 1) {
                cp_async_wait(p.ring - 2);
                ahead = own(slot1);
            }
            if (p.cluster > 1) cluster_wait();
            else __syncthreads();
            if (more && p.ring > 1) send(buf1, ahead);
            apply(row, slot, receive(buf));
            refill(slot);
            if (more && p.ring == 1) {
                cp_async_wait(0);
                send(buf1, own(slot1));
            }
            slot = slot1;
            buf = buf1;
        }
    }
    cp_async_wait(0);
}

// ---- backward ----------------------------------------------------------------
template <typename T, int VEC, int ITEMS, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowWarps * 32 : kMaxWarps * 32, WARP_ROW || VEC * ITEMS > 16 ? 1 : 2)
    norm_backward_kernel(const NormArgs p) {
    constexpr int E = VEC * ITEMS, NL = VEC > 1 ? VEC / 2 : 1;
    using V = Vec<T, VEC>;
    using L = Lanes<VEC>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 red[3][kMaxCluster * kMaxWarps];  // as in the forward
    const Place<T, VEC, ITEMS, WARP_ROW> at(p);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = at.threads / 32;
    const int slot_vecs = ITEMS * at.threads;
    V* ring_x = reinterpret_cast<V*>(smem) + threadIdx.x;
    V* ring_dy = ring_x + p.ring * slot_vecs;
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.dy);
    T* dx = static_cast<T*>(p.out);
    const float inv_c = 1.0f / float(p.cols);

    int64_t next = at.row;
    const T *next_x = x + next * p.ldx, *next_dy = dy + next * p.lddy;
    const int64_t step_x = at.stride * p.ldx, step_dy = at.stride * p.lddy;
    auto refill = [&](int slot) {
        if (next < p.rows) {
            fetch(at.c, next_x, ring_x + slot * slot_vecs, at.threads);
            fetch(at.c, next_dy, ring_dy + slot * slot_vecs, at.threads);
        }
        next += at.stride;
        next_x += step_x;
        next_dy += step_dy;
        cp_async_commit();
    };
    for (int s = 0; s < p.ring; ++s) refill(s);
    // the weight goes to shared memory: registers go to the two sums
    Param<VEC> weight(reinterpret_cast<float*>(smem + size_t(2 * p.ring) * slot_vecs * sizeof(V)), at.threads);
    weight.fill(at.c, p.weight, p.param_type, 1.0f);
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
        const V* sx = ring_x + slot * slot_vecs;
        const V* sd = ring_dy + slot * slot_vecs;
        L s1 = splat<L>(0), s2 = splat<L>(0);
        const L minus_m = splat<L>(-st.mean), r = splat<L>(st.rstd);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                L v[NL], d[NL], w[NL];
                unpack(sx[k * at.threads], v);
                unpack(sd[k * at.threads], d);
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
        const V* sx = ring_x + slot * slot_vecs;
        const V* sd = ring_dy + slot * slot_vecs;
        T* dst = dx + row * p.ldout;
        const L minus_m = splat<L>(-st.mean), r = splat<L>(st.rstd);
        const L minus_c1 = splat<L>(-s.x * inv_c), minus_c2 = splat<L>(-s.y * inv_c);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                L v[NL], d[NL], w[NL];
                unpack(sx[k * at.threads], v);
                unpack(sd[k * at.threads], d);
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
                *reinterpret_cast<V*>(dst + at.c.col(k)) = o;
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
            } else {
                if (lane < p.cluster) {
                    const uint32_t a = saddr(&red[buf][int(at.rank) * warps + warp]);
                    st_cluster_f32(a, uint32_t(lane), s.x);
                    st_cluster_f32(a + 4, uint32_t(lane), s.y);
                }
                cluster_arrive();
            }
        };
        auto receive = [&](int buf) {
            float2 s = make_float2(0.0f, 0.0f);
            for_entries(lane, p.cluster * warps, [&](int i) { s = add(s, red[buf][i]); });
            return make_float2(set_sum(s.x, p.cluster * warps), set_sum(s.y, p.cluster * warps));
        };
        if (p.cluster > 1) {
            cluster_arrive();
            cluster_wait();
        }
        int slot = 0, buf = 0;
        if (at.row < p.rows) {
            cp_async_wait(p.ring - 1);
            send(0, own(0, st));
        }
        for (int64_t row = at.row; row < p.rows; row += at.stride) {
            const int slot1 = slot + 1 == p.ring ? 0 : slot + 1, buf1 = buf == 2 ? 0 : buf + 1;
            const bool more = row + at.stride < p.rows;
            const Stat st1 = stat(row + at.stride);
            float2 ahead{};
            if (more && p.ring > 1) {
                cp_async_wait(p.ring - 2);
                ahead = own(slot1, st1);
            }
            if (p.cluster > 1) cluster_wait();
            else __syncthreads();
            if (more && p.ring > 1) send(buf1, ahead);
            apply(row, slot, st, receive(buf));
            refill(slot);
            if (more && p.ring == 1) {
                cp_async_wait(0);
                send(buf1, own(slot1, st1));
            }
            slot = slot1;
            buf = buf1;
            st = st1;
        }
    }
    cp_async_wait(0);
    if (!p.dweight && !p.dbias) return;

    if constexpr (WARP_ROW) {
        // join the warps' sums, one warp after another
        float* acc = reinterpret_cast<float*>(smem);  // the ring is done with
        __syncthreads();
        for (int w = 0; w < warps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int k = 0; k < ITEMS; ++k)
                    if (at.c.has(k))
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const int c = at.c.col(k) + e;
                            acc[c] = (w ? acc[c] : 0.0f) + lane_of(aw[k], e);
                            acc[p.cols + c] = (w ? acc[p.cols + c] : 0.0f) + lane_of(ab[k], e);
                        }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < p.cols; c += at.threads) {
            if (gridDim.x == 1) {
                if (p.dweight) p.dweight[c] = acc[c];
                if (p.dbias) p.dbias[c] = acc[p.cols + c];
            } else {
                p.partials[int64_t(blockIdx.x) * 2 * p.cols + c] = acc[c];
                p.partials[(int64_t(blockIdx.x) * 2 + 1) * p.cols + c] = acc[p.cols + c];
            }
        }
    } else {
        const bool whole = gridDim.x == uint32_t(p.cluster);
        float* to_w = whole ? p.dweight : p.partials + at.row * 2 * p.cols;
        float* to_b = whole ? p.dbias : p.partials + (at.row * 2 + 1) * p.cols;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k))
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int c = at.c.col(k) + e;
                    if (to_w) to_w[c] = lane_of(aw[k], e);
                    if (to_b) to_b[c] = lane_of(ab[k], e);
                }
    }
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

// Elements a thread has of each row (E): 8 or 32 where a warp has a row, 16
// where a CTA or cluster shares it, 32 in the rows that eight CTAs of 512
// threads cannot hold otherwise.
template <typename T, int VEC>
NormKernel pick(bool backward, bool warp_row, int e) {
    if (backward) {
        if (warp_row) return e == 8 ? norm_backward_kernel<T, VEC, 8 / VEC, true> : norm_backward_kernel<T, VEC, 32 / VEC, true>;
        return e == 16 ? norm_backward_kernel<T, VEC, 16 / VEC, false> : norm_backward_kernel<T, VEC, 32 / VEC, false>;
    }
    if (warp_row) return e == 8 ? norm_forward_kernel<T, VEC, 8 / VEC, true> : norm_forward_kernel<T, VEC, 32 / VEC, true>;
    return e == 16 ? norm_forward_kernel<T, VEC, 16 / VEC, false> : norm_forward_kernel<T, VEC, 32 / VEC, false>;
}

// CTAs that share a row: as few as hold it with 16 columns a thread.
int cluster_size(int64_t cols) {
    int c = 1;
    while (c < kMaxCluster && cols > int64_t(c) * kMaxWarps * 32 * 16) c *= 2;
    return c;
}

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
        e = d.cols <= int64_t(p.cluster) * kMaxWarps * 32 * 16 ? 16 : 32;
        const int64_t per = (d.cols + p.cluster - 1) / p.cluster;
        p.seg = int((per + vec - 1) / vec * vec);
        p.threads = int(((p.seg + e - 1) / e + 31) / 32 * 32);
    }
    const size_t row_bytes = size_t(p.threads) * e * esize * (backward ? 2 : 1);
    const size_t fixed = size_t(p.threads) * e * 4 * (backward ? 1 : 2);
    // only the vector copies are asynchronous: without them a longer ring
    // hides nothing
    auto fits = [&](size_t budget) { return budget < fixed ? 0 : int(std::min<size_t>(kMaxRing, (budget - fixed) / row_bytes)); };
    p.ring = vec == 1 ? 1 : fits(kSmemBudget / 2) >= 2 ? fits(kSmemBudget / 2) : std::max(1, fits(kSmemBudget));
    p.smem = p.ring * row_bytes + fixed;
    if (backward && p.warp_row) p.smem = std::max(p.smem, size_t(d.cols) * 8);
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
    const int64_t room = std::max<int64_t>(1, int64_t(std::min(num_sms, kMaxSms)) * per_sm / p.cluster);
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
    if (!(d.eps >= 0)) return "eps must be >= 0";
    if (d.rows == 0) return {};
    if (!d.x || !d.out || !d.mean || !d.rstd || (backward && !d.dy)) return "null pointer";
    if (off(d.x, es) || off(d.out, es) || off(d.dy, es)) return "a matrix is not aligned to its type";
    if (off(d.mean, 4) || off(d.rstd, 4)) return "mean or rstd is not aligned to fp32";
    if (d.ldx < d.cols || d.ldout < d.cols || (backward && d.lddy < d.cols)) return "a leading dimension is smaller than cols";
    return {};
}

cudaError_t norm_forward_launch(const NormDesc& d, int num_sms, cudaStream_t stream) {
    if (d.rows == 0) return cudaSuccess;
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
    norm_reduce_kernel<<<dim3(unsigned((d.cols + 31) / 32), 2), kReduceWarps * 32, 0, stream>>>(
        d.partials, n, int32_t(d.cols), d.dweight, d.dbias);
    return cudaGetLastError();
}

}  // namespace tl
