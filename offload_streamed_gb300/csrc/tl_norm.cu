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
// threads' sums of squares about their own means, which loses nothing to
// cancellation, whatever the row's mean.  Every order of summation is fixed by
// the sizes alone.
#include "tl_norm.h"
#include "tl_types.cuh"

#include <algorithm>

namespace tl {
namespace {

constexpr int kMaxRing = 4;         // rows in flight per thread
constexpr int kWarpRowWarps = 8;    // rows of a CTA at a time where a warp has a row
constexpr int kMaxWarps = 16;       // of a CTA that shares a row
constexpr int kMaxCluster = 8;
constexpr size_t kSmemBudget = 200 * 1024;
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

// Count, sum and sum of squares about the mean of a set of values, and the
// union of two such sets.
struct Moments {
    float n, sum, m2;
};
__device__ __forceinline__ Moments join(const Moments& a, const Moments& b) {
    const float n = a.n + b.n;
    if (b.n == 0.0f) return a;
    if (a.n == 0.0f) return b;
    const float d = b.sum / b.n - a.sum / a.n;
    return Moments{n, a.sum + b.sum, a.m2 + b.m2 + d * d * (a.n * b.n / n)};
}
__device__ __forceinline__ Moments warp_join(Moments v) {
#pragma unroll
    for (int s = 16; s; s >>= 1) {
        const Moments o{__shfl_xor_sync(~0u, v.n, s), __shfl_xor_sync(~0u, v.sum, s), __shfl_xor_sync(~0u, v.m2, s)};
        // both partners join in the same order, so that all lanes agree
        const bool low = (threadIdx.x & s) == 0;
        v = low ? join(v, o) : join(o, v);
    }
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(~0u, v, s);
    return v;
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
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowWarps * 32 : kMaxWarps * 32)
    norm_forward_kernel(const NormArgs p) {
    constexpr int E = VEC * ITEMS;
    using V = Vec<T, VEC>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Moments red[3][kMaxCluster][kMaxWarps];
    const Place<T, VEC, ITEMS, WARP_ROW> at(p);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = at.threads / 32;
    V* ring = reinterpret_cast<V*>(smem) + threadIdx.x;
    const int slot_vecs = ITEMS * at.threads;
    const T* x = static_cast<const T*>(p.x);
    T* y = static_cast<T*>(p.out);

    int64_t next = at.row;
    int filled = 0;
    for (int s = 0; s < p.ring; ++s, next += at.stride, ++filled) {
        if (next < p.rows) fetch(at.c, x + next * p.ldx, ring + s * slot_vecs, at.threads);
        cp_async_commit();
    }
    float w[E], b[E];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const bool in = at.c.has(k);
            w[k * VEC + e] = in && p.weight ? load_as_f32(p.weight, p.param_type, at.c.col(k) + e) : 1.0f;
            b[k * VEC + e] = in && p.bias ? load_as_f32(p.bias, p.param_type, at.c.col(k) + e) : 0.0f;
        }

    // Moments of the thread's own columns of the row in ring slot `slot`.
    auto own = [&](int slot) {
        const V* src = ring + slot * slot_vecs;
        float v[E], n = 0, sum = 0, m2 = 0;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                const V u = src[k * at.threads];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    v[k * VEC + e] = to_f32(u.v[e]);
                    sum += v[k * VEC + e];
                }
                n += VEC;
            }
        const float m = n > 0 ? sum / n : 0.0f;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k))
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = v[k * VEC + e] - m;
                    m2 += d * d;
                }
        return warp_join(Moments{n, sum, m2});
    };
    auto apply = [&](int64_t row, int slot, const Moments& s) {
        const float mean = s.sum / float(p.cols);
        const float rstd = rsqrtf(s.m2 / float(p.cols) + p.eps);
        const V* src = ring + slot * slot_vecs;
        T* dst = y + row * p.ldout;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                const V u = src[k * at.threads];
                V o;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    o.v[e] = from_f32<T>((to_f32(u.v[e]) - mean) * rstd * w[k * VEC + e] + b[k * VEC + e]);
                *reinterpret_cast<V*>(dst + at.c.col(k)) = o;
            }
        const bool writes = WARP_ROW ? lane == 0 : threadIdx.x == 0 && at.rank == 0;
        if (writes) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
    };
    auto refill = [&](int slot) {
        if (next < p.rows) fetch(at.c, x + next * p.ldx, ring + slot * slot_vecs, at.threads);
        next += at.stride;
        cp_async_commit();
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
                if (lane == 0) red[buf][0][warp] = s;
            } else {
                if (lane < p.cluster) {
                    const uint32_t a = saddr(&red[buf][at.rank][warp]);
                    st_cluster_f32(a, uint32_t(lane), s.n);
                    st_cluster_f32(a + 4, uint32_t(lane), s.sum);
                    st_cluster_f32(a + 8, uint32_t(lane), s.m2);
                }
                cluster_arrive();
            }
        };
        auto receive = [&](int buf) {
            Moments s{0, 0, 0};
            for (int i = lane; i < p.cluster * warps; i += 32) s = join(s, red[buf][i / warps][i % warps]);
            return warp_join(s);
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
__global__ void __launch_bounds__(WARP_ROW ? kWarpRowWarps * 32 : kMaxWarps * 32)
    norm_backward_kernel(const NormArgs p) {
    constexpr int E = VEC * ITEMS;
    using V = Vec<T, VEC>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 red[3][kMaxCluster][kMaxWarps];
    const Place<T, VEC, ITEMS, WARP_ROW> at(p);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = at.threads / 32;
    const int slot_vecs = ITEMS * at.threads;
    V* ring_x = reinterpret_cast<V*>(smem) + threadIdx.x;
    V* ring_dy = ring_x + p.ring * slot_vecs;
    float* wsm = reinterpret_cast<float*>(smem + size_t(2 * p.ring) * slot_vecs * sizeof(V)) + threadIdx.x;
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.dy);
    T* dx = static_cast<T*>(p.out);
    const float inv_c = 1.0f / float(p.cols);

    int64_t next = at.row;
    for (int s = 0; s < p.ring; ++s, next += at.stride) {
        if (next < p.rows) {
            fetch(at.c, x + next * p.ldx, ring_x + s * slot_vecs, at.threads);
            fetch(at.c, dy + next * p.lddy, ring_dy + s * slot_vecs, at.threads);
        }
        cp_async_commit();
    }
    // the weight as fp32 in the thread's own shared memory: registers go to
    // the two sums
    if (p.weight) {
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                wsm[(k * VEC + e) * at.threads] =
                    at.c.has(k) ? load_as_f32(p.weight, p.param_type, at.c.col(k) + e) : 0.0f;
    }
    auto weight = [&](int i) { return p.weight ? wsm[i * at.threads] : 1.0f; };
    float aw[E], ab[E];
#pragma unroll
    for (int i = 0; i < E; ++i) aw[i] = ab[i] = 0.0f;

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
        float s1 = 0, s2 = 0;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                const V u = sx[k * at.threads], g = sd[k * at.threads];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float gw = to_f32(g.v[e]) * weight(k * VEC + e);
                    s1 += gw;
                    s2 += gw * ((to_f32(u.v[e]) - st.mean) * st.rstd);
                }
            }
        return make_float2(warp_sum(s1), warp_sum(s2));
    };
    auto apply = [&](int64_t row, int slot, const Stat& st, float2 s) {
        const float c1 = s.x * inv_c, c2 = s.y * inv_c;
        const V* sx = ring_x + slot * slot_vecs;
        const V* sd = ring_dy + slot * slot_vecs;
        T* dst = dx + row * p.ldout;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
            if (at.c.has(k)) {
                const V u = sx[k * at.threads], g = sd[k * at.threads];
                V o;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = to_f32(g.v[e]), xh = (to_f32(u.v[e]) - st.mean) * st.rstd;
                    o.v[e] = from_f32<T>(st.rstd * (d * weight(k * VEC + e) - c1 - xh * c2));
                    aw[k * VEC + e] += d * xh;
                    ab[k * VEC + e] += d;
                }
                *reinterpret_cast<V*>(dst + at.c.col(k)) = o;
            }
    };
    auto refill = [&](int slot) {
        if (next < p.rows) {
            fetch(at.c, x + next * p.ldx, ring_x + slot * slot_vecs, at.threads);
            fetch(at.c, dy + next * p.lddy, ring_dy + slot * slot_vecs, at.threads);
        }
        next += at.stride;
        cp_async_commit();
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
                if (lane == 0) red[buf][0][warp] = s;
            } else {
                if (lane < p.cluster) {
                    const uint32_t a = saddr(&red[buf][at.rank][warp]);
                    st_cluster_f32(a, uint32_t(lane), s.x);
                    st_cluster_f32(a + 4, uint32_t(lane), s.y);
                }
                cluster_arrive();
            }
        };
        auto receive = [&](int buf) {
            float2 s = make_float2(0.0f, 0.0f);
            for (int i = lane; i < p.cluster * warps; i += 32) {
                const float2 v = red[buf][i / warps][i % warps];
                s.x += v.x;
                s.y += v.y;
            }
            return make_float2(warp_sum(s.x), warp_sum(s.y));
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
                            acc[c] = (w ? acc[c] : 0.0f) + aw[k * VEC + e];
                            acc[p.cols + c] = (w ? acc[p.cols + c] : 0.0f) + ab[k * VEC + e];
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
                    if (to_w) to_w[c] = aw[k * VEC + e];
                    if (to_b) to_b[c] = ab[k * VEC + e];
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
    const size_t fixed = backward && d.weight ? size_t(p.threads) * e * 4 : 0;
    // only the vector copies are asynchronous: without them a longer ring
    // hides nothing
    p.ring = vec == 1 ? 1 : int(std::max<size_t>(1, std::min<size_t>(kMaxRing, (kSmemBudget - fixed) / row_bytes)));
    p.smem = p.ring * row_bytes + fixed;
    if (backward && p.warp_row) p.smem = std::max(p.smem, size_t(d.cols) * 8);
    if (d.type == TL_TYPE_BF16)
        p.kernel = vec > 1 ? pick<__nv_bfloat16, 8>(backward, p.warp_row, e) : pick<__nv_bfloat16, 1>(backward, p.warp_row, e);
    else if (d.type == TL_TYPE_F16)
        p.kernel = vec > 1 ? pick<__half, 8>(backward, p.warp_row, e) : pick<__half, 1>(backward, p.warp_row, e);
    else
        p.kernel = vec > 1 ? pick<float, 4>(backward, p.warp_row, e) : pick<float, 1>(backward, p.warp_row, e);
    cudaError_t err = cudaFuncSetAttribute(p.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(p.smem));
    if (err != cudaSuccess) return err;
    int per_sm = 1;
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, p.kernel, p.threads, p.smem);
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
