// tl_route.cu -- the router around products grouped by expert: the k best
// experts of each token and their weights, the entries' order by expert, the
// weighted sum of the experts' answers, and the gradients of both.
//
// Choosing.  A warp holds a token's logits, logit e in lane e % 32, as keys whose
// order as unsigned integers is that of the logits (0: never chosen).  A round
// takes the warp's largest key with one integer reduction and removes it.  Keys
// of 16-bit logits carry the expert's index in their lower half, the lowest index
// the largest, so a round needs no second reduction for it.
//
// Order by expert.  A stable counting sort, whose places depend on nothing but
// the ids: each CTA counts its entries by expert; then each sums all CTAs' counts
// (those before its own apart), and its warps, whose entries lie one after
// another, rank theirs 32 at a time by the lanes of equal id, which a ballot for
// each bit of the ids gives.  Counting is fused into the choice, so a call is two
// launches, or one where a single CTA does it.
//
// 65536 x 256 bf16, top 8: 55 us among other calls, 50 repeated in a graph, for 6 of bytes.  The
// choice is about two thirds of it, bound by its instructions (some 400 a token; with scalar
// loads, and the next token's not under way meanwhile, it took 47 instead of 38); the order
// the rest, its passes' latency (the counts' loads of a warp are issued together).
#include "tl_launch.h"
#include "tl_route.h"
#include "tl_types.cuh"

#include <algorithm>
#include <climits>

namespace tl {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
// Tokens (or entries) are shared among as many CTAs as SMs, where there is work for them.
constexpr int kSortCtas = 152;

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependents_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- the entries' order ----------------------------------------------------

struct Sort {
    const int32_t* ids;
    int32_t* slots;
    int32_t* rows;
    int32_t* offsets;
    int32_t* counts;  // [groups + 1][kSortCtas]
    int32_t entries, k, groups;
    int32_t per;  // entries of a CTA
};

__device__ __forceinline__ int bin_of(int id, int groups) { return unsigned(id) < unsigned(groups) ? id : groups; }

// The lanes that hold the same b (0 .. 2^bits - 1) as this one.
__device__ __forceinline__ unsigned lanes_of(int b, int bits) {
    unsigned same = 0xffffffffu;
    for (int i = 0; i < bits; ++i) {
        const unsigned set = __ballot_sync(0xffffffffu, (b >> i) & 1);
        same &= (b >> i) & 1 ? set : ~set;
    }
    return same;
}

// Exclusive sum over the CTA's threads; *all is the total.
__device__ int scan_cta(int v, int* scratch, int* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += u;
    }
    if (lane == 31) scratch[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int w = lane < warps ? scratch[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += u;
        }
        scratch[lane] = w;
    }
    __syncthreads();
    *all = scratch[31];
    return s - v + (warp ? scratch[warp - 1] : 0);
}

// The places of entries first .. first + len - 1, `cta` of `ctas`.  at: [warps][groups + 1],
// start: [2 (groups + 1)].  With one CTA there are no counts to read.
__device__ void place_entries(const Sort& p, int first, int len, int cta, int ctas, int* at, int* start, int* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = p.groups + 1;
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) at[i] = 0;
    // all entries of a group in start, those in CTAs before this one in the second half of it
    int* before = start + bins;
    if (ctas > 1)
        for (int g = warp; g < bins; g += kSortWarps) {
            int v[(kSortCtas + 31) / 32], earlier = 0, total = 0;
#pragma unroll
            for (int i = 0; i < (kSortCtas + 31) / 32; ++i) v[i] = i * 32 + lane < ctas ? __ldcg(p.counts + int64_t(g) * kSortCtas + i * 32 + lane) : 0;
#pragma unroll
            for (int i = 0; i < (kSortCtas + 31) / 32; ++i) {
                total += v[i];
                earlier += i * 32 + lane < cta ? v[i] : 0;
            }
            total = __reduce_add_sync(0xffffffffu, total);
            earlier = __reduce_add_sync(0xffffffffu, earlier);
            if (lane == 0) {
                start[g] = total;
                before[g] = earlier;
            }
        }
    __syncthreads();
    // how many of each group a warp has, and each entry's rank among them; those of
    // the first rounds stay in registers
    constexpr int kKept = 8;
    const int span = (len + kSortThreads - 1) / kSortThreads * 32, rounds = span / 32;
    const int from = first + min(len, warp * span), to = first + min(len, (warp + 1) * span);
    int* mine = at + warp * bins;
    const int bits = 32 - __clz(bins);  // (bins itself stands for a lane without an entry)
    auto bin_at = [&](int i) { return i + lane < to ? bin_of(p.ids[i + lane], p.groups) : bins; };
    auto rank_of = [&](int bin) {
        const unsigned same = lanes_of(bin, bits), earlier = same & ((1u << lane) - 1);
        const int rank = bin < bins ? mine[bin] + __popc(earlier) : 0;
        __syncwarp();
        if (bin < bins && earlier == 0) mine[bin] += __popc(same);
        __syncwarp();
        return rank;
    };
    int rank[kKept], bin[kKept];
#pragma unroll
    for (int r = 0; r < kKept; ++r) bin[r] = r < rounds ? bin_at(from + 32 * r) : bins;
#pragma unroll
    for (int r = 0; r < kKept; ++r)
        if (r < rounds) rank[r] = rank_of(bin[r]);
    for (int r = kKept; r < rounds; ++r) rank_of(bin_at(from + 32 * r));
    __syncthreads();
    // where each warp's entries of a group begin, from the group's first in this CTA on
    for (int g = threadIdx.x; g < bins; g += kSortThreads) {
        int s = ctas > 1 ? before[g] : 0;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int v = at[w * bins + g];
            at[w * bins + g] = s;
            s += v;
        }
        if (ctas == 1) start[g] = s;
    }
    __syncthreads();
    int all;
    const int g = threadIdx.x, v = g < p.groups ? start[g] : 0;
    const int begin = scan_cta(v, scratch, &all);
    if (g < p.groups) start[g] = begin;
    if (g == 0) start[p.groups] = all;
    if (cta == 0) {
        if (g < p.groups) p.offsets[g] = begin;
        if (g == 0) p.offsets[p.groups] = all;
    }
    __syncthreads();
    auto put = [&](int i, int b, int in_warp) {
        if (b >= bins) return;
        const int place = start[b] + in_warp;
        p.slots[i + lane] = b < p.groups ? place : -1;
        p.rows[place] = (i + lane) / p.k;
    };
#pragma unroll
    for (int r = 0; r < kKept; ++r)
        if (r < rounds) put(from + 32 * r, bin[r], bin[r] < bins ? mine[bin[r]] + rank[r] : 0);
    if (rounds > kKept) {  // (the kept rounds count again, behind the warp's begin, which then grows)
        __syncwarp();
        for (int r = 0; r < rounds; ++r) {
            const int other = bin_at(from + 32 * r), k = rank_of(other);
            if (r >= kKept) put(from + 32 * r, other, k);
        }
    }
}

__device__ __forceinline__ void place_all(const Sort& p, bool alone) {
    extern __shared__ int sort_smem[];
    __shared__ int scratch[32];
    int* start = sort_smem + kSortWarps * (p.groups + 1);
    const int cta = alone ? 0 : int(blockIdx.x), first = cta * p.per;
    place_entries(p, first, min(p.per, p.entries - first), cta, alone ? 1 : int(gridDim.x), sort_smem, start, scratch);
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const Sort p) {
    extern __shared__ int sort_smem[];
    grid_dependents_go();
    for (int b = threadIdx.x; b <= p.groups; b += kSortThreads) sort_smem[b] = 0;
    __syncthreads();
    const int first = int(blockIdx.x) * p.per, last = min(p.entries, first + p.per);
    for (int i = first + int(threadIdx.x); i < last; i += kSortThreads) atomicAdd(sort_smem + bin_of(p.ids[i], p.groups), 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= p.groups; b += kSortThreads) p.counts[int64_t(b) * kSortCtas + blockIdx.x] = sort_smem[b];
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const Sort p) {
    grid_dependency_wait();  // the counts (and, of a route, the ids) are there
    place_all(p, gridDim.x == 1);
}

// ---- choosing --------------------------------------------------------------

// A logit as a key: larger logits have larger keys, zeros of both signs the same
// one, and -inf and NaN zero, which is never chosen.  16-bit logits (`inf`: the
// bits of infinity): the lower half holds the index.
__device__ __forceinline__ uint32_t key16(uint16_t raw, int e, uint32_t inf) {
    const uint32_t size = raw & 0x7fffu;
    if (size > inf || raw == (0x8000u | inf)) return 0;
    const uint32_t u = size == 0 ? 0x8000u : raw & 0x8000u ? 0xffffu ^ raw : raw | 0x8000u;
    return u << 16 | uint32_t(0xffff - e);
}
__device__ __forceinline__ uint16_t raw16(uint32_t key) {
    const uint32_t u = key >> 16;
    return uint16_t(u & 0x8000u ? u & 0x7fffu : 0xffffu ^ u);
}
template <typename T>
__device__ __forceinline__ uint32_t key_of(T v, int e);
template <>
__device__ __forceinline__ uint32_t key_of<__nv_bfloat16>(__nv_bfloat16 v, int e) {
    return key16(__bfloat16_as_ushort(v), e, 0x7f80u);
}
template <>
__device__ __forceinline__ uint32_t key_of<__half>(__half v, int e) {
    return key16(__half_as_ushort(v), e, 0x7c00u);
}
template <>
__device__ __forceinline__ uint32_t key_of<float>(float v, int) {
    const uint32_t raw = __float_as_uint(v), size = raw & 0x7fffffffu;
    if (size > 0x7f800000u || raw == 0xff800000u) return 0;
    return size == 0 ? 0x80000000u : raw & 0x80000000u ? ~raw : raw | 0x80000000u;
}
template <typename T>
__device__ __forceinline__ float key_value(uint32_t key);
template <>
__device__ __forceinline__ float key_value<__nv_bfloat16>(uint32_t key) {
    return to_f32(__ushort_as_bfloat16(raw16(key)));
}
template <>
__device__ __forceinline__ float key_value<__half>(uint32_t key) {
    return to_f32(__ushort_as_half(raw16(key)));
}
template <>
__device__ __forceinline__ float key_value<float>(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

// A lane's keys, largest first: a network of V (V - 1) / 2 comparisons at most, in which
// neighbours are exchanged.
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[V]) {
#pragma unroll
    for (int round = 0; round < V; ++round)
#pragma unroll
        for (int i = round & 1; i + 1 < V; i += 2) {
            const uint32_t a = key[i], b = key[i + 1];
            key[i] = max(a, b);
            key[i + 1] = min(a, b);
        }
}

struct Choice {
    const void* logits;
    int64_t ld;
    float* weights;
    int32_t tokens;
    int32_t normalize;
    int32_t per;  // tokens of a CTA
};

// A token's logits, V a lane (-inf past the last), as they lie in memory: lane e % 32 has
// logit e or, vectors of V, lane e / V.
template <typename T, int V, bool VECTORS>
__device__ __forceinline__ void load_logits(const T* row, int experts, T (&v)[V]) {
    const int lane = threadIdx.x & 31;
    if constexpr (VECTORS) {
        if (lane * V < experts) {
            const Vec<T, V> u = *reinterpret_cast<const Vec<T, V>*>(row + lane * V);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = u.v[i];
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = !VECTORS && i * 32 + lane < experts ? row[i * 32 + lane] : from_f32<T>(-INFINITY);
}

// V logits a lane.  Writes ids and weights of a CTA's tokens and its counts; alone: places the entries too.
template <typename T, int V, bool VECTORS>
__global__ void __launch_bounds__(kSortThreads) route_kernel(const Choice c, const Sort p, int32_t* ids, const bool alone) {
    extern __shared__ int sort_smem[];
    grid_dependents_go();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = p.k, experts = p.groups;
    for (int b = threadIdx.x; b <= experts; b += kSortThreads) sort_smem[b] = 0;
    __syncthreads();
    const int first = int(blockIdx.x) * c.per, last = min(c.tokens, first + c.per);
    const T* logits = static_cast<const T*>(c.logits);
    T next[V];  // the next token's, on their way
    if (first + warp < last) load_logits<T, V, VECTORS>(logits + int64_t(first + warp) * c.ld, experts, next);
    for (int t = first + warp; t < last; t += kSortWarps) {
        uint32_t key[V], top = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key_of<T>(next[i], VECTORS ? lane * V + i : i * 32 + lane);
        if (t + kSortWarps < last) load_logits<T, V, VECTORS>(logits + int64_t(t + kSortWarps) * c.ld, experts, next);
        float sum = 0, best = 0;
        if (!c.normalize) {
#pragma unroll
            for (int i = 0; i < V; ++i) top = max(top, key[i]);
            top = __reduce_max_sync(0xffffffffu, top);
            best = key_value<T>(top);
            if (top) {
#pragma unroll
                for (int i = 0; i < V; ++i) sum += key[i] ? expf(key_value<T>(key[i]) - best) : 0.0f;
            }
            sum = warp_sum(sum);
        }
        // lane j keeps the j-th best.  Few keys with their indexes are sorted first, and
        // the winner's lane moves up by one; others' are looked through again.
        constexpr bool kSorted = sizeof(T) == 2 && V <= 8;
        uint32_t won = 0;
        int id = -1;
        uint32_t local = 0;
        if constexpr (kSorted) {
            sort_keys(key);
            local = key[0];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) local = max(local, key[i]);
        }
        for (int j = 0; j < k; ++j) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, local);
            if (m == 0) break;
            int e;
            if constexpr (sizeof(T) == 2) {
                e = 0xffff - int(m & 0xffffu);
            } else {
                uint32_t at = ~0u;
                if (local == m) {
#pragma unroll
                    for (int i = V - 1; i >= 0; --i)
                        if (key[i] == m) at = uint32_t(i * 32 + lane);
                }
                e = int(__reduce_min_sync(0xffffffffu, at));
            }
            if (lane == j) {
                won = m;
                id = e;
            }
            if constexpr (kSorted) {
                const bool it = local == m;
#pragma unroll
                for (int i = 0; i + 1 < V; ++i) key[i] = it ? key[i + 1] : key[i];
                key[V - 1] = it ? 0 : key[V - 1];
                local = key[0];
            } else if ((e & 31) == lane) {  // remove the first of the lane's that holds it
                bool here = true;
                local = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const bool it = here && key[i] == m;
                    here = here && !it;
                    key[i] = it ? 0 : key[i];
                    local = max(local, key[i]);
                }
            }
        }
        const float v = key_value<T>(won);
        float w = 0;
        if (c.normalize) {
            best = __shfl_sync(0xffffffffu, v, 0);
            w = id >= 0 ? expf(v - best) : 0.0f;
            sum = warp_sum(w);
        } else if (id >= 0) {
            w = expf(v - best);
        }
        if (lane < k) {
            ids[int64_t(t) * k + lane] = id;
            c.weights[int64_t(t) * k + lane] = id >= 0 ? w / sum : 0.0f;
            if (!alone) atomicAdd(sort_smem + bin_of(id, experts), 1);
        }
    }
    __syncthreads();
    if (alone) {
        place_all(p, true);
        return;
    }
    for (int b = threadIdx.x; b <= experts; b += kSortThreads) p.counts[int64_t(b) * kSortCtas + blockIdx.x] = sort_smem[b];
}

// A warp for each token, whose row of gradients grows in shared memory.
constexpr int kBackThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kBackThreads) route_backward_kernel(const T* logits, int64_t ld, const int32_t* ids, const float* dweights,
                                                                      T* out, int64_t ldo, int tokens, int experts, int k, bool normalize) {
    extern __shared__ float back_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* row = back_smem + warp * experts;
    const int64_t t = int64_t(blockIdx.x) * (kBackThreads / 32) + warp;
    if (t >= tokens) return;
    const T* l = logits + t * ld;
    int id = lane < k ? ids[t * k + lane] : -1;
    if (unsigned(id) >= unsigned(experts)) id = -1;
    const float g = id >= 0 ? dweights[t * k + lane] : 0.0f;
    auto held = [](float v) { return v == v ? v : -INFINITY; };  // NaN counts as -inf
    for (int e = lane; e < experts; e += 32) row[e] = 0;
    float d, s = 0, best, sum = 0;
    if (normalize) {
        const float v = id >= 0 ? held(to_f32(l[id])) : -INFINITY;
        best = warp_max(v);
        const float w = v > -INFINITY ? expf(v - best) : 0.0f;
        sum = warp_sum(w);
        const float p = sum > 0 ? w / sum : w;
        s = warp_sum(p * g);
        d = p * (g - s);
    } else {
        d = g;
        best = -INFINITY;
        for (int e = lane; e < experts; e += 32) best = fmaxf(best, held(to_f32(l[e])));
        best = warp_max(best);
        if (best > -INFINITY)
            for (int e = lane; e < experts; e += 32) sum += expf(held(to_f32(l[e])) - best);
        sum = warp_sum(sum);
        const float v = id >= 0 ? held(to_f32(l[id])) : -INFINITY;
        s = warp_sum(v > -INFINITY ? expf(v - best) / sum * g : 0.0f);
    }
    __syncwarp();
    for (int j = 0; j < k; ++j) {  // in turn: an expert named twice gets both
        if (lane == j && id >= 0) row[id] += d;
        __syncwarp();
    }
    for (int e = lane; e < experts; e += 32) {
        float v = row[e];
        if (!normalize) {
            const float at = held(to_f32(l[e]));
            v = at > -INFINITY ? expf(at - best) / sum * (v - s) : 0.0f;
        }
        out[t * ldo + e] = from_f32<T>(v);
    }
}

// ---- the sum of the experts' answers ------------------------------------------

// `lanes` threads (a power of two) share a token's row, kVectors vectors of N elements
// each; the grid's second dimension walks the row's further vectors.  B entries at
// a time: their rows are all asked for before one is used.  Bound by memory: 8192 x
// 8192 bf16, two entries, 73 us among others, 5.5 TB/s (one vector a thread: 86).
constexpr int kCombineThreads = 256, kVectors = 2;
template <typename T, int N, int B>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const T* y, int64_t ldy, const int32_t* slots, const float* weights, T* out,
                                                                  int64_t ldo, int tokens, int k, int rows, int vectors, int lanes) {
    const int64_t t = int64_t(blockIdx.x) * (kCombineThreads / lanes) + threadIdx.x / lanes;
    const int v0 = int(blockIdx.y) * lanes * kVectors + int(threadIdx.x % lanes);
    if (t >= tokens || v0 >= vectors) return;
    using L = Lanes<N>;
    constexpr int M = N == 1 ? 1 : N / 2;
    L sum[kVectors][M];
#pragma unroll
    for (int q = 0; q < kVectors; ++q)
#pragma unroll
        for (int i = 0; i < M; ++i) sum[q][i] = splat<L>(0.0f);
    for (int j0 = 0; j0 < k; j0 += B) {
        Vec<T, N> u[B][kVectors];
        float w[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int s = j0 + j < k ? slots[t * k + j0 + j] : -1;
            const bool there = unsigned(s) < unsigned(rows);
            w[j] = there ? (weights ? weights[t * k + j0 + j] : 1.0f) : 0.0f;
#pragma unroll
            for (int q = 0; q < kVectors; ++q) {
                if (there && v0 + q * lanes < vectors) {
                    u[j][q] = *reinterpret_cast<const Vec<T, N>*>(y + int64_t(s) * ldy + int64_t(v0 + q * lanes) * N);
                } else {  // a missing answer adds nothing, whatever its weight
#pragma unroll
                    for (int i = 0; i < N; ++i) u[j][q].v[i] = from_f32<T>(0.0f);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j)
#pragma unroll
            for (int q = 0; q < kVectors; ++q) {
                L a[M];
                unpack(u[j][q], a);
#pragma unroll
                for (int i = 0; i < M; ++i) sum[q][i] = fma(a[i], splat<L>(w[j]), sum[q][i]);
            }
    }
#pragma unroll
    for (int q = 0; q < kVectors; ++q) {
        if (v0 + q * lanes >= vectors) break;
        Vec<T, N> o;
        pack(sum[q], o);
        *reinterpret_cast<Vec<T, N>*>(out + t * ldo + int64_t(v0 + q * lanes) * N) = o;
    }
}

// `lanes` threads walk a token's row, four of its entries at a time: dout is read
// once for four, from memory the first time.  8192 x 8192 bf16, two entries: 117 us,
// 5.7 TB/s; 4099 x 1000 fp16, eight: 29 us, 4.9 TB/s (an entry at a time: 37).
template <typename T, int N>
__global__ void __launch_bounds__(kCombineThreads) combine_backward_kernel(const T* dout, int64_t lddout, const T* y, int64_t ldy,
                                                                           const int32_t* slots, const float* weights, T* dy, int64_t lddy,
                                                                           float* dweights, int tokens, int k, int rows, int vectors, int lanes) {
    __shared__ float part[kMaxTop][kCombineThreads / 32];
    const int64_t t = int64_t(blockIdx.x) * (kCombineThreads / lanes) + threadIdx.x / lanes;
    const int first = int(threadIdx.x % lanes), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    using L = Lanes<N>;
    constexpr int M = N == 1 ? 1 : N / 2, B = 4;
    const bool mine = t < tokens;  // (whole warps: lanes is 32 at least)
    for (int j0 = 0; j0 < k; j0 += B) {
        L dot[B];
        int at[B];
        float w[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            dot[j] = splat<L>(0.0f);
            at[j] = mine && j0 + j < k ? slots[t * k + j0 + j] : -1;
            if (unsigned(at[j]) >= unsigned(rows)) at[j] = -1;
            w[j] = at[j] >= 0 && weights ? weights[t * k + j0 + j] : 1.0f;
        }
        if (mine)
            for (int v = first; v < vectors; v += lanes) {
                L g[M];
                Vec<T, N> u[B];
                unpack(*reinterpret_cast<const Vec<T, N>*>(dout + t * lddout + int64_t(v) * N), g);
                if (dweights) {
#pragma unroll
                    for (int j = 0; j < B; ++j)
                        if (at[j] >= 0) u[j] = *reinterpret_cast<const Vec<T, N>*>(y + int64_t(at[j]) * ldy + int64_t(v) * N);
                }
#pragma unroll
                for (int j = 0; j < B; ++j)
                    if (at[j] >= 0) {
                        if (dweights) {
                            L a[M];
                            unpack(u[j], a);
#pragma unroll
                            for (int i = 0; i < M; ++i) dot[j] = fma(g[i], a[i], dot[j]);
                        }
                        L f[M];
#pragma unroll
                        for (int i = 0; i < M; ++i) f[i] = mul(g[i], splat<L>(w[j]));
                        Vec<T, N> o;
                        pack(f, o);
                        *reinterpret_cast<Vec<T, N>*>(dy + int64_t(at[j]) * lddy + int64_t(v) * N) = o;
                    }
            }
        if (dweights)
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const float f = warp_sum(total(dot[j]));
                if (lane == 0 && j0 + j < k) part[j0 + j][warp] = f;
            }
    }
    if (!dweights) return;
    __syncthreads();
    const int per = lanes / 32, groups = kCombineThreads / lanes;  // warps of a token, tokens of a CTA
    for (int i = threadIdx.x; i < groups * k; i += kCombineThreads) {
        const int64_t token = int64_t(blockIdx.x) * groups + i / k;
        if (token >= tokens) continue;
        float f = 0;
        for (int w = 0; w < per; ++w) f += part[i % k][i / k * per + w];
        dweights[token * k + i % k] = f;
    }
}

bool off(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

int route_per(int64_t tokens) { return int(std::max<int64_t>(kSortWarps, (tokens + kSortCtas - 1) / kSortCtas)); }
int group_per(int64_t entries) { return int(std::max<int64_t>(2 * kSortThreads, (entries + kSortCtas - 1) / kSortCtas)); }
// One CTA does all: no second launch, and the further rounds are few (8192 entries by 8
// groups: 7 us; two launches for as many tokens of 64 experts 9).
constexpr int64_t kAloneTokens = 128, kAloneEntries = 8192;

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), unsigned grid, size_t smem, bool early, cudaStream_t stream, A... args) {
    int per_sm = 0;  // (asked for the shared memory that it allows)
    const cudaError_t e = ctas_per_sm(reinterpret_cast<const void*>(kern), kSortThreads, smem, &per_sm);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

size_t place_smem(int64_t groups) { return size_t(kSortWarps + 2) * size_t(groups + 1) * 4; }

Sort sort_of(const RouteDesc& d, int64_t per) {
    return Sort{d.ids, d.slots, d.rows, d.offsets, d.counts, int32_t(d.tokens * d.k), int32_t(d.k), int32_t(d.groups), int32_t(per)};
}

template <typename T>
cudaError_t route_typed(const RouteDesc& d, cudaStream_t stream) {
    const bool alone = d.tokens <= kAloneTokens;
    const int per = alone ? int(d.tokens) : route_per(d.tokens);
    const unsigned grid = unsigned((d.tokens + per - 1) / per);
    const Sort s = sort_of(d, int64_t(per) * d.k);
    const Choice c{d.logits, d.ld, d.weights, int32_t(d.tokens), d.normalize ? 1 : 0, per};
    const size_t smem = alone ? place_smem(d.groups) : size_t(d.groups + 1) * 4;
    auto run = [&](auto kern) { return launch(kern, grid, smem, false, stream, c, s, d.ids, alone); };
    // vectors of a lane, where rows are whole ones on their boundaries (16-bit logits: their order needs the index in the key)
    const auto whole = [&](int v) { return sizeof(T) == 2 && d.groups % v == 0 && d.ld % v == 0 && !off(d.logits, sizeof(T) * v); };
    constexpr bool V = sizeof(T) == 2;
    cudaError_t e;
    if (d.groups <= 32) e = run(route_kernel<T, 1, false>);
    else if (d.groups <= 64) e = whole(2) ? run(route_kernel<T, 2, V>) : run(route_kernel<T, 2, false>);
    else if (d.groups <= 128) e = whole(4) ? run(route_kernel<T, 4, V>) : run(route_kernel<T, 4, false>);
    else if (d.groups <= 256) e = whole(8) ? run(route_kernel<T, 8, V>) : run(route_kernel<T, 8, false>);
    else if (d.groups <= 512) e = run(route_kernel<T, 16, false>);
    else e = run(route_kernel<T, 32, false>);
    if (e != cudaSuccess || alone) return e;
    return launch(sort_place_kernel, grid, place_smem(d.groups), true, stream, s);
}

int row_lanes(int64_t vectors, int most) {
    int lanes = 32;
    while (lanes < most && lanes < vectors) lanes *= 2;
    return lanes;
}

// Vectors of 16 bytes where every row of every matrix starts on 16 bytes and holds whole ones.
template <typename T>
bool whole_vectors(const CombineDesc& d, bool backward) {
    const int64_t n = 16 / sizeof(T);
    if (d.cols % n || off(d.out, 16) || d.ldout % n) return false;
    if (d.y && (off(d.y, 16) || d.ldy % n)) return false;
    return !backward || (!off(d.dout, 16) && d.lddout % n == 0);
}

template <typename T, int N>
cudaError_t combine_vectors(const CombineDesc& d, bool backward, cudaStream_t stream) {
    const int64_t vectors = (d.cols + N - 1) / N;
    const int lanes = row_lanes(backward ? vectors : (vectors + kVectors - 1) / kVectors, kCombineThreads), tokens = kCombineThreads / lanes;
    dim3 grid(unsigned((d.tokens + tokens - 1) / tokens));
    if (!backward) {
        grid.y = unsigned((vectors + lanes * kVectors - 1) / (lanes * kVectors));
        const auto kern = d.k <= 2 ? combine_kernel<T, N, 2> : combine_kernel<T, N, 4>;
        kern<<<grid, kCombineThreads, 0, stream>>>(static_cast<const T*>(d.y), d.ldy, d.slots, d.weights, static_cast<T*>(d.out), d.ldout,
                                                                   int(d.tokens), int(d.k), int(d.rows), int(vectors), lanes);
    } else {
        combine_backward_kernel<T, N><<<grid, kCombineThreads, 0, stream>>>(static_cast<const T*>(d.dout), d.lddout, static_cast<const T*>(d.y), d.ldy, d.slots,
                                                                            d.weights, static_cast<T*>(d.out), d.ldout, d.dweights, int(d.tokens), int(d.k),
                                                                            int(d.rows), int(vectors), lanes);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t combine_typed(const CombineDesc& d, bool backward, cudaStream_t stream) {
    return whole_vectors<T>(d, backward) ? combine_vectors<T, 16 / sizeof(T)>(d, backward, stream) : combine_vectors<T, 1>(d, backward, stream);
}

template <typename F>
cudaError_t by_type(int32_t type, F&& f) {
    if (type == TL_TYPE_BF16) return f(__nv_bfloat16());
    if (type == TL_TYPE_F16) return f(__half());
    return f(float());
}

std::string entries_check(int64_t tokens, int64_t k, int64_t groups) {
    if (tokens < 0 || k < 1 || k > kMaxTop) return "tokens must be >= 0 and the entries of a token 1..32";
    if (groups < 1 || groups > kMaxGroups) return "groups must be 1..1024";
    if (tokens > INT32_MAX / 2 || tokens * k > INT32_MAX / 2) return "too many entries";
    return {};
}

}  // namespace

std::string route_check(const RouteDesc& d, bool with_logits) {
    std::string bad = entries_check(d.tokens, d.k, d.groups);
    if (!bad.empty()) return bad;
    if (with_logits && d.k > d.groups) return "more entries a token than experts";
    if (!d.offsets || off(d.offsets, 4)) return "offsets is null or not 4-byte aligned";
    if (d.tokens == 0) return {};
    if (!d.ids || !d.slots || !d.rows) return "null pointer";
    if (off(d.ids, 4) || off(d.slots, 4) || off(d.rows, 4)) return "ids, slots and rows must be 4-byte aligned";
    if (!with_logits) return {};
    if (!type_known(d.type)) return "unknown tl_type";
    if (!d.logits || !d.weights) return "null pointer";
    if (off(d.logits, type_bytes(d.type)) || off(d.weights, 4)) return "logits or weights are not aligned to their elements";
    if (d.ld < d.groups) return "the logits' leading dimension is smaller than a row";
    return {};
}

size_t route_workspace(int64_t tokens, int64_t k, int64_t groups) {
    if (!entries_check(tokens, k, groups).empty()) return 0;
    return size_t(groups + 1) * kSortCtas * 4;
}

cudaError_t group_rows_launch(const RouteDesc& d, cudaStream_t stream) {
    if (d.tokens == 0) return cudaMemsetAsync(d.offsets, 0, size_t(d.groups + 1) * 4, stream);
    const int64_t entries = d.tokens * d.k;
    const bool alone = entries <= kAloneEntries;
    const int per = alone ? int(entries) : group_per(entries);
    const unsigned grid = unsigned((entries + per - 1) / per);
    const Sort s = sort_of(d, per);
    if (grid > 1) {
        const cudaError_t e = launch(sort_count_kernel, grid, size_t(d.groups + 1) * 4, false, stream, s);
        if (e != cudaSuccess) return e;
    }
    return launch(sort_place_kernel, grid, place_smem(d.groups), grid > 1, stream, s);
}

cudaError_t route_launch(const RouteDesc& d, cudaStream_t stream) {
    if (d.tokens == 0) return cudaMemsetAsync(d.offsets, 0, size_t(d.groups + 1) * 4, stream);
    return by_type(d.type, [&](auto t) { return route_typed<decltype(t)>(d, stream); });
}

std::string route_backward_check(const RouteBackwardDesc& d) {
    std::string bad = entries_check(d.tokens, d.k, d.experts);
    if (!bad.empty()) return bad;
    if (d.k > d.experts) return "more entries a token than experts";
    if (!type_known(d.type)) return "unknown tl_type";
    if (d.tokens == 0) return {};
    if (!d.logits || !d.ids || !d.dweights || !d.dlogits) return "null pointer";
    if (off(d.logits, type_bytes(d.type)) || off(d.dlogits, type_bytes(d.type)) || off(d.ids, 4) || off(d.dweights, 4))
        return "an operand is not aligned to its elements";
    if (d.ld < d.experts || d.ldd < d.experts) return "a leading dimension is smaller than a row";
    return {};
}

cudaError_t route_backward_launch(const RouteBackwardDesc& d, cudaStream_t stream) {
    if (d.tokens == 0) return cudaSuccess;
    constexpr int tokens = kBackThreads / 32;
    const unsigned grid = unsigned((d.tokens + tokens - 1) / tokens);
    return by_type(d.type, [&](auto t) {
        using T = decltype(t);
        route_backward_kernel<T><<<grid, kBackThreads, size_t(tokens) * size_t(d.experts) * 4, stream>>>(
            static_cast<const T*>(d.logits), d.ld, d.ids, d.dweights, static_cast<T*>(d.dlogits), d.ldd, int(d.tokens), int(d.experts), int(d.k),
            d.normalize);
        return cudaGetLastError();
    });
}

std::string combine_check(const CombineDesc& d, bool backward) {
    if (d.tokens < 0 || d.k < 1 || d.k > kMaxTop) return "tokens must be >= 0 and the entries of a token 1..32";
    if (d.tokens > INT32_MAX / 2 || d.tokens * d.k > INT32_MAX / 2) return "too many entries";
    if (d.cols < 1 || d.cols > (1 << 20)) return "cols must be 1..1048576";
    if (d.rows < 0 || d.rows > INT32_MAX / 2) return "rows must be >= 0 and below 2^30";
    if (!type_known(d.type)) return "unknown tl_type";
    if (d.tokens == 0) return {};
    if (!d.slots || off(d.slots, 4) || off(d.weights, 4)) return "slots are null, or slots or weights not 4-byte aligned";
    const size_t e = type_bytes(d.type);
    if (!backward) {
        if (!d.out || off(d.out, e) || d.ldout < d.cols) return "out is null, not aligned to its elements, or its leading dimension too small";
        if (d.rows > 0 && (!d.y || off(d.y, e) || d.ldy < d.cols)) return "y is null, not aligned to its elements, or its leading dimension too small";
        return {};
    }
    if (!d.dout || off(d.dout, e) || d.lddout < d.cols) return "dout is null, not aligned to its elements, or its leading dimension too small";
    if (d.rows > 0 && (!d.out || off(d.out, e) || d.ldout < d.cols)) return "dy is null, not aligned to its elements, or its leading dimension too small";
    if (off(d.dweights, 4)) return "dweights is not 4-byte aligned";
    if (d.dweights && d.rows > 0 && (!d.y || off(d.y, e) || d.ldy < d.cols)) return "y is null, not aligned to its elements, or its leading dimension too small";
    return {};
}

cudaError_t combine_launch(const CombineDesc& d, cudaStream_t stream) {
    if (d.tokens == 0) return cudaSuccess;
    return by_type(d.type, [&](auto t) { return combine_typed<decltype(t)>(d, false, stream); });
}

cudaError_t combine_backward_launch(const CombineDesc& d, cudaStream_t stream) {
    if (d.tokens == 0) return cudaSuccess;
    return by_type(d.type, [&](auto t) { return combine_typed<decltype(t)>(d, true, stream); });
}

}  // namespace tl
