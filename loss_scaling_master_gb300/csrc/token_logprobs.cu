// token_logprobs.cu - log probabilities of given tokens, the entropy of each row
// and its most probable tokens; and the gradient at the logits.
//
//   m = max z, s = sum exp(z - m), w = sum exp(z - m) (z - m)
//   log p_j = (z_j - m) - log s,  H = log s - w / s
//   dz_j = S (dlogp (1[j = t] - p_j) - dent p_j (log p_j + H))
//
// Forward.  The logits are read once: each thread keeps a running maximum and the
// two sums relative to it, which are rescaled when the maximum grows, at most once
// for eight 16-byte loads.  Few rows are cut over the CTAs of a cluster, whose results
// the first of them joins from shared memory.
//
// The k most probable tokens.  The k-th largest of the threads' maxima is reached by at
// least k elements, so only threads whose maximum reaches it hold any of the k, and
// these are hardly more than k.  What they read is read once more (a thread's share of
// the row each, from L2), and what reaches the bound there is put in order.  (5 of 4096 x
// 128256 bf16 take 174 us so, none 158; lists kept by warps along the row took 703.)
//
// Every row starts where its address lies: a first and a last piece of less than 16
// bytes are taken by single elements, padded with -inf, which adds nothing.
#include <algorithm>

#include "f32x2.cuh"
#include "internal.h"
#include "mx.cuh"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace amp {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e+38f;
constexpr int kMaxParts = 8;  // CTAs of a cluster that share a row
constexpr int kLoads = 8, kBwdLoads = 2;  // 16-byte loads a thread has in flight

struct LogprobsFwd {
    const void *z;
    const int64_t *t;
    float *logp, *ent;
    float2 *stats;  // m, log s
    int64_t *ids;
    float *top;
    int64_t rows, ld;
    int cols, k;
};

__device__ __forceinline__ float exp2_flush(float u) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(u));
    return r;
}

// A row in pieces of 16 bytes: piece i holds the elements base + i * VN and on, of
// which those in [0, cols) exist; only the first and the last may lack some.
template <int XT>
struct Pieces {
    static constexpr int VN = XT == kF32 ? 4 : 8;
    const char *row;
    int base, count, cols;
    __device__ __forceinline__ Pieces(const void *z, int64_t at, int cols_) : cols(cols_) {
        constexpr int esz = XT == kF32 ? 4 : 2;
        row = static_cast<const char *>(z) + at * esz;
        const int past = int(reinterpret_cast<uintptr_t>(row) & 15) / esz;
        base = -past;
        count = int((int64_t(cols) + past + VN - 1) / VN);
    }
    __device__ __forceinline__ int first(int i) const { return base + i * VN; }
    __device__ __forceinline__ bool whole(int i) const { return first(i) >= 0 && first(i) <= cols - VN; }
    __device__ __forceinline__ uint4 load_whole(int i) const {
        return ld16(row + int64_t(first(i)) * (XT == kF32 ? 4 : 2));
    }
    // the raw words; -inf for what does not exist
    __device__ __forceinline__ uint4 load(int i) const {
        constexpr uint32_t none = XT == kF32 ? 0xFF800000u : XT == kF16 ? 0xFC00FC00u : 0xFF80FF80u;
        uint4 u = make_uint4(none, none, none, none);
        if (i >= count) return u;
        const int f = first(i);
        if (whole(i)) return load_whole(i);
        uint32_t w[4] = {none, none, none, none};
#pragma unroll
        for (int e = 0; e < VN; ++e) {
            if (f + e < 0 || f + e >= cols) continue;
            if constexpr (XT == kF32) {
                w[e] = reinterpret_cast<const uint32_t *>(row)[f + e];
            } else {
                const uint32_t v = reinterpret_cast<const uint16_t *>(row)[f + e];
                w[e / 2] = e % 2 ? (w[e / 2] & 0xFFFFu) | (v << 16) : (w[e / 2] & 0xFFFF0000u) | v;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <int XT>
__device__ __forceinline__ void widen(uint4 u, f2 (&y)[Pieces<XT>::VN / 2]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (XT == kF32) {
        y[0] = make_f2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        y[1] = make_f2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (XT == kBF16) y[j] = make_f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
            else y[j] = make_f2(f16_bits_to_f32(w[j] & 0xFFFFu), f16_bits_to_f32(w[j] >> 16));
        }
    }
}
// Largest of a piece's elements, NaN aside.
template <int XT>
__device__ __forceinline__ float largest(uint4 u) {
    if constexpr (XT == kF32) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)),
                     fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    } else {
        uint32_t a, b, c;
        if constexpr (XT == kF16) {
            asm("max.f16x2 %0, %1, %2;" : "=r"(a) : "r"(u.x), "r"(u.y));
            asm("max.f16x2 %0, %1, %2;" : "=r"(b) : "r"(u.z), "r"(u.w));
            asm("max.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
        } else {
            asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(u.x), "r"(u.y));
            asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(u.z), "r"(u.w));
            asm("max.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
        }
        return fmaxf(lowp_to_f32<XT>(c & 0xFFFFu), lowp_to_f32<XT>(c >> 16));
    }
}

// Differences are taken no lower than this in factors (its exponential is 0), so
// that a zero weight never meets an infinity.
constexpr float kFar = -1e4f;

__device__ __forceinline__ f2 exp2_both(f2 u) {
    const float2 s = split(u);
    return make_f2(exp2_flush(s.x), exp2_flush(s.y));
}
__device__ __forceinline__ f2 at_least(f2 u, float low) {
    const float2 s = split(u);
    return make_f2(fmaxf(s.x, low), fmaxf(s.y, low));
}

// The running maximum and the sums relative to it.  A NaN reaches the sums.
struct Sums {
    float m = kLowest, s = 0.0f, w = 0.0f;
    __device__ __forceinline__ void raise(float to) {  // to >= m
        const float d = fmaxf(m - to, kFar), c = exp2_flush(d * kLog2e);
        w = __fmaf_rn(s, d, w) * c;
        s *= c;
        m = to;
    }
    // n pieces' elements, of which big is the largest; ENT: with w
    template <int XT, bool ENT>
    __device__ __forceinline__ void add(const uint4 (&u)[kLoads], int n, float big) {
        if (__any_sync(0xFFFFFFFFu, big > m)) raise(fmaxf(m, big));  // soon rare
        const f2 nm = both(-m);
        f2 s2 = both(0.0f), w2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (j >= n) break;
            f2 y[Pieces<XT>::VN / 2];
            widen<XT>(u[j], y);
#pragma unroll
            for (int e = 0; e < Pieces<XT>::VN / 2; ++e) {
                const f2 d = add2(y[e], nm), x = exp2_both(mul2(d, both(kLog2e)));
                s2 = add2(s2, x);
                if (ENT) w2 = fma2(x, at_least(d, kFar), w2);
            }
        }
        s += sum2(s2);
        if (ENT) w += sum2(w2);
    }
    __device__ __forceinline__ void join(float m2, float s2, float w2) {
        raise(fmaxf(m, m2));
        const float d = fmaxf(m2 - m, kFar), c = exp2_flush(d * kLog2e);
        s = __fmaf_rn(s2, c, s);
        w = __fmaf_rn(__fmaf_rn(s2, d, w2), c, w);
    }
};

// An alternative: larger first, of equals the lower index.
struct Entry {
    float v;
    int i;
};
__device__ __forceinline__ bool before(float v, int i, Entry b) { return v > b.v || (v == b.v && i < b.i); }

// A warp's k best, lane l the l-th (32 are kept: what is behind the k-th does no harm).
struct Best {
    Entry mine{-INFINITY, -1};

    static __device__ __forceinline__ Entry other(Entry e, int mask) {
        return {__shfl_xor_sync(0xFFFFFFFFu, e.v, mask), __shfl_xor_sync(0xFFFFFFFFu, e.i, mask)};
    }
    // the earlier of the two in the lanes that `first` says, the later in the others
    static __device__ __forceinline__ Entry exchange(Entry e, int mask, bool first) {
        const Entry o = other(e, mask);
        return before(o.v, o.i, e) == first ? o : e;
    }
    // sorts a sequence that rises and falls
    static __device__ __forceinline__ Entry settle(Entry e) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 16; j > 0; j >>= 1) e = exchange(e, j, (lane & j) == 0);
        return e;
    }
    // with another sorted list
    __device__ __forceinline__ void merge(Entry e) {
        e = other(e, 31);
        if (before(e.v, e.i, mine)) mine = e;
        mine = settle(mine);
    }

    // one candidate, the same on all lanes
    __device__ __forceinline__ void insert(float v, int i) {
        const int lane = threadIdx.x & 31;
        const bool stays = !before(v, i, mine);
        const int at = __popc(__ballot_sync(0xFFFFFFFFu, stays));  // lanes that stay come first
        const float uv = __shfl_up_sync(0xFFFFFFFFu, mine.v, 1);
        const int ui = __shfl_up_sync(0xFFFFFFFFu, mine.i, 1);
        if (lane > at) mine = {uv, ui};
        if (lane == at) mine = {v, i};
    }
    __device__ __forceinline__ Entry last(int k) const {
        return {__shfl_sync(0xFFFFFFFFu, mine.v, k - 1), __shfl_sync(0xFFFFFFFFu, mine.i, k - 1)};
    }
    // a candidate of each lane
    __device__ __forceinline__ void offer(float v, int i, int k) {
        Entry b = last(k);
        uint32_t in = __ballot_sync(0xFFFFFFFFu, before(v, i, b));
        while (in) {
            const int src = __ffs(in) - 1;
            insert(__shfl_sync(0xFFFFFFFFu, v, src), __shfl_sync(0xFFFFFFFFu, i, src));
            b = last(k);
            in &= ~(1u << src);
            in &= __ballot_sync(0xFFFFFFFFu, before(v, i, b));
        }
    }
    // the elements of a piece a lane that reach the bound
    template <int XT>
    __device__ __forceinline__ void offer_piece(uint4 u, int first, float bound, int k) {
        constexpr int VN = Pieces<XT>::VN;
        const int lane = threadIdx.x & 31;
        const float big = largest<XT>(u);
        uint32_t hits = __ballot_sync(0xFFFFFFFFu, big >= bound && big > -INFINITY);
        while (hits) {
            const int src = __ffs(hits) - 1;
            hits &= hits - 1;
            const uint4 x = make_uint4(__shfl_sync(0xFFFFFFFFu, u.x, src), __shfl_sync(0xFFFFFFFFu, u.y, src),
                                       __shfl_sync(0xFFFFFFFFu, u.z, src), __shfl_sync(0xFFFFFFFFu, u.w, src));
            const int f = __shfl_sync(0xFFFFFFFFu, first, src);
            f2 y[VN / 2];
            float v = -INFINITY;
            widen<XT>(x, y);
#pragma unroll
            for (int e = 0; e < VN; ++e)
                if (lane == e) v = e % 2 ? split(y[e / 2]).y : split(y[e / 2]).x;
            // what is not there is -inf, which never enters
            offer(v >= bound ? v : -INFINITY, v >= bound && v > -INFINITY ? f + lane : INT32_MAX, k);
        }
    }
};

// Values alone, larger first, as Best does it with entries.
__device__ __forceinline__ float settle_values(float v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, v, j);
        v = (lane & j) == 0 ? fmaxf(v, o) : fminf(v, o);
    }
    return v;
}
__device__ __forceinline__ float sort_values(float v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 2; n < 32; n *= 2)
#pragma unroll
        for (int j = n / 2; j > 0; j >>= 1) {
            const float o = __shfl_xor_sync(0xFFFFFFFFu, v, j);
            v = ((lane & j) == 0) == ((lane & n) == 0) ? fmaxf(v, o) : fminf(v, o);
        }
    return settle_values(v);
}

// Of the threads that share a row.
template <int THREADS>
__device__ __forceinline__ void row_sync() {
    if constexpr (THREADS == 32) __syncwarp();
    else __syncthreads();
}

// Entries in order by counting those before each: `put(rank, entry)` for the first 32.
template <int THREADS, class F>
__device__ __forceinline__ void by_rank(const Entry *list, int n, F put) {
    for (int e = int(threadIdx.x); e < n; e += THREADS) {
        const Entry mine = list[e];
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < n; ++o) rank += before(list[o].v, list[o].i, mine);
        if (rank < 32) put(rank, mine);
    }
}

// The k best of what the row's threads of this CTA have read, big the largest that each
// has seen (not NaN), into s_top; filled up with -inf.
template <int XT, int THREADS, int ROWS>
__device__ __forceinline__ void top_of(const Pieces<XT> &row, int first_piece, int step, float big, int k,
                                       Entry (&s_top)[32]) {
    constexpr int WARPS = THREADS / 32, VN = Pieces<XT>::VN, QUEUE = WARPS == 1 ? 64 : 256;
    __shared__ float s_bigs[ROWS][THREADS];
    __shared__ int s_hots[ROWS][THREADS], s_counts[ROWS][2];
    __shared__ Entry s_queues[ROWS][QUEUE];
    float *s_big = s_bigs[threadIdx.y];
    int *s_hot = s_hots[threadIdx.y], *s_count = s_counts[threadIdx.y];
    Entry *queue = s_queues[threadIdx.y];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x < 2) s_count[threadIdx.x] = 0;
    if (threadIdx.x < 32) s_top[threadIdx.x] = {-INFINITY, -1};

    // the k-th largest of the threads' largest
    float bound;
    {
        float v = sort_values(big);
        if constexpr (WARPS > 1) {
            s_big[threadIdx.x] = v;
#pragma unroll
            for (int half = WARPS / 2; half > 0; half /= 2) {
                row_sync<THREADS>();
                if (warp < half) {
                    v = settle_values(fmaxf(v, s_big[32 * (warp + half) + 31 - lane]));
                    s_big[threadIdx.x] = v;
                }
            }
            row_sync<THREADS>();
            bound = s_big[k - 1];
        } else {
            bound = __shfl_sync(0xFFFFFFFFu, v, k - 1);
            __syncwarp();
        }
    }
    // who reached it (in any order: what follows is in one order whatever comes first)
    const uint32_t hot = __ballot_sync(0xFFFFFFFFu, big >= bound && big > -INFINITY);
    if (hot) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&s_count[0], __popc(hot));
        at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(hot & ((1u << lane) - 1));
        if ((hot >> lane) & 1) s_hot[at] = int(threadIdx.x);
    }
    row_sync<THREADS>();
    const int hots = s_count[0];
    for (int h = warp; h < hots; h += WARPS) {
        const int i0 = first_piece + s_hot[h];
        for (int i = i0 + lane * step; i < row.count; i += 32 * step) {
            const uint4 u = row.load(i);
            if (!(largest<XT>(u) >= bound)) continue;
            f2 y[VN / 2];
            widen<XT>(u, y);
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                const float v = e % 2 ? split(y[e / 2]).y : split(y[e / 2]).x;
                if (v >= bound && v > -INFINITY) {
                    const int at = atomicAdd(&s_count[1], 1);
                    if (at < QUEUE) queue[at] = {v, row.first(i) + e};
                }
            }
        }
    }
    row_sync<THREADS>();
    const int n = s_count[1];
    if (n <= QUEUE) {
        by_rank<THREADS>(queue, n, [&](int rank, Entry e) { s_top[rank] = e; });
        row_sync<THREADS>();
        return;
    }
    // too many (equal values, say): lists kept by warps, then joined in halves
    Best best;
    for (int h = warp; h < hots; h += WARPS) {
        const int i0 = first_piece + s_hot[h];
        for (int j = lane; i0 + (j - lane) * step < row.count; j += 32)
            best.offer_piece<XT>(row.load(i0 + j * step), row.first(i0 + j * step), bound, k);
    }
    if constexpr (WARPS > 1) {
        Entry(*list)[32] = reinterpret_cast<Entry(*)[32]>(queue);
        static_assert(QUEUE >= 32 * WARPS, "a list a warp");
        list[warp][lane] = best.mine;
#pragma unroll
        for (int half = WARPS / 2; half > 0; half /= 2) {
            row_sync<THREADS>();
            if (warp < half) {
                best.merge(list[warp + half][lane]);
                list[warp][lane] = best.mine;
            }
        }
    }
    if (warp == 0) s_top[lane] = best.mine;
    row_sync<THREADS>();
}

// THREADS share a row (x), ROWS rows a CTA (y; one where a row has more than a warp).
template <int XT, int THREADS, int ROWS, bool TOP>
__global__ void __launch_bounds__(THREADS *ROWS, 1024 / (THREADS * ROWS))
    logprobs_fwd_kernel(LogprobsFwd P) {
    constexpr int WARPS = THREADS / 32;
    __shared__ float s_m[WARPS], s_s[WARPS], s_w[WARPS];
    __shared__ Entry s_tops[TOP ? ROWS : 1][32], s_all[TOP && WARPS > 1 ? kMaxParts * 32 : 1];
    __shared__ float3 s_cta;
    pdl_wait();
    pdl_trigger();
    uint32_t parts;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
    const uint32_t rank = parts > 1 ? cluster_rank() : 0;
    const int64_t r = int64_t(blockIdx.x / parts) * ROWS + threadIdx.y;
    if (ROWS > 1 && r >= P.rows) return;  // whole warps, which wait for no other
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = P.t ? P.t[r] : 0;
    if (P.t && t < 0) {  // the same in all CTAs of the cluster
        if (rank == 0) {
            if (threadIdx.x == 0) {
                if (P.logp) P.logp[r] = 0.0f;
                if (P.ent) P.ent[r] = 0.0f;
                if (P.stats) P.stats[r] = make_float2(0.0f, 0.0f);
            }
            if (TOP && threadIdx.x < unsigned(P.k)) {
                P.ids[r * P.k + threadIdx.x] = -1;
                P.top[r * P.k + threadIdx.x] = -INFINITY;
            }
        }
        return;
    }
    const Pieces<XT> row(P.z, r * P.ld, P.cols);
    Sums a;
    float most = -INFINITY;  // the thread's largest
    const int step = int(parts) * THREADS;
    for (int i0 = int(rank) * THREADS; i0 < row.count; i0 += kLoads * step) {
        uint4 u[kLoads];
        int n = kLoads;  // loads that any thread has
        // (one test for all: with one a load, a load waited for the last)
        if (row.whole(i0) && row.whole(i0 + (kLoads - 1) * step + THREADS - 1)) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) u[j] = row.load_whole(i0 + j * step + int(threadIdx.x));
        } else {
            n = 0;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                u[j] = row.load(i0 + j * step + int(threadIdx.x));
                n += i0 + j * step < row.count;
            }
        }
        float big = largest<XT>(u[0]);
#pragma unroll
        for (int j = 1; j < kLoads; ++j) big = fmaxf(big, largest<XT>(u[j]));
        if (TOP) most = fmaxf(most, big);
        if (P.ent) a.add<XT, true>(u, n, big);
        else a.add<XT, false>(u, n, big);
    }
    Entry(&s_top)[32] = s_tops[TOP ? threadIdx.y : 0];
    if constexpr (TOP)
        top_of<XT, THREADS, ROWS>(row, int(rank) * THREADS, step, most, P.k, s_top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a.join(__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o),
               __shfl_xor_sync(0xFFFFFFFFu, a.w, o));
    if constexpr (WARPS > 1) {
        if (lane == 0) {
            s_m[warp] = a.m;
            s_s[warp] = a.s;
            s_w[warp] = a.w;
        }
        __syncthreads();
    }
    if (WARPS > 1 && warp == 0) {
        // the warps' sums, a lane each, in one order
        a = Sums();
        if (lane < WARPS) {
            a.m = s_m[lane];
            a.s = s_s[lane];
            a.w = s_w[lane];
        }
#pragma unroll
        for (int o = WARPS / 2; o > 0; o >>= 1)
            a.join(__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o),
                   __shfl_xor_sync(0xFFFFFFFFu, a.w, o));
        if (lane == 0) s_cta = make_float3(a.m, a.s, a.w);
    }
    if (WARPS > 1 && parts > 1) {
        __syncwarp();
        cluster_sync();
        if (rank == 0 && warp == 0) {
            // lane q: the sums of CTA q
            a = Sums();
            if (lane < int(parts)) {
                const uint32_t at = cluster_addr(&s_cta, lane);
                a.m = __uint_as_float(cluster_ld(at));
                a.s = __uint_as_float(cluster_ld(at + 4));
                a.w = __uint_as_float(cluster_ld(at + 8));
            }
#pragma unroll
            for (int o = kMaxParts / 2; o > 0; o >>= 1)
                a.join(__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.s, o),
                       __shfl_xor_sync(0xFFFFFFFFu, a.w, o));
        }
        if constexpr (TOP && WARPS > 1) {
            if (rank == 0) {
                // warp q: the list of CTA q; then in halves
                static_assert(WARPS >= kMaxParts || THREADS == 128, "a list a warp");
                Best best;
                if (warp < int(parts)) {
                    const uint32_t at = cluster_addr(&s_top[lane], warp);
                    best.mine = {__uint_as_float(cluster_ld(at)), int(cluster_ld(at + 4))};
                    s_all[32 * warp + lane] = best.mine;
                }
#pragma unroll
                for (int half = kMaxParts / 2; half > 0; half /= 2) {
                    __syncthreads();
                    if (warp < half && warp + half < int(parts)) {
                        best.merge(s_all[32 * (warp + half) + lane]);
                        s_all[32 * warp + lane] = best.mine;
                    }
                }
                if (warp == 0) s_top[lane] = best.mine;
            }
        }
        __syncwarp();
        cluster_sync();  // nobody leaves while its shared memory is read
    }
    if (rank != 0 || warp != 0) return;
    const float m = __shfl_sync(0xFFFFFFFFu, a.m, 0), logs = logf(__shfl_sync(0xFFFFFFFFu, a.s, 0));
    if (lane == 0) {
        if (P.logp)
            P.logp[r] = !P.t ? 0.0f
                        : t >= P.cols ? NAN
                                      : (load_elem<XT>(P.z, r * P.ld + t) - m) - logs;
        if (P.ent) P.ent[r] = logs - a.w / a.s;
        if (P.stats) P.stats[r] = make_float2(m, logs);
    }
    if (TOP && lane < P.k) {
        const Entry e = s_top[lane];
        const bool none = e.v == -INFINITY;
        P.ids[r * P.k + lane] = none ? -1 : e.i;
        P.top[r * P.k + lane] = none ? -INFINITY : (e.v - m) - logs;
    }
}

// ------------------------------------------------------------------ the gradient
struct LogprobsBwd {
    const void *z;
    const int64_t *t;
    const float2 *stats;
    const float *dlogp, *ent, *dent, *scale;
    void *dz;
    int64_t rows, ld, dld;
    int cols, chunks;
};

// One CTA a share of a row: every element is read and written once, and what the row
// adds are five numbers.  With u = log p:
//   dz = p (A + B u) [+ S dlogp for the token],  A = -S (dlogp + dent H), B = -S dent
template <int XT, int THREADS, int ROWS>
__global__ void __launch_bounds__(THREADS *ROWS) logprobs_bwd_kernel(LogprobsBwd P) {
    constexpr int VN = Pieces<XT>::VN, esz = XT == kF32 ? 4 : 2, U = kBwdLoads;
    pdl_wait();
    pdl_trigger();
    const int64_t r = int64_t(blockIdx.x / unsigned(P.chunks)) * ROWS + threadIdx.y;
    if (ROWS > 1 && r >= P.rows) return;
    const int chunk = int(blockIdx.x % unsigned(P.chunks));
    const Pieces<XT> row(P.z, r * P.ld, P.cols);
    char *out = static_cast<char *>(P.dz) + r * P.dld * esz;
    const bool aligned = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.row)) & 15) == 0;
    const int64_t t = P.t ? P.t[r] : 0;
    const float scale = P.scale ? *P.scale : 1.0f;
    const float dl = P.dlogp ? P.dlogp[r] : 0.0f, de = P.dent ? P.dent[r] : 0.0f, ent = P.dent ? P.ent[r] : 0.0f;
    const float2 st = P.stats[r];
    const bool used = t >= 0;
    const int per = (row.count + P.chunks - 1) / P.chunks, end = min(row.count, (chunk + 1) * per);
    const float dlogp = dl * scale, dent = de * scale, B = -dent, BH = B * ent;
    float A = BH - dlogp;
    if (t >= P.cols && P.t) A = NAN;
    const int at = P.dlogp && used && t < P.cols ? int(t) : -VN;
    const f2 nm = both(-st.x), nl = both(-st.y), nl2 = both(-st.y * kLog2e), A2 = both(A), B2 = both(B);

    auto gradient = [&](const uint4 &u, int f, f2 (&y)[VN / 2]) {
        if (!used) {
#pragma unroll
            for (int e = 0; e < VN / 2; ++e) y[e] = both(0.0f);
            return;
        }
        widen<XT>(u, y);
        float token = 0.0f;
        const bool here = unsigned(at - f) < unsigned(VN);
        if (here) {
#pragma unroll
            for (int e = 0; e < VN; ++e)
                if (f + e == at) token = e % 2 ? split(y[e / 2]).y : split(y[e / 2]).x;
        }
#pragma unroll
        for (int e = 0; e < VN / 2; ++e) {
            const f2 d = add2(y[e], nm), p = exp2_both(fma2(d, both(kLog2e), nl2));
            y[e] = mul2(p, P.dent ? fma2(B2, at_least(add2(d, nl), kFar), A2) : A2);
        }
        if (here) {
            // dlogp (1 - p), without the difference's rounding where p is near 1
            const float lp = (token - st.x) - st.y;
            const float g =
                __fmaf_rn(-dlogp, expm1f(lp), exp2_flush(lp * kLog2e) * __fmaf_rn(B, fmaxf(lp, kFar), BH));
#pragma unroll
            for (int e = 0; e < VN / 2; ++e) {
                const float2 v = split(y[e]);
                y[e] = make_f2(f + 2 * e == at ? g : v.x, f + 2 * e + 1 == at ? g : v.y);
            }
        }
    };
    auto store_whole = [&](int f, const f2 (&y)[VN / 2]) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 v = split(y[XT == kF32 ? q / 2 : q]);
            if constexpr (XT == kF32) w[q] = __float_as_uint(q % 2 ? v.y : v.x);
            else w[q] = f32x2_to_16x2<XT>(v.x, v.y);
        }
        st16(out + int64_t(f) * esz, make_uint4(w[0], w[1], w[2], w[3]));
    };
    for (int i0 = chunk * per; i0 < end; i0 += U * THREADS) {
        const int last = i0 + U * THREADS - 1;
        if (aligned && last < end && row.whole(i0) && row.whole(last)) {
            uint4 u[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                u[j] = used ? row.load_whole(i0 + j * THREADS + int(threadIdx.x)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int f = row.first(i0 + j * THREADS + int(threadIdx.x));
                f2 y[VN / 2];
                gradient(u[j], f, y);
                store_whole(f, y);
            }
            continue;
        }
#pragma unroll 1
        for (int i = i0 + int(threadIdx.x); i < min(end, i0 + U * THREADS); i += THREADS) {
            const int f = row.first(i);
            f2 y[VN / 2];
            gradient(used ? row.load(i) : make_uint4(0, 0, 0, 0), f, y);
            if (aligned && row.whole(i)) {
                store_whole(f, y);
                continue;
            }
#pragma unroll
            for (int e = 0; e < VN; ++e)
                if (f + e >= 0 && f + e < P.cols)
                    store_elem<XT>(out, f + e, e % 2 ? split(y[e / 2]).y : split(y[e / 2]).x);
        }
    }
}

constexpr int kShortRows = 4;  // a CTA, a warp each
template <int XT, int THREADS, int ROWS>
cudaError_t fwd(const LogprobsFwd &P, int parts, int dev, cudaStream_t s) {
    const dim3 grid(unsigned((P.rows + ROWS - 1) / ROWS * parts)), block(THREADS, ROWS);
    return P.k ? launch_pdl_cluster<&logprobs_fwd_kernel<XT, THREADS, ROWS, true>, kAnyShared>(dev, grid, block, parts, s, P)
               : launch_pdl_cluster<&logprobs_fwd_kernel<XT, THREADS, ROWS, false>, kAnyShared>(dev, grid, block, parts, s, P);
}
template <int XT>
cudaError_t fwd_x(const LogprobsFwd &P, int device, cudaStream_t s) {
    const int pieces = P.cols / Pieces<XT>::VN + 1, sms = sm_count(device);
    // A warp a short row, up to 8 alternatives.  Beyond that a lane's maximum bounds little,
    // and one warp orders what reaches the bound: no gain in few rows, up to 20 alternatives
    // one in many, then its queue overflows.  us by a warp and by 128 threads, bf16:
    //     alternatives    0            5            8            20           32
    //     64 x 1000       2.3   2.4    5.7   4.4    6.7   4.7    12.5  6.1    46    7.4
    //     300 x 2000      2.7   2.7    5.8   4.8    7.4   5.1    13.1  6.7    54    8.2
    //     3000 x 4000     7.9   9.3    13.2  15.3   15.0  16.2   23.4  21.3   106   27.0
    //     8192 x 1000     6.7   17.3   14.2  31.9   17.3  34.1   31.6  45.3   130   57.7
    if (P.k <= 8 && (pieces <= 260 || (pieces <= 520 && P.rows >= 16 * sms))) return fwd<XT, 32, kShortRows>(P, 1, device, s);
    // 128 threads a row where those CTAs fill the SMs, 8 each (1023 x 50257 fp16 22.8 us with
    // 128, 21.9 with 256), and rows are not too long; shorter rows already when they are fewer.
    // us with 128 and with 256, bf16:
    //     tokens               32000         50257         64000         80000         128256
    //     1216, alone          13.6  14.8    23.9  26.4    27.5  29.2    33.3  34.6    50.8  52.3
    //     4096, alone          45.5  50.2    71.4  76.4    83.6  86.2    102   105     161   159
    //     1216, 5 alternatives 17.1  19.3    27.4  30.3    32.1  33.8    39.8  40.3    63.0  59.1
    //     4096, 5 alternatives 53.4  64.3    83.6  89.8    98.9  99.3    124   119     202   177
    //     2048, 20             34.6  40.3    56.3  54.5    68.7  59.4    89.2  74.2    143   113
    //     4096, 20             62.9  73.3    104   99.2    129   109     168   134     277   210
    // So the two cross beyond 100000 tokens alone, next to 64000 with 5 alternatives (8000
    // pieces) and between 32000 and 50257 with 20; the limits in pieces are below each.
    const int fits = P.rows >= 8 * sms ? (P.k <= 8 ? 6500 : 4200) : P.rows >= 2 * sms ? 1030 : 260;
    if (pieces <= fits) return fwd<XT, 128, 1>(P, 1, device, s);
    // Until there is a CTA for each SM: a second one there costs the joined rows more than
    // it gives (5 tokens, 1, 2, 4 and 8 CTAs a row: 1 x 128256 bf16 12.0, 9.1, 7.2, 6.3 us;
    // 64 x 50257 fp32 8.8, 7.7, 7.2, 8.2; 150 x 128256 bf16 12.4, 11.6, 15.5, 19.9;
    // 200 x 50257 fp16 9.6, 12.4 with two).
    int parts = 1;
    while (parts < kMaxParts && P.rows * parts <= sms && pieces > parts * 1024) parts *= 2;
    return fwd<XT, 256, 1>(P, parts, device, s);
}
template <int XT>
cudaError_t bwd_x(LogprobsBwd P, int device, cudaStream_t s) {
    const int sms = sm_count(device);
    const int64_t pieces = P.cols / Pieces<XT>::VN + 2;  // a row that starts inside a piece has one more
    P.chunks = 1;
    if (pieces <= 260)
        return launch_pdl_cluster<&logprobs_bwd_kernel<XT, 32, kShortRows>, kAnyShared>(
            device, dim3(unsigned((P.rows + kShortRows - 1) / kShortRows)), dim3(32, kShortRows), 1, s, P);
    if (pieces <= 1030 && P.rows >= 2 * sms)
        return launch_pdl_cluster<&logprobs_bwd_kernel<XT, 128, 1>, kAnyShared>(device, dim3(unsigned(P.rows)), dim3(128), 1, s, P);
    // shares of 8 loads a thread, smaller ones where rows are few
    int64_t chunks = (pieces + 8 * 256 - 1) / (8 * 256);
    while (chunks * P.rows < 4 * sms && chunks * 512 < pieces) chunks *= 2;
    P.chunks = int(chunks);
    return launch_pdl_cluster<&logprobs_bwd_kernel<XT, 256, 1>, kAnyShared>(device, dim3(unsigned(P.rows * P.chunks)), dim3(256), 1, s, P);
}

}  // namespace

cudaError_t launch_logprobs_fwd(const void *z, int elem, int64_t rows, int64_t cols, int64_t ld, const int64_t *t,
                                float *logp, float *ent, float *stats, int64_t *ids, float *top, int k, int device,
                                cudaStream_t s) {
    const LogprobsFwd P{z, t, logp, ent, reinterpret_cast<float2 *>(stats), ids, top, rows, ld, int(cols), k};
    const cudaError_t e = elem == kF32   ? fwd_x<kF32>(P, device, s)
                          : elem == kF16 ? fwd_x<kF16>(P, device, s)
                                         : fwd_x<kBF16>(P, device, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_logprobs_bwd(const void *z, int elem, int64_t rows, int64_t cols, int64_t ld, const int64_t *t,
                                const float *stats, const float *dlogp, const float *ent, const float *dent,
                                const float *scale, void *dz, int64_t dld, int device, cudaStream_t s) {
    const LogprobsBwd P{z, t, reinterpret_cast<const float2 *>(stats), dlogp, ent, dent, scale, dz, rows, ld, dld,
                        int(cols), 1};
    const cudaError_t e = elem == kF32   ? bwd_x<kF32>(P, device, s)
                          : elem == kF16 ? bwd_x<kF16>(P, device, s)
                                         : bwd_x<kBF16>(P, device, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace amp
