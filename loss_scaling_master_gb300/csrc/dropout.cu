// dropout.cu - dropout whose mask is a function of the element's place and never
// stored, added to a residual; its gradient, alone or with that of the bias that was
// added before it.
//
//   y = residual + (bits(k) >= T ? x * 65536 / (65536 - T) : 0),  T = RNE(65536 p)
//
// bits(k): 16 bits of Philox4x32-10 (philox.cuh), one call of the generator for 8
// consecutive elements, so the backward pass makes the same mask again in whichever
// order it walks.  The generator's 20 wide multiplications and 60 other instructions
// for 8 elements are a third of what the issue rate leaves an element at the rate of
// memory.
#include "column_sums.cuh"
#include "internal.h"
#include "philox.cuh"

namespace amp {
namespace {

struct Dropout {
    const void *x, *res;
    void *y, *db;
    const int32_t *step;
    uint64_t seed;
    int64_t rows, cols;  // flat: rows = 1
    float scale;
    uint32_t drop, last;  // T, and 65536 T - 1: of 32 bits whose upper half is u, u >= T where they are above it
    uint32_t site;
    int otype;
};

// What becomes of 8 elements x of the group.  ALL: T = 0.
template <bool ALL>
__device__ __forceinline__ void drop8(const Dropout &P, int32_t step, int64_t group, float (&x)[8]) {
    if constexpr (ALL) return;
    const uint4 r = sr_random8(P.seed, step, int32_t(P.site), group);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = x[2 * j] * P.scale, b = x[2 * j + 1] * P.scale;
        x[2 * j] = (w[j] << 16) > P.last ? a : 0.0f;
        x[2 * j + 1] = w[j] > P.last ? b : 0.0f;
    }
}
// Bit j: element j of the group stays.
template <bool ALL>
__device__ __forceinline__ uint32_t keep8(const Dropout &P, int32_t step, int64_t group) {
    if constexpr (ALL) return 0xFFu;
    const uint4 r = sr_random8(P.seed, step, int32_t(P.site), group);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if ((w[j] << 16) > P.last) m |= 1u << (2 * j);
        if (w[j] > P.last) m |= 2u << (2 * j);
    }
    return m;
}

// 8 elements a thread, every address aligned; the last ones one at a time.
template <int XT, bool RES, bool ALL>
__global__ void __launch_bounds__(kThreads) dropout_vec_kernel(Dropout P) {
    pdl_wait();
    pdl_trigger();
    const int32_t step = P.step ? *P.step : 0;
    const int64_t groups = P.cols >> 3;
    for (int64_t g = int64_t(blockIdx.x) * kThreads + threadIdx.x; g < groups; g += int64_t(gridDim.x) * kThreads) {
        float x[8], r[8];
        ldv<XT>(P.x, 8 * g, x);
        if (RES) ldv<XT>(P.res, 8 * g, r);
        drop8<ALL>(P, step, g, x);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (RES) x[j] = r[j] + x[j];
        stv<XT>(P.y, 8 * g, x);
    }
    const int64_t k = 8 * groups + threadIdx.x;
    if (blockIdx.x == 0 && k < P.cols) {
        float v = (keep8<ALL>(P, step, groups) >> threadIdx.x) & 1 ? load_elem<XT>(P.x, k) * P.scale : 0.0f;
        if (RES) v = load_elem<XT>(P.res, k) + v;
        store_elem<XT>(P.y, k, v);
    }
}

// Any address: a warp takes 256 elements, a lane makes the mask of 8 consecutive ones
// and applies that of every 32nd.
template <int XT, bool RES, bool ALL>
__global__ void __launch_bounds__(kThreads) dropout_elem_kernel(Dropout P) {
    pdl_wait();
    pdl_trigger();
    const int32_t step = P.step ? *P.step : 0;
    const int lane = threadIdx.x & 31;
    const int64_t stride = int64_t(gridDim.x) * kThreads * 8;
    for (int64_t k0 = (int64_t(blockIdx.x) * kThreads + (threadIdx.x & ~31)) * 8; k0 < P.cols; k0 += stride) {
        const uint32_t m = keep8<ALL>(P, step, (k0 >> 3) + lane);
        float x[8], r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t k = k0 + 32 * j + lane;
            x[j] = k < P.cols ? load_elem<XT>(P.x, k) : 0.0f;
            r[j] = RES && k < P.cols ? load_elem<XT>(P.res, k) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t k = k0 + 32 * j + lane;
            const uint32_t b = __shfl_sync(0xFFFFFFFFu, m, 4 * j + lane / 8);
            float v = (b >> (lane & 7)) & 1 ? x[j] * P.scale : 0.0f;
            if (RES) v = r[j] + v;
            if (k < P.cols) store_elem<XT>(P.y, k, v);
        }
    }
}

// The gradient with the bias's: by columns (column_sums.cuh).  16-bit rows come kAhead
// ahead through shared memory (16384 x 5120 bf16 59 us, after a forward pass 74; by
// registers, three rows at once, 66.5 and 88; 4 rows ahead 59.2 and 77, 8 63 and 73).
constexpr int kAhead = 6, kRingShared = 132;  // KB an SM: 4 CTAs of 29
template <bool ALL, int XT, class S>
__global__ void __launch_bounds__(S::threads, S::ctas) dropout_bias_ring_kernel(Dropout P) {
    static_assert(XT != kF32);
    __shared__ uint4 s_ring[kAhead][S::threads];
    pdl_wait();
    pdl_trigger();
    const SumShare<S> at(P.rows);
    const int32_t step = P.step ? *P.step : 0;
    const int64_t c = at.col0 + int(threadIdx.x) % S::across * 8, hop = S::groups * P.cols;
    const int64_t end = c < P.cols ? at.row1 * P.cols : 0;
    int64_t k = (at.row0 + int(threadIdx.x) / S::across) * P.cols + c;
    float a[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const auto ask = [&](int64_t at_k, int slot) {
        if (at_k < end) copy_ahead<16>(&s_ring[slot][threadIdx.x], static_cast<const char *>(P.x) + 2 * at_k);
        copies_of_row();
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ask(k + i * hop, i);
    for (int slot = 0; k < end; k += hop) {
        copies_wait<kAhead - 1>();
        const uint4 g[1] = {s_ring[slot][threadIdx.x]};
        float y[8];
        raw8_to_f32<XT>(g, y);
        drop8<ALL>(P, step, k >> 3, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += y[j];
        stv<XT>(P.y, k, y);
        ask(k + kAhead * hop, slot);
        slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
    sum_join<S>(at, P.cols, a, P.db, P.otype);
}
// fp32 rows go through registers, two a step (8192 x 2048 22.8 us; through shared memory,
// where a thread's two copies each take half of every 32 bytes, 35).
template <bool ALL, class S>
__global__ void __launch_bounds__(S::threads, S::ctas) dropout_bias_f32_kernel(Dropout P) {
    constexpr int U = 2;
    pdl_wait();
    pdl_trigger();
    const SumShare<S> at(P.rows);
    const int32_t step = P.step ? *P.step : 0;
    const int64_t c = at.col0 + int(threadIdx.x) % S::across * 8;
    const bool in = c < P.cols;
    float a[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t r0 = at.row0 + int(threadIdx.x) / S::across; in && r0 < at.row1; r0 += U * S::groups) {
        float y[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * S::groups;
            if (r >= at.row1) break;
            ldv<kF32>(P.x, r * P.cols + c, y[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * S::groups, k = r * P.cols + c;
            if (r >= at.row1) break;
            drop8<ALL>(P, step, k >> 3, y[u]);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] += y[u][j];
            stv<kF32>(P.y, k, y[u]);
        }
    }
    sum_join<S>(at, P.cols, a, P.db, P.otype);
}
// Rows of any length (flat_sums): a group of elements is one of the generator's.
template <int XT, bool ALL>
struct DropoutFlat {
    const Dropout &P;
    int64_t all;
    int32_t step;
    using Raw = RawGroup<XT>;
    __device__ __forceinline__ Raw load(int64_t g, bool whole) const {
        Raw r;
        r.load(P.x, g, whole, all);
        return r;
    }
    __device__ __forceinline__ void values(const Raw &raw, int64_t g, int64_t, int64_t, float (&y)[8]) const {
        raw8_to_f32<XT>(raw.u, y);
        drop8<ALL>(P, step, g, y);
    }
    __device__ __forceinline__ void store(int64_t g, int lo, int hi, const float (&y)[8]) const {
        store_group<XT>(P.y, g, lo, hi, y);
    }
};
template <int XT, bool ALL>
__global__ void __launch_bounds__(SumFlat::threads, SumFlat::ctas) dropout_bias_flat_kernel(Dropout P) {
    pdl_wait();
    pdl_trigger();
    const SumShare<SumFlat> at(P.rows);
    DropoutFlat<XT, ALL> op{P, P.rows * P.cols, P.step ? *P.step : 0};
    flat_sums(at, P.rows, P.cols, op, P.db, P.otype);
}
// Any size and address.  A warp's 32 columns of a row lie in at most 5 of the
// generator's groups: 30 lanes make the masks of 6 rows.
template <int XT, bool ALL>
__global__ void __launch_bounds__(SumElem::threads, SumElem::ctas) dropout_bias_elem_kernel(Dropout P) {
    using S = SumElem;
    constexpr int U = 6;
    pdl_wait();
    pdl_trigger();
    const SumShare<S> at(P.rows);
    const int32_t step = P.step ? *P.step : 0;
    const int lane = threadIdx.x & 31;
    const int64_t c0 = at.col0, c = c0 + lane;  // a warp is a row of the tile
    const bool in = c < P.cols;
    float a[1] = {0.0f};
    for (int64_t r0 = at.row0 + int(threadIdx.x) / S::across; r0 < at.row1; r0 += U * S::groups) {
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * S::groups;
            x[u] = in && r < at.row1 ? load_elem<XT>(P.x, r * P.cols + c) : 0.0f;
        }
        const int64_t k0 = (r0 + int64_t(min(lane / 5, U - 1)) * S::groups) * P.cols + c0;
        const uint32_t m = keep8<ALL>(P, step, (k0 >> 3) + lane % 5);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * S::groups, k = r * P.cols + c0;
            const int off = int(k & 7) + lane;
            const uint32_t b = __shfl_sync(0xFFFFFFFFu, m, 5 * u + off / 8);
            const float v = (b >> (off & 7)) & 1 ? x[u] * P.scale : 0.0f;
            if (in && r < at.row1) {
                a[0] += v;
                store_elem<XT>(P.y, k + lane, v);
            }
        }
    }
    sum_join<S>(at, P.cols, a, P.db, P.otype);
}

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

template <int XT, bool ALL>
cudaError_t go(const Dropout &P, int dev, cudaStream_t s) {
    const bool vec = !off16(P.x) && !off16(P.res) && !off16(P.y);
    if (P.db) {
        if (!vec) return launch_sums<SumElem, &dropout_bias_elem_kernel<XT, ALL>>(P.rows, P.cols, dev, s, P);
        if (P.cols % 8) return launch_sums<SumFlat, &dropout_bias_flat_kernel<XT, ALL>>(P.rows, P.cols, dev, s, P);
        if constexpr (XT == kF32)
            return launch_sums<SumVec<32>, &dropout_bias_f32_kernel<ALL, SumVec<32>>>(P.rows, P.cols, dev, s, P);
        else if (narrow_tiles(P.cols, dev))
            return launch_sums<SumVec<32>, &dropout_bias_ring_kernel<ALL, XT, SumVec<32>>, kRingShared>(P.rows, P.cols, dev, s, P);
        else
            return launch_sums<SumVec<64>, &dropout_bias_ring_kernel<ALL, XT, SumVec<64>>, kRingShared>(P.rows, P.cols, dev, s, P);
    }
    Dropout F = P;
    F.cols = P.rows * P.cols;
    F.rows = 1;
    const int64_t want = (F.cols + kThreads * 8 - 1) / (kThreads * 8);
    const dim3 grid(unsigned(std::min<int64_t>(want, int64_t(sm_count(dev)) * 64))), block(kThreads);
    if (vec)
        return F.res ? launch_pdl_cluster<&dropout_vec_kernel<XT, true, ALL>, kSmallShared>(dev, grid, block, 1, s, F)
                     : launch_pdl_cluster<&dropout_vec_kernel<XT, false, ALL>, kSmallShared>(dev, grid, block, 1, s, F);
    return F.res ? launch_pdl_cluster<&dropout_elem_kernel<XT, true, ALL>, kSmallShared>(dev, grid, block, 1, s, F)
                 : launch_pdl_cluster<&dropout_elem_kernel<XT, false, ALL>, kSmallShared>(dev, grid, block, 1, s, F);
}
template <int XT>
cudaError_t go_all(const Dropout &P, int dev, cudaStream_t s) {
    return P.drop == 0 ? go<XT, true>(P, dev, s) : go<XT, false>(P, dev, s);
}

}  // namespace

cudaError_t launch_dropout(const void *x, const void *res, int elem, int64_t rows, int64_t cols, uint32_t drop,
                           uint64_t seed, const int32_t *step, uint32_t site, void *y, void *db, int dbelem,
                           int device, cudaStream_t s) {
    const float scale = drop < 65536u ? float(65536.0 / double(65536u - drop)) : 0.0f;
    const Dropout P{x, res, y, db, step, seed, rows, cols, scale, drop, (drop << 16) - 1, site, dbelem};
    const cudaError_t e = elem == kF32   ? go_all<kF32>(P, device, s)
                          : elem == kF16 ? go_all<kF16>(P, device, s)
                                         : go_all<kBF16>(P, device, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace amp
