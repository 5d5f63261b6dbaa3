// column_sums.cuh - sums over the rows of a matrix, for the gradient of a bias: what
// its kernels share.
//
// A CTA takes a few columns of a share of the rows, the CTAs of a cluster the shares of
// the same columns; each adds its rows in registers, then its row groups in shared
// memory, and sends each of the cluster's CTAs the part of the columns that that one
// adds up.  The order of every sum depends on the shape and on whether rows are taken
// by 16 bytes (no atomics, so equal calls give equal bits), and nothing goes through
// global memory or a second launch.
#pragma once

#include <algorithm>

#include "internal.h"
#include "mx.cuh"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace amp {

constexpr int kSumParts = 8;  // CTAs of a cluster, at most (16 are slower to start and meet: 1024 x 768 + 0.6 us)

// How a CTA takes its columns: threads, CTAs an SM holds, columns, threads beside one
// another on a row, row groups, and the lines of partial sums in shared memory.
template <int COLS>
struct SumVec {  // rows of whole groups of 8 elements, aligned: 8 columns a thread
    static constexpr int threads = 256, ctas = 4, cols = COLS, across = COLS / 8, groups = threads / across;
    static constexpr int each = 8, lines = threads / 32, pitch = cols;
};
struct SumFlat {  // rows of any length: see flat_sums
    static constexpr int threads = 256, ctas = 4, cols = 56, across = 8, groups = 32;
    static constexpr int each = 2, lines = threads / 32, pitch = 64;
};
struct SumElem {  // any address: a column a thread
    static constexpr int threads = 512, ctas = 2, cols = 32, across = cols, groups = 16;
    static constexpr int each = 1, lines = groups, pitch = cols;
};

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// This CTA's columns and rows.  Every thread makes one as it starts: the other CTAs learn
// that this one has.
template <class S>
struct SumShare {
    uint32_t rank, parts;
    int64_t col0, row0, row1;
    __device__ __forceinline__ explicit SumShare(int64_t rows) {
        parts = cluster_size();
        rank = parts > 1 ? cluster_rank() : 0;
        col0 = int64_t(blockIdx.x / parts) * S::cols;
        row0 = rows * rank / parts;
        row1 = rows * (rank + 1) / parts;
        if (parts > 1) cluster_arrive_all();
    }
};

// Adds up all threads' a[] (8 columns from 8 x, or column x, x the thread's place on
// the row; SumFlat: the lane's column and the 32nd after it) and stores the columns' sums.
// Every thread of every CTA of the cluster calls it once.
template <class S>
__device__ __forceinline__ void sum_join(const SumShare<S> &at, int64_t cols, const float (&a)[S::each], void *out,
                                         int otype) {
    __shared__ __align__(16) float s_line[S::lines][S::pitch];
    __shared__ float s_recv[kSumParts][S::cols];
    if constexpr (S::each == 8) {
        // the row groups of a warp
        float b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            b[j] = a[j];
#pragma unroll
            for (int o = S::across; o < 32; o *= 2) b[j] += __shfl_xor_sync(0xFFFFFFFFu, b[j], o);
        }
        if ((threadIdx.x & 31) < S::across) {
            float4 *to = reinterpret_cast<float4 *>(&s_line[threadIdx.x >> 5][8 * (threadIdx.x & 31)]);
            to[0] = make_float4(b[0], b[1], b[2], b[3]);
            to[1] = make_float4(b[4], b[5], b[6], b[7]);
        }
    } else if constexpr (S::each == 2) {
        s_line[threadIdx.x >> 5][threadIdx.x & 31] = a[0];
        s_line[threadIdx.x >> 5][32 + (threadIdx.x & 31)] = a[1];
    } else {
        s_line[threadIdx.x / S::pitch][threadIdx.x % S::pitch] = a[0];
    }
    __syncthreads();
    if (at.parts > 1) cluster_wait_all();  // every CTA has started
    const int mine = (S::cols + int(at.parts) - 1) / int(at.parts);  // columns that a CTA adds up
    if (threadIdx.x < S::cols) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < S::lines; ++i) t += s_line[i][threadIdx.x];
        const int q = int(threadIdx.x) / mine;
        if (at.parts > 1) cluster_st(cluster_addr(&s_recv[at.rank][threadIdx.x - q * mine], uint32_t(q)), t);
        else s_recv[0][threadIdx.x] = t;
    }
    __syncwarp();
    if (at.parts > 1) {
        cluster_arrive_all();
        cluster_wait_all();  // what was sent is here; nobody reaches into another CTA from now on
    }
    const int c = int(at.rank) * mine + int(threadIdx.x);
    if (threadIdx.x < unsigned(mine) && c < S::cols && at.col0 + c < cols) {
        float t = s_recv[0][threadIdx.x];
#pragma unroll
        for (uint32_t q = 1; q < kSumParts; ++q)
            if (q < at.parts) t += s_recv[q][threadIdx.x];
        if (otype == kF32) store_elem<kF32>(out, at.col0 + c, t);
        else if (otype == kF16) store_elem<kF16>(out, at.col0 + c, t);
        else store_elem<kBF16>(out, at.col0 + c, t);
    }
}

// Rows on their way to shared memory, which takes no registers: N bytes a thread, for itself
// alone, so that no barrier is needed.
template <int N>
__device__ __forceinline__ void copy_ahead(void *to, const void *from) {
    const uint32_t at = uint32_t(__cvta_generic_to_shared(to));
    if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(N) : "memory");
}
// What was asked for since the last call belongs to one row.
__device__ __forceinline__ void copies_of_row() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LATER>  // all rows but the last LATER are there
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory"); }

// Rows of any length, tensors aligned to 16 bytes: the matrix is taken as a flat run of
// groups of 8 elements, of which a tile's part of a row holds at most `across`, the first
// and the last perhaps in part.  What the op makes of a warp's groups goes through shared
// memory to a column or two a lane.  (By single elements 16383 x 5121 bf16 dropout 189 us,
// so 129; with GELU 383 and 198.  Tiles of 24 columns, four groups, take 2047 x 1111 fp32
// dropout from 8.8 us to 10.1, 8192 x 257 bf16 from 17.1 to 13.8, wider ones to twice as long.)
//
// Op: Raw load(g, whole), void values(raw, g, r, c, y) (c: the column of element 0, may
// lie before the tile), void store(g, lo, hi, y); g counts groups, whole: all 8 exist.
template <class Op>
__device__ __forceinline__ void flat_sums(const SumShare<SumFlat> &at, int64_t rows, int64_t cols, Op &op, void *out,
                                          int otype) {
    using S = SumFlat;
    constexpr int U = 2, PITCH = 68, WARP_ROWS = 32 / S::across;
    __shared__ __align__(16) float s_rows[S::threads / 32][U][WARP_ROWS][PITCH];
    const int64_t all = rows * cols;
    const int width = int(min(int64_t(S::cols), cols - at.col0));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tx = lane % S::across, ty = lane / S::across;
    float a[2] = {0.0f, 0.0f};
    for (int64_t base = at.row0 + warp * WARP_ROWS; base < at.row1; base += U * S::groups) {
        typename Op::Raw raw[U];
        int64_t g[U];
        int lo[U], hi[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = base + u * S::groups + ty, k0 = r * cols + at.col0;
            const int off = int(k0 & 7);
            g[u] = (k0 >> 3) + tx;
            lo[u] = max(0, off - 8 * tx);
            hi[u] = r < at.row1 ? max(0, min(8, off + width - 8 * tx)) : 0;
            if (hi[u] > lo[u]) raw[u] = op.load(g[u], 8 * g[u] + 8 <= all);
        }
        __syncwarp();  // the last rows are read
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = base + u * S::groups + ty;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = 0.0f;
            if (hi[u] > lo[u]) {
                op.values(raw[u], g[u], r, 8 * g[u] - r * cols, y);
                op.store(g[u], lo[u], hi[u], y);
            }
            float4 *to = reinterpret_cast<float4 *>(&s_rows[warp][u][ty][8 * tx]);
            to[0] = make_float4(y[0], y[1], y[2], y[3]);
            to[1] = make_float4(y[4], y[5], y[6], y[7]);
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t off = uint32_t((base + u * S::groups) * cols + at.col0);
#pragma unroll
            for (int i = 0; i < WARP_ROWS; ++i) {  // rows behind the last are zeros
                const float *from = s_rows[warp][u][i] + ((off + uint32_t(i) * uint32_t(cols)) & 7);
                if (lane < width) a[0] += from[lane];
                if (lane + 32 < width) a[1] += from[lane + 32];
            }
        }
    }
    sum_join<S>(at, cols, a, out, otype);
}

// Shares of the rows: as many as make the rounds of CTAs that the GPU holds at once
// shortest, while all but one of them would have more than a row a group.  CTAs of clusters start one after another, 5 ns each, so
// beyond two an SM a share is at least four rows a group (1000 x 2304 dropout by 576 CTAs
// 5.2 us, by 288 4.3).
template <class S>
int sum_parts(int64_t rows, int64_t tiles, int sms) {
    const int64_t room = int64_t(sms) * S::ctas;
    int parts = 1;
    double least = 0.0;
    for (int p = 1; p <= kSumParts; ++p) {
        if (p > 1 && rows <= int64_t(S::groups) * (p - 1)) break;
        if (p > 1 && tiles * p > 2 * sms && rows < int64_t(4 * S::groups) * p) break;
        const double t = double((tiles * p + room - 1) / room) / p;
        if (p == 1 || t < least) {
            least = t;
            parts = p;
        }
    }
    return parts;
}
template <class S, auto Kernel, int SharedKB = kSmallShared, class A>
cudaError_t launch_sums(int64_t rows, int64_t cols, int device, cudaStream_t s, const A &args) {
    const int64_t tiles = (cols + S::cols - 1) / S::cols;
    const int parts = sum_parts<S>(rows, tiles, sm_count(device));
    return launch_pdl_cluster<Kernel, SharedKB>(device, dim3(unsigned(tiles * parts)), dim3(S::threads), parts, s, args);
}
// 16-bit rows in tiles of 32 columns where 64 would leave CTAs unused (1024 x 768 dropout
// 3.3 us, by 64 3.6; 16384 x 768 14.6 and 20.4; but 4096 x 8192 32.8 and 27.3); fp32 ones always
// (8192 x 2048 22.8 and 27.2).
inline bool narrow_tiles(int64_t cols, int device) {
    return cols < int64_t(sm_count(device)) * SumVec<64>::ctas * 64 / kSumParts;
}

// 8 elements of a group as raw words; a group that ends behind the tensor's last element
// (`all` of them) by single ones.
template <int XT>
struct RawGroup {
    uint4 u[kWords8<XT>];
    __device__ __forceinline__ void load(const void *x, int64_t g, bool whole, int64_t all) {
        if (whole) {
#pragma unroll
            for (int w = 0; w < kWords8<XT>; ++w)
                u[w] = ld16(static_cast<const char *>(x) + g * (XT == kF32 ? 32 : 16) + 16 * w);
        } else {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = 8 * g + j < all ? load_elem<XT>(x, 8 * g + j) : 0.0f;
            f32_to_raw8<XT>(y, u);
        }
    }
};
// Elements lo .. hi - 1 of a group.
template <int XT>
__device__ __forceinline__ void store_group(void *x, int64_t g, int lo, int hi, const float (&y)[8]) {
    if (hi - lo == 8) return stv<XT>(x, 8 * g, y);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j >= lo && j < hi) store_elem<XT>(x, 8 * g + j, y[j]);
}

}  // namespace amp
