// column_sums.cuh - sums over the rows of a matrix, for the gradient of a bias: what
// its kernels share.
//
// A CTA takes 64 columns of a share of the rows, the CTAs of a cluster the shares of
// the same columns; each adds its rows in registers, then its row groups in shared
// memory, and the cluster's CTAs add one another's sums from there, each a part of
// the columns.  The order of every sum depends on the shape and on whether rows are
// taken by 16 bytes (no atomics, so equal calls give equal bits), and nothing goes through global memory or a second
// launch.
#pragma once

#include <algorithm>

#include "mx.cuh"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace amp {

constexpr int kSumThreads = 256, kSumCols = 64, kSumCtas = 4;  // CTAs an SM holds
// Threads beside one another on a row and row groups: 8 columns a thread, or one.
template <bool VEC>
struct SumShape {
    static constexpr int across = VEC ? kSumCols / 8 : kSumCols, groups = kSumThreads / across;
};

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// This CTA's columns and rows.
struct SumShare {
    uint32_t rank, parts;
    int64_t col0, row0, row1;
    __device__ __forceinline__ explicit SumShare(int64_t rows) {
        parts = cluster_size();
        rank = parts > 1 ? cluster_rank() : 0;
        col0 = int64_t(blockIdx.x / parts) * kSumCols;
        row0 = rows * rank / parts;
        row1 = rows * (rank + 1) / parts;
    }
};

// Adds up all threads' a[] (VEC: of the columns 8 x, ...; else of column x, x the
// thread's place on the row) and stores the columns' sums.  Every thread of every CTA
// of the cluster calls it once.
template <bool VEC>
__device__ __forceinline__ void sum_join(const SumShare &at, int64_t cols, const float (&a)[VEC ? 8 : 1], void *out,
                                         int otype) {
    constexpr int LINES = VEC ? kSumThreads / 32 : SumShape<VEC>::groups;
    __shared__ __align__(16) float s_line[LINES][kSumCols];
    __shared__ __align__(16) float s_part[kSumCols];
    if constexpr (VEC) {
        // the 4 row groups of a warp
        float b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            b[j] = a[j] + __shfl_xor_sync(0xFFFFFFFFu, a[j], 8);
            b[j] += __shfl_xor_sync(0xFFFFFFFFu, b[j], 16);
        }
        if ((threadIdx.x & 31) < 8) {
            float4 *to = reinterpret_cast<float4 *>(&s_line[threadIdx.x >> 5][8 * (threadIdx.x & 7)]);
            to[0] = make_float4(b[0], b[1], b[2], b[3]);
            to[1] = make_float4(b[4], b[5], b[6], b[7]);
        }
    } else {
        s_line[threadIdx.x / kSumCols][threadIdx.x % kSumCols] = a[0];
    }
    __syncthreads();
    if (threadIdx.x < kSumCols) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < LINES; ++i) t += s_line[i][threadIdx.x];
        s_part[threadIdx.x] = t;
    }
    __syncwarp();
    if (at.parts > 1) cluster_sync();  // every CTA's sums are written
    const int mine = (kSumCols + int(at.parts) - 1) / int(at.parts), c = int(at.rank) * mine + int(threadIdx.x);
    if (threadIdx.x < unsigned(mine) && c < kSumCols && at.col0 + c < cols) {
        float t = s_part[c];
        if (at.parts > 1) {
            t = 0.0f;
            for (uint32_t q = 0; q < at.parts; ++q) t += __uint_as_float(cluster_ld(cluster_addr(&s_part[c], q)));
        }
        if (otype == kF32) store_elem<kF32>(out, at.col0 + c, t);
        else if (otype == kF16) store_elem<kF16>(out, at.col0 + c, t);
        else store_elem<kBF16>(out, at.col0 + c, t);
    }
    __syncwarp();
    if (at.parts > 1) cluster_sync();  // nobody leaves while its shared memory is read
}

// Shares of the rows, at most 8 of at least a row a group: as many as make the rounds
// of CTAs that the GPU holds at once shortest.
inline int sum_parts(int64_t rows, int64_t cols, int groups, int sms) {
    const int64_t tiles = (cols + kSumCols - 1) / kSumCols, room = int64_t(sms) * kSumCtas;
    int parts = 1;
    double least = 0.0;
    for (int p = 1; p <= 8 && (p == 1 || rows > int64_t(groups) * (p - 1)); ++p) {
        const double t = double((tiles * p + room - 1) / room) / p;
        if (p == 1 || t < least) {
            least = t;
            parts = p;
        }
    }
    return parts;
}
template <class K, class A>
cudaError_t launch_sums(K kernel, int64_t rows, int64_t cols, int groups, int sms, cudaStream_t s, const A &args) {
    const int parts = sum_parts(rows, cols, groups, sms);
    const int64_t tiles = (cols + kSumCols - 1) / kSumCols;
    return launch_pdl_cluster(kernel, dim3(unsigned(tiles * parts)), dim3(kSumThreads), 0, parts, s, args);
}

}  // namespace amp
