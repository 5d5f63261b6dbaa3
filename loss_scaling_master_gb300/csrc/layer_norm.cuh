// layer_norm.cuh - what the forward and the backward layer norm share: how a
// row is spread over threads, its loads and its sums.
//
// A row of up to 16384 elements is held in registers by TPR threads, thread t
// taking the groups of 8 elements t, t + TPR, ..., NV of them (row_shape
// picks the smallest such pair).  Four neighbouring threads hold one block of
// the 8-bit checkpoint.  Longer rows are walked in pieces (the *_long
// kernels).
#pragma once

#include "internal.h"
#include "mx.cuh"
#include "pdl.cuh"

namespace amp {

constexpr int64_t kNormRegCols = 16384;  // the longest row held in registers

// 16-byte access to every group of 8 elements of rows of this length
inline bool norm_vec(const void *p, int64_t cols, int esz) {
    return cols % 8 == 0 && (cols * esz) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

// The group of 8 elements from k, of which n (<= 0: none) are in the row.
template <int XT>
__device__ __forceinline__ void ld_group(const void *x, int64_t k, int n, bool vec,
                                         uint4 (&u)[kWords8<XT>]) {
    constexpr int esz = XT == kF32 ? 4 : 2;
    if (vec) {
#pragma unroll
        for (int j = 0; j < kWords8<XT>; ++j)
            u[j] = n > 0 ? ld16(static_cast<const char *>(x) + k * esz + 16 * j) : make_uint4(0, 0, 0, 0);
    } else {
        load_raw8_tail<XT>(x, k, n, u);
    }
}
template <int XT>
__device__ __forceinline__ void st_group(void *x, int64_t k, int n, bool vec, const float (&y)[8]) {
    constexpr int esz = XT == kF32 ? 4 : 2;
    if (n <= 0) return;
    if (vec) {
        uint4 u[kWords8<XT>];
        f32_to_raw8<XT>(y, u);
#pragma unroll
        for (int j = 0; j < kWords8<XT>; ++j) st16(static_cast<char *>(x) + k * esz + 16 * j, u[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) store_elem<XT>(x, k + j, y[j]);
    }
}

// A parameter vector of its own type (wt: an ElemType); `fill` where it is NULL.
__device__ __forceinline__ void ld_param(const void *w, int wt, int64_t c, int n, bool vec, float fill,
                                         float (&y)[8]) {
    if (w == nullptr || n <= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = fill;
    } else if (wt == kF32) {
        uint4 u[2];
        ld_group<kF32>(w, c, n, vec, u);
        raw8_to_f32<kF32>(u, y);
    } else if (wt == kF16) {
        uint4 u[1];
        ld_group<kF16>(w, c, n, vec, u);
        raw8_to_f32<kF16>(u, y);
    } else {
        uint4 u[1];
        ld_group<kBF16>(w, c, n, vec, u);
        raw8_to_f32<kBF16>(u, y);
    }
}
__device__ __forceinline__ void st_param(void *w, int wt, int64_t c, float v) {
    if (wt == kF32) store_elem<kF32>(w, c, v);
    else if (wt == kF16) store_elem<kF16>(w, c, v);
    else store_elem<kBF16>(w, c, v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The sums of N values over the TPR threads of a row, given to all of them.
// Every thread of the CTA calls it (it synchronises); s: CTA scratch of at
// least N * 32 floats, a different one for calls that follow one another
// without a barrier between.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float *s) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5, first = warp / W * W;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) s[i * 32 + warp] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) t += s[i * 32 + first + w];
            v[i] = t;
        }
    }
}

__host__ __device__ constexpr int norm_cta(int tpr) { return tpr > 256 ? tpr : 256; }

}  // namespace amp

// Calls F<TPR, NV>(...) for the row length: the rule is the smallest number of
// threads that holds the row in two groups each (one for the shortest), four
// for the longest rows, whose CTA could not be larger.
#define AMP_NORM_SHAPE(cols, F)          \
    do {                                 \
        if ((cols) <= 256) { F(32, 1); } \
        else if ((cols) <= 512) { F(32, 2); } \
        else if ((cols) <= 1024) { F(64, 2); } \
        else if ((cols) <= 2048) { F(128, 2); } \
        else if ((cols) <= 4096) { F(256, 2); } \
        else if ((cols) <= 8192) { F(512, 2); } \
        else { F(512, 4); }              \
    } while (0)
