// layer_norm.cuh - what the forward and the backward layer norm share: how a
// row is spread over threads, loads and stores, packed fp32 arithmetic, sums.
//
// A row of up to 16384 elements is read once and kept by TPR threads, NV groups of
// 8 elements each (AMP_NORM_SHAPE picks the pair): in registers up to 8192 elements,
// above that partly in local memory (512 threads have 128 registers each, and four
// groups do not fit: 360 to 640 bytes of spills a thread forward, 624 to 1396
// backward, and 8 to 196 in some of the backward's shapes below).  Where rows are whole,
// 16-byte aligned groups of 8 (VEC), thread t takes the groups t, t + TPR, ...,
// one 16-byte access each of a 16-bit tensor, and 4 neighbouring threads hold
// one block of the 8-bit checkpoint.  Otherwise a thread takes single elements
// TPR apart, so that a warp's accesses stay side by side whatever the row
// length; a warp then holds one block at a time.  Longer rows are walked in
// pieces (the *_long kernels).
//
// The arithmetic runs two elements an instruction (fp32x2), each rounded as a
// scalar one: what bounds these kernels besides memory is instruction issue
// (34 instructions an element in scalar form with per-element guards took 84 us
// for the forward pass of 16384 x 4096 bf16 with a checkpoint, 50 us of memory).
#pragma once

#include "f32x2.cuh"
#include "internal.h"
#include "mx.cuh"
#include "pdl.cuh"

namespace amp {

constexpr int64_t kNormRegCols = 16384;  // the longest row that a CTA keeps

// 16-byte access to every group of 8 elements of rows of this length
inline bool norm_vec(const void *p, int64_t cols, int esz) {
    return cols % 8 == 0 && (cols * esz) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

// ---- a thread's 8 elements: group v of thread t ------------------------------
// Element j's column, and how many of the 8 are in the row (VEC: all or none).
template <bool VEC, int TPR>
__device__ __forceinline__ int norm_col(int v, int t, int j) {
    return VEC ? 8 * (v * TPR + t) + j : (8 * v + j) * TPR + t;
}
template <bool VEC, int TPR>
__device__ __forceinline__ int norm_count(int v, int t, int cols) {
    if (VEC) return 8 * (v * TPR + t) < cols ? 8 : 0;
    const int left = cols - 8 * v * TPR - t;  // of elements TPR apart
    return left <= 0 ? 0 : min(8, (left + TPR - 1) / TPR);
}

// Elements from a thread's first element of a row to element j of its group v.
// (The kernels keep a pointer to that first element and move it on by a row:
// with an index worked out for every access, address arithmetic was a quarter
// of the instructions.)
template <bool VEC, int TPR>
__host__ __device__ constexpr int norm_step(int v, int j) {
    return VEC ? 8 * v * TPR + j : (8 * v + j) * TPR;
}

// The 8 elements of group v behind x as loaded (VEC: raw words; else one element
// a word, so that nothing waits for the loads before the row's turn); n of them
// are in the row, the rest are zeros.
template <int XT, bool VEC>
constexpr int kNormWords = VEC ? kWords8<XT> : 2;

template <int XT, bool VEC, int TPR>
__device__ __forceinline__ void ld8(const void *x, int v, int n, uint4 (&u)[kNormWords<XT, VEC>]) {
    constexpr int esz = XT == kF32 ? 4 : 2;
    const int k = norm_step<VEC, TPR>(v, 0);
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kWords8<XT>; ++i)
            u[i] = n > 0 ? ld16(static_cast<const char *>(x) + k * esz + 16 * i) : make_uint4(0, 0, 0, 0);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (XT == kF32) w[j] = j < n ? static_cast<const uint32_t *>(x)[k + j * TPR] : 0u;
            else w[j] = j < n ? static_cast<const uint16_t *>(x)[k + j * TPR] : 0u;
        }
        u[0] = make_uint4(w[0], w[1], w[2], w[3]);
        u[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
template <int XT>
__device__ __forceinline__ void to_f32(const uint4 (&u)[kWords8<XT>], f2 (&y)[4]) {
    float f[8];
    raw8_to_f32<XT>(u, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = make_f2(f[2 * i], f[2 * i + 1]);
}
// What ld8 loaded.
template <int XT, bool VEC>
__device__ __forceinline__ void widen8(const uint4 (&u)[kNormWords<XT, VEC>], f2 (&y)[4]) {
    if constexpr (VEC) {
        to_f32<XT>(u, y);
    } else {
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (XT == kF32) f[j] = __uint_as_float(w[j]);
            else f[j] = lowp_to_f32<XT>(w[j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = make_f2(f[2 * i], f[2 * i + 1]);
    }
}
__device__ __forceinline__ void split8(const f2 (&y)[4], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 s = split(y[i]);
        f[2 * i] = s.x;
        f[2 * i + 1] = s.y;
    }
}
template <int XT, bool VEC, int TPR>
__device__ __forceinline__ void st8(void *x, int v, int n, const f2 (&y)[4]) {
    constexpr int esz = XT == kF32 ? 4 : 2;
    const int k = norm_step<VEC, TPR>(v, 0);
    float f[8];
    split8(y, f);
    if constexpr (VEC) {
        if (n <= 0) return;
        uint4 u[kWords8<XT>];
        f32_to_raw8<XT>(f, u);
#pragma unroll
        for (int i = 0; i < kWords8<XT>; ++i) st16(static_cast<char *>(x) + k * esz + 16 * i, u[i]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) store_elem<XT>(x, k + j * TPR, f[j]);
    }
}

// A parameter vector (wt: its ElemType); `fill` where it is NULL.
__device__ __forceinline__ float ld_param(const void *w, int wt, int64_t c, float fill) {
    if (w == nullptr) return fill;
    return wt == kF32 ? load_elem<kF32>(w, c) : wt == kF16 ? load_elem<kF16>(w, c) : load_elem<kBF16>(w, c);
}
template <bool VEC, int TPR>
__device__ __forceinline__ void ld_params(const void *w, int wt, int v, int t, int n, float fill, f2 (&y)[4]) {
    float f[8];
    // (by single elements, 1024 x 768 with fp32 parameters 3.5 us instead of 2.6)
    if (VEC && w != nullptr && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {
        const int c = norm_col<true, TPR>(v, t, 0);
        uint4 u[2] = {};
        if (n > 0) {
            u[0] = ld16(static_cast<const char *>(w) + c * (wt == kF32 ? 4 : 2));
            if (wt == kF32) u[1] = ld16(static_cast<const char *>(w) + c * 4 + 16);
        }
        if (wt == kF32) raw8_to_f32<kF32>(u, f);
        else if (wt == kF16) raw8_to_f32<kF16>(u, f);
        else raw8_to_f32<kBF16>(u, f);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = j < n ? ld_param(w, wt, norm_col<VEC, TPR>(v, t, j), fill) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = make_f2(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void st_param(void *w, int wt, int64_t c, float v) {
    if (wt == kF32) store_elem<kF32>(w, c, v);
    else if (wt == kF16) store_elem<kF16>(w, c, v);
    else store_elem<kBF16>(w, c, v);
}

// The sums of one or two values over the TPR threads of a row, given to all of
// them.  Every thread of the CTA calls it (it synchronises); s: CTA scratch of
// N * 32 floats, another one for the next call.  Two values share the steps:
// after the first, each half of a warp carries one of them.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float *s) {
    static_assert(N == 1 || N == 2, "values");
    constexpr uint32_t all = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float a = v[0];
    if constexpr (N == 2) {
        const bool hi = lane & 16;
        a = (hi ? v[1] : v[0]) + __shfl_xor_sync(all, hi ? v[0] : v[1], 16);
    } else {
        a += __shfl_xor_sync(all, a, 16);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(all, a, o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        if ((lane & 15) == 0 && (N == 2 || lane == 0)) s[(lane >> 4) * 32 + warp] = a;
        __syncthreads();
        // lane i of each half takes warp i's part of the half's value
        const float p = s[(N == 2 ? lane & 16 : 0) * 2 + warp / W * W + (lane & (W - 1))];
        a = p;
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) a += __shfl_xor_sync(all, a, o);
    }
    v[0] = N == 2 || TPR == 32 ? __shfl_sync(all, a, 0) : a;
    if constexpr (N == 2) v[1] = __shfl_sync(all, a, 16);
}

__host__ __device__ constexpr int norm_cta(int tpr) { return tpr > 256 ? tpr : 256; }
__host__ __device__ constexpr int norm_rpc(int tpr) { return norm_cta(tpr) / tpr; }  // rows a CTA holds

}  // namespace amp

// Runs F(TPR, NV) for the row length: the smallest CTA that holds the row in two
// groups a thread, and four for the longest rows, which spill (4096 x 16384 bf16
// forward 61 us, memory 39.6, backward 121 of 59.3; a row over a cluster's CTAs
// would not, and is not built).
// T1, V1 and T2, V2: the shapes up to 1024 and 2048 elements.  Forward 128 x 1 (8
// rows of 768 1.8 us, with a warp a row, whose code is four times as long and run
// once, over 3 us; 8192 x 768 the same either way) and 256 x 1 (16384 x 2048 with a
// checkpoint 33.3 us, 128 x 2 40.5 with spills, 100 x 2048 2.0 and 2.7 us); backward
// 64 x 2 (8 x 768 4.3 us, 16384 x 1024 25.6, a warp a row 5.5 and 26.6, 128 x 1 3.6
// and 28.5) and 128 x 2.
#define AMP_NORM_SHAPE(cols, F, T1, V1, T2, V2) \
    do {                                        \
        if ((cols) <= 256) { F(32, 1); }        \
        else if ((cols) <= 1024) { F(T1, V1); } \
        else if ((cols) <= 2048) { F(T2, V2); } \
        else if ((cols) <= 4096) { F(256, 2); } \
        else if ((cols) <= 8192) { F(512, 2); } \
        else { F(512, 4); }                     \
    } while (0)
// Rows taken by single elements, whose loads each hold a register until their
// turn: one group a thread as long as the CTA can grow.
#define AMP_NORM_SHAPE_ODD(cols, F)             \
    do {                                        \
        if ((cols) <= 256) { F(32, 1); }        \
        else if ((cols) <= 1024) { F(128, 1); } \
        else if ((cols) <= 2048) { F(256, 1); } \
        else if ((cols) <= 4096) { F(512, 1); } \
        else if ((cols) <= 8192) { F(512, 2); } \
        else { F(512, 4); }                     \
    } while (0)
