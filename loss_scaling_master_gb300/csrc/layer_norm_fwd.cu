// layer_norm_fwd.cu - layer norm over rows, forward.
//
//   mean = sum x / d;  var = sum (x - mean)^2 / d;  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd w + b, and optionally the 8-bit checkpoint of x
//
// The row sits in registers (layer_norm.cuh), so x is read once although the
// variance is taken about the finished mean (no cancellation for rows far from
// zero): read + write of the row is all the traffic, and memory bounds it.
#include <algorithm>

#include "layer_norm.cuh"

namespace amp {
namespace {

struct NormFwd {
    const void *x, *w, *b;
    void *y;
    float *mean, *rstd;
    uint8_t *q, *s;
    int64_t rows, cols;
    float eps, inv_d;
    int wt, xvec, yvec, wvec, bvec, qvec;
};

// The checkpoint of one group of 8 (n of them in the row); the 4 lanes of a
// block call it together.  c: the group's first column.
__device__ __forceinline__ void keep_group(const NormFwd &P, int64_t r, int64_t c, int n, const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (n <= 0) return;
    const uint32_t e = mx_scale_code<MxE4M3>(m);
    const float f = mx_unscale(e);
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        h[j] = f32x2_to_fp8x2_raw<kE4M3>(__fmul_rn(x[2 * j], f), __fmul_rn(x[2 * j + 1], f));
    uint8_t *q = P.q + r * P.cols + c;
    if (P.qvec) {
        *reinterpret_cast<uint2 *>(q) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) q[j] = uint8_t(h[j / 2] >> (8 * (j & 1)));
    }
    if ((c & 31) == 0) P.s[r * ((P.cols + 31) / 32) + c / 32] = uint8_t(e);
}

template <int XT, int TPR, int NV>
__global__ void __launch_bounds__(norm_cta(TPR)) norm_fwd_kernel(NormFwd P) {
    __shared__ float s1[32], s2[32];
    pdl_wait();
    pdl_trigger();
    constexpr int RPC = norm_cta(TPR) / TPR;
    const int t = threadIdx.x % TPR;
    const int64_t r = int64_t(blockIdx.x) * RPC + threadIdx.x / TPR;
    const bool in = r < P.rows;
    uint4 raw[NV][kWords8<XT>];
    int n[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = 8 * (v * TPR + t);
        n[v] = in ? int(P.cols) - c : 0;
        ld_group<XT>(P.x, r * P.cols + c, n[v], P.xvec, raw[v]);
    }
    float x[NV][8], a[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        raw8_to_f32<XT>(raw[v], x[v]);
        a[0] += ((x[v][0] + x[v][1]) + (x[v][2] + x[v][3])) + ((x[v][4] + x[v][5]) + (x[v][6] + x[v][7]));
    }
    row_sums<TPR>(a, s1);
    const float mean = a[0] * P.inv_d;
    float b[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = j < n[v] ? x[v][j] - mean : 0.0f;
            b[0] = __fmaf_rn(d, d, b[0]);
        }
    row_sums<TPR>(b, s2);
    const float rstd = 1.0f / sqrtf(__fmaf_rn(b[0], P.inv_d, P.eps));
    if (in && t == 0) {
        if (P.mean) P.mean[r] = mean;
        if (P.rstd) P.rstd[r] = rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = 8 * (v * TPR + t);
        if (P.q) keep_group(P, r, c, n[v], x[v]);
        float w[8], o[8];
        ld_param(P.w, P.wt, c, n[v], P.wvec, 1.0f, w);
        ld_param(P.b, P.wt, c, n[v], P.bvec, 0.0f, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __fmaf_rn((x[v][j] - mean) * rstd, w[j], o[j]);
        st_group<XT>(P.y, r * P.cols + c, n[v], P.yvec, o);
    }
}

// Rows past kNormRegCols: one CTA a row, walked three times (the second and
// third reads come from L2).
template <int XT>
__global__ void __launch_bounds__(512) norm_fwd_long(NormFwd P) {
    __shared__ float s1[32], s2[32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = blockIdx.x;
    const int64_t steps = (P.cols + 8 * 512 - 1) / (8 * 512);
    float a[1] = {0.0f}, b[1] = {0.0f}, x[8];
    auto get = [&](int64_t i, int64_t &c) {
        uint4 raw[kWords8<XT>];
        c = 8 * (i * 512 + threadIdx.x);
        const int n = int(min(int64_t(8), P.cols - c));
        ld_group<XT>(P.x, r * P.cols + c, n, P.xvec, raw);
        raw8_to_f32<XT>(raw, x);
        return n;
    };
    int64_t c;
    for (int64_t i = 0; i < steps; ++i) {
        get(i, c);
        a[0] += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
    }
    row_sums<512>(a, s1);
    const float mean = a[0] * P.inv_d;
    for (int64_t i = 0; i < steps; ++i) {
        const int n = get(i, c);
        float q = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = j < n ? x[j] - mean : 0.0f;
            q = __fmaf_rn(d, d, q);
        }
        b[0] += q;
    }
    row_sums<512>(b, s2);
    const float rstd = 1.0f / sqrtf(__fmaf_rn(b[0], P.inv_d, P.eps));
    if (threadIdx.x == 0) {
        if (P.mean) P.mean[r] = mean;
        if (P.rstd) P.rstd[r] = rstd;
    }
    for (int64_t i = 0; i < steps; ++i) {
        const int n = get(i, c);
        if (P.q) keep_group(P, r, c, n, x);
        float w[8], o[8];
        ld_param(P.w, P.wt, c, n, P.wvec, 1.0f, w);
        ld_param(P.b, P.wt, c, n, P.bvec, 0.0f, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __fmaf_rn((x[j] - mean) * rstd, w[j], o[j]);
        st_group<XT>(P.y, r * P.cols + c, n, P.yvec, o);
    }
}

template <int XT>
cudaError_t go(const NormFwd &P, cudaStream_t s) {
    if (P.cols > kNormRegCols)
        return launch_pdl(norm_fwd_long<XT>, dim3((unsigned)P.rows), dim3(512), 0, s, P);
#define F(TPR, NV)                                                                                  \
    return launch_pdl(norm_fwd_kernel<XT, TPR, NV>,                                                 \
                      dim3((unsigned)((P.rows + norm_cta(TPR) / TPR - 1) / (norm_cta(TPR) / TPR))), \
                      dim3(norm_cta(TPR)), 0, s, P)
    AMP_NORM_SHAPE(P.cols, F);
#undef F
}

}  // namespace

cudaError_t launch_norm_fwd(const void *x, int xelem, int64_t rows, int64_t cols, const void *w,
                            const void *b, int welem, float eps, void *y, float *mean, float *rstd,
                            uint8_t *q, uint8_t *sc, cudaStream_t s) {
    NormFwd P{x, w, b, y, mean, rstd, q, sc, rows, cols, eps, float(1.0 / double(cols)), welem, 0, 0, 0, 0, 0};
    const int esz = xelem == kF32 ? 4 : 2, wsz = welem == kF32 ? 4 : 2;
    P.xvec = norm_vec(x, cols, esz);
    P.yvec = norm_vec(y, cols, esz);
    P.wvec = norm_vec(w, cols, wsz);
    P.bvec = norm_vec(b, cols, wsz);
    P.qvec = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    cudaError_t e = xelem == kF32 ? go<kF32>(P, s) : xelem == kF16 ? go<kF16>(P, s) : go<kBF16>(P, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace amp
