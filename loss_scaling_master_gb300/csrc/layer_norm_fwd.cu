// layer_norm_fwd.cu - layer norm over rows, forward.
//
//   mean = sum x / d;  var = sum (x - mean)^2 / d;  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd w + b, and optionally the 8-bit checkpoint of x
//
// The row stays with its CTA (layer_norm.cuh), so x is read once although the
// variance is taken about the finished mean (no cancellation for rows far from
// zero): read + write of the row is all the traffic.  CTAs stay and walk rows;
// a thread's parameters are loaded once, and the next row's loads are issued
// before the present row is worked on.
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
    int wt;
};

// CTAs an SM holds (and the register bound that lets it).  16384 x 4096 bf16
// with a checkpoint: 2 CTAs 64 us, 3 59 us, 4 (spills) 68 us; 16383 x 4095, by
// single elements, 1 CTA of 512 141 us, 2 117 us.
template <int XT, bool VEC>
__host__ __device__ constexpr int fwd_ctas(int tpr, int nv) {
    if (nv == 1) return norm_cta(tpr) > 256 ? 2 : 4;
    return norm_cta(tpr) > 256 ? 1 : VEC && XT != kF32 ? 3 : 2;
}

// 1 / sqrt(var + eps) from the sum of squares, the same at every row length, within 2
// ulp.  (A square root and a division rounded one by one lengthen a row's chain of
// dependent steps: 16384 x 4096 bf16 49.3 -> 50.2 us, with a checkpoint 58.7 -> 60.4,
// 16384 x 2048 28.4 -> 29.9.)
__device__ __forceinline__ float row_rstd(float sumsq, const NormFwd &P) {
    return rsqrtf(__fmaf_rn(sumsq, P.inv_d, P.eps));
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The checkpoint of a thread's group v; the warp calls it together.  q, sc: the
// places of the thread's first element's code and scale byte.
template <int XT, bool VEC, int TPR>
__device__ __forceinline__ void keep8(uint8_t *q, uint8_t *sc, int v, int n, const uint4 (&raw)[kNormWords<XT, VEC>],
                                      const f2 (&x)[4]) {
    float f[8];
    split8(x, f);
    if constexpr (VEC) {
        uint32_t m;
        if constexpr (XT == kF32) {
            m = max(max(max(abs_bits(f[0]), abs_bits(f[1])), max(abs_bits(f[2]), abs_bits(f[3]))),
                    max(max(abs_bits(f[4]), abs_bits(f[5])), max(abs_bits(f[6]), abs_bits(f[7]))));
        } else {  // maxima on packed pairs
            const uint32_t p = absmax2<XT>(absmax2<XT>(raw[0].x, raw[0].y), absmax2<XT>(raw[0].z, raw[0].w));
            m = abs_bits(lowp_to_f32<XT>(absmax2<XT>(p, p >> 16) & 0xFFFFu));
        }
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        if (n <= 0) return;
        const uint32_t e = mx_scale_code<MxE4M3>(m);
        const f2 u = both(mx_unscale(e));
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 z = split(mul2(x[i], u));
            h[i] = f32x2_to_fp8x2_raw<kE4M3>(z.x, z.y);
        }
        *reinterpret_cast<uint2 *>(q + norm_step<true, TPR>(v, 0)) =
            make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        if ((threadIdx.x & 3) == 0) sc[norm_step<true, TPR>(v, 0) / kMxBlock] = uint8_t(e);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t e = mx_scale_code<MxE4M3>(warp_max_u32(abs_bits(f[j])));
            if (j >= n) continue;
            q[norm_step<false, TPR>(v, j)] =
                uint8_t(f32x2_to_fp8x2_raw<kE4M3>(__fmul_rn(f[j], mx_unscale(e)), 0.0f));
            if ((threadIdx.x & 31) == 0) sc[norm_step<false, TPR>(v, j) / kMxBlock] = uint8_t(e);
        }
    }
}

template <int XT, bool VEC, int TPR, int NV>
__global__ void __launch_bounds__(norm_cta(TPR), (fwd_ctas<XT, VEC>(TPR, NV)))
    norm_fwd_kernel(NormFwd P) {
    __shared__ float scratch[2][2][32];
    pdl_wait();
    pdl_trigger();
    constexpr int RPC = norm_rpc(TPR);
    const int t = threadIdx.x % TPR;
    constexpr int esz = XT == kF32 ? 4 : 2;
    const int64_t step = int64_t(gridDim.x) * RPC, kb = (P.cols + kMxBlock - 1) / kMxBlock;
    int64_t r = int64_t(blockIdx.x) * RPC + threadIdx.x / TPR;
    const int c0 = norm_col<VEC, TPR>(0, t, 0);
    const int64_t hop = step * P.cols;
    const char *xp = static_cast<const char *>(P.x) + (r * P.cols + c0) * esz;
    char *yp = static_cast<char *>(P.y) + (r * P.cols + c0) * esz;
    uint8_t *qp = P.q + r * P.cols + c0, *sp = P.s + r * kb + c0 / kMxBlock;
    int n[NV];
    f2 w[NV][4], b[NV][4];
    uint4 nxt[NV][kNormWords<XT, VEC>];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        n[v] = norm_count<VEC, TPR>(v, t, int(P.cols));
        ld8<XT, VEC, TPR>(xp, v, r < P.rows ? n[v] : 0, nxt[v]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        ld_params<VEC, TPR>(P.w, P.wt, v, t, n[v], 1.0f, w[v]);
        ld_params<VEC, TPR>(P.b, P.wt, v, t, n[v], 0.0f, b[v]);
    }
    int buf = 0;
    // every thread of the CTA walks the same number of steps
    for (int64_t base = int64_t(blockIdx.x) * RPC; base < P.rows; base += step, r += step, buf ^= 1) {
        const bool in = r < P.rows;
        uint4 raw[NV][kNormWords<XT, VEC>];
        f2 x[NV][4];
        float a[1];
        f2 s2 = both(0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < kNormWords<XT, VEC>; ++i) raw[v][i] = nxt[v][i];
            widen8<XT, VEC>(raw[v], x[v]);
            s2 = add2(s2, add2(add2(x[v][0], x[v][1]), add2(x[v][2], x[v][3])));
        }
        const bool more = r + step < P.rows;
        xp += hop * esz;
#pragma unroll
        for (int v = 0; v < NV; ++v) ld8<XT, VEC, TPR>(xp, v, more ? n[v] : 0, nxt[v]);
        a[0] = sum2(s2);
        row_sums<TPR>(a, scratch[buf][0]);
        const float mean = a[0] * P.inv_d;
        if (P.q) {
#pragma unroll
            for (int v = 0; v < NV; ++v) keep8<XT, VEC, TPR>(qp, sp, v, in ? n[v] : 0, raw[v], x[v]);
            qp += hop;
            sp += step * kb;
        }
        s2 = both(0.0f);
        const f2 off = both(-mean);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (VEC && n[v] == 0) continue;
            f2 q = both(0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[v][i] = add2(x[v][i], off);
                if (!VEC) {  // elements behind the row's end
                    const float2 p = split(x[v][i]);
                    x[v][i] = make_f2(2 * i < n[v] ? p.x : 0.0f, 2 * i + 1 < n[v] ? p.y : 0.0f);
                }
                q = fma2(x[v][i], x[v][i], q);
            }
            s2 = add2(s2, q);
        }
        a[0] = sum2(s2);
        row_sums<TPR>(a, scratch[buf][1]);
        const float rstd = row_rstd(a[0], P);
        if (in && t == 0) {
            if (P.mean) P.mean[r] = mean;
            if (P.rstd) P.rstd[r] = rstd;
        }
        const f2 rs = both(rstd);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (n[v] == 0) continue;
            f2 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = fma2(mul2(x[v][i], rs), w[v][i], b[v][i]);
            st8<XT, VEC, TPR>(yp, v, in ? n[v] : 0, o);
        }
        yp += hop * esz;
    }
}

// Rows past kNormRegCols: one CTA a row, walked three times, an element a
// thread and step (the second and third reads come from L2): 2048 x 32768 bf16
// 258 us, memory 39.6.
template <int XT>
__global__ void __launch_bounds__(512) norm_fwd_long(NormFwd P) {
    __shared__ float s1[32], s2[32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = blockIdx.x, row = r * P.cols, kb = (P.cols + kMxBlock - 1) / kMxBlock;
    float a[1] = {0.0f};
    for (int64_t c0 = 0; c0 < P.cols; c0 += 4096) {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = c0 + 512 * j + threadIdx.x;
            part += c < P.cols ? load_elem<XT>(P.x, row + c) : 0.0f;
        }
        a[0] += part;
    }
    row_sums<512>(a, s1);
    const float mean = a[0] * P.inv_d;
    a[0] = 0.0f;
    for (int64_t c0 = 0; c0 < P.cols; c0 += 4096) {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = c0 + 512 * j + threadIdx.x;
            const float d = c < P.cols ? load_elem<XT>(P.x, row + c) - mean : 0.0f;
            part = __fmaf_rn(d, d, part);
        }
        a[0] += part;
    }
    row_sums<512>(a, s2);
    const float rstd = row_rstd(a[0], P);
    if (threadIdx.x == 0) {
        if (P.mean) P.mean[r] = mean;
        if (P.rstd) P.rstd[r] = rstd;
    }
    for (int64_t c0 = 0; c0 < P.cols; c0 += 512) {
        const int64_t c = c0 + threadIdx.x;
        const bool in = c < P.cols;
        const float x = in ? load_elem<XT>(P.x, row + c) : 0.0f;
        if (P.q) {
            const uint32_t e = mx_scale_code<MxE4M3>(warp_max_u32(abs_bits(x)));
            if (in) P.q[row + c] = uint8_t(f32x2_to_fp8x2_raw<kE4M3>(__fmul_rn(x, mx_unscale(e)), 0.0f));
            if (in && (c & 31) == 0) P.s[r * kb + c / 32] = uint8_t(e);
        }
        if (in)
            store_elem<XT>(P.y, row + c,
                           __fmaf_rn((x - mean) * rstd, ld_param(P.w, P.wt, c, 1.0f), ld_param(P.b, P.wt, c, 0.0f)));
    }
}

template <int XT, bool VEC>
cudaError_t go(const NormFwd &P, int device, cudaStream_t s) {
    const int64_t sms = sm_count(device);
#define F(TPR, NV)                                                                                       \
    return launch_pdl(norm_fwd_kernel<XT, VEC, TPR, NV>,                                                 \
                      dim3((unsigned)std::min<int64_t>((P.rows + norm_rpc(TPR) - 1) / norm_rpc(TPR),     \
                                                       sms * (fwd_ctas<XT, VEC>(TPR, NV)))), \
                      dim3(norm_cta(TPR)), 0, s, P)
    if constexpr (VEC) AMP_NORM_SHAPE(P.cols, F, 128, 1, 256, 1);
    else AMP_NORM_SHAPE_ODD(P.cols, F);
#undef F
}
template <int XT>
cudaError_t go_x(const NormFwd &P, bool vec, int device, cudaStream_t s) {
    if (P.cols > kNormRegCols)
        return launch_pdl(norm_fwd_long<XT>, dim3((unsigned)P.rows), dim3(512), 0, s, P);
    return vec ? go<XT, true>(P, device, s) : go<XT, false>(P, device, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const void *x, int xelem, int64_t rows, int64_t cols, const void *w,
                            const void *b, int welem, float eps, void *y, float *mean, float *rstd,
                            uint8_t *q, uint8_t *sc, int device, cudaStream_t s) {
    const NormFwd P{x, w, b, y, mean, rstd, q, sc, rows, cols, eps, float(1.0 / double(cols)), welem};
    const int esz = xelem == kF32 ? 4 : 2;
    const bool vec = norm_vec(x, cols, esz) && norm_vec(y, cols, esz) && (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    const cudaError_t e = xelem == kF32   ? go_x<kF32>(P, vec, device, s)
                          : xelem == kF16 ? go_x<kF16>(P, vec, device, s)
                                          : go_x<kBF16>(P, vec, device, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace amp
