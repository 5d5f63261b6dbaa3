// layer_norm_bwd.cu - gradients of the layer norm.
//
//   xh = (x - mean) rstd, g = dy w
//   dx = rstd (g - sum(g) / d - xh sum(g xh) / d)
//   dw = sum over rows dy xh,  db = sum over rows dy
//
// dy and x (or its 8-bit checkpoint) are read once.  CTAs stay and walk rows
// blockIdx, blockIdx + grid, ..., each thread adding its columns' dy xh and dy
// in registers, so a row costs its own traffic only; the next row's loads are
// issued before the present row is worked on.  At the end a CTA joins its row
// groups' sums in a fixed order and writes one row of partial sums; a second
// kernel adds those rows, again in a fixed order (no atomics, so equal calls
// give equal bits).
#include <algorithm>

#include "layer_norm.cuh"

namespace amp {
namespace {

struct NormBwd {
    const void *dy, *x, *w;
    const uint8_t *q, *s;
    const float *mean, *rstd;
    void *dx;
    float *part;  // [grid][2][cols]: dw then db
    int64_t rows, cols;
    float inv_d;
    int wt, dyvec, xvec, wvec, dxvec, qvec;
};

// x of one group: raw words, or 8 codes and the block's scale byte.
template <int XT, bool CK>
struct Group {
    uint4 dy[kWords8<XT>];
    uint4 x[CK ? 1 : kWords8<XT>];  // CK: codes in x, y; scale byte in z
};

template <int XT, bool CK>
__device__ __forceinline__ void load_pair(const NormBwd &P, int64_t r, int64_t c, int n, Group<XT, CK> &g) {
    const int64_t k = r * P.cols + c;
    ld_group<XT>(P.dy, k, n, P.dyvec, g.dy);
    if constexpr (CK) {
        uint2 u = make_uint2(0, 0);
        uint32_t e = 0;
        if (n > 0) {
            if (P.qvec) {
                u = *reinterpret_cast<const uint2 *>(P.q + k);
            } else {
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n) w[j / 4] |= uint32_t(P.q[k + j]) << (8 * (j & 3));
                u = make_uint2(w[0], w[1]);
            }
            e = P.s[r * ((P.cols + 31) / 32) + c / 32];
        }
        g.x[0] = make_uint4(u.x, u.y, e, 0);
    } else {
        ld_group<XT>(P.x, k, n, P.xvec, g.x);
    }
}
template <int XT, bool CK>
__device__ __forceinline__ void unpack_pair(const Group<XT, CK> &g, float (&dy)[8], float (&x)[8]) {
    raw8_to_f32<XT>(g.dy, dy);
    if constexpr (CK) {
        const float s = mx_scale(g.x[0].z);
        e4m3x4_to_f32x4(g.x[0].x, x);
        e4m3x4_to_f32x4(g.x[0].y, x + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(x[j], s);
    } else {
        raw8_to_f32<XT>(g.x, x);
    }
}

template <int XT, bool CK, int TPR, int NV>
__global__ void __launch_bounds__(norm_cta(TPR)) norm_bwd_kernel(NormBwd P) {
    constexpr int RPC = norm_cta(TPR) / TPR;
    __shared__ float scratch[2][2 * 32];
    extern __shared__ float s_join[];  // RPC > 1: 2 * cols floats
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    float aw[NV][8], ab[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) aw[v][j] = ab[v][j] = 0.0f;
    const int64_t step = int64_t(gridDim.x) * RPC;
    Group<XT, CK> nxt[NV];
    int64_t r = int64_t(blockIdx.x) * RPC + sub;
    int len[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        len[v] = int(P.cols) - 8 * (v * TPR + t);
        load_pair<XT, CK>(P, r, 8 * (v * TPR + t), r < P.rows ? len[v] : 0, nxt[v]);
    }
    float nmean = r < P.rows ? P.mean[r] : 0.0f, nrstd = r < P.rows ? P.rstd[r] : 0.0f;
    int buf = 0;
    // every thread of the CTA walks the same number of steps
    for (int64_t base = int64_t(blockIdx.x) * RPC; base < P.rows; base += step, r += step, buf ^= 1) {
        const bool in = r < P.rows;
        const float mean = nmean, rstd = nrstd;
        float g[NV][8], xh[NV][8], sums[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float w[8];
            ld_param(P.w, P.wt, 8 * (v * TPR + t), len[v], P.wvec, 1.0f, w);
            unpack_pair<XT, CK>(nxt[v], g[v], xh[v]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[v][j] = in && j < len[v] ? (xh[v][j] - mean) * rstd : 0.0f;
                const float dy = g[v][j];
                aw[v][j] = __fmaf_rn(dy, xh[v][j], aw[v][j]);
                ab[v][j] += dy;
                g[v][j] = dy * w[j];
                sums[0] += g[v][j];
                sums[1] = __fmaf_rn(g[v][j], xh[v][j], sums[1]);
            }
        }
        const int64_t rn = r + step;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            load_pair<XT, CK>(P, rn, 8 * (v * TPR + t), rn < P.rows ? len[v] : 0, nxt[v]);
        if (rn < P.rows) {
            nmean = P.mean[rn];
            nrstd = P.rstd[rn];
        }
        row_sums<TPR>(sums, scratch[buf]);
        if (P.dx && in) {
            const float c0 = sums[0] * P.inv_d, c1 = sums[1] * P.inv_d;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = rstd * (g[v][j] - __fmaf_rn(xh[v][j], c1, c0));
                st_group<XT>(P.dx, r * P.cols + 8 * (v * TPR + t), len[v], P.dxvec, o);
            }
        }
    }
    if (!P.part) return;
    float *out = P.part + int64_t(blockIdx.x) * 2 * P.cols;
    if constexpr (RPC > 1) {
        // the row groups add in turn
        const int d = int(P.cols);
        for (int i = 0; i < RPC; ++i) {
            if (sub == i) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (j >= len[v]) continue;
                        const int c = 8 * (v * TPR + t) + j;
                        s_join[c] = (i ? s_join[c] : 0.0f) + aw[v][j];
                        s_join[d + c] = (i ? s_join[d + c] : 0.0f) + ab[v][j];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * d; c += norm_cta(TPR)) out[c] = s_join[c];
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= len[v]) continue;
                const int c = 8 * (v * TPR + t) + j;
                out[c] = aw[v][j];
                out[P.cols + c] = ab[v][j];
            }
    }
}

// Rows past kNormRegCols.  dx: one CTA a row, walked twice.
template <int XT, bool CK>
__global__ void __launch_bounds__(512) norm_bwd_long_dx(NormBwd P) {
    __shared__ float scratch[2 * 32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = blockIdx.x;
    const int64_t steps = (P.cols + 8 * 512 - 1) / (8 * 512);
    const float mean = P.mean[r], rstd = P.rstd[r];
    float sums[2] = {0.0f, 0.0f}, g[8], xh[8];
    auto get = [&](int64_t i, int64_t &c) {
        c = 8 * (i * 512 + threadIdx.x);
        const int n = int(min(int64_t(8), P.cols - c));
        Group<XT, CK> p;
        load_pair<XT, CK>(P, r, c, n, p);
        float w[8];
        ld_param(P.w, P.wt, c, n, P.wvec, 1.0f, w);
        unpack_pair<XT, CK>(p, g, xh);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            xh[j] = j < n ? (xh[j] - mean) * rstd : 0.0f;
            g[j] *= w[j];
        }
        return n;
    };
    int64_t c;
    for (int64_t i = 0; i < steps; ++i) {
        get(i, c);
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a += g[j];
            b = __fmaf_rn(g[j], xh[j], b);
        }
        sums[0] += a;
        sums[1] += b;
    }
    row_sums<512>(sums, scratch);
    const float c0 = sums[0] * P.inv_d, c1 = sums[1] * P.inv_d;
    for (int64_t i = 0; i < steps; ++i) {
        const int n = get(i, c);
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = rstd * (g[j] - __fmaf_rn(xh[j], c1, c0));
        st_group<XT>(P.dx, r * P.cols + c, n, P.dxvec, o);
    }
}
// The parameter sums of long rows: thread = one column, blockIdx.y = a share
// of the rows.
template <int XT, bool CK>
__global__ void __launch_bounds__(kThreads) norm_bwd_long_params(NormBwd P) {
    pdl_wait();
    pdl_trigger();
    const int64_t c = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (c >= P.cols) return;
    float a = 0.0f, b = 0.0f;
    for (int64_t r = blockIdx.y; r < P.rows; r += gridDim.y) {
        const float dy = load_elem<XT>(P.dy, r * P.cols + c);
        float x;
        if constexpr (CK) {
            float v[4];
            e4m3x4_to_f32x4(P.q[r * P.cols + c], v);
            x = __fmul_rn(v[0], mx_scale(P.s[r * ((P.cols + 31) / 32) + c / 32]));
        } else {
            x = load_elem<XT>(P.x, r * P.cols + c);
        }
        a = __fmaf_rn(dy, (x - P.mean[r]) * P.rstd[r], a);
        b += dy;
    }
    float *out = P.part + int64_t(blockIdx.y) * 2 * P.cols;
    out[c] = a;
    out[P.cols + c] = b;
}

// Adds the partial rows.  A CTA takes 32 columns; warp w the rows w, w + 8, ...
struct NormJoin {
    const float *part;
    int64_t parts, cols;
    void *dw, *db;
    int wt;
};
__global__ void __launch_bounds__(kThreads) norm_join_kernel(NormJoin P) {
    __shared__ float s[2][kThreads / 32][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float a = 0.0f, b = 0.0f;
    if (c < P.cols) {
#pragma unroll 4
        for (int64_t p = warp; p < P.parts; p += kThreads / 32) {
            a += P.part[p * 2 * P.cols + c];
            b += P.part[p * 2 * P.cols + P.cols + c];
        }
    }
    s[0][warp][lane] = a;
    s[1][warp][lane] = b;
    __syncthreads();
    if (warp < 2 && c < P.cols) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) t += s[warp][w][lane];
        void *out = warp ? P.db : P.dw;
        if (out) st_param(out, P.wt, c, t);
    }
}

template <int XT, bool CK>
cudaError_t go(NormBwd &P, int64_t parts, cudaStream_t s) {
    if (P.cols > kNormRegCols) {
        // the parameters first: dx may overwrite dy
        if (P.part) {
            cudaError_t e = launch_pdl(norm_bwd_long_params<XT, CK>,
                                       dim3((unsigned)((P.cols + kThreads - 1) / kThreads), (unsigned)parts),
                                       dim3(kThreads), 0, s, P);
            if (e != cudaSuccess) return e;
        }
        if (!P.dx || P.rows == 0) return cudaSuccess;
        return launch_pdl(norm_bwd_long_dx<XT, CK>, dim3((unsigned)P.rows), dim3(512), 0, s, P);
    }
#define F(TPR, NV)                                                                              \
    return launch_pdl(norm_bwd_kernel<XT, CK, TPR, NV>, dim3((unsigned)parts), dim3(norm_cta(TPR)), \
                      norm_cta(TPR) > TPR ? size_t(P.cols) * 8 : 0, s, P)
    AMP_NORM_SHAPE(P.cols, F);
#undef F
}

}  // namespace

// Rows of partial sums: as many CTAs as the device holds at once (2 of 256
// threads an SM, 1 of 512), at most one for each group of rows.
int64_t norm_parts(int64_t rows, int64_t cols, int device) {
    const int64_t sms = sm_count(device);
    if (cols > kNormRegCols) return std::max<int64_t>(1, std::min<int64_t>(rows, 32));
#define F(TPR, NV)                                                    \
    return std::max<int64_t>(                                         \
        1, std::min<int64_t>((rows + norm_cta(TPR) / TPR - 1) / (norm_cta(TPR) / TPR), \
                             norm_cta(TPR) > 256 ? sms : 2 * sms))
    AMP_NORM_SHAPE(cols, F);
#undef F
}

cudaError_t launch_norm_bwd(const void *dy, const void *x, int elem, const uint8_t *q, const uint8_t *sc,
                            int64_t rows, int64_t cols, const void *w, int welem, const float *mean,
                            const float *rstd, void *dx, void *dw, void *db, float *part, int device,
                            cudaStream_t s) {
    NormBwd P{dy, x, w, q, sc, mean, rstd, dx, dw || db ? part : nullptr, rows, cols,
              float(1.0 / double(cols)), welem, 0, 0, 0, 0, 0};
    const int esz = elem == kF32 ? 4 : 2, wsz = welem == kF32 ? 4 : 2;
    P.dyvec = norm_vec(dy, cols, esz);
    P.xvec = norm_vec(x, cols, esz);
    P.wvec = norm_vec(w, cols, wsz);
    P.dxvec = norm_vec(dx, cols, esz);
    P.qvec = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    const int64_t parts = norm_parts(rows, cols, device);
    cudaError_t e = cudaSuccess;
    if (q)
        e = elem == kF32   ? go<kF32, true>(P, parts, s)
            : elem == kF16 ? go<kF16, true>(P, parts, s)
                           : go<kBF16, true>(P, parts, s);
    else
        e = elem == kF32   ? go<kF32, false>(P, parts, s)
            : elem == kF16 ? go<kF16, false>(P, parts, s)
                           : go<kBF16, false>(P, parts, s);
    if (e == cudaSuccess && P.part) {
        const NormJoin J{part, parts, cols, dw, db, welem};
        e = launch_pdl(norm_join_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(kThreads), 0, s, J);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace amp
