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
//
// 16384 x 4096 bf16 from the checkpoint: 75 us with the join's 6, memory 50 us.
// What bounds it is the latency of a row's phases (sums, barrier, sums) at 2 CTAs
// an SM, which the column sums' registers allow.
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
    int wt;
};

// CTAs of the backward kernel an SM holds: 2 of 256 threads, 1 of 512.
__host__ __device__ constexpr int bwd_ctas(int tpr, int nv) { return norm_cta(tpr) == 256 && nv <= 2 ? 2 : 1; }

// A thread's 8 elements of dy and of x as loaded, or of x's codes with their
// scale bytes (VEC: 8 codes in x, y and one byte in z; else one a word).
template <int XT, bool CK, bool VEC>
struct Group {
    uint4 dy[kNormWords<XT, VEC>];
    uint4 x[!CK ? kNormWords<XT, VEC> : VEC ? 1 : 2];
    uint4 s[CK && !VEC ? 2 : 1];
};

// dy, x, q, s: the places of the thread's first element.
template <int XT, bool CK, bool VEC, int TPR>
__device__ __forceinline__ void load_pair(const char *dy, const char *x, const uint8_t *q, const uint8_t *s, int v,
                                          int n, Group<XT, CK, VEC> &g) {
    ld8<XT, VEC, TPR>(dy, v, n, g.dy);
    if constexpr (!CK) {
        ld8<XT, VEC, TPR>(x, v, n, g.x);
    } else if constexpr (VEC) {
        uint2 u = make_uint2(0, 0);
        uint32_t e = 0;
        if (n > 0) {
            u = *reinterpret_cast<const uint2 *>(q + norm_step<true, TPR>(v, 0));
            e = s[norm_step<true, TPR>(v, 0) / kMxBlock];
        }
        g.x[0] = make_uint4(u.x, u.y, e, 0);
    } else {
        uint32_t w[8], e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = norm_step<false, TPR>(v, j);
            w[j] = j < n ? q[k] : 0u;
            e[j] = j < n ? s[k / kMxBlock] : 0u;
        }
        g.x[0] = make_uint4(w[0], w[1], w[2], w[3]);
        g.x[1] = make_uint4(w[4], w[5], w[6], w[7]);
        g.s[0] = make_uint4(e[0], e[1], e[2], e[3]);
        g.s[1] = make_uint4(e[4], e[5], e[6], e[7]);
    }
}
// dy and x - mean (a code times its power of two is exact, so one fused
// multiply-add rounds as the subtraction does).
template <int XT, bool CK, bool VEC>
__device__ __forceinline__ void unpack_pair(const Group<XT, CK, VEC> &g, f2 off, f2 (&dy)[4], f2 (&x)[4]) {
    widen8<XT, VEC>(g.dy, dy);
    if constexpr (!CK) {
        widen8<XT, VEC>(g.x, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = add2(x[i], off);
    } else if constexpr (VEC) {
        float f[8];
        e4m3x4_to_f32x4(g.x[0].x, f);
        e4m3x4_to_f32x4(g.x[0].y, f + 4);
        const f2 s = both(mx_scale(g.x[0].z));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fma2(make_f2(f[2 * i], f[2 * i + 1]), s, off);
    } else {
        const uint32_t w[8] = {g.x[0].x, g.x[0].y, g.x[0].z, g.x[0].w, g.x[1].x, g.x[1].y, g.x[1].z, g.x[1].w};
        const uint32_t e[8] = {g.s[0].x, g.s[0].y, g.s[0].z, g.s[0].w, g.s[1].x, g.s[1].y, g.s[1].z, g.s[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[4];
            e4m3x4_to_f32x4(w[2 * i] | (w[2 * i + 1] << 8), f);
            x[i] = fma2(make_f2(f[0], f[1]), make_f2(mx_scale(e[2 * i]), mx_scale(e[2 * i + 1])), off);
        }
    }
}

template <int XT, bool CK, bool VEC, int TPR, int NV>
__global__ void __launch_bounds__(norm_cta(TPR), bwd_ctas(TPR, NV)) norm_bwd_kernel(NormBwd P) {
    constexpr int RPC = norm_rpc(TPR);
    constexpr bool HOLD = TPR < 512 || NV < 4;  // weights in registers
    __shared__ float scratch[2][2 * 32];
    extern __shared__ __align__(16) float s_join[];  // RPC > 1: RPC * cols floats
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    f2 aw[NV][4], ab[NV][4], w[HOLD ? NV : 1][4];
    constexpr int esz = XT == kF32 ? 4 : 2;
    const int64_t step = int64_t(gridDim.x) * RPC, hop = step * P.cols, kb = (P.cols + kMxBlock - 1) / kMxBlock;
    int64_t r = int64_t(blockIdx.x) * RPC + sub;
    const int c0 = norm_col<VEC, TPR>(0, t, 0);
    const int64_t k0 = r * P.cols + c0;
    const char *dyp = static_cast<const char *>(P.dy) + k0 * esz, *xp = static_cast<const char *>(P.x) + k0 * esz;
    const uint8_t *qp = P.q + k0, *sp = P.s + r * kb + c0 / kMxBlock;
    char *dxp = static_cast<char *>(P.dx) + k0 * esz;
    int len[NV];
    Group<XT, CK, VEC> nxt[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        len[v] = norm_count<VEC, TPR>(v, t, int(P.cols));
        load_pair<XT, CK, VEC, TPR>(dyp, xp, qp, sp, v, r < P.rows ? len[v] : 0, nxt[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) aw[v][i] = ab[v][i] = both(0.0f);
        if (HOLD) ld_params<VEC, TPR>(P.w, P.wt, v, t, len[v], 1.0f, w[HOLD ? v : 0]);
    }
    float nmean = r < P.rows ? P.mean[r] : 0.0f, nrstd = r < P.rows ? P.rstd[r] : 0.0f;
    int buf = 0;
    // every thread of the CTA walks the same number of steps
    for (int64_t base = int64_t(blockIdx.x) * RPC; base < P.rows; base += step, r += step, buf ^= 1) {
        const bool in = r < P.rows;
        const float mean = in ? nmean : 0.0f, rstd = in ? nrstd : 0.0f;
        const f2 off = both(-mean), rs = both(rstd);
        f2 g[NV][4], xh[NV][4], s0 = both(0.0f), s1 = both(0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!HOLD) ld_params<VEC, TPR>(P.w, P.wt, v, t, len[v], 1.0f, w[0]);
            if (len[v] == 0) continue;
            // elements behind the row's end have dy = w = 0 and a finite xh
            // (with the row's own mean and rstd), a row behind the last one
            // has zeros throughout: neither changes a sum
            unpack_pair<XT, CK, VEC>(nxt[v], off, g[v], xh[v]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xh[v][i] = mul2(xh[v][i], rs);
                aw[v][i] = fma2(g[v][i], xh[v][i], aw[v][i]);
                ab[v][i] = add2(ab[v][i], g[v][i]);
                g[v][i] = mul2(g[v][i], w[HOLD ? v : 0][i]);
                s0 = add2(s0, g[v][i]);
                s1 = fma2(g[v][i], xh[v][i], s1);
            }
        }
        const bool more = r + step < P.rows;
        dyp += hop * esz;
        xp += hop * esz;
        qp += hop;
        sp += step * kb;
#pragma unroll
        for (int v = 0; v < NV; ++v) load_pair<XT, CK, VEC, TPR>(dyp, xp, qp, sp, v, more ? len[v] : 0, nxt[v]);
        if (more) {
            nmean = P.mean[r + step];
            nrstd = P.rstd[r + step];
        }
        float sums[2] = {sum2(s0), sum2(s1)};
        row_sums<TPR>(sums, scratch[buf]);
        if (P.dx && in) {
            const f2 c0 = both(-sums[0] * P.inv_d * rstd), c1 = both(-sums[1] * P.inv_d * rstd);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (len[v] == 0) continue;
                f2 o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = fma2(g[v][i], rs, fma2(xh[v][i], c1, c0));
                st8<XT, VEC, TPR>(dxp, v, len[v], o);
            }
        }
        dxp += hop * esz;
    }
    if (!P.part) return;
    float *out = P.part + int64_t(blockIdx.x) * 2 * P.cols;
    const int d = int(P.cols);
    if constexpr (RPC > 1) {
        // every row group leaves its sums, then a thread adds a column's
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float a[8];
                split8(k ? ab[v] : aw[v], a);
                float *to = s_join + sub * d + norm_col<VEC, TPR>(v, t, 0);
                if constexpr (VEC) {
                    if (len[v] == 0) continue;
                    reinterpret_cast<float4 *>(to)[0] = make_float4(a[0], a[1], a[2], a[3]);
                    reinterpret_cast<float4 *>(to)[1] = make_float4(a[4], a[5], a[6], a[7]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < len[v]) to[j * TPR] = a[j];
                }
            }
            __syncthreads();
            for (int c = threadIdx.x; c < d; c += norm_cta(TPR)) {
                float a = 0.0f;
#pragma unroll
                for (int i = 0; i < RPC; ++i) a += s_join[i * d + c];
                out[k * d + c] = a;
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float a[8], b[8];
            split8(aw[v], a);
            split8(ab[v], b);
            const int c = norm_col<VEC, TPR>(v, t, 0);
            if constexpr (VEC) {
                // (by single elements, 32 bytes apart over a warp: 128 x 4096 13.9 us
                // instead of 7.4, 16384 x 4096 82 instead of 75)
                if (len[v] == 0) continue;
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    *reinterpret_cast<float4 *>(out + c + j) = make_float4(a[j], a[j + 1], a[j + 2], a[j + 3]);
                    *reinterpret_cast<float4 *>(out + d + c + j) = make_float4(b[j], b[j + 1], b[j + 2], b[j + 3]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (j >= len[v]) continue;
                    out[c + j * TPR] = a[j];
                    out[d + c + j * TPR] = b[j];
                }
            }
        }
    }
}

// Rows past kNormRegCols, an element a thread and step: 2048 x 32768 bf16 295 us,
// memory 59.3.
template <int XT, bool CK>
__device__ __forceinline__ float long_x(const NormBwd &P, int64_t r, int64_t c) {
    if constexpr (CK) {
        float v[4];
        e4m3x4_to_f32x4(P.q[r * P.cols + c], v);
        return __fmul_rn(v[0], mx_scale(P.s[r * ((P.cols + kMxBlock - 1) / kMxBlock) + c / kMxBlock]));
    } else {
        return load_elem<XT>(P.x, r * P.cols + c);
    }
}
// dx: one CTA a row, walked twice.
template <int XT, bool CK>
__global__ void __launch_bounds__(512) norm_bwd_long_dx(NormBwd P) {
    __shared__ float scratch[2 * 32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = blockIdx.x;
    const float mean = P.mean[r], rstd = P.rstd[r];
    float sums[2] = {0.0f, 0.0f};
    for (int64_t c0 = 0; c0 < P.cols; c0 += 4096) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = c0 + 512 * j + threadIdx.x;
            if (c < P.cols) {
                const float g = load_elem<XT>(P.dy, r * P.cols + c) * ld_param(P.w, P.wt, c, 1.0f);
                a += g;
                b = __fmaf_rn(g, (long_x<XT, CK>(P, r, c) - mean) * rstd, b);
            }
        }
        sums[0] += a;
        sums[1] += b;
    }
    row_sums<512>(sums, scratch);
    const float c0 = sums[0] * P.inv_d, c1 = sums[1] * P.inv_d;
    for (int64_t c = threadIdx.x; c < P.cols; c += 512) {
        const float g = load_elem<XT>(P.dy, r * P.cols + c) * ld_param(P.w, P.wt, c, 1.0f);
        const float xh = (long_x<XT, CK>(P, r, c) - mean) * rstd;
        store_elem<XT>(P.dx, r * P.cols + c, rstd * (g - __fmaf_rn(xh, c1, c0)));
    }
}
// The parameter sums: thread = one column, blockIdx.y = a share of the rows.
template <int XT, bool CK>
__global__ void __launch_bounds__(kThreads) norm_bwd_long_params(NormBwd P) {
    pdl_wait();
    pdl_trigger();
    const int64_t c = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (c >= P.cols) return;
    float a = 0.0f, b = 0.0f;
    for (int64_t r = blockIdx.y; r < P.rows; r += gridDim.y) {
        const float dy = load_elem<XT>(P.dy, r * P.cols + c);
        a = __fmaf_rn(dy, (long_x<XT, CK>(P, r, c) - P.mean[r]) * P.rstd[r], a);
        b += dy;
    }
    float *out = P.part + int64_t(blockIdx.y) * 2 * P.cols;
    out[c] = a;
    out[P.cols + c] = b;
}

// Adds the partial rows.  A CTA takes 32 of the 2 cols columns, warp w the rows
// w, w + warps, ...: the loads of a warp are independent, so a column costs a few
// load latencies.  16 warps up to 160 rows (32 x 4096 with its gradients 5.0 us, by 32
// warps 6.3; 4096 x 8192 42 and 44 us), 32 above (1024 x 768 6.3 us, by 16 6.7).
struct NormJoin {
    const float *part;
    int64_t parts, cols;
    void *dw, *db;
    int wt;
};
template <int THREADS>
__global__ void __launch_bounds__(THREADS) norm_join_kernel(NormJoin P) {
    __shared__ float s[THREADS / 32][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float a = 0.0f;
    if (c < 2 * P.cols) {
#pragma unroll 8
        for (int64_t p = warp; p < P.parts; p += THREADS / 32) a += P.part[p * 2 * P.cols + c];
    }
    s[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && c < 2 * P.cols) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) t += s[w][lane];
        void *out = c < P.cols ? P.dw : P.db;
        if (out) st_param(out, P.wt, c < P.cols ? c : c - P.cols, t);
    }
}

// CTAs of the backward pass, and so rows of partial sums: as many as the device
// holds at once, at most one for each group of rows.
int64_t norm_grid(int64_t rows, int64_t cols, bool vec, int device) {
    if (cols > kNormRegCols) return std::max<int64_t>(1, std::min<int64_t>(rows, 32));
    const int64_t sms = sm_count(device);
#define F(TPR, NV)                                                                             \
    return std::max<int64_t>(1, std::min<int64_t>((rows + norm_rpc(TPR) - 1) / norm_rpc(TPR),  \
                                                  sms * bwd_ctas(TPR, NV)))
    if (vec) AMP_NORM_SHAPE(cols, F, 64, 2, 128, 2);
    else AMP_NORM_SHAPE_ODD(cols, F);
#undef F
}

template <int XT, bool CK, bool VEC>
cudaError_t go(const NormBwd &P, int64_t parts, cudaStream_t s) {
#define F(TPR, NV)                                                                                           \
    return launch_pdl(norm_bwd_kernel<XT, CK, VEC, TPR, NV>, dim3((unsigned)parts), dim3(norm_cta(TPR)),     \
                      norm_rpc(TPR) > 1 ? size_t(P.cols) * 4 * norm_rpc(TPR) : 0, s, P)
    if constexpr (VEC) AMP_NORM_SHAPE(P.cols, F, 64, 2, 128, 2);
    else AMP_NORM_SHAPE_ODD(P.cols, F);
#undef F
}
template <int XT, bool CK>
cudaError_t go_x(const NormBwd &P, bool vec, int64_t parts, cudaStream_t s) {
    if (P.cols <= kNormRegCols) return vec ? go<XT, CK, true>(P, parts, s) : go<XT, CK, false>(P, parts, s);
    // the parameters first: dx may overwrite dy
    if (P.part) {
        const cudaError_t e = launch_pdl(norm_bwd_long_params<XT, CK>,
                                         dim3((unsigned)((P.cols + kThreads - 1) / kThreads), (unsigned)parts),
                                         dim3(kThreads), 0, s, P);
        if (e != cudaSuccess) return e;
    }
    if (!P.dx || P.rows == 0) return cudaSuccess;
    return launch_pdl(norm_bwd_long_dx<XT, CK>, dim3((unsigned)P.rows), dim3(512), 0, s, P);
}

}  // namespace

// Rows of partial sums that a workspace has room for, whichever way the rows are
// taken.
int64_t norm_parts(int64_t rows, int64_t cols, int device) {
    return std::max(norm_grid(rows, cols, true, device), norm_grid(rows, cols, false, device));
}

cudaError_t launch_norm_bwd(const void *dy, const void *x, int elem, const uint8_t *q, const uint8_t *sc,
                            int64_t rows, int64_t cols, const void *w, int welem, const float *mean,
                            const float *rstd, void *dx, void *dw, void *db, float *part, int device,
                            cudaStream_t s) {
    const NormBwd P{dy, x, w, q, sc, mean, rstd, dx, dw || db ? part : nullptr, rows, cols,
                    float(1.0 / double(cols)), welem};
    const int esz = elem == kF32 ? 4 : 2;
    const bool vec = norm_vec(dy, cols, esz) && norm_vec(x, cols, esz) && norm_vec(dx, cols, esz) &&
                     (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    const int64_t parts = norm_grid(rows, cols, vec, device);
    cudaError_t e = cudaSuccess;
    if (q)
        e = elem == kF32   ? go_x<kF32, true>(P, vec, parts, s)
            : elem == kF16 ? go_x<kF16, true>(P, vec, parts, s)
                           : go_x<kBF16, true>(P, vec, parts, s);
    else
        e = elem == kF32   ? go_x<kF32, false>(P, vec, parts, s)
            : elem == kF16 ? go_x<kF16, false>(P, vec, parts, s)
                           : go_x<kBF16, false>(P, vec, parts, s);
    if (e == cudaSuccess && P.part) {
        const NormJoin J{part, parts, cols, dw, db, welem};
        const dim3 grid((unsigned)((2 * cols + 31) / 32));
        e = parts <= 160 ? launch_pdl(norm_join_kernel<512>, grid, dim3(512), 0, s, J)
                         : launch_pdl(norm_join_kernel<1024>, grid, dim3(1024), 0, s, J);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace amp
