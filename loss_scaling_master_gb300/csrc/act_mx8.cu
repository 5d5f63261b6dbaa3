// act_mx8.cu - activations whose inputs are kept as 8-bit checkpoints (e4m3,
// blocks of 32 with a power-of-two scale: mx.cuh), their gradients from those
// checkpoints, and the checkpoint on its own.
//
//   forward   y = f(x) [* u];  x [, u] -> codes and scales in the same pass
//   backward  xh, uh = the checkpoint's values;
//             dx = dy f'(xh) [* uh], du = dy f(xh)
//   f(x) = x Phi(x), x sigma(2 z(x)) with z = sqrt(2/pi) (x + 0.044715 x^3)
//          (= x/2 (1 + tanh z)), or x sigma(x)
//
// Every element is read and written once, so memory bounds the kernels as long
// as the arithmetic stays under the issue rate.  A thread takes 8 elements
// (one 16-byte access of a 16-bit tensor), 4 threads a block, whose maximum
// takes two shuffles.  Rows that are not whole groups of 8 elements, or not
// 16-byte aligned, are taken by single elements, a block across a warp.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "internal.h"
#include "mx.cuh"
#include "pdl.cuh"

namespace amp {
namespace {

enum Mode : int { kSave = 3 };  // after the three amp_act values: no activation

struct ActFwd {
    const void *x, *u;
    void *y;
    uint8_t *q, *s, *qu, *su;
    int64_t rows, cols;
    int kb;  // blocks a row
};
struct ActBwd {
    const void *dy;
    const uint8_t *q, *s, *qu, *su;
    void *dx, *du;
    int64_t rows, cols;
    int kb;
};

// CTAs an SM holds (0: as many as the compiler's registers leave): see bwd_vec_ctas.
__host__ __device__ constexpr int fwd_vec_ctas(int xt, int act, bool gated) {
    return act == AMP_ACT_GELU && !gated && xt == kF32 ? 8 : 0;
}
// 8 elements a thread; rows are whole groups of 8 and every address aligned.
template <int XT, int ACT, bool GATED, bool KEEP>
__global__ void __launch_bounds__(kThreads, fwd_vec_ctas(XT, ACT, GATED))
    act_fwd_vec(ActFwd P) {
    pdl_wait();
    pdl_trigger();
    // the 4 threads of a block run together, so every thread of a warp walks
    // until the warp's first row is past the end, and guards
    RowWalk at((blockIdx.x * kThreads + threadIdx.x) / 4, gridDim.x * (kThreads / 4), P.kb);
    for (; __any_sync(0xFFFFFFFFu, at.row < P.rows); at.next()) {
        const bool row = at.row < P.rows;
        const int64_t b = at.row * P.kb + at.at;
        const int col = at.at * kMxBlock + 8 * (threadIdx.x & 3);
        const bool in = row && col < P.cols;
        const int64_t k = at.row * P.cols + col;
        float x[8], u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = u[j] = 0.0f;
        if (in) {
            ldv<XT>(P.x, k, x);
            if (GATED) ldv<XT>(P.u, k, u);
        }
        if (KEEP) {
            const uint32_t e = mx_scale_code<MxE4M3>(block_max8(x));
            if (in) *reinterpret_cast<uint2 *>(P.q + k) = codes8(x, mx_unscale(e));
            if (row && (threadIdx.x & 3) == 0) P.s[b] = uint8_t(e);
            if (GATED) {
                const uint32_t eu = mx_scale_code<MxE4M3>(block_max8(u));
                if (in) *reinterpret_cast<uint2 *>(P.qu + k) = codes8(u, mx_unscale(eu));
                if (row && (threadIdx.x & 3) == 0) P.su[b] = uint8_t(eu);
            }
        }
        if (ACT != kSave && in) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 v = act_apply<XT, ACT, GATED>(x[j], x[j + 1], u[j], u[j + 1]);
                x[j] = v.x;
                x[j + 1] = v.y;
            }
            stv<XT>(P.y, k, x);
        }
    }
}

// block_max8 by integers, as large bits are large magnitudes.
__device__ __forceinline__ uint32_t block_max8_ints(const float (&y)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
}

// Any size, any address: a warp takes EB blocks of a row at a time, a lane one
// element of each, so accesses stay side by side and a row's place is worked out
// once for EB elements (with one block a step, 100 instructions an element bound
// the kernel: 2047 x 1111 f16 GELU forward 8.6 us, with four 5.3 us, with eight 4.7 us;
// 4095 x 8191 bf16 50.8 us with four, 42.4 with eight).  Eight where rows are long and
// many enough; 20000 x 100 takes 5.7 us by four and 6.8 by eight, 33 x 1111 1.5 and 1.8.
template <int XT>
using Elem = std::conditional_t<XT == kF32, uint32_t, uint16_t>;
template <int XT>
__device__ __forceinline__ float widen1(Elem<XT> v) {
    if constexpr (XT == kF32) return __uint_as_float(v);
    else return lowp_to_f32<XT>(v);
}

// The checkpoint of a warp's EB blocks, x[i] the lane's element of block i.  By
// four: a block's maximum by one reduction over the warp.  By eight: the warp's
// 256 elements go through shared memory (s, 1 KB, and b, 256 bytes) to 8
// consecutive ones a lane and their codes come back as bytes, so that scales and
// conversions serve 8 elements (fp32: 16-byte pieces exchanged in every other
// block, against bank conflicts).  n > 32 i: element i is in the row; kb: blocks
// left in it.  INTS: the blocks' maxima by integers.
template <int XT, int EB, bool INTS>
__device__ __forceinline__ void keep_elems(const Elem<XT> (&x)[EB], int n, int kb, uint8_t *q, uint8_t *sc,
                                           uint4 *s, uint2 *b) {
    const int lane = threadIdx.x & 31;
    if constexpr (EB == 8) {
        constexpr int W = kWords8<XT>;
        __syncwarp();  // the last values of s and b are read
#pragma unroll
        for (int i = 0; i < 8; ++i)
            reinterpret_cast<Elem<XT> *>(s)[32 * i + (W == 2 ? lane ^ (4 * (i & 1)) : lane)] = x[i];
        __syncwarp();
        uint4 u[W];
#pragma unroll
        for (int i = 0; i < W; ++i) u[i] = s[(W * lane + i) ^ (W == 2 ? (lane >> 2) & 1 : 0)];
        float y[8];
        raw8_to_f32<XT>(u, y);
        const uint32_t e = mx_scale_code<MxE4M3>(INTS ? block_max8_ints(y) : block_max8(y));
        b[lane] = codes8(y, mx_unscale(e));
        if ((lane & 3) == 0 && lane / 4 < kb) sc[lane / 4] = uint8_t(e);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n > 32 * i) q[32 * i] = reinterpret_cast<const uint8_t *>(b)[32 * i + lane];
    } else {
        uint32_t mine = 0;  // lane i: block i's scale byte
#pragma unroll
        for (int i = 0; i < EB; ++i) {
            const float v = widen1<XT>(x[i]);
            const uint32_t e = mx_scale_code<MxE4M3>(warp_max_u32(__float_as_uint(v) & 0x7FFFFFFFu));
            if (n > 32 * i) q[32 * i] = uint8_t(f32x2_to_fp8x2_raw<kE4M3>(__fmul_rn(v, mx_unscale(e)), 0.0f));
            if (lane == i) mine = e;
        }
        if (lane < EB && lane < kb) sc[lane] = uint8_t(mine);
    }
}

template <int XT, int ACT, bool GATED, bool KEEP, int EB>
__global__ void __launch_bounds__(kThreads) act_fwd_elem(ActFwd P) {
    __shared__ uint4 s_x[EB == 8 && KEEP ? kThreads / 32 : 1][32 * kWords8<XT>];
    __shared__ uint2 s_q[EB == 8 && KEEP ? kThreads / 32 : 1][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = EB == 8 && KEEP ? threadIdx.x >> 5 : 0;
    RowWalk at(blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32), (P.kb + EB - 1) / EB);
    for (; at.row < P.rows; at.next()) {
        const int b0 = at.at * EB, n = int(P.cols) - b0 * kMxBlock - lane;  // n > 32 i: element i is in the row
        const int64_t k = at.row * P.cols + b0 * kMxBlock + lane, sb = at.row * P.kb + b0;
        const Elem<XT> *xp = static_cast<const Elem<XT> *>(P.x) + k, *up = static_cast<const Elem<XT> *>(P.u) + k;
        Elem<XT> x[EB], u[EB];
#pragma unroll
        for (int i = 0; i < EB; ++i) {
            x[i] = n > 32 * i ? xp[32 * i] : Elem<XT>(0);
            u[i] = GATED && n > 32 * i ? up[32 * i] : Elem<XT>(0);
        }
        if constexpr (KEEP) {
            // Maxima by integers leave plain 16-bit activations 40 registers, by three magnitudes
            // an instruction 42, and an SM 5 CTAs instead of 6 (4095 x 8191 bf16 GELU 42.6 and
            // 44.0 us, tanh 45.9 and 46.6, SiLU 40.9 and 42.4).  Elsewhere they are slower:
            // the checkpoint alone 25.9 and 25.1 us, gated SiLU 66.1 and 64.8, fp32 GELU 57.1 and 53.3.
            constexpr bool INTS = ACT != kSave && !GATED && XT != kF32;
            keep_elems<XT, EB, INTS>(x, n, P.kb - b0, P.q + k, P.s + sb, s_x[warp], s_q[warp]);
            if (GATED) keep_elems<XT, EB, INTS>(u, n, P.kb - b0, P.qu + k, P.su + sb, s_x[warp], s_q[warp]);
        }
        if constexpr (ACT != kSave) {
            char *yp = static_cast<char *>(P.y) + k * int(sizeof(Elem<XT>));
#pragma unroll
            for (int i = 0; i < EB; i += 2) {
                if (n <= 32 * i) break;
                const float2 v = act_apply<XT, ACT, GATED>(widen1<XT>(x[i]), widen1<XT>(x[i + 1]), widen1<XT>(u[i]),
                                                       widen1<XT>(u[i + 1]));
                store_elem<XT>(yp, 32 * i, v.x);
                if (n > 32 * (i + 1)) store_elem<XT>(yp, 32 * (i + 1), v.y);
            }
        }
    }
}

// CTAs an SM holds: GELU's backward is a register or more above 32 (gated: 40) where the
// compiler is left to itself, and slower by an SM's missing CTAs (4096 x 8192 bf16 35.7
// instead of 31.9 us, gated 44.8 and 42.4, fp32 53.4 and 46.6; fp32 forward 46.7 and 44.7).
// The others are slower with any bound here.  0: none.
__host__ __device__ constexpr int bwd_vec_ctas(int act, bool gated) {
    return act == AMP_ACT_GELU ? (gated ? 6 : 8) : 0;
}
template <int XT, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, bwd_vec_ctas(ACT, GATED)) act_bwd_vec(ActBwd P) {
    pdl_wait();
    pdl_trigger();
    RowWalk at((blockIdx.x * kThreads + threadIdx.x) / 4, gridDim.x * (kThreads / 4), P.kb);
    for (; at.row < P.rows; at.next()) {
        const int64_t b = at.row * P.kb + at.at;
        const int col = at.at * kMxBlock + 8 * (threadIdx.x & 3);
        if (col >= P.cols) continue;
        const int64_t k = at.row * P.cols + col;
        float x[8], u[8], g[8], o[8];
        values8(*reinterpret_cast<const uint2 *>(P.q + k), mx_scale(P.s[b]), x);
        if (GATED) values8(*reinterpret_cast<const uint2 *>(P.qu + k), mx_scale(P.su[b]), u);
        if (ACT != kSave) ldv<XT>(P.dy, k, g);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            if constexpr (ACT == kSave) {
                g[j] = x[j];
                g[j + 1] = x[j + 1];
            } else {
                float2 dx, du;
                act_grads<XT, ACT, GATED>(x[j], x[j + 1], u[j], u[j + 1], g[j], g[j + 1], dx, du);
                o[j] = du.x;
                o[j + 1] = du.y;
                g[j] = dx.x;
                g[j + 1] = dx.y;
            }
        }
        stv<XT>(P.dx, k, g);
        if (GATED) stv<XT>(P.du, k, o);
    }
}

template <int XT, int ACT, bool GATED, int EB>
__global__ void __launch_bounds__(kThreads) act_bwd_elem(ActBwd P) {
    pdl_wait();
    pdl_trigger();
    constexpr int esz = XT == kF32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    RowWalk at(blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32),
               (P.kb + EB - 1) / EB);
    for (; at.row < P.rows; at.next()) {
        const int b0 = at.at * EB, n = int(P.cols) - b0 * kMxBlock - lane;
        const int64_t k = at.row * P.cols + b0 * kMxBlock + lane, sb = at.row * P.kb + b0;
        const char *gp = static_cast<const char *>(P.dy) + k * esz;
        char *dxp = static_cast<char *>(P.dx) + k * esz, *dup = static_cast<char *>(P.du) + k * esz;
        const uint8_t *qp = P.q + k, *qup = P.qu + k;
        uint32_t q[EB], qu[EB];
        float g[EB];
        // lane i: block i's scale
        const bool scales = lane < EB && lane < P.kb - b0;
        const float sx = scales ? mx_scale(P.s[sb + lane]) : 0.0f;
        const float su = GATED && scales ? mx_scale(P.su[sb + lane]) : 0.0f;
#pragma unroll
        for (int i = 0; i < EB; ++i) {
            q[i] = qu[i] = 0;
            g[i] = 0.0f;
            if (n <= 32 * i) continue;
            q[i] = qp[32 * i];
            if (GATED) qu[i] = qup[32 * i];
            if (ACT != kSave) g[i] = load_elem<XT>(gp, 32 * i);
        }
#pragma unroll
        for (int i = 0; i < EB; i += 2) {
            constexpr uint32_t all = 0xFFFFFFFFu;
            const float s0 = __shfl_sync(all, sx, i), s1 = __shfl_sync(all, sx, i + 1);
            const float t0 = GATED ? __shfl_sync(all, su, i) : 0.0f, t1 = GATED ? __shfl_sync(all, su, i + 1) : 0.0f;
            if (n <= 32 * i) continue;
            const bool two = n > 32 * (i + 1);
            float v[4], w[4];
            e4m3x4_to_f32x4(q[i] | (q[i + 1] << 8), v);
            const float x0 = __fmul_rn(v[0], s0), x1 = __fmul_rn(v[1], s1);
            if constexpr (ACT == kSave) {
                store_elem<XT>(dxp, 32 * i, x0);
                if (two) store_elem<XT>(dxp, 32 * (i + 1), x1);
            } else {
                float2 dx, du;
                if (GATED) e4m3x4_to_f32x4(qu[i] | (qu[i + 1] << 8), w);
                const float u0 = GATED ? __fmul_rn(w[0], t0) : 0.0f;
                const float u1 = GATED ? __fmul_rn(w[1], t1) : 0.0f;
                act_grads<XT, ACT, GATED>(x0, x1, u0, u1, g[i], g[i + 1], dx, du);
                store_elem<XT>(dxp, 32 * i, dx.x);
                if (two) store_elem<XT>(dxp, 32 * (i + 1), dx.y);
                if (GATED) {
                    store_elem<XT>(dup, 32 * i, du.x);
                    if (two) store_elem<XT>(dup, 32 * (i + 1), du.y);
                }
            }
        }
    }
}

bool ptr_ok(const void *p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) == 0; }

// CTAs for that many threads' work, at most `most` an SM.
unsigned grid_of(int64_t threads, int most, int device) {
    const int64_t want = (threads + kThreads - 1) / kThreads;
    return unsigned(std::min<int64_t>(want, int64_t(sm_count(device)) * most));
}

// CTAs an SM, resident or waiting: 64 of the 16-byte kernels (8192 x 14336 gated
// 142 us, with 8 of them 171 us) and 32 of the others (4095 x 8191 bf16 GELU 42 us,
// with 8 of them 47 us; 20000 x 100 5.7 and 5.3 us).
constexpr int kVecCtas = 64, kElemCtas = 32;
int64_t vec_threads(int64_t rows, int kb) { return rows * kb * 4; }
int64_t elem_threads(int64_t rows, int kb, int eb) { return rows * ((kb + eb - 1) / eb) * 32; }
// eight blocks a step: rows of 32 blocks or more, and 16 warps for every SM
bool eight_blocks(int64_t rows, int kb, int device) {
    return kb >= 32 && elem_threads(rows, kb, 8) >= int64_t(sm_count(device)) * 512;
}

template <int XT, int ACT, bool GATED, bool KEEP>
cudaError_t fwd_keep(const ActFwd &P, bool vec, int dev, cudaStream_t s) {
    const dim3 block(kThreads);
    if (vec)
        return launch_pdl(act_fwd_vec<XT, ACT, GATED, KEEP>, dim3(grid_of(vec_threads(P.rows, P.kb), kVecCtas, dev)),
                          block, 0, s, P);
    if (eight_blocks(P.rows, P.kb, dev))
        return launch_pdl(act_fwd_elem<XT, ACT, GATED, KEEP, 8>,
                          dim3(grid_of(elem_threads(P.rows, P.kb, 8), kElemCtas, dev)), block, 0, s, P);
    return launch_pdl(act_fwd_elem<XT, ACT, GATED, KEEP, 4>,
                      dim3(grid_of(elem_threads(P.rows, P.kb, 4), kElemCtas, dev)), block, 0, s, P);
}
template <int XT, int ACT, bool GATED>
cudaError_t fwd(const ActFwd &P, bool keep, bool vec, int dev, cudaStream_t s) {
    if constexpr (ACT != kSave)
        if (!keep) return fwd_keep<XT, ACT, GATED, false>(P, vec, dev, s);
    return fwd_keep<XT, ACT, GATED, true>(P, vec, dev, s);
}
template <int XT, int ACT, bool GATED>
cudaError_t bwd(const ActBwd &P, bool vec, int dev, cudaStream_t s) {
    const dim3 block(kThreads);
    if (vec)
        return launch_pdl(act_bwd_vec<XT, ACT, GATED>, dim3(grid_of(vec_threads(P.rows, P.kb), kVecCtas, dev)), block, 0,
                          s, P);
    if (eight_blocks(P.rows, P.kb, dev))
        return launch_pdl(act_bwd_elem<XT, ACT, GATED, 8>, dim3(grid_of(elem_threads(P.rows, P.kb, 8), kElemCtas, dev)),
                          block, 0, s, P);
    return launch_pdl(act_bwd_elem<XT, ACT, GATED, 4>, dim3(grid_of(elem_threads(P.rows, P.kb, 4), kElemCtas, dev)),
                      block, 0, s, P);
}

template <int XT>
cudaError_t fwd_x(const ActFwd &P, int act, bool keep, bool vec, int dev, cudaStream_t s) {
    if (act == kSave) return fwd<XT, kSave, false>(P, keep, vec, dev, s);
    if (P.u) {
        if (act == AMP_ACT_GELU) return fwd<XT, AMP_ACT_GELU, true>(P, keep, vec, dev, s);
        if (act == AMP_ACT_GELU_TANH) return fwd<XT, AMP_ACT_GELU_TANH, true>(P, keep, vec, dev, s);
        return fwd<XT, AMP_ACT_SILU, true>(P, keep, vec, dev, s);
    }
    if (act == AMP_ACT_GELU) return fwd<XT, AMP_ACT_GELU, false>(P, keep, vec, dev, s);
    if (act == AMP_ACT_GELU_TANH) return fwd<XT, AMP_ACT_GELU_TANH, false>(P, keep, vec, dev, s);
    return fwd<XT, AMP_ACT_SILU, false>(P, keep, vec, dev, s);
}
template <int XT>
cudaError_t bwd_x(const ActBwd &P, int act, bool vec, int dev, cudaStream_t s) {
    if (act == kSave) return bwd<XT, kSave, false>(P, vec, dev, s);
    if (P.qu) {
        if (act == AMP_ACT_GELU) return bwd<XT, AMP_ACT_GELU, true>(P, vec, dev, s);
        if (act == AMP_ACT_GELU_TANH) return bwd<XT, AMP_ACT_GELU_TANH, true>(P, vec, dev, s);
        return bwd<XT, AMP_ACT_SILU, true>(P, vec, dev, s);
    }
    if (act == AMP_ACT_GELU) return bwd<XT, AMP_ACT_GELU, false>(P, vec, dev, s);
    if (act == AMP_ACT_GELU_TANH) return bwd<XT, AMP_ACT_GELU_TANH, false>(P, vec, dev, s);
    return bwd<XT, AMP_ACT_SILU, false>(P, vec, dev, s);
}

}  // namespace

cudaError_t launch_act_fwd(int act, const void *x, const void *u, int elem, int64_t rows, int64_t cols,
                           void *y, uint8_t *q, uint8_t *sc, uint8_t *qu, uint8_t *su, int device,
                           cudaStream_t s) {
    const ActFwd P{x, u, y, q, sc, qu, su, rows, cols, int((cols + kMxBlock - 1) / kMxBlock)};
    const bool vec = cols % 8 == 0 && ptr_ok(x, 15) && ptr_ok(u, 15) && ptr_ok(y, 15) && ptr_ok(q, 7) && ptr_ok(qu, 7);
    const int a = act < 0 ? int(kSave) : act;
    cudaError_t e = elem == kF32   ? fwd_x<kF32>(P, a, q != nullptr, vec, device, s)
                    : elem == kF16 ? fwd_x<kF16>(P, a, q != nullptr, vec, device, s)
                                   : fwd_x<kBF16>(P, a, q != nullptr, vec, device, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_act_bwd(int act, const void *dy, int elem, int64_t rows, int64_t cols,
                           const uint8_t *q, const uint8_t *sc, const uint8_t *qu, const uint8_t *su,
                           void *dx, void *du, int device, cudaStream_t s) {
    const ActBwd P{dy, q, sc, qu, su, dx, du, rows, cols, int((cols + kMxBlock - 1) / kMxBlock)};
    const bool vec = cols % 8 == 0 && ptr_ok(dy, 15) && ptr_ok(dx, 15) && ptr_ok(du, 15) && ptr_ok(q, 7) && ptr_ok(qu, 7);
    const int a = act < 0 ? int(kSave) : act;
    cudaError_t e = elem == kF32   ? bwd_x<kF32>(P, a, vec, device, s)
                    : elem == kF16 ? bwd_x<kF16>(P, a, vec, device, s)
                                   : bwd_x<kBF16>(P, a, vec, device, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace amp
