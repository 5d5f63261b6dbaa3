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

#include "ampops.h"
#include "f32x2.cuh"
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

// ---- f and f' ----------------------------------------------------------------
// How far each is from 64 bits is in ampops.h.  The functions take two elements at a
// time, and in the GELUs what is not a lookup of the special function unit, a comparison
// or a selection runs as one instruction for both (f32x2.cuh; GELU over 4096 x 8192 bf16
// 34 instead of 39 us).  SiLU has too little of that to pay for the moves into pairs
// (8192 x 14336 gated 143 us scalar, 149 us in pairs).
//
// fp32 tensors have forms of their own, whose errors are as small as the type's rounding.
// Relative norm of the error over N(0, 1.5), f and f' (in brackets: the elementary fp32
// forms with erf, tanh and exp):
//     GELU       3.3e-8 and 3.5e-8 (3.7e-8, 3.6e-8)
//     GELU tanh  3.3e-8 and 4.5e-8 (3.6e-8, 7.9e-8)
//     SiLU       3.5e-8 and 4.4e-8 (4.5e-8, 5.1e-8)
// With normcdff() and expf() GELU is no nearer and takes 84 + 90 us for 4096 x 8192
// instead of 45 + 47.
//
// 2^u and 1 / x, each within 2 ulp; exp2_flush gives 0 below 2^-126
__device__ __forceinline__ float exp2_approx(float u) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(u));
    return r;
}
__device__ __forceinline__ float exp2_flush(float u) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(u));
    return r;
}
__device__ __forceinline__ float recip_approx(float x) {  // 0 above 2^126
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 recip2(f2 a) {
    const float2 s = split(a);
    return make_f2(recip_approx(s.x), recip_approx(s.y));
}
__device__ __forceinline__ f2 abs2(f2 a) { return a & 0x7FFFFFFF7FFFFFFFull; }
constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.9259629911e-8f, kLn2 = 0.6931471805599453f;

// 1 / (1 + exp(-t)) as 1 / (1 + e) or e / (1 + e), e = exp(-|t|): the
// denominator stays in [1, 2], so neither overflow nor the flush to zero of a
// large one's reciprocal cuts the tail off (it keeps its relative precision
// down to the subnormals).  n = 1 - the result; in fp32 the larger of the two is
// 1 - the smaller, which has no error of the division left (16 bits: the smaller
// may be the difference, absolutely good to 2^-23).
template <int XT>
__device__ __forceinline__ f2 sigmoid2(f2 t, f2 &n) {
    const float2 u = split(mul2(abs2(t), both(-kLog2e))), s = split(t);
    const float ex = exp2_approx(u.x), ey = exp2_approx(u.y);
    const f2 e = make_f2(ex, ey), one = both(1.0f), r = recip2(add2(e, one));
    if constexpr (XT == kF32) {
        const f2 lo = mul2(e, r);
        const float2 l = split(lo), h = split(fma2(lo, both(-1.0f), one));
        n = make_f2(s.x >= 0.0f ? l.x : h.x, s.y >= 0.0f ? l.y : h.y);
        return make_f2(s.x >= 0.0f ? h.x : l.x, s.y >= 0.0f ? h.y : l.y);
    }
    const f2 v = mul2(make_f2(s.x >= 0.0f ? 1.0f : ex, s.y >= 0.0f ? 1.0f : ey), r);
    n = fma2(v, both(-1.0f), one);
    return v;
}
template <int XT>
__device__ __forceinline__ float sigmoid1(float t, float &n) {
    if constexpr (XT == kF32) {
        // exp(-a) = 2^-(a log2 e), and what the product was rounded by made good
        const float a = fminf(fabsf(t), 120.0f), u = a * kLog2e;
        const float m = __fmaf_rn(a, -kLog2eLow, __fmaf_rn(a, -kLog2e, u)), e0 = exp2_approx(-u);
        const float e = __fmaf_rn(e0 * m, kLn2, e0), lo = e * recip_approx(1.0f + e), hi = 1.0f - lo;
        n = t >= 0.0f ? lo : hi;
        return t >= 0.0f ? hi : lo;
    }
    const float e = exp2_approx(fabsf(t) * -kLog2e), v = (t >= 0.0f ? 1.0f : e) * recip_approx(1.0f + e);
    n = 1.0f - v;
    return v;
}

// The magnitude past which sigma(2z) is 0 or 1 to the last bit, so cubes and squares of
// larger x need not be formed (they would overflow and meet a zero factor).  NaN stays.
__device__ __forceinline__ float act_clamp(float x) { return fabsf(x) > 30.0f ? copysignf(30.0f, x) : x; }
__device__ __forceinline__ f2 act_clamp2(f2 x) {
    const float2 s = split(x);
    return make_f2(act_clamp(s.x), act_clamp(s.y));
}

// Phi(x) and e = exp(-x^2/2).  Phi(-a) / e is a polynomial in t = 1 / (1 + p a) as far as
// e goes, so Phi(-|x|) keeps its relative precision into the tail, and the exponential is
// the one that the derivative needs.  (An error function of bounded absolute error, whose
// Phi is 0.4 % off at x = -6 and 2 % at -10, takes as long.)  The coefficients here are
// least-maximum fits of the relative error, made for this file.
//
// 16 bits: one polynomial, good to 1.9e-6.  e = 0 where x^2 overflows.
// fp32: one good to 4.5e-8 for a >= 1.25; below, where Phi is not small and the roundings
// of that one would show, 1/2 - a P(a^2) good to 9.6e-9 of a P.
template <int XT>
__device__ __forceinline__ f2 gauss_cdf2(f2 x, f2 &e) {
    const float2 s = split(x);
    f2 v;
    if constexpr (XT == kF32) {
        const f2 a = make_f2(fminf(fabsf(s.x), 15.0f), fminf(fabsf(s.y), 15.0f)), q = mul2(a, a);
        const float2 u = split(mul2(q, both(-0.5f * kLog2e)));
        e = make_f2(exp2_flush(u.x), exp2_flush(u.y));
        const f2 t = recip2(fma2(a, both(0.625f), both(1.0f)));
        f2 o = fma2(t, both(-0.2584007978f), both(0.7364913225f));
        o = fma2(o, t, both(-0.7159850597f));
        o = fma2(o, t, both(0.1085906923f));
        o = fma2(o, t, both(0.1240824759f));
        o = fma2(o, t, both(0.2523988783f));
        o = fma2(o, t, both(0.2491545975f));
        o = mul2(fma2(o, t, both(4.668735983e-06f)), e);
        f2 i = fma2(q, both(-6.809503247e-06f), both(0.0001110411758f));
        i = fma2(i, q, both(-0.001183837187f));
        i = fma2(i, q, both(0.009972282685f));
        i = fma2(i, q, both(-0.06649021059f));
        i = fma2(mul2(fma2(i, q, both(0.3989422619f)), a), both(-1.0f), both(0.5f));
        const float2 so = split(o), si = split(i), sa = split(a);
        v = make_f2(sa.x < 1.25f ? si.x : so.x, sa.y < 1.25f ? si.y : so.y);
    } else {
        const float2 u = split(mul2(mul2(x, x), both(-0.5f * kLog2e)));
        e = make_f2(exp2_flush(u.x), exp2_flush(u.y));
        const f2 t = recip2(fma2(abs2(x), both(0.3f), both(1.0f)));
        v = fma2(t, both(-0.0845924839f), both(0.2405701131f));
        v = fma2(v, t, both(-0.0486405641f));
        v = fma2(v, t, both(0.1647616178f));
        v = fma2(v, t, both(0.1067056805f));
        v = fma2(v, t, both(0.1212744638f));
        v = mul2(fma2(v, t, both(-7.9769998e-05f)), e);
    }
    const float2 sv = split(v);
    return make_f2(s.x >= 0.0f ? 1.0f - sv.x : sv.x, s.y >= 0.0f ? 1.0f - sv.y : sv.y);
}

// 2 sqrt(2/pi) = 1.5957691216, times 0.044715 = 0.0713548163
constexpr float kTanhA = 1.5957691216057308f, kTanhB = 0.07135481627159954f;

template <int XT, int ACT>
__device__ __forceinline__ f2 act_value2(f2 x) {
    f2 e;
    if constexpr (ACT == AMP_ACT_GELU) return mul2(x, gauss_cdf2<XT>(x, e));
    const f2 c = act_clamp2(x);
    return mul2(x, sigmoid2<XT>(mul2(c, fma2(mul2(c, c), both(kTanhB), both(kTanhA))), e));
}
// f(x) and f'(x)
template <int XT, int ACT>
__device__ __forceinline__ void act_both2(f2 x, f2 &f, f2 &d) {
    if constexpr (ACT == AMP_ACT_GELU) {
        f2 e;
        const f2 p = gauss_cdf2<XT>(x, e);
        f = mul2(x, p);
        d = fma2(mul2(x, both(0.3989422804014327f)), e, p);
    } else {
        const f2 c = act_clamp2(x), q = mul2(c, c);
        f2 n;
        const f2 s = sigmoid2<XT>(mul2(c, fma2(q, both(kTanhB), both(kTanhA))), n);
        f = mul2(x, s);
        d = fma2(mul2(mul2(c, s), n), fma2(q, both(3.0f * kTanhB), both(kTanhA)), s);
    }
}

// y = f(x) [* u] for two elements.
template <int XT, int ACT, bool GATED>
__device__ __forceinline__ float2 act_apply(float x0, float x1, float u0, float u1) {
    if constexpr (ACT == AMP_ACT_SILU) {
        float n;
        const float a = x0 * sigmoid1<XT>(x0, n), b = x1 * sigmoid1<XT>(x1, n);
        return GATED ? make_float2(a * u0, b * u1) : make_float2(a, b);
    }
    const f2 y = act_value2<XT, ACT>(make_f2(x0, x1));
    return split(GATED ? mul2(y, make_f2(u0, u1)) : y);
}
// dx = g f'(x) [* u] and du = g f(x) for two elements.
template <int XT, int ACT, bool GATED>
__device__ __forceinline__ void act_grads(float x0, float x1, float u0, float u1, float g0, float g1, float2 &dx,
                                          float2 &du) {
    if constexpr (ACT == AMP_ACT_SILU) {
        float n0, n1;
        const float s0 = sigmoid1<XT>(x0, n0), s1 = sigmoid1<XT>(x1, n1);
        const float f0 = x0 * s0, f1 = x1 * s1;
        du = make_float2(g0 * f0, g1 * f1);
        dx = make_float2((GATED ? g0 * u0 : g0) * __fmaf_rn(f0, n0, s0), (GATED ? g1 * u1 : g1) * __fmaf_rn(f1, n1, s1));
    } else {
        f2 f, d, g = make_f2(g0, g1);
        act_both2<XT, ACT>(make_f2(x0, x1), f, d);
        du = split(mul2(g, f));
        if (GATED) g = mul2(g, make_f2(u0, u1));
        dx = split(mul2(g, d));
    }
}

// fp32 bits of max |y| over the 8 elements and the 4 lanes of the block
__device__ __forceinline__ uint32_t block_max8(const float (&y)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
}

__device__ __forceinline__ uint2 codes8(const float (&y)[8], float f) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a, b;
        mul2_rn(y[2 * j], y[2 * j + 1], f, f, a, b);
        h[j] = f32x2_to_fp8x2_raw<kE4M3>(a, b);
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ void values8(uint2 q, float s, float (&y)[8]) {
    e4m3x4_to_f32x4(q.x, y);
    e4m3x4_to_f32x4(q.y, y + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(y[j], s);
}

template <int XT>
__device__ __forceinline__ void ldv(const void *p, int64_t k, float (&y)[8]) {
    constexpr int esz = XT == kF32 ? 4 : 2;
    uint4 u[kWords8<XT>];
#pragma unroll
    for (int j = 0; j < kWords8<XT>; ++j) u[j] = ld16(static_cast<const char *>(p) + k * esz + 16 * j);
    raw8_to_f32<XT>(u, y);
}
template <int XT>
__device__ __forceinline__ void stv(void *p, int64_t k, const float (&y)[8]) {
    constexpr int esz = XT == kF32 ? 4 : 2;
    uint4 u[kWords8<XT>];
    f32_to_raw8<XT>(y, u);
#pragma unroll
    for (int j = 0; j < kWords8<XT>; ++j) st16(static_cast<char *>(p) + k * esz + 16 * j, u[j]);
}

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
// left in it.
template <int XT, int EB>
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
        const uint32_t e = mx_scale_code<MxE4M3>(block_max8(y));
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
            keep_elems<XT, EB>(x, n, P.kb - b0, P.q + k, P.s + sb, s_x[warp], s_q[warp]);
            if (GATED) keep_elems<XT, EB>(u, n, P.kb - b0, P.qu + k, P.su + sb, s_x[warp], s_q[warp]);
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
