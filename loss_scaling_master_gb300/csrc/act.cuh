// act.cuh - the activations of ampops.h and their derivatives, two elements at a time:
//   f(x) = x Phi(x), x sigma(2 z(x)) with z = sqrt(2/pi) (x + 0.044715 x^3)
//          (= x/2 (1 + tanh z)), or x sigma(x)
#pragma once

#include "ampops.h"
#include "common.cuh"
#include "f32x2.cuh"

namespace amp {

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

}  // namespace amp
