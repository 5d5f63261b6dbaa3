// fp4_linear.cuh - what the kernels of fp4_product.cuh make of their accumulators in a
// linear layer:
//
//   z = A B^T + bias,  out = f(z) + residual (one rounding),  8-bit checkpoint of z
//
// A lane holds one column of C and consecutive tokens.  32 lanes are then one block of
// the checkpoint for each token, whose maximum is one reduction over the warp.  The
// residual comes in the layout in which store16 stores (two neighbouring elements of a
// row a lane, even lanes the even tokens) and is turned over by one shuffle for two
// elements; the words of the first 16 tokens are asked for before the accumulators are
// waited for, the others 16 tokens ahead.
#pragma once

#include "act.cuh"
#include "fp4_product.cuh"

namespace amp {
namespace {

enum : int { kNoAct = 3 };  // after the three amp_act values

struct Fp4Linear : Fp4Product {
    const void *bias, *res;
    uint8_t *q, *s;
    int kb;          // blocks of 32 columns
    uint8_t bt;      // ElemType of bias
    uint8_t act;     // amp_act or kNoAct
    uint8_t rpacked; // packed, and the residual 4-byte aligned too
    uint8_t qpacked; // q 4-byte aligned, and n % 4 == 0
};

template <int OT>
__device__ __forceinline__ float bias_at(const Fp4Linear &P, int64_t nn) {
    if (!P.bias || nn >= P.n) return 0.0f;
    return P.bt == kF32 ? static_cast<const float *>(P.bias)[nn] : load_elem<OT>(P.bias, nn);
}

// The checkpoint's scales of cnt tokens from m0 for the 32 columns that hold nn: NaN.
__device__ __forceinline__ void scales_nan(const Fp4Linear &P, int64_t m0, int cnt, int64_t nn) {
    if (!P.q || (threadIdx.x & 31) != 0) return;
#pragma unroll 1
    for (int64_t m = m0; m < m0 + cnt && m < P.m; ++m) P.s[m * P.kb + nn / kMxBlock] = 255;
}

template <int OT, int ACT>
struct EpOne {
    using Args = Fp4Linear;
    static constexpr bool none = false;
    static constexpr int CH = 16, WORDS = OT == kF32 ? CH : CH / 2;
    struct State {
        uint32_t r[WORDS];  // the residual of CH tokens
        float bias;
    };

    // the residual's elements of CH tokens from m0, of which `rows` are in C
    static __device__ __forceinline__ void residual(const Args &P, int64_t m0, int rows, int64_t nn,
                                                    uint32_t (&r)[WORDS]) {
        if constexpr (OT == kF32) {
            const float *at = static_cast<const float *>(P.res) + m0 * P.n + nn;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                r[i] = nn < P.n && i < rows ? __float_as_uint(*at) : 0u;
                at += P.n;
            }
        } else if (P.rpacked) {
            const int odd = threadIdx.x & 1;
            const char *at = static_cast<const char *>(P.res) + ((m0 + odd) * P.n + (nn - odd)) * 2;
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
                r[i] = nn < P.n && 2 * i + odd < rows ? *reinterpret_cast<const uint32_t *>(at) : 0u;
                at += 4 * P.n;
            }
        } else {
            const uint16_t *at = static_cast<const uint16_t *>(P.res) + m0 * P.n + nn;
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
                uint32_t a = 0, b = 0;
                if (nn < P.n && 2 * i < rows) a = *at;
                at += P.n;
                if (nn < P.n && 2 * i + 1 < rows) b = *at;
                at += P.n;
                r[i] = a | (b << 16);
            }
        }
    }
    static __device__ __forceinline__ void begin(const Args &P, int64_t m0, int rows, int64_t nn, State &ep) {
        ep.bias = bias_at<OT>(P, nn);
        if (P.res) residual(P, m0, rows, nn, ep.r);
    }

    // The checkpoint of CH tokens' z (0 in columns behind the last one).
    static __device__ __forceinline__ void save(const Args &P, int64_t m0, int rows, int64_t nn,
                                                const float (&z)[CH]) {
        const int lane = threadIdx.x & 31;
        uint8_t *at = P.q + m0 * P.n + nn;
        uint32_t mine = 0;  // lane i: token i's scale byte
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const uint32_t e = mx_scale_code<MxE4M3>(warp_max_u32(__float_as_uint(z[i]) & 0x7FFFFFFFu));
            if (nn < P.n && i < rows)
                *at = uint8_t(f32x2_to_fp8x2_raw<kE4M3>(__fmul_rn(z[i], mx_unscale(e)), 0.0f));
            at += P.n;
            if (lane == i) mine = e;
        }
        if (lane < CH && lane < rows && nn - lane < P.n) P.s[(m0 + lane) * P.kb + (nn - lane) / kMxBlock] = uint8_t(mine);
    }

    // f(z) + residual for two tokens, elements 2 i and 2 i + 1 of the residual's words
    static __device__ __forceinline__ float2 value(const Args &P, float z0, float z1, int i,
                                                   const uint32_t (&r)[WORDS]) {
        float2 y = make_float2(z0, z1);
        if constexpr (ACT != kNoAct) y = act_apply<OT, ACT, false>(z0, z1, 0.0f, 0.0f);
        if (P.res) {
            if constexpr (OT == kF32) {
                y.x += __uint_as_float(r[2 * i]);
                y.y += __uint_as_float(r[2 * i + 1]);
            } else {
                uint32_t w = r[i];
                if (P.rpacked) {
                    const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
                    w = threadIdx.x & 1 ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
                }
                y.x += lowp_to_f32<OT>(w & 0xFFFFu);
                y.y += lowp_to_f32<OT>(w >> 16);
            }
        }
        return y;
    }

    // ep: as begin() left it for the same place
    template <int CNT>
    static __device__ __forceinline__ void finish(const Args &P, int64_t m0, int rows, int64_t nn,
                                                  const uint32_t (&v)[CNT], State &ep) {
#pragma unroll
        for (int c = 0; c < CNT; c += CH) {
            if (c >= rows) break;
            State nxt;
            if (P.res && c + CH < CNT) residual(P, m0 + c + CH, rows - c - CH, nn, nxt.r);
            float z[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) z[i] = __uint_as_float(v[c + i]) + ep.bias;
            if (P.q) save(P, m0 + c, rows - c, nn, z);
            if constexpr (OT == kF32) {
                uint32_t o[CH];
#pragma unroll
                for (int i = 0; i < CH; i += 2) {
                    const float2 y = value(P, z[i], z[i + 1], i / 2, ep.r);
                    o[i] = __float_as_uint(y.x);
                    o[i + 1] = __float_as_uint(y.y);
                }
                store32<CH>(P, m0 + c, rows - c, nn, o);
            } else {
                uint32_t o[CH / 2];
#pragma unroll
                for (int i = 0; i < CH / 2; ++i) {
                    const float2 y = value(P, z[2 * i], z[2 * i + 1], i, ep.r);
                    o[i] = f32x2_to_16x2<OT>(y.x, y.y);
                }
                store16<CH>(P, m0 + c, rows - c, nn, o);
            }
            if (c + CH < CNT) {
#pragma unroll
                for (int i = 0; i < WORDS; ++i) ep.r[i] = nxt.r[i];
            }
        }
    }
    static __device__ __forceinline__ void saved_nan(const Args &P, int64_t m0, int cnt, int64_t nn) {
        scales_nan(P, m0, cnt, nn);
    }
};

// The element type and the activation looked up for every 16 tokens: for the kernels of
// one CTA a tile, whose time is the operands'.
struct EpAny {
    using Args = Fp4Linear;
    static constexpr bool none = false;
    struct State {};
    static __device__ __forceinline__ void begin(const Args &, int64_t, int, int64_t, State &) {}
    template <int OT, int ACT, int CNT>
    static __device__ __forceinline__ void run(const Args &P, int64_t m0, int rows, int64_t nn,
                                               const uint32_t (&v)[CNT]) {
        typename EpOne<OT, ACT>::State ep;
        EpOne<OT, ACT>::begin(P, m0, rows, nn, ep);
        EpOne<OT, ACT>::template finish<CNT>(P, m0, rows, nn, v, ep);
    }
    template <int OT, int CNT>
    static __device__ __forceinline__ void run_act(const Args &P, int64_t m0, int rows, int64_t nn,
                                                   const uint32_t (&v)[CNT]) {
        switch (P.act) {
        case AMP_ACT_GELU: return run<OT, AMP_ACT_GELU, CNT>(P, m0, rows, nn, v);
        case AMP_ACT_GELU_TANH: return run<OT, AMP_ACT_GELU_TANH, CNT>(P, m0, rows, nn, v);
        case AMP_ACT_SILU: return run<OT, AMP_ACT_SILU, CNT>(P, m0, rows, nn, v);
        default: return run<OT, kNoAct, CNT>(P, m0, rows, nn, v);
        }
    }
    template <int CNT>
    static __device__ __forceinline__ void finish(const Args &P, int64_t m0, int rows, int64_t nn,
                                                  const uint32_t (&v)[CNT], State &) {
        if (P.ot == kF32) run_act<kF32, CNT>(P, m0, rows, nn, v);
        else if (P.ot == kF16) run_act<kF16, CNT>(P, m0, rows, nn, v);
        else run_act<kBF16, CNT>(P, m0, rows, nn, v);
    }

    // Four neighbouring columns of one token; a warp holds 128, so 8 lanes a block.
    template <int OT>
    static __device__ __forceinline__ void four(const Args &P, int64_t m, int64_t nn, float (&z)[4]) {
        const int64_t k = m * P.n + nn;
        float r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            z[j] += bias_at<OT>(P, nn + j);
            r[j] = P.res && nn + j < P.n ? load_elem<OT>(P.res, k + j) : 0.0f;
        }
        if (P.q) {
            uint32_t b = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) b = max(b, __float_as_uint(z[j]) & 0x7FFFFFFFu);
#pragma unroll
            for (int o = 1; o < 8; o *= 2) b = max(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
            const uint32_t e = mx_scale_code<MxE4M3>(b);
            const float f = mx_unscale(e);
            const uint32_t c = f32x2_to_fp8x2_raw<kE4M3>(__fmul_rn(z[0], f), __fmul_rn(z[1], f)) |
                               (f32x2_to_fp8x2_raw<kE4M3>(__fmul_rn(z[2], f), __fmul_rn(z[3], f)) << 16);
            if (P.qpacked && nn < P.n) {
                *reinterpret_cast<uint32_t *>(P.q + k) = c;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (nn + j < P.n) P.q[k + j] = uint8_t(c >> (8 * j));
            }
            if (nn % kMxBlock == 0 && nn < P.n) P.s[m * P.kb + nn / kMxBlock] = uint8_t(e);
        }
        float2 a = make_float2(z[0], z[1]), b = make_float2(z[2], z[3]);
        if (P.act == AMP_ACT_GELU) {
            a = act_apply<OT, AMP_ACT_GELU, false>(a.x, a.y, 0.0f, 0.0f);
            b = act_apply<OT, AMP_ACT_GELU, false>(b.x, b.y, 0.0f, 0.0f);
        } else if (P.act == AMP_ACT_GELU_TANH) {
            a = act_apply<OT, AMP_ACT_GELU_TANH, false>(a.x, a.y, 0.0f, 0.0f);
            b = act_apply<OT, AMP_ACT_GELU_TANH, false>(b.x, b.y, 0.0f, 0.0f);
        } else if (P.act == AMP_ACT_SILU) {
            a = act_apply<OT, AMP_ACT_SILU, false>(a.x, a.y, 0.0f, 0.0f);
            b = act_apply<OT, AMP_ACT_SILU, false>(b.x, b.y, 0.0f, 0.0f);
        }
        const float y[4] = {a.x + r[0], a.y + r[1], b.x + r[2], b.y + r[3]};
        if (OT != kF32 && P.packed && nn + 4 <= P.n) {
            uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(P.out) + k);
            o[0] = f32x2_to_16x2<OT == kF32 ? kBF16 : OT>(y[0], y[1]);
            o[1] = f32x2_to_16x2<OT == kF32 ? kBF16 : OT>(y[2], y[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (nn + j < P.n) store_elem<OT>(P.out, k + j, y[j]);
        }
    }
    static __device__ __forceinline__ void finish4(const Args &P, int64_t m, int64_t nn, float (&z)[4]) {
        if (P.ot == kF32) four<kF32>(P, m, nn, z);
        else if (P.ot == kF16) four<kF16>(P, m, nn, z);
        else four<kBF16>(P, m, nn, z);
    }
    static __device__ __forceinline__ void saved_nan(const Args &P, int64_t m0, int cnt, int64_t nn) {
        scales_nan(P, m0, cnt, nn);
    }
};

}  // namespace
}  // namespace amp
