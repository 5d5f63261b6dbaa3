// mx.cuh - the block formats of ampops.h: 32 elements with one E8M0 scale.
//
// The scale byte comes from the bits of the block's largest magnitude alone:
// with a = m * 2^p (1 <= m < 2) and M = M_m * 2^M_p the format's maximum, the
// smallest k with a <= M * 2^k is p - M_p, or one more if m > M_m.  Adding
// (2^23 - 1 - mantissa(M)) to a's bits carries into the exponent field exactly
// when mantissa(a) > mantissa(M), so e = field(bits + over) - M_p, clamped at
// 0 (a block whose maximum is below M * 2^-127).  Every scale is a power of
// two, so x * 2^(127-e) is exact and the conversion's is the only rounding.
#pragma once

#include "common.cuh"

namespace amp {

constexpr int kMxBlock = 32;

// e2m1: maximum 6 = 1.5 * 2^2 (mantissa 0x400000).
// e4m3: maximum 448 = 1.75 * 2^8 (mantissa 0x600000).
struct MxE2M1 {
    static constexpr uint32_t over = 0x3FFFFFu;
    static constexpr int low = 2;
};
struct MxE4M3 {
    static constexpr uint32_t over = 0x1FFFFFu;
    static constexpr int low = 8;
};

// Scale byte of a block from the fp32 bits of max |x| (NaN above inf above all).
template <class F>
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t abs_bits) {
    const int e = max(int((abs_bits + F::over) >> 23) - F::low, 0);
    return abs_bits >= 0x7F800000u ? 255u : uint32_t(e);
}
// 2^(127 - e) for e <= 253; -inf for 255, whose codes mean nothing.
__device__ __forceinline__ float mx_unscale(uint32_t e) { return __uint_as_float((254u - e) << 23); }
// 2^(e - 127), subnormal for e = 0, NaN for e = 255.
__device__ __forceinline__ float mx_scale(uint32_t e) {
    uint32_t b = e == 0 ? 0x00400000u : e << 23;
    return __uint_as_float(e == 255u ? 0x7FC00000u : b);
}

// Of two pairs of f16 or bf16, the larger magnitude each; its sign bit means
// nothing, and a NaN wins.
template <int XT>
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (XT == kF16) asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two fp32 -> one byte of two e2m1 codes (lo in bits 0-3), RNE.  Only values
// of magnitude at most 6 matter.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
        "cvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
// Eight fp32 -> four bytes of e2m1 codes, element 0 in bits 0-3.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&y)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}
// Four e2m1 codes (the low half of w), or eight -> fp32 values.
__device__ __forceinline__ void e2m1x4_to_f32x4(uint32_t w, float *y) {
    uint32_t h0, h1;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(w));
    y[0] = f16_bits_to_f32(h0 & 0xFFFFu);
    y[1] = f16_bits_to_f32(h0 >> 16);
    y[2] = f16_bits_to_f32(h1 & 0xFFFFu);
    y[3] = f16_bits_to_f32(h1 >> 16);
}
__device__ __forceinline__ void e2m1x8_to_f32x8(uint32_t w, float (&y)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[2 * j] = f16_bits_to_f32(h[j] & 0xFFFFu);
        y[2 * j + 1] = f16_bits_to_f32(h[j] >> 16);
    }
}
// Four e4m3 codes (one word) -> fp32 values.
__device__ __forceinline__ void e4m3x4_to_f32x4(uint32_t w, float *y) {
    uint32_t h0, h1;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(w));
    y[0] = f16_bits_to_f32(h0 & 0xFFFFu);
    y[1] = f16_bits_to_f32(h0 >> 16);
    y[2] = f16_bits_to_f32(h1 & 0xFFFFu);
    y[3] = f16_bits_to_f32(h1 >> 16);
}

// 8 consecutive elements held as raw words (one uint4 for 16-bit types, two
// for fp32) <-> fp32.
template <int XT>
constexpr int kWords8 = XT == kF32 ? 2 : 1;

template <int XT>
__device__ __forceinline__ void raw8_to_f32(const uint4 *u, float (&y)[8]) {
    if constexpr (XT == kF32) {
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __uint_as_float(w[j]);
    } else {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (XT == kBF16) {
                y[2 * j] = __uint_as_float(w[j] << 16);
                y[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            } else {
                y[2 * j] = f16_bits_to_f32(w[j] & 0xFFFFu);
                y[2 * j + 1] = f16_bits_to_f32(w[j] >> 16);
            }
        }
    }
}

// Two fp32 -> two elements of a 16-bit type in one word (RNE).
template <int XT>
__device__ __forceinline__ uint32_t f32x2_to_16x2(float lo, float hi) {
    uint32_t r;
    if constexpr (XT == kBF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int XT>
__device__ __forceinline__ void f32_to_raw8(const float (&y)[8], uint4 *u) {
    if constexpr (XT == kF32) {
        u[0] = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                          __float_as_uint(y[3]));
        u[1] = make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]),
                          __float_as_uint(y[7]));
    } else {
        u[0] = make_uint4(f32x2_to_16x2<XT>(y[0], y[1]), f32x2_to_16x2<XT>(y[2], y[3]),
                          f32x2_to_16x2<XT>(y[4], y[5]), f32x2_to_16x2<XT>(y[6], y[7]));
    }
}

// One element of a type at index k.
template <int XT>
__device__ __forceinline__ float load_elem(const void *x, int64_t k) {
    if constexpr (XT == kF32) return static_cast<const float *>(x)[k];
    else return lowp_to_f32<XT>(static_cast<const uint16_t *>(x)[k]);
}
template <int XT>
__device__ __forceinline__ void store_elem(void *x, int64_t k, float v) {
    if constexpr (XT == kF32) static_cast<float *>(x)[k] = v;
    else static_cast<uint16_t *>(x)[k] = uint16_t(f32x2_to_16x2<XT>(v, 0.0f) & 0xFFFFu);
}

// Items 0 .. rows * per_row - 1 taken `step` apart (a grid's worth, so below
// 2^32): an item's row and place in it, by 32-bit divisions at the start and
// additions from then on.
struct RowWalk {
    int64_t row;
    int at, step_row, step_at, per_row;
    __device__ __forceinline__ RowWalk(uint32_t first, uint32_t step, int per_row_) : per_row(per_row_) {
        const uint32_t r = first / uint32_t(per_row), s = step / uint32_t(per_row);
        row = r;
        at = int(first - r * uint32_t(per_row));
        step_row = int(s);
        step_at = int(step - s * uint32_t(per_row));
    }
    __device__ __forceinline__ void next() {
        row += step_row;
        at += step_at;
        if (at >= per_row) {
            at -= per_row;
            ++row;
        }
    }
};

}  // namespace amp
