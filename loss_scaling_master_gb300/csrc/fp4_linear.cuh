// fp4_linear.cuh - what the kernels of fp4_product.cuh make of their accumulators in a
// linear layer:
//
//   z = A B^T + bias,  out = f(z) + residual (one rounding),  8-bit checkpoint of z
//
// A lane holds one column of C and consecutive tokens.  A bias and a residual are added so
// (EpOne): the residual comes in the layout in which store16 stores (two neighbouring
// elements of a row a lane, even lanes the even tokens) and is turned over by one shuffle
// for two elements; the words of the first 16 tokens (fp32: 8) are asked for before the
// accumulators are waited for, the others as many tokens ahead.  An activation and the checkpoint want
// neighbouring columns in a lane (Stage).
#pragma once

#include "act.cuh"
#include "fp4_product.cuh"

namespace amp {

struct Fp4Linear : Fp4Product {
    const void *bias, *res;
    uint8_t *q, *s;
    int kb;          // blocks of 32 columns
    uint8_t bt;      // ElemType of bias
    uint8_t act;     // amp_act or kNoAct
    uint8_t rpacked; // packed, and the residual 4-byte aligned too
    uint8_t vec;     // rows are whole groups of 8 elements, and every address is aligned for one
};

// The kernels of pairs of CTAs (fp4_linear_pair.cu), and that file's error word.
cudaError_t linear_pairs(const Fp4Linear &P, const void *a, const void *b, int64_t row_bytes, int device,
                         cudaStream_t s);
cudaError_t linear_pairs_error_take(int32_t *v, int device, cudaStream_t s);

namespace {

enum : int { kNoAct = 3 };  // after the three amp_act values

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

// A bias and a residual alone, added a column a lane as the columns come.
template <int OT>
struct EpOne {
    using Args = Fp4Linear;
    using Split = EpOne;
    static constexpr bool none = false;
    static constexpr int staged = 0;
    static constexpr int CH = OT == kF32 ? 8 : 16, WORDS = 8;
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

    // z + residual for two tokens, elements 2 i and 2 i + 1 of the residual's words
    static __device__ __forceinline__ float2 add(const Args &P, float z0, float z1, int i,
                                                 const uint32_t (&r)[WORDS]) {
        float2 y = make_float2(z0, z1);
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
    static __device__ __forceinline__ void pack(float2 y, int i, uint32_t (&o)[WORDS]) {
        if constexpr (OT == kF32) {
            o[2 * i] = __float_as_uint(y.x);
            o[2 * i + 1] = __float_as_uint(y.y);
        } else {
            o[i] = f32x2_to_16x2<OT>(y.x, y.y);
        }
    }
    static __device__ __forceinline__ void store(const Args &P, int64_t m0, int rows, int64_t nn,
                                                 const uint32_t (&o)[WORDS]) {
        if constexpr (OT == kF32) store32<CH>(P, m0, rows, nn, o);
        else store16<CH>(P, m0, rows, nn, o);
    }

    // ep: as begin() left it for the same place
    template <int CNT>
    static __device__ __forceinline__ void finish(const Args &P, int64_t m0, int rows, int64_t nn,
                                                  const uint32_t (&v)[CNT], State &ep, uint8_t *) {
#pragma unroll
        for (int c = 0; c < CNT; c += CH) {
            if (c >= rows) break;
            State nxt;
            if (P.res && c + CH < CNT) residual(P, m0 + c + CH, rows - c - CH, nn, nxt.r);
            uint32_t o[WORDS];
#pragma unroll
            for (int i = 0; i < CH / 2; ++i)
                pack(add(P, __uint_as_float(v[c + 2 * i]) + ep.bias, __uint_as_float(v[c + 2 * i + 1]) + ep.bias, i,
                         ep.r),
                     i, o);
            store(P, m0 + c, rows - c, nn, o);
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

// Eight neighbouring columns of one token, four lanes a block of the checkpoint.
template <int OT>
struct Eight {
    uint4 r[kWords8<OT>];  // the residual's (rows of whole groups of eight)
    __device__ __forceinline__ void load(const Fp4Linear &P, bool in, int64_t k) {
#pragma unroll
        for (int w = 0; w < kWords8<OT>; ++w) {
            r[w] = make_uint4(0, 0, 0, 0);
            if (P.res && in) r[w] = ld16(static_cast<const char *>(P.res) + k * (OT == kF32 ? 4 : 2) + 16 * w);
        }
    }
    // The checkpoint's codes of z (0 where `in` is false and behind the last column), its
    // scale stored; z becomes f(z).
    template <int ACT>
    static __device__ __forceinline__ uint2 apply(const Fp4Linear &P, bool in, int64_t scale_at, float (&z)[8]) {
        uint2 c = make_uint2(0, 0);
        if (P.q) {
            const uint32_t e = mx_scale_code<MxE4M3>(block_max8(z));
            c = codes8(z, mx_unscale(e));
            if (in && (threadIdx.x & 3) == 0) P.s[scale_at] = uint8_t(e);
        }
        if constexpr (ACT != kNoAct) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 v = act_apply<OT, ACT, false>(z[j], z[j + 1], 0.0f, 0.0f);
                z[j] = v.x;
                z[j + 1] = v.y;
            }
        }
        return c;
    }
    // out = y + residual, and the codes
    __device__ __forceinline__ void store(const Fp4Linear &P, bool in, int64_t k, float (&y)[8], uint2 c) const {
        if (P.res) {
            float b[8];
            raw8_to_f32<OT>(r, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += b[j];
        }
        if (!in) return;
        if (P.q) *reinterpret_cast<uint2 *>(P.q + k) = c;
        stv<OT>(P.out, k, y);
    }
};

// 16 tokens at a time through shared memory, so that a lane gets eight neighbouring columns:
// scales serve eight elements, and accesses are 16 bytes (4096 x 8192 x 2048 bf16 with bias,
// GELU and checkpoint 51 us, a column a lane 82).  Rows that are not whole groups of eight
// come back the same way, values and codes, to a column a lane (1000 x 2303 x 768 8.8 us,
// single elements eight a lane 24).  The rows of 36 floats keep the accesses free of bank
// conflicts.
struct Stage {
    static constexpr int CH = 16, PITCH = 36, bytes = CH * PITCH * 4 + CH * 32;
    float *z;
    uint8_t *codes;
    __device__ __forceinline__ explicit Stage(uint8_t *mem)
        : z(reinterpret_cast<float *>(mem)), codes(mem + CH * PITCH * 4) {}

    // the lane's two groups: tokens lane / 4 and 8 + lane / 4, columns from 8 (lane % 4)
    static __device__ __forceinline__ int64_t column(int64_t nn) {
        const int lane = threadIdx.x & 31;
        return nn - lane + 8 * (lane & 3);
    }
    template <int OT>
    static __device__ __forceinline__ void residual(const Fp4Linear &P, int64_t m0, int rows, int64_t nn,
                                                    Eight<OT> (&e)[2]) {
        const int64_t c = column(nn);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = 8 * h + (threadIdx.x & 31) / 4;
            e[h].load(P, t < rows && c < P.n, int64_t(int(m0) + t) * int(P.n) + c);
        }
    }
    __device__ __forceinline__ void put(const uint32_t (&v)[CH], float bias) const {
        __syncwarp();  // the last tokens are read
#pragma unroll
        for (int i = 0; i < CH; ++i) z[i * PITCH + (threadIdx.x & 31)] = __uint_as_float(v[i]) + bias;
        __syncwarp();
    }
    // VEC: rows of whole groups of eight.  PAIR: in the kernel of pairs of CTAs, whose
    // unrolled steps the others have no registers for.
    template <int OT, int ACT, bool VEC, bool PAIR>
    __device__ __forceinline__ void finish(const Fp4Linear &P, int64_t m0, int rows, int64_t nn,
                                           const Eight<OT> (&e)[2]) const {
        const int lane = threadIdx.x & 31;
        const int64_t c = column(nn);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = 8 * h + lane / 4, m = int(m0) + t;
            const bool in = t < rows && c < P.n;
            float4 *at = reinterpret_cast<float4 *>(z + t * PITCH + 8 * (lane & 3));
            const float4 a = at[0], b = at[1];
            float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            const uint2 code = Eight<OT>::template apply<ACT>(P, in, int64_t(m) * P.kb + int(c) / kMxBlock, y);
            if constexpr (VEC) {
                e[h].store(P, in, int64_t(m) * int(P.n) + c, y, code);
            } else {
                at[0] = make_float4(y[0], y[1], y[2], y[3]);
                at[1] = make_float4(y[4], y[5], y[6], y[7]);
                *reinterpret_cast<uint2 *>(codes + 32 * t + 8 * (lane & 3)) = code;
            }
        }
        if constexpr (VEC) return;
        __syncwarp();
        if constexpr (!PAIR) {
            const int64_t n = P.n;
            int64_t k = m0 * n + nn;
#pragma unroll 1
            for (int i0 = 0; i0 < min(rows, CH) && nn < n; i0 += 8, k += 8 * n) {
                float r[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = P.res && i0 + i < rows ? load_elem<OT>(P.res, k + i * n) : 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (i0 + i >= rows) break;
                    const float v = z[(i0 + i) * PITCH + lane];
                    store_elem<OT>(P.out, k + i * n, P.res ? v + r[i] : v);
                    if (P.q) P.q[k + i * n] = codes[32 * (i0 + i) + lane];
                }
            }
        } else {
            using One = EpOne<OT>;
#pragma unroll
            for (int h = 0; h < CH; h += One::CH) {
                uint32_t r[One::WORDS], o[One::WORDS];
                if (P.res) One::residual(P, m0 + h, rows - h, nn, r);
#pragma unroll
                for (int i = 0; i < One::CH / 2; ++i)
                    One::pack(One::add(P, z[(h + 2 * i) * PITCH + lane], z[(h + 2 * i + 1) * PITCH + lane], i, r), i, o);
                One::store(P, m0 + h, rows - h, nn, o);
            }
            if (P.q && nn < P.n) {
                uint8_t *at = P.q + m0 * P.n + nn;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    if (i < rows) *at = codes[32 * i + lane];
                    at += P.n;
                }
            }
        }
    }
};

// For pairs of CTAs.
template <int OT, int ACT, bool VEC>
struct EpStaged {
    using Args = Fp4Linear;
    using Split = EpStaged;
    static constexpr bool none = false;
    static constexpr int CH = Stage::CH, staged = Stage::bytes;
    struct State {
        Eight<OT> e[2];
        float bias;
    };
    static __device__ __forceinline__ void begin(const Args &P, int64_t m0, int rows, int64_t nn, State &ep) {
        ep.bias = bias_at<OT>(P, nn);
        if (VEC) Stage::residual(P, m0, rows, nn, ep.e);
    }
    template <int CNT>
    static __device__ __forceinline__ void finish(const Args &P, int64_t m0, int rows, int64_t nn,
                                                  const uint32_t (&v)[CNT], State &ep, uint8_t *mem) {
        const Stage stage(mem);
#pragma unroll
        for (int s = 0; s < CNT; s += CH) {
            if (s >= rows) break;
            uint32_t part[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) part[i] = v[s + i];
            stage.put(part, ep.bias);
            // 16-bit types: 16 tokens ahead (fp32 has no registers for that)
            Eight<OT> nxt[2];
            if constexpr (VEC && OT != kF32)
                if (s + CH < CNT) Stage::residual(P, m0 + s + CH, rows - s - CH, nn, nxt);
            stage.template finish<OT, ACT, VEC, true>(P, m0 + s, rows - s, nn, ep.e);
            if constexpr (VEC) {
                if (s + CH == CNT) break;
                if constexpr (OT == kF32) {
                    Stage::residual(P, m0 + s + CH, rows - s - CH, nn, ep.e);
                } else {
                    ep.e[0] = nxt[0];
                    ep.e[1] = nxt[1];
                }
            }
        }
    }
    static __device__ __forceinline__ void saved_nan(const Args &P, int64_t m0, int cnt, int64_t nn) {
        scales_nan(P, m0, cnt, nn);
    }
};

// For one CTA a tile: as EpStaged, with the element type and the activation looked up for
// every 16 tokens.
template <bool VEC>
struct EpAny {
    using Args = Fp4Linear;
    using Split = EpAny<true>;  // joining a cut reduction's parts looks up VEC itself
    static constexpr bool none = false;
    static constexpr int CH = Stage::CH, staged = Stage::bytes;
    struct State {};
    static __device__ __forceinline__ void begin(const Args &, int64_t, int, int64_t, State &) {}

    template <int OT>
    static __device__ __forceinline__ void run(const Args &P, int64_t m0, int rows, int64_t nn,
                                               const uint32_t (&v)[CH], const Stage &stage) {
        Eight<OT> e[2];
        if (VEC) Stage::residual(P, m0, rows, nn, e);
        stage.put(v, bias_at<OT>(P, nn));
        switch (P.act) {
        case AMP_ACT_GELU: return stage.finish<OT, AMP_ACT_GELU, VEC, false>(P, m0, rows, nn, e);
        case AMP_ACT_GELU_TANH: return stage.finish<OT, AMP_ACT_GELU_TANH, VEC, false>(P, m0, rows, nn, e);
        case AMP_ACT_SILU: return stage.finish<OT, AMP_ACT_SILU, VEC, false>(P, m0, rows, nn, e);
        default: return stage.finish<OT, kNoAct, VEC, false>(P, m0, rows, nn, e);
        }
    }
    template <int CNT>
    static __device__ __forceinline__ void finish(const Args &P, int64_t m0, int rows, int64_t nn,
                                                  const uint32_t (&v)[CNT], State &, uint8_t *mem) {
        static_assert(CNT == CH, "16 tokens");
        const Stage stage(mem);
        if (P.ot == kF32) run<kF32>(P, m0, rows, nn, v, stage);
        else if (P.ot == kF16) run<kF16>(P, m0, rows, nn, v, stage);
        else run<kBF16>(P, m0, rows, nn, v, stage);
    }

    // Four neighbouring columns of one token, for tiles whose reduction was cut (a warp
    // holds 128 columns, so 8 lanes a block of the checkpoint; eight columns a thread,
    // half of the threads idle, took 1.3 us longer at 48 x 4096 x 4096).
    template <int OT>
    static __device__ __forceinline__ void four(const Args &P, int64_t m, int64_t nn, float (&z)[4],
                                                const float (&bias)[4], const float (&r)[4]) {
        const int64_t k = m * P.n + nn;
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] += bias[j];
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
            if (P.vec && nn < P.n) {
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
    // The partial tiles of a cluster's CTAs in shared memory, [token][128 columns]: rank by
    // rank, so the order of the sum is fixed; one group's loads are issued together.
    template <int THREADS, int OT>
    static __device__ __forceinline__ void join_as(const Args &P, const uint32_t (&part)[kMaxParts], uint32_t parts,
                                                   uint32_t rank, int64_t m0, int64_t n0, int cols) {
        // a thread's columns stay: the step is whole rows of 32 groups
        const int l = 4 * (threadIdx.x % (kLanes / 4));
        const int64_t nn = n0 + l;
        float bias[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) bias[j] = bias_at<OT>(P, nn + j);
        for (int i = int(rank) * THREADS + int(threadIdx.x); i < cols * (kLanes / 4); i += int(parts) * THREADS) {
            const int t = i / (kLanes / 4);
            float4 v[kMaxParts];
            float r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[j] = P.res && nn + j < P.n ? load_elem<OT>(P.res, (m0 + t) * P.n + nn + j) : 0.0f;
#pragma unroll
            for (uint32_t q = 0; q < kMaxParts; ++q)
                if (q < parts) v[q] = cluster_ld4(part[q] + uint32_t(t * kLanes + l) * 4);
            float z[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (uint32_t q = 1; q < kMaxParts; ++q)
                if (q < parts) {
                    z[0] += v[q].x;
                    z[1] += v[q].y;
                    z[2] += v[q].z;
                    z[3] += v[q].w;
                }
            four<OT>(P, m0 + t, nn, z, bias, r);
        }
    }
    template <int THREADS>
    static __device__ __forceinline__ void join(const Args &P, const uint32_t (&part)[kMaxParts], uint32_t parts,
                                                uint32_t rank, int64_t m0, int64_t n0, int cols) {
        if (P.ot == kF32) join_as<THREADS, kF32>(P, part, parts, rank, m0, n0, cols);
        else if (P.ot == kF16) join_as<THREADS, kF16>(P, part, parts, rank, m0, n0, cols);
        else join_as<THREADS, kBF16>(P, part, parts, rank, m0, n0, cols);
    }
    static __device__ __forceinline__ void saved_nan(const Args &P, int64_t m0, int cnt, int64_t nn) {
        scales_nan(P, m0, cnt, nn);
    }
};

}  // namespace
}  // namespace amp
