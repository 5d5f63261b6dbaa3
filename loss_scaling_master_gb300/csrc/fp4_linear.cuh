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
cudaError_t linear_pairs_error_take(int32_t *v, cudaStream_t s);

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

template <int OT, int ACT>
struct EpOne {
    using Args = Fp4Linear;
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
                                                  const uint32_t (&v)[CNT], State &ep, uint8_t *) {
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

// Eight neighbouring columns of one token, four lanes a block of the checkpoint.
template <int OT>
struct Eight {
    uint4 r[kWords8<OT>];  // the residual's
    // vec: the whole row is groups of eight, and aligned
    __device__ __forceinline__ void load(const Fp4Linear &P, bool in, int64_t k, int left) {
#pragma unroll
        for (int w = 0; w < kWords8<OT>; ++w) r[w] = make_uint4(0, 0, 0, 0);
        if (!P.res || !in) return;
        if (P.vec) {
#pragma unroll
            for (int w = 0; w < kWords8<OT>; ++w)
                r[w] = ld16(static_cast<const char *>(P.res) + k * (OT == kF32 ? 4 : 2) + 16 * w);
        } else {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = j < left ? load_elem<OT>(P.res, k + j) : 0.0f;
            f32_to_raw8<OT>(y, r);
        }
    }
    // z: with the bias, 0 where in is false or behind the last column (left: columns from here)
    template <int ACT>
    __device__ __forceinline__ void finish(const Fp4Linear &P, bool in, int64_t k, int left, int64_t scale_at,
                                           float (&z)[8]) const {
        if (P.q) {
            const uint32_t e = mx_scale_code<MxE4M3>(block_max8(z));
            const uint2 c = codes8(z, mx_unscale(e));
            if (in) {
                if (P.vec) {
                    *reinterpret_cast<uint2 *>(P.q + k) = c;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < left) P.q[k + j] = uint8_t((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
                }
                if ((threadIdx.x & 3) == 0) P.s[scale_at] = uint8_t(e);
            }
        }
        float y[8], b[8];
        raw8_to_f32<OT>(r, b);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float2 v = make_float2(z[j], z[j + 1]);
            if constexpr (ACT != kNoAct) v = act_apply<OT, ACT, false>(v.x, v.y, 0.0f, 0.0f);
            y[j] = v.x;
            y[j + 1] = v.y;
        }
        if (P.res) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += b[j];
        }
        if (!in) return;
        if (P.vec) {
            stv<OT>(P.out, k, y);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < left) store_elem<OT>(P.out, k + j, y[j]);
        }
    }
};

// For pairs of CTAs: 16 tokens at a time go through shared memory, so that a lane gets
// eight neighbouring columns: scales serve eight elements, and accesses are 16 bytes.
// (4096 x 8192 x 2048 bf16 with bias, GELU and checkpoint 51 us, a column a lane 82.)
// The rows of 36 floats keep both accesses free of bank conflicts.
template <int OT, int ACT>
struct EpStaged {
    using Args = Fp4Linear;
    static constexpr bool none = false;
    static constexpr int CH = 16, PITCH = 36, staged = CH * PITCH * 4;
    struct State {
        Eight<OT> e[2];
        float bias;
    };
    static __device__ __forceinline__ void residual(const Args &P, int64_t m0, int rows, int64_t nn, Eight<OT> (&e)[2]) {
        const int lane = threadIdx.x & 31;
        const int64_t c = nn - lane + 8 * (lane & 3);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = 8 * h + lane / 4;
            e[h].load(P, t < rows && c < P.n, int64_t(int(m0) + t) * int(P.n) + c, 8);
        }
    }
    static __device__ __forceinline__ void begin(const Args &P, int64_t m0, int rows, int64_t nn, State &ep) {
        ep.bias = bias_at<OT>(P, nn);
        residual(P, m0, rows, nn, ep.e);
    }
    template <int CNT>
    static __device__ __forceinline__ void finish(const Args &P, int64_t m0, int rows, int64_t nn,
                                                  const uint32_t (&v)[CNT], State &ep, uint8_t *mem) {
        float *stage = reinterpret_cast<float *>(mem);
        const int lane = threadIdx.x & 31;
        const int64_t c = nn - lane + 8 * (lane & 3);
#pragma unroll
        for (int s = 0; s < CNT; s += CH) {
            if (s >= rows) break;
            __syncwarp();  // the last tokens are read
#pragma unroll
            for (int i = 0; i < CH; ++i) stage[i * PITCH + lane] = __uint_as_float(v[s + i]) + ep.bias;
            __syncwarp();
            // 16-bit types: 16 tokens ahead (fp32 has no registers for that)
            Eight<OT> nxt[OT == kF32 ? 1 : 2];
            if constexpr (OT != kF32)
                if (s + CH < CNT) residual(P, m0 + s + CH, rows - s - CH, nn, nxt);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = 8 * h + lane / 4;
                const bool in = s + t < rows && c < P.n;
                const int m = int(m0) + s + t;
                const float4 *at = reinterpret_cast<const float4 *>(stage + t * PITCH + 8 * (lane & 3));
                const float4 a = at[0], b = at[1];
                float z[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                ep.e[h].template finish<ACT>(P, in, int64_t(m) * int(P.n) + c, 8,
                                             int64_t(m) * P.kb + int(c) / kMxBlock, z);
            }
            if (s + CH < CNT) {
                if constexpr (OT == kF32) {
                    residual(P, m0 + s + CH, rows - s - CH, nn, ep.e);
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
// every 16 tokens, and rows of any length.
struct EpAny {
    using Args = Fp4Linear;
    static constexpr bool none = false;
    static constexpr int CH = 16, PITCH = 36, staged = CH * PITCH * 4;
    struct State {};
    static __device__ __forceinline__ void begin(const Args &, int64_t, int, int64_t, State &) {}

    // 16 tokens from m0; stage: their z, a row of PITCH a token
    template <int OT, int ACT>
    static __device__ __forceinline__ void tokens(const Args &P, int64_t m0, int rows, int64_t c,
                                                  const float *stage, const Eight<OT> (&e)[2]) {
        const int lane = threadIdx.x & 31, left = int(min(int64_t(8), P.n - c));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = 8 * h + lane / 4;
            const float4 *at = reinterpret_cast<const float4 *>(stage + t * PITCH + 8 * (lane & 3));
            const float4 a = at[0], b = at[1];
            float z[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            e[h].template finish<ACT>(P, t < rows && left > 0, (m0 + t) * P.n + c, left, (m0 + t) * P.kb + c / kMxBlock,
                                      z);
        }
    }
    template <int OT>
    static __device__ __forceinline__ void run(const Args &P, int64_t m0, int rows, int64_t nn,
                                               const uint32_t (&v)[CH], float *stage) {
        const int lane = threadIdx.x & 31;
        const int64_t c = nn - lane + 8 * (lane & 3);
        Eight<OT> e[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = 8 * h + lane / 4;
            e[h].load(P, t < rows && c < P.n, (m0 + t) * P.n + c, int(min(int64_t(8), P.n - c)));
        }
        const float bias = bias_at<OT>(P, nn);
        __syncwarp();  // the last tokens are read
#pragma unroll
        for (int i = 0; i < CH; ++i) stage[i * PITCH + lane] = __uint_as_float(v[i]) + bias;
        __syncwarp();
        switch (P.act) {
        case AMP_ACT_GELU: return tokens<OT, AMP_ACT_GELU>(P, m0, rows, c, stage, e);
        case AMP_ACT_GELU_TANH: return tokens<OT, AMP_ACT_GELU_TANH>(P, m0, rows, c, stage, e);
        case AMP_ACT_SILU: return tokens<OT, AMP_ACT_SILU>(P, m0, rows, c, stage, e);
        default: return tokens<OT, kNoAct>(P, m0, rows, c, stage, e);
        }
    }
    template <int CNT>
    static __device__ __forceinline__ void finish(const Args &P, int64_t m0, int rows, int64_t nn,
                                                  const uint32_t (&v)[CNT], State &, uint8_t *mem) {
        static_assert(CNT == CH, "16 tokens");
        float *stage = reinterpret_cast<float *>(mem);
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
