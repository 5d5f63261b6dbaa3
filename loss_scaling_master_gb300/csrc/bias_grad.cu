// bias_grad.cu - the gradient of a bias, alone or with that of the activation that
// follows it (from the 8-bit checkpoint of the activation's input):
//
//   dz = dy f'(zh)  (or dz = dy),   db = sum over rows dz
//
// dy and the checkpoint are read once and dz is written once; the sums are of dz as
// computed, before its rounding.  See column_sums.cuh.
#include "act.cuh"
#include "column_sums.cuh"
#include "internal.h"

namespace amp {
namespace {

enum : int { kNoAct = 3 };  // after the three amp_act values

struct BiasBwd {
    const void *dy;
    const uint8_t *q, *s;
    void *dz, *db;
    int64_t rows, cols;
    int kb, otype;
};

template <int XT, int ACT, class S>
__global__ void __launch_bounds__(S::threads, S::ctas) bias_bwd_kernel(BiasBwd P) {
    constexpr bool VEC = S::each == 8;
    static_assert(!VEC || XT == kF32, "16-bit ones by bias_bwd_ring_kernel");
    // Elements a thread and row, and rows a step, as many as 64 registers hold (8192 x 2048
    // fp32: the sums alone 2, 4, 8 rows 9.0, 7.8, 18 us, with GELU 2, 3 rows 29.2, 33.8).
    constexpr int N = VEC ? 8 : 1, U = !VEC ? 8 : ACT == kNoAct ? 4 : 2;
    pdl_wait();
    pdl_trigger();
    const SumShare<S> at(P.rows);
    const int64_t c = at.col0 + int(threadIdx.x) % S::across * N;
    const bool in = c < P.cols;
    float a[N];
#pragma unroll
    for (int j = 0; j < N; ++j) a[j] = 0.0f;
    for (int64_t r0 = at.row0 + int(threadIdx.x) / S::across; in && r0 < at.row1; r0 += U * S::groups) {
        if constexpr (VEC) {
            uint4 g[U][kWords8<XT>];
            uint2 q[U];
            uint32_t e[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + u * S::groups, k = r * P.cols + c;
                if (r >= at.row1) break;
#pragma unroll
                for (int w = 0; w < kWords8<XT>; ++w)
                    g[u][w] = ld16(static_cast<const char *>(P.dy) + k * (XT == kF32 ? 4 : 2) + 16 * w);
                if (ACT != kNoAct) {
                    q[u] = *reinterpret_cast<const uint2 *>(P.q + k);
                    e[u] = P.s[r * P.kb + c / kMxBlock];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + u * S::groups, k = r * P.cols + c;
                if (r >= at.row1) break;
                float y[8];
                raw8_to_f32<XT>(g[u], y);
                if constexpr (ACT != kNoAct) {
                    float x[8];
                    values8(q[u], mx_scale(e[u]), x);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        float2 dz, unused;
                        act_grads<XT, ACT, false>(x[j], x[j + 1], 0.0f, 0.0f, y[j], y[j + 1], dz, unused);
                        y[j] = dz.x;
                        y[j + 1] = dz.y;
                    }
                    stv<XT>(P.dz, k, y);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] += y[j];
            }
        } else {
            float g[U];
            uint32_t q[U], e[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + u * S::groups, k = r * P.cols + c;
                g[u] = 0.0f;
                q[u] = e[u] = 0;
                if (r >= at.row1) continue;
                g[u] = load_elem<XT>(P.dy, k);
                if (ACT != kNoAct) {
                    q[u] = P.q[k];
                    e[u] = P.s[r * P.kb + c / kMxBlock];
                }
            }
#pragma unroll
            for (int u = 0; u < U; u += 2) {
                float2 dz = make_float2(g[u], g[u + 1]);
                if constexpr (ACT != kNoAct) {
                    float x[4];
                    float2 unused;
                    e4m3x4_to_f32x4(q[u] | (q[u + 1] << 8), x);
                    act_grads<XT, ACT, false>(__fmul_rn(x[0], mx_scale(e[u])), __fmul_rn(x[1], mx_scale(e[u + 1])),
                                              0.0f, 0.0f, g[u], g[u + 1], dz, unused);
                }
                const int64_t r = r0 + u * S::groups, k = r * P.cols + c;
                if (r < at.row1) {
                    if (ACT != kNoAct) store_elem<XT>(P.dz, k, dz.x);
                    a[0] += dz.x;
                }
                if (r + S::groups < at.row1) {
                    if (ACT != kNoAct) store_elem<XT>(P.dz, k + S::groups * P.cols, dz.y);
                    a[0] += dz.y;
                }
            }
        }
    }
    sum_join<S>(at, P.cols, a, P.db, P.otype);
}

// 16-bit rows of whole groups come ahead through shared memory; a block's scale, read by a
// plain load, one row ahead.  (16384 x 5120 bf16 with GELU, 2, 3, 4, 6 rows: 76, 76, 81,
// 124 us, the last by three CTAs an SM; by registers, three rows at once, 79.3.  The sums
// alone, 16384 x 768, 3, 4, 6, 8 rows: 5.5, 5.2, 5.7, 5.6; eight by registers 5.9.)
constexpr int kRingShared = 100;  // KB an SM: 4 CTAs of 17 or 21
template <int XT, int ACT, class S>
__global__ void __launch_bounds__(S::threads, S::ctas) bias_bwd_ring_kernel(BiasBwd P) {
    static_assert(XT != kF32);
    constexpr bool DO = ACT != kNoAct;
    constexpr int AHEAD = DO ? 2 : 4;
    __shared__ uint4 s_dy[AHEAD][S::threads];
    __shared__ uint2 s_q[DO ? AHEAD : 1][DO ? S::threads : 1];
    pdl_wait();
    pdl_trigger();
    const SumShare<S> at(P.rows);
    const int64_t c = at.col0 + int(threadIdx.x) % S::across * 8, hop = S::groups * P.cols;
    const int64_t r0 = at.row0 + int(threadIdx.x) / S::across, end = c < P.cols ? at.row1 * P.cols : 0;
    int64_t k = r0 * P.cols + c;
    const uint8_t *sc = DO ? P.s + r0 * P.kb + c / kMxBlock : nullptr;
    const int64_t sc_hop = int64_t(S::groups) * P.kb;
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = 0.0f;
    const auto ask = [&](int64_t at_k, int slot) {
        if (at_k < end) {
            copy_ahead<16>(&s_dy[slot][threadIdx.x], static_cast<const char *>(P.dy) + 2 * at_k);
            if (DO) copy_ahead<8>(&s_q[DO ? slot : 0][DO ? threadIdx.x : 0], P.q + at_k);
        }
        copies_of_row();
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) ask(k + i * hop, i);
    uint32_t e_next = DO && k < end ? *sc : 0;
    for (int slot = 0; k < end; k += hop) {
        const uint32_t e = e_next;
        if (DO && k + hop < end) e_next = *(sc += sc_hop);
        copies_wait<AHEAD - 1>();
        const uint4 g[1] = {s_dy[slot][threadIdx.x]};
        float y[8];
        raw8_to_f32<XT>(g, y);
        if constexpr (DO) {
            float x[8];
            values8(s_q[slot][threadIdx.x], mx_scale(e), x);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float2 dz, unused;
                act_grads<XT, ACT, false>(x[j], x[j + 1], 0.0f, 0.0f, y[j], y[j + 1], dz, unused);
                y[j] = dz.x;
                y[j + 1] = dz.y;
            }
            stv<XT>(P.dz, k, y);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += y[j];
        ask(k + AHEAD * hop, slot);
        slot = slot + 1 == AHEAD ? 0 : slot + 1;
    }
    sum_join<S>(at, P.cols, a, P.db, P.otype);
}

template <int XT, int ACT>
struct BiasFlat {
    const BiasBwd &P;
    int64_t all;
    struct Raw {
        RawGroup<XT> g;
        uint2 q;
    };
    __device__ __forceinline__ Raw load(int64_t g, bool whole) const {
        Raw r;
        r.g.load(P.dy, g, whole, all);
        r.q = make_uint2(0, 0);
        if constexpr (ACT != kNoAct) {
            if (whole) {
                r.q = *reinterpret_cast<const uint2 *>(P.q + 8 * g);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t b = 8 * g + j < all ? P.q[8 * g + j] : 0u;
                    if (j < 4) r.q.x |= b << (8 * j);
                    else r.q.y |= b << (8 * (j - 4));
                }
            }
        }
        return r;
    }
    // c: column of element 0; elements before column 0 or behind the last one count for nothing
    __device__ __forceinline__ void values(const Raw &raw, int64_t, int64_t r, int64_t c, float (&y)[8]) const {
        raw8_to_f32<XT>(raw.g.u, y);
        if constexpr (ACT != kNoAct) {
            // 8 elements lie in at most two blocks
            const int64_t c0 = max(c, int64_t(0)), b0 = c0 / kMxBlock, b1 = min(c + 7, P.cols - 1) / kMxBlock;
            const float s0 = mx_scale(P.s[r * P.kb + b0]), s1 = mx_scale(P.s[r * P.kb + b1]);
            float x[8];
            e4m3x4_to_f32x4(raw.q.x, x);
            e4m3x4_to_f32x4(raw.q.y, x + 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(x[j], c + j < (b0 + 1) * kMxBlock ? s0 : s1);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float2 dz, unused;
                act_grads<XT, ACT, false>(x[j], x[j + 1], 0.0f, 0.0f, y[j], y[j + 1], dz, unused);
                y[j] = dz.x;
                y[j + 1] = dz.y;
            }
        }
    }
    __device__ __forceinline__ void store(int64_t g, int lo, int hi, const float (&y)[8]) const {
        if constexpr (ACT != kNoAct) store_group<XT>(P.dz, g, lo, hi, y);
    }
};
template <int XT, int ACT>
__global__ void __launch_bounds__(SumFlat::threads, SumFlat::ctas) bias_bwd_flat_kernel(BiasBwd P) {
    pdl_wait();
    pdl_trigger();
    const SumShare<SumFlat> at(P.rows);
    BiasFlat<XT, ACT> op{P, P.rows * P.cols};
    flat_sums(at, P.rows, P.cols, op, P.db, P.otype);
}

template <int XT, int ACT>
cudaError_t go(const BiasBwd &P, bool aligned, int dev, cudaStream_t s) {
    if (!aligned) return launch_sums<SumElem, &bias_bwd_kernel<XT, ACT, SumElem>>(P.rows, P.cols, dev, s, P);
    // the activations' longer way to a group's values needs CTAs enough to hide it (2047 x
    // 1111 bf16 GELU 13.3 us, by single elements 10.4; 16383 x 5121 198 and 383)
    if (P.cols % 8 && (ACT == kNoAct || !narrow_tiles(P.cols, dev)))
        return launch_sums<SumFlat, &bias_bwd_flat_kernel<XT, ACT>>(P.rows, P.cols, dev, s, P);
    if (P.cols % 8) return launch_sums<SumElem, &bias_bwd_kernel<XT, ACT, SumElem>>(P.rows, P.cols, dev, s, P);
    if constexpr (XT == kF32)
        return launch_sums<SumVec<32>, &bias_bwd_kernel<XT, ACT, SumVec<32>>>(P.rows, P.cols, dev, s, P);
    else if (narrow_tiles(P.cols, dev))
        return launch_sums<SumVec<32>, &bias_bwd_ring_kernel<XT, ACT, SumVec<32>>, kRingShared>(P.rows, P.cols, dev, s, P);
    else
        return launch_sums<SumVec<64>, &bias_bwd_ring_kernel<XT, ACT, SumVec<64>>, kRingShared>(P.rows, P.cols, dev, s, P);
}
template <int XT>
cudaError_t go_x(const BiasBwd &P, int act, bool aligned, int dev, cudaStream_t s) {
    switch (act) {
    case AMP_ACT_GELU: return go<XT, AMP_ACT_GELU>(P, aligned, dev, s);
    case AMP_ACT_GELU_TANH: return go<XT, AMP_ACT_GELU_TANH>(P, aligned, dev, s);
    case AMP_ACT_SILU: return go<XT, AMP_ACT_SILU>(P, aligned, dev, s);
    default: return go<XT, kNoAct>(P, aligned, dev, s);
    }
}

}  // namespace

cudaError_t launch_bias_bwd(int act, const void *dy, int elem, int64_t rows, int64_t cols, const uint8_t *q,
                            const uint8_t *sc, void *dz, void *db, int dbelem, int device, cudaStream_t s) {
    const BiasBwd P{dy, q, sc, dz, db, rows, cols, int((cols + kMxBlock - 1) / kMxBlock), dbelem};
    const auto off = [](const void *p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
    const bool aligned = !off(dy, 15) && !off(dz, 15) && !off(q, 7);
    const int a = act < 0 ? int(kNoAct) : act;
    const cudaError_t e = elem == kF32   ? go_x<kF32>(P, a, aligned, device, s)
                          : elem == kF16 ? go_x<kF16>(P, a, aligned, device, s)
                                         : go_x<kBF16>(P, a, aligned, device, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace amp
