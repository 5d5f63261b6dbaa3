// fp4_linear_pair.cu - the linear layer's kernels of pairs of CTAs (fp4_linear.cuh), one
// for each element type and activation.
#include "fp4_linear.cuh"

namespace amp {
namespace {

Launched g_launched;

// Pairs of CTAs: staged where there is something to compute, or a residual and a short
// reduction to hide it behind (bf16 with a residual, a column a lane and staged: 4096 x 8192
// x 2048 44.8 and 40.3 us, 4096 x 4096 x 4096 32.0 and 29.7, 8192 x 4096 x 8192 80.1 and
// 80.7); else a column a lane.
template <int OT, int ACT>
cudaError_t pair_act(const Fp4Linear &P, const void *a, const void *b, int64_t row_bytes, int device, cudaStream_t s) {
    if constexpr (ACT == kNoAct)
        if (!P.q && !(P.vec && P.res && P.k64 <= 64)) return go_pair<EpOne<OT>>(P, a, b, row_bytes, device, s);
    return P.vec ? go_pair<EpStaged<OT, ACT, true>>(P, a, b, row_bytes, device, s)
                 : go_pair<EpStaged<OT, ACT, false>>(P, a, b, row_bytes, device, s);
}
template <int OT>
cudaError_t pair_of(const Fp4Linear &P, const void *a, const void *b, int64_t row_bytes, int device, cudaStream_t s) {
    switch (P.act) {
    case AMP_ACT_GELU: return pair_act<OT, AMP_ACT_GELU>(P, a, b, row_bytes, device, s);
    case AMP_ACT_GELU_TANH: return pair_act<OT, AMP_ACT_GELU_TANH>(P, a, b, row_bytes, device, s);
    case AMP_ACT_SILU: return pair_act<OT, AMP_ACT_SILU>(P, a, b, row_bytes, device, s);
    default: return pair_act<OT, kNoAct>(P, a, b, row_bytes, device, s);
    }
}

}  // namespace

cudaError_t linear_pairs(const Fp4Linear &P, const void *a, const void *b, int64_t row_bytes, int device,
                         cudaStream_t s) {
    g_launched.mark(device);
    return P.ot == kF32   ? pair_of<kF32>(P, a, b, row_bytes, device, s)
           : P.ot == kF16 ? pair_of<kF16>(P, a, b, row_bytes, device, s)
                          : pair_of<kBF16>(P, a, b, row_bytes, device, s);
}

cudaError_t linear_pairs_error_take(int32_t *v, int device, cudaStream_t s) {
    return g_launched.any(device) ? error_take(v, s) : cudaSuccess;
}

}  // namespace amp
