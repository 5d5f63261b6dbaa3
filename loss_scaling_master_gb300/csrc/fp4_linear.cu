// fp4_linear.cu - a linear layer of two 4-bit block-scaled matrices with bias,
// activation and residual (fp4_linear.cuh) on the kernels of fp4_product.cuh; those of
// pairs of CTAs are compiled in fp4_linear_pair.cu.
#include "fp4_linear.cuh"

namespace amp {
namespace {

Launched g_launched;

// z = bias for an empty reduction: a warp takes 32 columns of 16 tokens.
__global__ void __launch_bounds__(kThreads) linear_empty_kernel(Fp4Linear P) {
    __shared__ __align__(16) uint8_t s_stage[kThreads / 32][EpAny<false>::staged];
    pdl_wait();
    pdl_trigger();
    const int64_t items = (int64_t(P.m) + 15) / 16 * P.kb;
    for (int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / 32; i < items;
         i += int64_t(gridDim.x) * (kThreads / 32)) {
        const int64_t m0 = i / P.kb * 16;
        const uint32_t zero[16] = {};
        EpAny<false>::State ep;
        EpAny<false>::finish<16>(P, m0, int(min(int64_t(16), P.m - m0)), i % P.kb * kMxBlock + (threadIdx.x & 31), zero, ep,
                          s_stage[threadIdx.x / 32]);
    }
}

}  // namespace

cudaError_t launch_fp4_linear(const void *a, const uint8_t *sa, const void *b, const uint8_t *sb, int64_t m, int64_t n,
                              int64_t k, const void *bias, int belem, int act, const void *res, void *out, int oelem,
                              uint8_t *q, uint8_t *sc, int device, cudaStream_t s, Fp4Limits limits) {
    Fp4Linear P{};
    describe(P, sa, sb, m, n, k, out, oelem, limits);
    P.bias = bias;
    P.res = res;
    P.q = q;
    P.s = sc;
    P.kb = int((n + kMxBlock - 1) / kMxBlock);
    P.bt = uint8_t(belem);
    P.act = uint8_t(act < 0 ? int(kNoAct) : act);
    P.rpacked = P.packed && (reinterpret_cast<uintptr_t>(res) & 3) == 0;
    const auto off = [](const void *p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
    P.vec = n % 8 == 0 && !off(out, 15) && !off(res, 15) && !off(q, 7);
    cudaError_t e;
    const int64_t row_bytes = (k + kMxBlock - 1) / kMxBlock * 16;
    if (k == 0) {
        const int64_t want = ((m + 15) / 16 * P.kb * 32 + kThreads - 1) / kThreads;
        e = launch_pdl(linear_empty_kernel, dim3(unsigned(std::min<int64_t>(want, 4096))), dim3(kThreads), 0, s, P);
    } else if (!takes_pairs(m, n, device)) {
        g_launched.mark(device);
        e = P.vec ? go_solo<EpAny<true>>(P, a, b, row_bytes, device, s)
                  : go_solo<EpAny<false>>(P, a, b, row_bytes, device, s);
    } else {
        e = linear_pairs(P, a, b, row_bytes, device, s);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t fp4_linear_error_take(int32_t *v, cudaStream_t s) {
    *v = 0;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess && g_launched.any(device)) e = error_take(v, s);
    int32_t pairs = 0;
    if (e == cudaSuccess) e = linear_pairs_error_take(&pairs, device, s);
    *v |= pairs;
    return e;
}

}  // namespace amp
