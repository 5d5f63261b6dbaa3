// fp4_product.cu - C = A B^T of two 4-bit block-scaled matrices: the kernels of
// fp4_product.cuh with the accumulators stored as they are.
#include "fp4_product.cuh"

namespace amp {
namespace {

// C = 0 for an empty reduction.
__global__ void __launch_bounds__(kThreads) fp4_zero_kernel(uint8_t *out, int64_t bytes) {
    pdl_wait();
    pdl_trigger();
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < bytes; i += int64_t(gridDim.x) * kThreads)
        out[i] = 0;
}

}  // namespace

cudaError_t launch_fp4_product(const void *a, const uint8_t *sa, const void *b, const uint8_t *sb, int64_t m,
                               int64_t n, int64_t k, void *out, int oelem, int device, cudaStream_t s,
                               Fp4Limits limits) {
    cudaError_t e;
    if (k == 0) {
        const int64_t bytes = m * n * (oelem == kF32 ? 4 : 2);
        const int64_t want = (bytes + kThreads - 1) / kThreads;
        e = launch_pdl(fp4_zero_kernel, dim3(unsigned(std::min<int64_t>(want, 4096))), dim3(kThreads), 0, s,
                       static_cast<uint8_t *>(out), bytes);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    Fp4Product P{};
    describe(P, sa, sb, m, n, k, out, oelem, limits);
    const int64_t row_bytes = (k + kMxBlock - 1) / kMxBlock * 16;
    e = takes_pairs(m, n, device) ? go_pair<EpNone>(P, a, b, row_bytes, device, s)
                                  : go_solo<EpNone>(P, a, b, row_bytes, device, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t fp4_error_take(int32_t *v, cudaStream_t s) {
    int32_t linear = 0;
    cudaError_t e = error_take(v, s);
    if (e == cudaSuccess) e = fp4_linear_error_take(&linear, s);
    *v |= linear;
    return e;
}

}  // namespace amp
