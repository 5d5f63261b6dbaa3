// fp4_product.cu - C = A B^T of two 4-bit block-scaled matrices on the
// tensor cores (tcgen05.mma kind::mxf4, E8M0 scales over blocks of 32).
//
//   C[i,j] = sum_k A[i,k] B[j,k],  fp32 accumulators, one rounding at the end
//
// Orientation.  The rows of B (the columns of C, a weight's outputs) go on the
// 128 lanes of tensor memory and the rows of A (tokens) on its columns: lanes
// are then consecutive elements of a row of C, and few tokens only narrow the
// instruction (N = 16, 32, 64) instead of leaving lanes empty.
//
// Pipeline.  One warp's thread loads (tensor-map loads of 128 bytes = 256
// elements a row, plain bulk copies of the scale tiles, whose layout is already
// the one the copy to tensor memory takes), one issues the scale copies and the
// products, four warps read finished accumulators and store.  Stages are handed
// over with mbarriers.  CTAs stay and walk tiles.
//
// Few tiles.  Where the tiles of C do not fill the GPU, the reduction axis is
// cut over the CTAs of a cluster; each leaves its fp32 partial tile in shared
// memory and the cluster's CTAs add them, rank by rank, from there (so the
// order of the sum is fixed and nothing goes through global memory).
//
// Every wait gives up after a second of GPU time: the thread sets the error
// word, the others see the CTA's flag, copies in flight are waited for, tensor
// memory is freed, and the kernel returns.
#include <cudaTypedefs.h>

#include <algorithm>

#include "internal.h"
#include "mx.cuh"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace amp {
namespace {

__device__ int32_t g_fp4_error;

constexpr int kLanes = 128;        // rows of B a tile
constexpr int kStageBytes = 128;   // bytes of a row a stage: 256 elements
constexpr int kProductThreads = 256;

struct Fp4Product {
    const uint8_t *sa, *sb;  // scale tiles of A and B
    void *out;
    int64_t m, n;
    int ot;             // ElemType of out
    int kt;             // scale tiles (128 elements) along the reduction
    int k64;            // products of 64 along the reduction
    int tiles_m, tiles_n;
};

template <int BN>
struct Shape {
    static constexpr int tok_tiles = BN > 128 ? BN / 128 : 1;  // scale tiles along the tokens
    static constexpr int w_bytes = kLanes * kStageBytes;
    static constexpr int t_bytes = BN * kStageBytes;
    static constexpr int t_room = (t_bytes + 1023) / 1024 * 1024;
    static constexpr int stage = w_bytes + t_room + 1024 + 1024 * tok_tiles;
    static constexpr int stages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
    static constexpr int acc_bufs = BN == 256 ? 1 : 2;
    static constexpr int sf_cols = 8 + 8 * tok_tiles;  // columns of a stage's scales
    static constexpr int sf_base = BN * acc_bufs < 32 ? 32 : BN * acc_bufs;
    static constexpr int tmem_cols = sf_base + stages * sf_cols > 256 ? 512 : 256;
    static_assert(sf_base + stages * sf_cols <= 512, "tensor memory");
    static constexpr int smem = stages * stage + 1024;  // and the alignment to 1024
};

template <int OT>
__device__ __forceinline__ void store_chunk(const Fp4Product &P, int64_t m0, int64_t nn, int cols,
                                            const float *v) {
    if (nn >= P.n) return;
#pragma unroll
    for (int c = 0; c < 16; ++c)
        if (c < cols) store_elem<OT>(P.out, (m0 + c) * P.n + nn, v[c]);
}

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kProductThreads, 1)
    fp4_product_kernel(const __grid_constant__ CUtensorMap map_t, const __grid_constant__ CUtensorMap map_w,
                       Fp4Product P) {
    using S = Shape<BN>;
    constexpr int NS = S::stages, NA = S::acc_bufs;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], empty[NS], acc_full[NA], acc_empty[NA], drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_fail;
    uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 128);
        }
        mbar_init(&drain, 1);
        s_fail = 0;
        mbar_fence_init();
        tma_prefetch_map(&map_t);
        tma_prefetch_map(&map_w);
    }
    if (warp == 2) tmem_alloc<S::tmem_cols>(&s_tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    pdl_trigger();

    // this CTA's tiles and its share of the reduction (in stages of 256)
    const int tiles = P.tiles_m * P.tiles_n;
    const uint32_t rank = SPLIT ? cluster_rank() : 0;
    uint32_t parts = 1;
    if (SPLIT) asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
    const int stride = SPLIT ? tiles : int(gridDim.x);
    const int first = SPLIT ? int(blockIdx.x / parts) : int(blockIdx.x);
    const int ks_all = (P.kt + 1) / 2;
    const int ks0 = int(int64_t(ks_all) * rank / parts), ks1 = int(int64_t(ks_all) * (rank + 1) / parts);
    // tile -> (token tile, output tile): 16 output tiles side by side, so the
    // CTAs that run together share operands in L2
    auto where = [&](int tile, int &tm, int &tn) {
        const int per = 16 * P.tiles_m, g = tile / per, in = tile - g * per;
        const int w = min(16, P.tiles_n - 16 * g);
        tm = in / w;
        tn = 16 * g + in % w;
    };
    auto give_up = [&]() {
        s_fail = 1;
        g_fp4_error = 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            int st = 0;
            uint32_t ph = 0;
            int issued = 0;
            for (int tile = first; tile < tiles && !s_fail; tile += stride) {
                int tm, tn;
                where(tile, tm, tn);
                for (int ks = ks0; ks < ks1; ++ks) {
                    if (!mbar_wait(&empty[st], ph ^ 1)) {
                        give_up();
                        break;
                    }
                    uint8_t *b = smem + st * S::stage;
                    const int na = min(2, P.kt - 2 * ks);
                    const int tt = BN > 128 ? min(S::tok_tiles, int((P.m + 127) / 128) - tm * S::tok_tiles) : 1;
                    mbar_arrive_expect_tx(&full[st], S::w_bytes + S::t_bytes + uint32_t(na) * 512u * uint32_t(1 + tt));
                    tma_load_2d(b, &map_w, ks * kStageBytes, tn * kLanes, &full[st]);
                    tma_load_2d(b + S::w_bytes, &map_t, ks * kStageBytes, tm * BN, &full[st]);
                    uint8_t *sf = b + S::w_bytes + S::t_room;
                    bulk_g2s(sf, P.sb + (int64_t(tn) * P.kt + 2 * ks) * 512, na * 512, &full[st]);
                    for (int h = 0; h < tt; ++h)
                        bulk_g2s(sf + 1024 + 1024 * h,
                                 P.sa + ((int64_t(tm) * S::tok_tiles + h) * P.kt + 2 * ks) * 512, na * 512,
                                 &full[st]);
                    ++issued;
                    if (++st == NS) {
                        st = 0;
                        ph ^= 1;
                    }
                    if (s_fail) break;
                }
            }
            if (s_fail) {  // wait for the copies still in flight
                for (int i = 0; i < min(issued, NS); ++i) {
                    st = st == 0 ? NS - 1 : st - 1;
                    if (st == NS - 1) ph ^= 1;
                    mbar_wait(&full[st], ph);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int st = 0, ab = 0;
            uint32_t ph = 0, aph = 0;
            constexpr uint32_t instr = mxf4_instr(kLanes, BN);
            bool ok = true;
            for (int tile = first; tile < tiles && ok && !s_fail; tile += stride) {
                ok = mbar_wait(&acc_empty[ab], aph ^ 1);
                tc_fence_after();
                const uint32_t acc = tmem + ab * BN;
                for (int ks = ks0; ks < ks1 && ok; ++ks) {
                    ok = mbar_wait(&full[st], ph);
                    if (!ok || s_fail) break;
                    tc_fence_after();
                    const uint32_t b = smem_addr(smem + st * S::stage);
                    const uint32_t sf = b + S::w_bytes + S::t_room;
                    const uint32_t tw = tmem + S::sf_base + st * S::sf_cols, tt = tw + 8;
                    const int na = min(2, P.kt - 2 * ks);
                    for (int a = 0; a < na; ++a) {
                        copy_scales(tw + 4 * a, scale_desc(sf + 512 * a));
#pragma unroll
                        for (int h = 0; h < S::tok_tiles; ++h)
                            copy_scales(tt + 4 * (a * S::tok_tiles + h), scale_desc(sf + 1024 + 1024 * h + 512 * a));
                    }
                    const uint64_t dw = operand_desc(b), dt = operand_desc(b + S::w_bytes);
                    const int nj = min(4, P.k64 - 4 * ks);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < nj)
                            mma_mxf4(acc, dw + 2 * j, dt + 2 * j, instr | mxf4_half(j & 1), tw + 4 * (j / 2),
                                     tt + 4 * (j / 2) * S::tok_tiles, ks > ks0 || j > 0);
                    tc_commit(&empty[st]);
                    if (++st == NS) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                tc_commit(&acc_full[ab]);
                if (++ab == NA) {
                    ab = 0;
                    aph ^= 1;
                }
            }
            if (!ok) give_up();
            if (s_fail) {  // wait for the products still in flight
                tc_commit(&drain);
                mbar_wait(&drain, 0);
            }
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3;
        int ab = 0;
        uint32_t aph = 0;
        for (int tile = first; tile < tiles; tile += stride) {
            int tm, tn;
            where(tile, tm, tn);
            bool ok = mbar_wait(&acc_full[ab], aph);
            if (!__all_sync(0xFFFFFFFFu, ok && !s_fail)) {
                if (!ok) give_up();
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ab * BN + (uint32_t(32 * quarter) << 16);
            const int64_t nn = int64_t(tn) * kLanes + 32 * quarter + lane, m0 = int64_t(tm) * BN;
            const int cols = int(min(int64_t(BN), P.m - m0));
#pragma unroll 1
            for (int c = 0; c < BN; c += 16) {
                if (c >= cols) break;
                uint32_t v[16];
                tmem_ld16(acc + c, v);
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]);
                if (SPLIT) {
                    // partial tile [column][lane] over the stages' buffers: every
                    // product of this CTA has finished reading them
                    float *part = reinterpret_cast<float *>(smem);
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(c + i) * kLanes + 32 * quarter + lane] = f[i];
                } else if (P.ot == kF32) {
                    store_chunk<kF32>(P, m0 + c, nn, cols - c, f);
                } else if (P.ot == kF16) {
                    store_chunk<kF16>(P, m0 + c, nn, cols - c, f);
                } else {
                    store_chunk<kBF16>(P, m0 + c, nn, cols - c, f);
                }
            }
            tc_fence_before();
            mbar_arrive(&acc_empty[ab]);
            if (++ab == NA) {
                ab = 0;
                aph ^= 1;
            }
        }
    }

    if constexpr (SPLIT) {
        __syncwarp();
        cluster_sync();  // every CTA's partial tile is written
        int tm, tn;
        where(first, tm, tn);
        const int64_t m0 = int64_t(tm) * BN;
        const int cols = int(min(int64_t(BN), P.m - m0));
        const uint32_t part = smem_addr(smem);
        const int l = threadIdx.x & 127;
        const int64_t nn = int64_t(tn) * kLanes + l;
        if (nn < P.n) {
            // columns go round the CTAs and their two halves of threads
            for (int c = int(rank) * 2 + (threadIdx.x >> 7); c < cols; c += 2 * int(parts)) {
                float v = 0.0f;
                for (uint32_t r = 0; r < parts; ++r) v += cluster_ld(part + (c * kLanes + l) * 4, r);
                const int64_t k = (m0 + c) * P.n + nn;
                if (P.ot == kF32) store_elem<kF32>(P.out, k, v);
                else if (P.ot == kF16) store_elem<kF16>(P.out, k, v);
                else store_elem<kBF16>(P.out, k, v);
            }
        }
        cluster_sync();  // nobody leaves while its shared memory is read
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_free<S::tmem_cols>(tmem);
}

// C = 0 for an empty reduction.
__global__ void __launch_bounds__(kThreads) fp4_zero_kernel(uint8_t *out, int64_t bytes) {
    pdl_wait();
    pdl_trigger();
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < bytes; i += int64_t(gridDim.x) * kThreads)
        out[i] = 0;
}

// cuTensorMapEncodeTiled, through the runtime so the library needs no libcuda
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) !=
                cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// Packed rows [rows, row_bytes], boxes of box_rows x 128 bytes, swizzled over
// 128 bytes; what lies outside reads as zero.
cudaError_t make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t row_bytes, int box_rows) {
    const auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cuuint64_t(row_bytes), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(row_bytes)};
    const cuuint32_t box[2] = {kStageBytes, cuuint32_t(box_rows)}, es[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BN>
cudaError_t go(Fp4Product P, const void *a, const void *b, int64_t row_bytes, int device, cudaStream_t s) {
    using S = Shape<BN>;
    CUtensorMap mt, mw;
    cudaError_t e = make_map(&mt, a, P.m, row_bytes, BN);
    if (e == cudaSuccess) e = make_map(&mw, b, P.n, row_bytes, kLanes);
    if (e != cudaSuccess) return e;
    P.tiles_m = int((P.m + BN - 1) / BN);
    P.tiles_n = int((P.n + kLanes - 1) / kLanes);
    const int64_t tiles = int64_t(P.tiles_m) * P.tiles_n;
    const int sms = sm_count(device), ks = (P.kt + 1) / 2;
    int parts = 1;
    while (parts < 8 && tiles * parts * 2 <= sms && parts * 2 <= ks) parts *= 2;
    auto *kernel = parts > 1 ? &fp4_product_kernel<BN, true> : &fp4_product_kernel<BN, false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(parts > 1 ? tiles * parts : std::min<int64_t>(tiles, sms)));
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = S::smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(parts);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, mt, mw, P);
}

}  // namespace

cudaError_t launch_fp4_product(const void *a, const uint8_t *sa, const void *b, const uint8_t *sb, int64_t m,
                               int64_t n, int64_t k, void *out, int oelem, int device, cudaStream_t s) {
    cudaError_t e;
    if (k == 0) {
        const int64_t bytes = m * n * (oelem == kF32 ? 4 : 2);
        const int64_t want = (bytes + kThreads - 1) / kThreads;
        e = launch_pdl(fp4_zero_kernel, dim3(unsigned(std::min<int64_t>(want, 4096))), dim3(kThreads), 0, s,
                       static_cast<uint8_t *>(out), bytes);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    Fp4Product P{};
    P.sa = sa;
    P.sb = sb;
    P.out = out;
    P.m = m;
    P.n = n;
    P.ot = oelem;
    P.kt = int((k + 127) / 128);
    P.k64 = int((k + 63) / 64);
    const int64_t row_bytes = (k + kMxBlock - 1) / kMxBlock * 16;
    if (m <= 16) e = go<16>(P, a, b, row_bytes, device, s);
    else if (m <= 32) e = go<32>(P, a, b, row_bytes, device, s);
    else if (m <= 64) e = go<64>(P, a, b, row_bytes, device, s);
    else if (m <= 128 || ((m + 255) / 256) * ((n + 127) / 128) < sm_count(device)) e = go<128>(P, a, b, row_bytes, device, s);
    else e = go<256>(P, a, b, row_bytes, device, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t fp4_error_take(int32_t *v, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(v, g_fp4_error, sizeof *v, 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || *v == 0) return e;
    const int32_t zero = 0;
    e = cudaMemcpyToSymbolAsync(g_fp4_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
    return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace amp
