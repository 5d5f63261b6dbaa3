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
// elements a row; the scales come in the order that the copy to tensor memory
// takes), one issues the scale copies and the products, the other warps read
// finished accumulators and store.  Stages are handed over with mbarriers.
// CTAs stay and walk tiles.
//
// Many tiles: pairs of CTAs (cta_group::2) share 256 x 256 tiles.  Each loads
// half of both operands and the products read the other half from the
// neighbour, so a product of 256 x 256 x 64 costs each SM 8 KB of shared-memory
// reads and 8 KB of fills instead of 12 and 12 for a tile of its own.
//
// Few tiles: one CTA a tile, and where the tiles do not fill the GPU the
// reduction axis is cut over the CTAs of a cluster; each leaves its fp32
// partial tile in shared memory and the cluster's CTAs add them, rank by rank,
// from there (so the order of the sum is fixed and nothing goes through global
// memory).
//
// 8192 x 14336 x 4096 bf16 (pairs): 138 us, 6.97 PFLOP/s, the tensor pipe busy
// 73 % of the time: a stage of four products takes 402 clocks alone and 550 while
// the store warps write the previous tile, and the hand-over of the accumulators
// (all of tensor memory that the scales leave is one tile) idles it 0.3 us a tile.
// 48 x 4096 x 4096 (four parts): 5.3 us, of which 1.5 are memory.
//
// Every wait gives up after a second (2^30 ns) of GPU time: the role sets the error word and
// ends, and the roles that wait for it give up in turn.  Whoever gave up, the CTA
// (both of a pair) waits, again bounded, for every load and product that is in
// flight, frees its tensor memory and returns.  An accumulator is handed over only
// when all of its products were issued; what is not handed over is stored as NaN.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "mx.cuh"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace amp {
namespace {

__device__ int32_t g_fp4_error;

constexpr int kLanes = 128;       // rows of B a CTA
constexpr int kStageBytes = 128;  // bytes of a row a stage: 256 elements

struct Fp4Product {
    const uint8_t *sa, *sb;  // scale tiles of A and B
    void *out;
    int64_t n;
    int m;
    int kt;   // scale tiles (128 elements) along the reduction
    int k64;  // products of 64 along the reduction
    int tiles_m, tiles_n;
    uint8_t ot;      // ElemType of out
    uint8_t packed;  // 16-bit out with even rows and 4-byte alignment: two elements a store
    Fp4Limits lim;
};
// One line of the constant cache: a second one is missed at every start (0.15 us a
// call of a few tokens).
static_assert(sizeof(Fp4Product) == 64, "one line of constants");

// Stages after which a role ends early.
__device__ __forceinline__ int stop_after(const Fp4Product &P, uint32_t role) {
    return P.lim.role == role ? int(P.lim.stages) : INT32_MAX;
}
__device__ __forceinline__ unsigned long long limit_ns(const Fp4Product &P) { return 1ull << P.lim.log2_ns; }
// A role's wait, by its whole warp.
__device__ __forceinline__ bool role_wait(const Fp4Product &P, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, limit_ns(P)));
}
constexpr uint32_t kNaN = 0x7FC00000u;
// NaN for one column of C and cnt tokens from m0.
__device__ __forceinline__ void store_nan(const Fp4Product &P, int64_t m0, int cnt, int64_t nn) {
    if (nn >= P.n) return;
#pragma unroll 1
    for (int64_t m = m0; m < m0 + cnt && m < P.m; ++m) {
        if (P.ot == kF32) static_cast<uint32_t *>(P.out)[m * P.n + nn] = kNaN;
        else static_cast<uint16_t *>(P.out)[m * P.n + nn] = P.ot == kF16 ? 0x7E00 : 0x7FC0;
    }
}

// tile -> (token tile, output tile): `side` output tiles side by side, so the
// CTAs that run together share operands in L2
__device__ __forceinline__ void tile_at(const Fp4Product &P, int side, int tile, int &tm, int &tn) {
    const int per = side * P.tiles_m, g = tile / per, in = tile - g * per;
    const int w = min(side, P.tiles_n - side * g);
    tm = in / w;
    tn = side * g + in % w;
}

// The 16-bit results of one lane (column nn of C) for CNT tokens from m0, of
// which `rows` are in C; p[i]: tokens 2 i and 2 i + 1.  Packed: neighbouring
// lanes swap halves, so each stores two neighbouring elements of one row.
template <int CNT>
__device__ __forceinline__ void store16(const Fp4Product &P, int64_t m0, int rows, int64_t nn,
                                        const uint32_t (&p)[CNT / 2]) {
    uint16_t *out = static_cast<uint16_t *>(P.out);
    if (P.packed) {
        const int odd = threadIdx.x & 1;
        char *at = reinterpret_cast<char *>(out + (m0 + odd) * P.n + (nn - odd));
        const int64_t step = 4 * P.n;
#pragma unroll
        for (int i = 0; i < CNT / 2; ++i) {
            const uint32_t r = __shfl_xor_sync(0xFFFFFFFFu, p[i], 1);
            const uint32_t v = odd ? __byte_perm(r, p[i], 0x7632) : __byte_perm(p[i], r, 0x5410);
            if (nn < P.n && 2 * i + odd < rows) *reinterpret_cast<uint32_t *>(at) = v;
            at += step;
        }
    } else if (nn < P.n) {
        uint16_t *at = out + m0 * P.n + nn;
#pragma unroll
        for (int i = 0; i < CNT / 2; ++i) {
            if (2 * i < rows) *at = uint16_t(p[i]);
            at += P.n;
            if (2 * i + 1 < rows) *at = uint16_t(p[i] >> 16);
            at += P.n;
        }
    }
}
template <int CNT>
__device__ __forceinline__ void store32(const Fp4Product &P, int64_t m0, int rows, int64_t nn,
                                        const uint32_t (&v)[CNT]) {
    if (nn >= P.n) return;
    float *at = static_cast<float *>(P.out) + m0 * P.n + nn;
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
        if (i < rows) *at = __uint_as_float(v[i]);
        at += P.n;
    }
}
template <int OT, int CNT>
__device__ __forceinline__ void pack16(const uint32_t (&v)[CNT], uint32_t *p) {
#pragma unroll
    for (int i = 0; i < CNT / 2; ++i)
        p[i] = f32x2_to_16x2<OT>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}

// ------------------------------------------------------------------ a pair of CTAs a tile
constexpr int kPairThreads = 640;  // load, issue, allocate, (idle), 16 store warps
struct Pair {
    static constexpr int w_bytes = kLanes * kStageBytes;  // this CTA's half of the tile's rows of B
    static constexpr int t_bytes = 128 * kStageBytes;     // and of its rows of A
    static constexpr int loads = w_bytes + t_bytes + 1024 + 2048;
    static constexpr int stage = loads;
    static constexpr int stages = 6;
    static constexpr int sf_base = 256, sf_cols = 8 + 16;  // columns of a stage's scales
    static constexpr int smem = stages * stage + 1024;
    static_assert(sf_base + stages * sf_cols <= 512, "tensor memory");
};

__global__ void __launch_bounds__(kPairThreads, 1)
    fp4_product_pair_kernel(const __grid_constant__ CUtensorMap map_t, const __grid_constant__ CUtensorMap map_w,
                            const __grid_constant__ CUtensorMap map_st,
                            const __grid_constant__ CUtensorMap map_sw, Fp4Product P) {
    using S = Pair;
    constexpr int NS = S::stages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], empty[NS], acc_full, acc_empty, drain, loaded;
    __shared__ uint32_t s_tmem, s_issued;
    uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);   // the first CTA's: its arrival, and the bytes of both
            mbar_init(&empty[i], 1);  // both: the products' commit
        }
        mbar_init(&acc_full, 1);
        mbar_init(&acc_empty, 32);  // the first CTA's: the 16 store warps of both
        mbar_init(&drain, 1);       // both: everything that was issued
        mbar_init(&loaded, 2);      // the first CTA's: both loading warps have ended
        mbar_fence_init();
        tma_prefetch_map(&map_t);
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_st);
        tma_prefetch_map(&map_sw);
    }
    if (warp == 2) tmem_alloc<2, 512>(&s_tmem);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the barriers exist in both CTAs
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    pdl_trigger();

    const int tiles = P.tiles_m * P.tiles_n;
    const int first = int(blockIdx.x >> 1), stride = int(gridDim.x >> 1);
    const int ks_all = (P.kt + 1) / 2;
    auto give_up = [&]() { g_fp4_error = 1; };

    if (warp == 0) {
        const int stop = stop_after(P, rank);
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += stride) {
            int tm, tn;
            tile_at(P, 8, tile, tm, tn);
            for (int ks = 0; ks < ks_all; ++ks) {
                ok = role_wait(P, &empty[st], ph ^ 1) & (issued != stop);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t *b = smem + st * S::stage;
                    if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * S::loads);
                    const uint32_t bar = cluster_addr(&full[st], 0);
                    const int x = ks * kStageBytes;
                    tma_load_2d_pair(b, &map_w, x, tn * 256 + int(rank) * 128, bar);
                    tma_load_2d_pair(b + S::w_bytes, &map_t, x, tm * 256 + int(rank) * 128, bar);
                    uint8_t *sf = b + S::w_bytes + S::t_bytes;
                    tma_load_2d_pair(sf, &map_sw, ks * 256, tn * 2 + int(rank), bar);
                    tma_load_2d_pair(sf + 1024, &map_st, ks * 256, tm * 2, bar);
                }
                __syncwarp();
                ++issued;
                if (++st == NS) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok) give_up();
        if (lane == 0) {
            s_issued = issued;
            cluster_arrive_release(cluster_addr(&loaded, 0));
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const int stop = stop_after(P, 2);
            int st = 0, taken = 0;
            uint32_t ph = 0, aph = 0;
            constexpr uint32_t instr = mxf4_instr(256, 256);
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += stride) {
                for (int ks = 0; ks < ks_all; ++ks) {
                    ok = role_wait(P, &full[st], ph) & (taken != stop);
                    if (!ok) break;
                    ++taken;
                    tc_fence_after();
                    const uint32_t b = smem_addr(smem) + st * S::stage;
                    const uint32_t sf = b + S::w_bytes + S::t_bytes;
                    const uint32_t tw = tmem + S::sf_base + st * S::sf_cols, tt = tw + 8;
                    const uint64_t ds = scale_desc(sf), dw = operand_desc(b), dt = operand_desc(b + S::w_bytes);
                    const int nj = min(4, P.k64 - 4 * ks);
                    if (elect_one()) {
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            copy_scales<2>(tw + 4 * a, ds + 32 * a);  // 512 bytes on
                            copy_scales<2>(tt + 8 * a, ds + 64 + 32 * a);
                            copy_scales<2>(tt + 8 * a + 4, ds + 128 + 32 * a);
                        }
                    }
                    __syncwarp();
                    if (ks == 0) {
                        // only now are the accumulators needed: with this wait
                        // first, the products of a tile began 0.2 us later
                        ok = role_wait(P, &acc_empty, aph ^ 1);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < nj)
                                mma_mxf4<2>(tmem, dw + 2 * j, dt + 2 * j, instr | mxf4_half(j & 1), tw + 4 * (j / 2),
                                            tt + 8 * (j / 2), ks > 0 || j > 0);
                        tc_commit_pair(&empty[st]);
                    }
                    __syncwarp();
                    if (++st == NS) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair(&acc_full);
                __syncwarp();
                aph ^= 1;
            }
            if (!ok) give_up();
            if (elect_one()) tc_commit_pair(&drain);
            __syncwarp();
            mbar_wait(&drain, 0);
            if (!ok) {
                // Wait for the loads that no product waited for, of both CTAs: the
                // last NS stages.  A stage that only one of the CTAs has loaded is
                // made whole on its barrier first (the stage's last use is behind it:
                // its products were committed before that CTA loaded it again).
                const bool known =
                    __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&loaded, 0, 2 * limit_ns(P) + kWaitLimitNs));
                const int one = known ? int(s_issued) : 0, two = known ? int(cluster_ld(cluster_addr(&s_issued, 1))) : 0;
                bool landed = true;  // after one that did not, the rest are only looked at
                for (int f = max(0, max(one, two) - NS); f < max(one, two); ++f) {
                    uint64_t *bar = &full[f % NS];
                    if (elect_one()) {
                        if (f >= one) mbar_arrive_expect_tx(bar, S::loads);
                        else if (f >= two) mbar_complete_tx(bar, S::loads);
                    }
                    __syncwarp();
                    landed = __all_sync(0xFFFFFFFFu, mbar_wait(bar, (f / NS) & 1, landed ? kWaitLimitNs : 0));
                }
            }
        }
    } else if (warp >= 4) {
        // a quarter of the lanes and 64 of the 256 columns a warp: into
        // registers at once, so the accumulators are free for the next tile's
        // products while this one is rounded and stored
        const int quarter = warp & 3, c0 = 64 * ((warp - 4) >> 2);
        const uint32_t acc = tmem + c0 + (uint32_t(32 * quarter) << 16);
        const uint32_t done = cluster_addr(&acc_empty, 0);
        uint32_t aph = 0;
        int tile = first;
        for (; tile < tiles; tile += stride) {
            int tm, tn;
            tile_at(P, 8, tile, tm, tn);
            if (!role_wait(P, &acc_full, aph)) break;
            aph ^= 1;
            tc_fence_after();
            uint32_t v[64];
            tmem_ld<64>(acc, v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) cluster_arrive(done);
            const int64_t nn = int64_t(tn) * 256 + rank * 128 + 32 * quarter + lane;
            const int64_t m0 = int64_t(tm) * 256 + c0;
            const int rows = int(max(int64_t(0), min(int64_t(64), P.m - m0)));
            if (P.ot == kF32) {
                store32<64>(P, m0, rows, nn, v);
            } else {
                uint32_t p[32];
                if (P.ot == kF16) pack16<kF16>(v, p);
                else pack16<kBF16>(v, p);
                store16<64>(P, m0, rows, nn, p);
            }
        }
        if (tile < tiles) give_up();
        for (; tile < tiles; tile += stride) {
            int tm, tn;
            tile_at(P, 8, tile, tm, tn);
            store_nan(P, int64_t(tm) * 256 + c0, 64, int64_t(tn) * 256 + rank * 128 + 32 * quarter + lane);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // nobody leaves while the other's barriers or memory are in use
    tc_fence_after();
    if (warp == 2) {
        if (rank == 1) mbar_wait(&drain, 0);  // the last arrival from the first CTA is in
        tmem_free<2, 512>(tmem);
    }
}

// ------------------------------------------------------------------ one CTA a tile
constexpr uint32_t kMaxParts = 4;  // CTAs that share one tile's reduction
constexpr int kSoloThreads = 384;  // load, issue, allocate, (idle), 8 store warps

template <int BN>
struct Solo {
    static constexpr int w_bytes = kLanes * kStageBytes;
    static constexpr int t_bytes = BN * kStageBytes;
    static constexpr int stage = w_bytes + t_bytes + 2048;  // and 1 KB of scales of each operand
    static constexpr int stages = BN == 128 ? 6 : BN == 64 ? 4 : 5;
    static constexpr int ctas = BN == 128 ? 1 : 2;  // CTAs an SM holds
    static constexpr int sf_base = 2 * BN;          // two accumulators
    static constexpr int sf_cols = 16;
    static constexpr int tmem_cols = BN == 128 ? 512 : 256;
    static_assert(sf_base + stages * sf_cols <= tmem_cols, "tensor memory");
    static constexpr int smem = stages * stage + 1024;  // and the alignment to 1024
    static_assert(BN * kLanes * 4 <= stages * stage, "the partial tile");
};

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kSoloThreads, Solo<BN>::ctas)
    fp4_product_kernel(const __grid_constant__ CUtensorMap map_t, const __grid_constant__ CUtensorMap map_w,
                       Fp4Product P) {
    using S = Solo<BN>;
    constexpr int NS = S::stages, NA = 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], empty[NS], acc_full[NA], acc_empty[NA], drain, ended;
    __shared__ uint32_t s_tmem;
    uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 256);
        }
        mbar_init(&drain, 1);  // everything that was issued
        mbar_init(&ended, 2);  // loads and products: nothing is in flight
        mbar_fence_init();
        tma_prefetch_map(&map_t);
        tma_prefetch_map(&map_w);
    }
    if (warp == 2) tmem_alloc<1, S::tmem_cols>(&s_tmem);
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
    auto give_up = [&]() { g_fp4_error = 1; };

    if (warp == 0) {
        const int stop = stop_after(P, 0);
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += stride) {
            int tm, tn;
            tile_at(P, 16, tile, tm, tn);
            for (int ks = ks0; ks < ks1; ++ks) {
                ok = role_wait(P, &empty[st], ph ^ 1) & (issued != stop);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t *b = smem + st * S::stage;
                    const int sfb = min(2, P.kt - 2 * ks) * 512;
                    mbar_arrive_expect_tx(&full[st], S::w_bytes + S::t_bytes + 2 * sfb);
                    tma_load_2d(b, &map_w, ks * kStageBytes, tn * kLanes, &full[st]);
                    tma_load_2d(b + S::w_bytes, &map_t, ks * kStageBytes, tm * BN, &full[st]);
                    uint8_t *sf = b + S::w_bytes + S::t_bytes;
                    bulk_g2s(sf, P.sb + (int64_t(tn) * P.kt + 2 * ks) * 512, sfb, &full[st]);
                    bulk_g2s(sf + 1024, P.sa + (int64_t(tm) * P.kt + 2 * ks) * 512, sfb, &full[st]);
                }
                __syncwarp();
                ++issued;
                if (++st == NS) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok) give_up();
        // every load lands before the CTA ends, whether its products wait for it or
        // have given up
        bool landed = true;  // after one that did not, the rest are only looked at
        for (int i = 0; i < min(issued, NS); ++i) {
            st = st == 0 ? NS - 1 : st - 1;
            if (st == NS - 1) ph ^= 1;
            landed = __all_sync(0xFFFFFFFFu, mbar_wait(&full[st], ph, landed ? kWaitLimitNs : 0));
        }
        if (lane == 0) mbar_arrive(&ended);
    } else if (warp == 1) {
        const int stop = stop_after(P, 2);
        int st = 0, ab = 0, taken = 0;
        uint32_t ph = 0, aph = 0;
        constexpr uint32_t instr = mxf4_instr(kLanes, BN);
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += stride) {
            ok = role_wait(P, &acc_empty[ab], aph ^ 1);
            tc_fence_after();
            const uint32_t acc = tmem + ab * BN;
            for (int ks = ks0; ks < ks1 && ok; ++ks) {
                ok = role_wait(P, &full[st], ph) & (taken != stop);
                if (!ok) break;
                ++taken;
                tc_fence_after();
                const uint32_t b = smem_addr(smem) + st * S::stage;
                const uint32_t tw = tmem + S::sf_base + st * S::sf_cols, tt = tw + 8;
                const uint64_t ds = scale_desc(b + S::w_bytes + S::t_bytes);
                const uint64_t dw = operand_desc(b), dt = operand_desc(b + S::w_bytes);
                const int nj = min(4, P.k64 - 4 * ks);
                if (elect_one()) {
#pragma unroll
                    for (int a = 0; a < 2; ++a)
                        if (2 * a < nj) {
                            copy_scales<1>(tw + 4 * a, ds + 32 * a);  // 512 bytes on
                            copy_scales<1>(tt + 4 * a, ds + 64 + 32 * a);
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < nj)
                            mma_mxf4<1>(acc, dw + 2 * j, dt + 2 * j, instr | mxf4_half(j & 1), tw + 4 * (j / 2),
                                        tt + 4 * (j / 2), ks > ks0 || j > 0);
                    tc_commit(&empty[st]);
                }
                __syncwarp();
                if (++st == NS) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!ok) break;
            if (elect_one()) tc_commit(&acc_full[ab]);
            __syncwarp();
            if (++ab == NA) {
                ab = 0;
                aph ^= 1;
            }
        }
        if (!ok) give_up();
        if (elect_one()) tc_commit(&drain);
        __syncwarp();
        mbar_wait(&drain, 0);
        if (lane == 0) mbar_arrive(&ended);
    } else if (warp >= 4) {
        // a quarter of the lanes and half of the columns a warp (all of 16)
        constexpr int HALF = BN > 16 ? BN / 2 : BN, CH = HALF < 32 ? HALF : 32;  // CH: columns at a time
        const int quarter = warp & 3, c0 = (warp - 4) / 4 * HALF;
        int ab = 0;
        uint32_t aph = 0;
        int tile = first;
        for (; tile < tiles; tile += stride) {
            int tm, tn;
            tile_at(P, 16, tile, tm, tn);
            if (!role_wait(P, &acc_full[ab], aph)) break;
            tc_fence_after();
            const uint32_t acc = tmem + ab * BN + (uint32_t(32 * quarter) << 16);
            const int64_t nn = int64_t(tn) * kLanes + 32 * quarter + lane, m0 = int64_t(tm) * BN;
            const int rows = int(min(int64_t(BN), P.m - m0));
#pragma unroll 1
            for (int c = c0; c < min(rows, c0 + HALF) && c < BN; c += CH) {
                uint32_t v[CH];
                tmem_ld<CH>(acc + c, v);
                if (SPLIT) {
                    // partial tile [column][lane] over the stages' buffers: every
                    // product of this CTA has finished reading them
                    float *part = reinterpret_cast<float *>(smem);
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        part[(c + i) * kLanes + 32 * quarter + lane] = __uint_as_float(v[i]);
                } else if (P.ot == kF32) {
                    store32<CH>(P, m0 + c, rows - c, nn, v);
                } else {
                    uint32_t p[CH / 2];
                    if (P.ot == kF16) pack16<kF16>(v, p);
                    else pack16<kBF16>(v, p);
                    store16<CH>(P, m0 + c, rows - c, nn, p);
                }
            }
            tc_fence_before();
            mbar_arrive(&acc_empty[ab]);
            if (++ab == NA) {
                ab = 0;
                aph ^= 1;
            }
        }
        if (tile < tiles) give_up();
        if (SPLIT && tile < tiles) {
            // the partial tile takes the place of loads that may be in flight
            mbar_wait(&ended, 0, 3 * limit_ns(P) + 3 * kWaitLimitNs);
            for (int c = c0; c < c0 + HALF && c < BN; ++c)
                reinterpret_cast<uint32_t *>(smem)[c * kLanes + 32 * quarter + lane] = kNaN;
        }
        for (; !SPLIT && tile < tiles; tile += stride) {
            int tm, tn;
            tile_at(P, 16, tile, tm, tn);
            if (c0 < BN) store_nan(P, int64_t(tm) * BN + c0, HALF, int64_t(tn) * kLanes + 32 * quarter + lane);
        }
    }

    if constexpr (SPLIT) {
        __syncwarp();
        cluster_sync();  // every CTA's partial tile is written
        int tm, tn;
        tile_at(P, 16, first, tm, tn);
        const int64_t m0 = int64_t(tm) * BN;
        const int cols = int(min(int64_t(BN), P.m - m0));
        uint32_t part[kMaxParts];
#pragma unroll
        for (uint32_t r = 0; r < kMaxParts; ++r) part[r] = cluster_addr(smem, r < parts ? r : 0);
        // groups of four neighbouring elements go round the CTAs' threads; the
        // loads of one group's parts are issued together
        for (int i = int(rank) * kSoloThreads + int(threadIdx.x); i < cols * (kLanes / 4);
             i += int(parts) * kSoloThreads) {
            const int c = i / (kLanes / 4), l = 4 * (i % (kLanes / 4));
            float4 v[kMaxParts];
#pragma unroll
            for (uint32_t r = 0; r < kMaxParts; ++r)
                if (r < parts) v[r] = cluster_ld4(part[r] + uint32_t(c * kLanes + l) * 4);
            float s[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (uint32_t r = 1; r < kMaxParts; ++r)
                if (r < parts) {
                    s[0] += v[r].x;
                    s[1] += v[r].y;
                    s[2] += v[r].z;
                    s[3] += v[r].w;
                }
            const int64_t nn = int64_t(tn) * kLanes + l, k = (m0 + c) * P.n + nn;
            if (P.packed && nn + 4 <= P.n) {
                uint16_t *o = static_cast<uint16_t *>(P.out) + k;
                const uint32_t a = P.ot == kF16 ? f32x2_to_16x2<kF16>(s[0], s[1]) : f32x2_to_16x2<kBF16>(s[0], s[1]);
                const uint32_t b = P.ot == kF16 ? f32x2_to_16x2<kF16>(s[2], s[3]) : f32x2_to_16x2<kBF16>(s[2], s[3]);
                reinterpret_cast<uint32_t *>(o)[0] = a;
                reinterpret_cast<uint32_t *>(o)[1] = b;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (nn + j >= P.n) break;
                    if (P.ot == kF32) store_elem<kF32>(P.out, k + j, s[j]);
                    else if (P.ot == kF16) store_elem<kF16>(P.out, k + j, s[j]);
                    else store_elem<kBF16>(P.out, k + j, s[j]);
                }
            }
        }
        cluster_sync();  // nobody leaves while its shared memory is read
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_free<1, S::tmem_cols>(tmem);
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

// [rows, row_elems] of es-byte elements, boxes of box_rows x box_elems; what
// lies outside reads as zero.
cudaError_t make_map(CUtensorMap *m, CUtensorMapDataType type, int es, const void *base, int64_t rows,
                     int64_t row_elems, int box_elems, int box_rows, CUtensorMapSwizzle swizzle) {
    const auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {cuuint64_t(row_elems), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(row_elems * es)};
    const cuuint32_t box[2] = {cuuint32_t(box_elems), cuuint32_t(box_rows)}, one[2] = {1, 1};
    const CUresult r = enc(m, type, 2, const_cast<void *>(base), dims, strides, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// Packed rows, 128 bytes wide boxes, swizzled over 128 bytes.
cudaError_t rows_map(CUtensorMap *m, const void *base, int64_t rows, int64_t row_bytes, int box_rows) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, rows, row_bytes, kStageBytes, box_rows,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}
// Scale tiles: a row of kt tiles of 128 words; boxes of two tiles.
cudaError_t scales_map(CUtensorMap *m, const void *base, int64_t tile_rows, int kt, int box_rows) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, base, tile_rows, int64_t(kt) * 128, 256, box_rows,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
}

// ready: one bit a device, set once the kernel's shared memory is granted there
cudaError_t launch(const void *kernel, std::atomic<uint64_t> &ready, int device, unsigned grid, int threads, int smem,
                   int cluster, cudaStream_t s, void **args) {
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if ((ready.load(std::memory_order_relaxed) & bit) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(cluster);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t go_pair(Fp4Product P, const void *a, const void *b, int64_t row_bytes, int device, cudaStream_t s) {
    CUtensorMap mt, mw, mst, msw;
    cudaError_t e = rows_map(&mt, a, P.m, row_bytes, 128);
    if (e == cudaSuccess) e = rows_map(&mw, b, P.n, row_bytes, 128);
    if (e == cudaSuccess) e = scales_map(&mst, P.sa, (P.m + 127) / 128, P.kt, 2);
    if (e == cudaSuccess) e = scales_map(&msw, P.sb, (P.n + 127) / 128, P.kt, 1);
    if (e != cudaSuccess) return e;
    P.tiles_m = int((P.m + 255) / 256);
    P.tiles_n = int((P.n + 255) / 256);
    const int64_t tiles = int64_t(P.tiles_m) * P.tiles_n;
    void *args[] = {&mt, &mw, &mst, &msw, &P};
    static std::atomic<uint64_t> ready{0};
    return launch(reinterpret_cast<const void *>(&fp4_product_pair_kernel), ready, device,
                  unsigned(2 * std::min<int64_t>(tiles, sm_count(device) / 2)), kPairThreads, Pair::smem, 2, s, args);
}

template <int BN>
cudaError_t go(Fp4Product P, const void *a, const void *b, int64_t row_bytes, int device, cudaStream_t s) {
    using S = Solo<BN>;
    // a narrower tile takes all tokens: the kernel finds a token tile's scales as
    // the scale tile (128 rows) of the same index
    if (BN < 128 && P.m > BN) return cudaErrorInvalidValue;
    CUtensorMap mt, mw;
    cudaError_t e = rows_map(&mt, a, P.m, row_bytes, BN);
    if (e == cudaSuccess) e = rows_map(&mw, b, P.n, row_bytes, kLanes);
    if (e != cudaSuccess) return e;
    P.tiles_m = int((P.m + BN - 1) / BN);
    P.tiles_n = int((P.n + kLanes - 1) / kLanes);
    const int64_t tiles = int64_t(P.tiles_m) * P.tiles_n, room = int64_t(sm_count(device)) * S::ctas;
    // Cutting the reduction pays where the CTAs still find an SM each and the
    // stages saved (0.2 us each) outweigh the exchange, which grows with the
    // tokens: 1 x 2048 x 2560 4.4 us whole, 4.1 us in four; 64 x 1024 x 1536 3.7
    // whole, 4.8 in four; 48 x 4096 x 4096 5.9 and 5.3; 128 x 4096 x 4096 6.5 and
    // 6.7; 128 x 4096 x 5120 7.4 and 6.9.  On shared SMs it does not: 1 x 14336 x
    // 4096 6.5 us whole, 8.0 us in two.  Eight parts are slower than four (clusters
    // of 8 large CTAs do not fill every part of the GPU: 512 x 512 x 8192 12.7 us,
    // in four 7.1).
    const int ks = (P.kt + 1) / 2, pays = 7 + int(std::min<int64_t>(P.m, BN)) / 16;
    int parts = 1;
    for (int p = 2; p <= int(kMaxParts) && tiles * p <= sm_count(device); p *= 2)
        if (ks - (ks + p - 1) / p >= pays) parts = p;
    void *args[] = {&mt, &mw, &P};
    static std::atomic<uint64_t> ready[2];
    if (parts > 1)
        return launch(reinterpret_cast<const void *>(&fp4_product_kernel<BN, true>), ready[1], device, unsigned(tiles * parts),
                      kSoloThreads, S::smem, parts, s, args);
    return launch(reinterpret_cast<const void *>(&fp4_product_kernel<BN, false>), ready[0], device,
                  unsigned(std::min<int64_t>(tiles, room)), kSoloThreads, S::smem, 1, s, args);
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
    P.sa = sa;
    P.sb = sb;
    P.out = out;
    P.m = int(m);
    P.n = n;
    P.lim = limits;
    P.ot = uint8_t(oelem);
    P.packed = oelem != kF32 && n % 2 == 0 && (reinterpret_cast<uintptr_t>(out) & 3) == 0;
    P.kt = int((k + 127) / 128);
    P.k64 = int((k + 63) / 64);
    const int64_t row_bytes = (k + kMxBlock - 1) / kMxBlock * 16;
    const int64_t pair_tiles = ((m + 255) / 256) * ((n + 255) / 256);
    if (m <= 16) e = go<16>(P, a, b, row_bytes, device, s);
    else if (m <= 32) e = go<32>(P, a, b, row_bytes, device, s);
    else if (m <= 64) e = go<64>(P, a, b, row_bytes, device, s);
    else if (m <= 128 || pair_tiles * 2 < sm_count(device)) e = go<128>(P, a, b, row_bytes, device, s);
    else e = go_pair(P, a, b, row_bytes, device, s);
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
