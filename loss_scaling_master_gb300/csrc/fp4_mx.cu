// fp4_mx.cu - microscaled 4-bit quantisation (both orientations in one pass)
// and its inverse.
//
// Mathematics: mx.cuh.  One CTA takes a 128x128 tile of x, which holds whole
// blocks of both orientations and exactly one 512-byte scale tile of each, so
// x is read once: 2 bytes (16-bit x) in and 17/32 byte out per element and
// orientation.
//
// A warp takes 32 rows x 64 columns, a lane 8 rows x 8 columns of it (16-byte
// loads), all in registers.  The 4 lanes side by side hold a row block, the 4
// lanes below one another a column block.  Their maxima are exchanged by a
// transposing reduction (each step halves the number of words a lane still
// carries), after which every lane holds the finished maxima of two rows and
// two columns, forms their scale bytes and hands them round with 4 shuffles.
// The lane's 8 consecutive rows make the transposed copy's nibbles without an
// exchange; only the 16-byte pieces of that copy go through shared memory, so
// that a column's 64 bytes leave together.
//
// 16384 x 5120 bf16, both orientations: 45.4 us, 83 % of memory's rate; what is
// left is instruction issue (15 an element, 2.6 of 4 a clock) with 4 CTAs an SM
// (2 CTAs 57 us, 3 50 us).  8192 x 4096, rows only: 15.4 us, 3.4 rounds of CTAs.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "mx.cuh"
#include "pdl.cuh"

namespace amp {
namespace {

struct Fp4Quant {
    const void *x;
    int64_t rows, cols;
    uint8_t *out, *scales, *out_t, *scales_t;
    const int32_t *skip;
    int64_t tiles_c;  // tiles along the columns
};

// Words w[0..N) over the 4 lanes of two lane bits -> the maxima of words
// i * N / 4 .. for the lane with index i in the group.  `Op` is an associative
// maximum; hi and lo are the lane masks of the group's two index bits.
template <int N, class Op>
__device__ __forceinline__ void transposing_max4(uint32_t (&w)[N], uint32_t (&r)[N / 4], int hi,
                                                 int lo, int lane, Op op) {
    const bool bh = lane & hi, bl = lane & lo;
    uint32_t h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const uint32_t mine = bh ? w[N / 2 + i] : w[i], other = bh ? w[i] : w[N / 2 + i];
        h[i] = op(mine, __shfl_xor_sync(0xFFFFFFFFu, other, hi));
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const uint32_t mine = bl ? h[N / 4 + i] : h[i], other = bl ? h[i] : h[N / 4 + i];
        r[i] = op(mine, __shfl_xor_sync(0xFFFFFFFFu, other, lo));
    }
}

// A warp's 32 rows x 64 columns of x from rows at any address: loaded by single
// elements, 32 of a row side by side, and turned over to the lanes' 8 x 8 pieces
// in shared memory (s: the warp's 4 KB; fp32 takes two turns of 16 rows, its
// 16-byte pieces exchanged in the right half of a row so that 8 lanes' reads
// fall into 32 banks).  16383 x 5121 bf16, both orientations: 64 us, 87 us with a
// lane loading its own piece element by element (a warp's load then touches 16 to
// 32 sectors for 32 elements); 1537 x 1111 fp32 3.7 and 5.1 us.  x: the warp's
// first element; rows, cols: how many of the matrix are there.
template <int XT>
__device__ __forceinline__ void load_any(const void *x, int64_t stride, int rows, int cols, uint8_t *s, int lane,
                                         uint4 (&raw)[8][kWords8<XT>]) {
    constexpr int TURNS = kWords8<XT>, R = 8 / TURNS;  // rows a lane and turn
    constexpr int B = 8;                               // rows whose loads are issued together
    using E = std::conditional_t<XT == kF32, uint32_t, uint16_t>;
    const E *at = static_cast<const E *>(x) + lane;
    const bool in0 = lane < cols, in1 = lane + 32 < cols;
    E *put = reinterpret_cast<E *>(s) + lane;
    E *put1 = XT == kF32 ? reinterpret_cast<E *>(s) + 32 + (lane ^ 4) : put + 32;
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
        if (t) __syncwarp();
#pragma unroll
        for (int m0 = 0; m0 < 4 * R; m0 += B) {
            E v[B][2];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int m = m0 + b, r = m / R * 8 + t * R + m % R;
                v[b][0] = r < rows && in0 ? at[r * stride] : E(0);
                v[b][1] = r < rows && in1 ? at[r * stride + 32] : E(0);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                put[64 * (m0 + b)] = v[b][0];
                put1[64 * (m0 + b)] = v[b][1];
            }
        }
        __syncwarp();
        const int cl = lane & 7, rl = lane >> 3;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int u = 0; u < kWords8<XT>; ++u)
                raw[t * R + i][u] = reinterpret_cast<const uint4 *>(
                    s + (rl * R + i) * 64 * sizeof(E))[XT == kF32 ? (2 * cl + u) ^ (cl >> 2) : cl];
    }
}

template <int XT, bool T, bool VEC>
__global__ void __launch_bounds__(kThreads, XT == kF32 ? 2 : 4) fp4_quant_kernel(Fp4Quant P) {
    __shared__ __align__(16) uint8_t s_x[VEC ? 16 : 8 * 4096];
    __shared__ __align__(16) uint32_t s_t[T ? 128 * 16 : 4];  // transposed codes, 64 B a column
    __shared__ __align__(16) uint8_t s_rs[512];
    __shared__ __align__(16) uint8_t s_cs[T ? 512 : 16];
    constexpr int W = kWords8<XT>;
    pdl_wait();
    pdl_trigger();
    if (P.skip && *P.skip != 0) return;
    const int64_t tr = int64_t(blockIdx.x) / P.tiles_c, tc = int64_t(blockIdx.x) % P.tiles_c;
    const int64_t r0 = tr * kTile, c0 = tc * kTile;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cl = lane & 7, rl = lane >> 3;
    const int lr = 32 * (warp >> 1) + 8 * rl;  // first of the lane's 8 rows in the tile
    const int lc = 64 * (warp & 1) + 8 * cl;   // first of its 8 columns
    const int64_t row = r0 + lr, col = c0 + lc;
    constexpr int esz = XT == kF32 ? 4 : 2;

    uint4 raw[8][W];
    if constexpr (VEC) {
        // a row's length is a multiple of 8 here
        const int n = col < P.cols ? int(max(int64_t(0), min(int64_t(8), P.rows - row))) : 0;
        const char *p = static_cast<const char *>(P.x) + (row * P.cols + col) * esz;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int u = 0; u < W; ++u)
                raw[i][u] = i < n ? ld16(p + i * P.cols * esz + 16 * u) : make_uint4(0, 0, 0, 0);
    } else {
        const int64_t wr = r0 + 32 * (warp >> 1), wc = c0 + 64 * (warp & 1);
        load_any<XT>(static_cast<const char *>(P.x) + (wr * P.cols + wc) * esz, P.cols,
                     int(max(int64_t(0), min(int64_t(32), P.rows - wr))),
                     int(max(int64_t(0), min(int64_t(64), P.cols - wc))), s_x + 4096 * warp, lane, raw);
    }

    // rmax[k]: fp32 bits of the maximum of row 2 (cl % 4) + k's block; cmax[k]:
    // of column 2 rl + k's
    uint32_t rmax[2], cmax[2] = {0, 0};
    if constexpr (XT == kF32) {
        uint32_t rw[8], cw[8];
        auto op = [](uint32_t a, uint32_t b) { return max(a, b); };
#pragma unroll
        for (int i = 0; i < 8; ++i) rw[i] = cw[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                                   raw[i][W - 1].x, raw[i][W - 1].y, raw[i][W - 1].z, raw[i][W - 1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t a = w[j] & 0x7FFFFFFFu;
                rw[i] = max(rw[i], a);
                if (T) cw[j] = max(cw[j], a);
            }
        }
        transposing_max4<8>(rw, rmax, 2, 1, lane, op);
        if (T) transposing_max4<8>(cw, cmax, 16, 8, lane, op);
    } else {
        // maxima on packed pairs, their signs cleared when they are widened (on
        // the bits as integers, signs cleared first: 45.7 against 45.4 us at 16384
        // x 5120, 15.8 against 15.4 us at 8192 x 4096 rows only)
        uint32_t m[8], rw[4], cw[4], r1[1], c1[1] = {0};
        auto op = [](uint32_t a, uint32_t b) { return absmax2<XT>(a, b); };
        auto widen = [](uint32_t h) { return __float_as_uint(lowp_to_f32<XT>(h & 0xFFFFu)) & 0x7FFFFFFFu; };
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w[4] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w};
            m[i] = op(op(w[0], w[1]), op(w[2], w[3]));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (T) cw[j] = i ? op(cw[j], w[j]) : w[j];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            rw[i] = op(__byte_perm(m[2 * i], m[2 * i + 1], 0x5410), __byte_perm(m[2 * i], m[2 * i + 1], 0x7632));
        transposing_max4<4>(rw, r1, 2, 1, lane, op);
        rmax[0] = widen(r1[0]);
        rmax[1] = widen(r1[0] >> 16);
        if (T) {
            transposing_max4<4>(cw, c1, 16, 8, lane, op);
            cmax[0] = widen(c1[0]);
            cmax[1] = widen(c1[0] >> 16);
        }
    }

    // ---- scale bytes
    const uint32_t e0 = mx_scale_code<MxE2M1>(rmax[0]), e1 = mx_scale_code<MxE2M1>(rmax[1]);
    {
        // byte (r % 32) * 16 + r / 32 * 4 + block, rows lr + 2 (cl % 4) + {0, 1}
        uint8_t *s = s_rs + (8 * rl + 2 * (cl & 3)) * 16 + (warp >> 1) * 4 + 2 * (warp & 1) + (cl >> 2);
        s[0] = uint8_t(e0);
        s[16] = uint8_t(e1);
    }
    float fc[T ? 8 : 1];  // the lane's columns' multipliers
    if constexpr (T) {
        const uint32_t d0 = mx_scale_code<MxE2M1>(cmax[0]), d1 = mx_scale_code<MxE2M1>(cmax[1]);
        const int c = lc + 2 * rl;  // c and c + 1 are in the same group of 32 columns
        uint8_t *s = s_cs + (c % 32) * 16 + (c / 32) * 4 + (warp >> 1);
        s[0] = uint8_t(d0);
        s[16] = uint8_t(d1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t e = __shfl_sync(0xFFFFFFFFu, d0 | (d1 << 16), cl + 8 * k);
            fc[2 * k] = mx_unscale(e & 0xFFFFu);
            fc[2 * k + 1] = mx_unscale(e >> 16);
        }
    }

    // ---- codes, two rows at a time: each element is widened once for both
    // orientations; the two rows make one byte of each column's word
    const int64_t rowb = (P.cols + kMxBlock - 1) / kMxBlock * 16;  // bytes a packed row
    const bool colin = col / 2 < rowb;
    uint8_t *out = P.out + row * rowb + col / 2;
    uint32_t cw[T ? 8 : 1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t e = __shfl_sync(0xFFFFFFFFu, e0 | (e1 << 16), (lane & ~3) + k);
        float y[2][8], z[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 2 * k + h;
            const float f = mx_unscale(h ? e >> 16 : e & 0xFFFFu);
            raw8_to_f32<XT>(raw[i], y[h]);
#pragma unroll
            for (int j = 0; j < 8; j += 2) mul2_rn(y[h][j], y[h][j + 1], f, f, z[j], z[j + 1]);
            const uint32_t w = f32x8_to_e2m1x8(z);
            if (colin && row + i < P.rows) *reinterpret_cast<uint32_t *>(out + i * rowb) = w;
        }
        if constexpr (T) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float a0, a1, b0, b1;
                mul2_rn(y[0][j], y[0][j + 1], fc[j], fc[j + 1], a0, a1);
                mul2_rn(y[1][j], y[1][j + 1], fc[j], fc[j + 1], b0, b1);
                const uint32_t p = f32x2_to_e2m1x2(a0, b0), q = f32x2_to_e2m1x2(a1, b1);
                cw[j] = k == 0 ? p : cw[j] + (p << (8 * k));
                cw[j + 1] = k == 0 ? q : cw[j + 1] + (q << (8 * k));
            }
        }
    }
    if constexpr (T) {
        // column lc + j, row group lr / 8; 16-byte pieces permuted by cl, and
        // odd and even columns exchanged in every other group of 32, so that a
        // warp's words fall into 32 banks
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s_t[((lc + j) ^ ((cl >> 2) & 1)) * 16 + ((lr / 8) ^ ((cl & 3) << 2))] = cw[j];
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int64_t tile = tr * P.tiles_c + tc;
        st16(P.scales + tile * 512 + 16 * threadIdx.x, reinterpret_cast<const uint4 *>(s_rs)[threadIdx.x]);
    }
    if constexpr (T) {
        const int64_t tiles_r = (P.rows + kTile - 1) / kTile;
        if (threadIdx.x >= 32 && threadIdx.x < 64) {
            const int64_t tile = tc * tiles_r + tr;
            st16(P.scales_t + tile * 512 + 16 * (threadIdx.x - 32),
                 reinterpret_cast<const uint4 *>(s_cs)[threadIdx.x - 32]);
        }
        const int64_t rowb_t = (P.rows + kMxBlock - 1) / kMxBlock * 16;
        const int q = threadIdx.x & 3;
        const int64_t at = r0 / 2 + 16 * q;  // byte in the transposed row
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = (threadIdx.x >> 2) + 64 * k;
            if (c0 + c < P.cols && at < rowb_t)
                st16(P.out_t + (c0 + c) * rowb_t + at,
                     *reinterpret_cast<const uint4 *>(
                         &s_t[(c ^ ((c >> 5) & 1)) * 16 + ((q ^ ((c >> 3) & 3)) << 2)]));
        }
    }
}

// ---- values of the codes -------------------------------------------------
// With U = 4 a step takes the rows r, r + 32, r + 64 and r + 96 of a tile of 128
// at one place: their scales are one 16-byte line of a scale tile, and their
// addresses a fixed distance apart.  (With a row's place worked out for every 8
// elements, 12 instructions an element bound the kernel: 16384 x 5120 bf16 36.2
// against 33.4 us, memory 31.4 us; 1000 x 2304 3.2 against 2.1 us.)  Where that
// leaves SMs without a CTA, U = 1: a row a step (32 x 4096 1.3 against 1.4 us, 33 x
// 1111 1.3 against 1.6 us).
struct Fp4Dequant {
    const uint8_t *q, *scales;
    int64_t rows, cols;
    int64_t groups;  // of rows: U = 4: 32 a whole tile; else the rows
    int pieces;      // of a packed row: of 16 bytes of output, or of 256 elements
    void *out;
};
template <int U>
struct RowGroup {
    int64_t row;  // the first
    int n;        // how many of the U are there
    __device__ __forceinline__ RowGroup(const Fp4Dequant &P, int64_t g) {
        row = U == 4 ? (g >> 5) * kTile + (g & 31) : g;
        n = U == 4 ? int(min(int64_t(4), (P.rows - row + 31) / 32)) : 1;
    }
};
// the rows' scale bytes of block b
template <int U>
__device__ __forceinline__ void group_scales(const Fp4Dequant &P, int64_t row, int b, uint32_t (&e)[U]) {
    const int64_t tile = (row >> 7) * ((P.cols + kTile - 1) / kTile) + (b >> 2);
    const uint8_t *line = P.scales + tile * 512 + (row & 31) * 16;
    if constexpr (U == 4) {
        const uint4 w = ld16(line);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = (u[i] >> (8 * (b & 3))) & 0xFFu;
    } else {
        e[0] = line[((row >> 5) & 3) * 4 + (b & 3)];
    }
}

// Rows that are whole, aligned 16-byte pieces: one of them a thread, step and
// row.  (Two pieces side by side a thread in fp32 would write every sector by
// halves: 16384 x 5120 83 us, one 59 us, memory 56 us.)
template <int XT, int U>
__global__ void __launch_bounds__(kThreads) fp4_dequant_vec(Fp4Dequant P) {
    pdl_wait();
    pdl_trigger();
    constexpr int N = XT == kF32 ? 4 : 8;  // elements a piece
    using Codes = std::conditional_t<XT == kF32, uint16_t, uint32_t>;
    RowWalk at(blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads, P.pieces);
    for (; at.row < P.groups; at.next()) {
        if (N * at.at >= P.cols) continue;
        const RowGroup<U> r(P, at.row);
        const Codes *q = reinterpret_cast<const Codes *>(P.q) + r.row * P.pieces + at.at;
        uint32_t codes[U], e[U];
#pragma unroll
        for (int i = 0; i < U; ++i) codes[i] = i < r.n ? q[32 * i * int64_t(P.pieces)] : 0u;
        group_scales<U>(P, r.row, at.at / (kMxBlock / N), e);
        char *out = static_cast<char *>(P.out) + (r.row * P.cols + N * at.at) * (16 / N);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i >= r.n) break;
            const float s = mx_scale(e[i]);
            float y[8];
            if constexpr (N == 4) e2m1x4_to_f32x4(codes[i], y);
            else e2m1x8_to_f32x8(codes[i], y);
#pragma unroll
            for (int j = 0; j < N; j += 2) mul2_rn(y[j], y[j + 1], s, s, y[j], y[j + 1]);
            uint4 u[1];
            if constexpr (N == 4)
                u[0] = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                                  __float_as_uint(y[3]));
            else f32_to_raw8<XT>(y, u);
            st16(out + 32 * i * P.cols * (16 / N), u[0]);
        }
    }
}

// Any row length and address: a warp takes 256 elements of each row, a lane one
// packed word of them; the values are turned over in shared memory so that each
// store of the warp is 32 elements side by side (fp32: 16-byte pieces exchanged
// in every other 32 elements, against bank conflicts): 16383 x 5121 bf16 39 us,
// 79 us with a word decoded for each element.
template <int XT, int U>
__global__ void __launch_bounds__(kThreads) fp4_dequant_elem(Fp4Dequant P) {
    using E = std::conditional_t<XT == kF32, uint32_t, uint16_t>;
    constexpr int W = kWords8<XT>;
    __shared__ uint4 s_y[kThreads / 32][32 * W];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    uint4 *const put = s_y[threadIdx.x >> 5];
    const E *const get = reinterpret_cast<const E *>(put);
    const int64_t rowb = (P.cols + kMxBlock - 1) / kMxBlock * 16;
    RowWalk at(blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32), P.pieces);
    for (; at.row < P.groups; at.next()) {
        const RowGroup<U> r(P, at.row);
        const int c0 = 256 * at.at;
        uint32_t codes[U] = {}, e[U] = {};
        if (c0 / 2 + 4 * lane < rowb) {
            const uint8_t *q = P.q + r.row * rowb + c0 / 2 + 4 * lane;
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (i < r.n) codes[i] = *reinterpret_cast<const uint32_t *>(q + 32 * i * rowb);
            group_scales<U>(P, r.row, c0 / 32 + lane / 4, e);
        }
        E *out = static_cast<E *>(P.out) + r.row * P.cols + c0 + lane;
        const int n = int(P.cols) - c0 - lane;  // n > 32 j: element j is in the row
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i >= r.n) break;
            const float s = mx_scale(e[i]);
            float y[8];
            e2m1x8_to_f32x8(codes[i], y);
#pragma unroll
            for (int j = 0; j < 8; j += 2) mul2_rn(y[j], y[j + 1], s, s, y[j], y[j + 1]);
            uint4 u[W];
            f32_to_raw8<XT>(y, u);
            __syncwarp();  // the last row's words are out
#pragma unroll
            for (int j = 0; j < W; ++j) put[(W * lane + j) ^ (W == 2 ? (lane >> 2) & 1 : 0)] = u[j];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (n > 32 * j) out[32 * j] = get[32 * j + (W == 2 ? lane ^ (4 * (j & 1)) : lane)];
            out += 32 * P.cols;
        }
    }
}

}  // namespace

cudaError_t launch_fp4_quant(const void *x, int xelem, int64_t rows, int64_t cols, uint8_t *out,
                             uint8_t *scales, uint8_t *out_t, uint8_t *scales_t,
                             const int32_t *skip_if, cudaStream_t s) {
    Fp4Quant P;
    P.x = x;
    P.rows = rows;
    P.cols = cols;
    P.out = out;
    P.scales = scales;
    P.out_t = out_t;
    P.scales_t = scales_t;
    P.skip = skip_if;
    P.tiles_c = (cols + kTile - 1) / kTile;
    const int esz = xelem == kF32 ? 4 : 2;
    // whole groups of 8 elements: every group of 8 columns lies inside the row
    const bool vec = cols % 8 == 0 && (cols * esz) % 16 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
    const int64_t tiles = ((rows + kTile - 1) / kTile) * P.tiles_c;
    const dim3 grid((unsigned)tiles), block(kThreads);
    cudaError_t e;
#define FP4_Q1(XT, T)                                                               \
    e = vec ? launch_pdl(fp4_quant_kernel<XT, T, true>, grid, block, 0, s, P)        \
            : launch_pdl(fp4_quant_kernel<XT, T, false>, grid, block, 0, s, P)
#define FP4_Q(XT)                    \
    do {                             \
        if (out_t) FP4_Q1(XT, true); \
        else FP4_Q1(XT, false);      \
    } while (0)
    if (xelem == kF32) FP4_Q(kF32);
    else if (xelem == kF16) FP4_Q(kF16);
    else FP4_Q(kBF16);
#undef FP4_Q
#undef FP4_Q1
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_fp4_dequant(const uint8_t *q, const uint8_t *scales, int64_t rows, int64_t cols,
                               void *out, int oelem, int device, cudaStream_t s) {
    const int esz = oelem == kF32 ? 4 : 2;
    const bool vec = (cols * esz) % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    Fp4Dequant P{q, scales, rows, cols, rows / kTile * 32 + std::min<int64_t>(32, rows % kTile), 0, out};
    P.pieces = int(vec ? (cols + kMxBlock - 1) / kMxBlock * (kMxBlock * esz / 16) : (cols + 255) / 256);
    const int64_t sms = sm_count(device), per_cta = vec ? kThreads : kThreads / 32;
    const bool four = P.groups * P.pieces >= sms * per_cta;
    if (!four) P.groups = rows;
    const int64_t want = (P.groups * P.pieces + per_cta - 1) / per_cta;
    const dim3 grid((unsigned)std::min<int64_t>(want, sms * 32)), block(kThreads);
    cudaError_t e;
#define FP4_D1(XT, U)                                                         \
    e = vec ? launch_pdl(fp4_dequant_vec<XT, U>, grid, block, 0, s, P)        \
            : launch_pdl(fp4_dequant_elem<XT, U>, grid, block, 0, s, P)
#define FP4_D(XT)                \
    do {                         \
        if (four) FP4_D1(XT, 4); \
        else FP4_D1(XT, 1);      \
    } while (0)
    if (oelem == kF32) FP4_D(kF32);
    else if (oelem == kF16) FP4_D(kF16);
    else FP4_D(kBF16);
#undef FP4_D1
#undef FP4_D
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace amp
