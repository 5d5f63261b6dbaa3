// ops_api.cu - the extern "C" boundary of the operators of ampops.h: argument
// checks and launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <utility>

#include "ampops.h"
#include "internal.h"
#include "mx.cuh"

namespace {

amp_status fail(amp_status st, const char *fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    amp::set_last_error(msg);
    return st;
}
amp_status finish(cudaError_t e, const char *fn) {
    return e == cudaSuccess ? AMP_OK : fail(AMP_ECUDA, "%s: %s", fn, cudaGetErrorString(e));
}

int elem_code(amp_dtype d) {
    switch (d) {
    case AMP_DT_F32: return amp::kF32;
    case AMP_DT_F16: return amp::kF16;
    case AMP_DT_BF16: return amp::kBF16;
    default: return -1;
    }
}

// Sizes the launch arithmetic can hold: sides below 2^31, rows * cols below
// 2^60, tiles of 128 x 128 below 2^31.
bool bad_shape(int64_t rows, int64_t cols) {
    const int64_t lim = (int64_t(1) << 31) - 256;
    if (rows < 0 || cols < 0 || rows >= lim || cols >= lim) return true;
    if (cols > 0 && rows > (int64_t(1) << 60) / cols) return true;
    return ((rows + 127) / 128) * ((cols + 127) / 128) > (int64_t(1) << 30);
}
bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
// Tensors of one element type (NULL passes): on the GPU an address between two
// elements is a fault, not a status.
template <class... Ps>
bool off_type(int elem, Ps... p) {
    return (misaligned(p, elem == amp::kF32 ? 4 : 2) || ...);
}

cudaStream_t cu(amp_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
uint8_t *u8(void *p) { return static_cast<uint8_t *>(p); }
const uint8_t *u8(const void *p) { return static_cast<const uint8_t *>(p); }

const char *kShape = "%s: negative or too large size";
const char *kNull = "%s: NULL argument";
const char *kType = "%s: unsupported dtype";
const char *kOff = "%s: a tensor is not aligned to its type";

}  // namespace

extern "C" {

int64_t fp4_mx_bytes(int64_t rows, int64_t cols) {
    return bad_shape(rows, cols) ? -1 : rows * ((cols + 31) / 32) * 16;
}
int64_t fp4_mx_scale_bytes(int64_t rows, int64_t cols) {
    return bad_shape(rows, cols) ? -1 : ((rows + 127) / 128) * ((cols + 127) / 128) * 512;
}

amp_status fp4_quant_mx(const void *x, amp_dtype x_dtype, int64_t rows, int64_t cols, void *out,
                        void *scales, void *out_t, void *scales_t, const int32_t *skip_if_dev,
                        amp_stream_t stream) {
    AMP_TRACE("fp4_quant_mx");
    const char *fn = "fp4_quant_mx";
    if (bad_shape(rows, cols)) return fail(AMP_EINVAL, kShape, fn);
    const int xc = elem_code(x_dtype);
    if (xc < 0) return fail(AMP_EDTYPE, kType, fn);
    if ((out_t == nullptr) != (scales_t == nullptr))
        return fail(AMP_EINVAL, "%s: out_t and scales_t go together", fn);
    if (rows * cols == 0) return AMP_OK;
    if (!x || !out || !scales) return fail(AMP_EINVAL, kNull, fn);
    if (misaligned(out, 16) || misaligned(scales, 16) || misaligned(out_t, 16) || misaligned(scales_t, 16))
        return fail(AMP_EINVAL, "%s: outputs must be 16-byte aligned", fn);
    if (off_type(xc, x) || off_type(amp::kF32, skip_if_dev)) return fail(AMP_EINVAL, kOff, fn);
    return finish(amp::launch_fp4_quant(x, xc, rows, cols, u8(out), u8(scales), u8(out_t), u8(scales_t),
                                        skip_if_dev, cu(stream)),
                  fn);
}

amp_status fp4_dequant_mx(const void *q, const void *scales, int64_t rows, int64_t cols, void *out,
                          amp_dtype out_dtype, amp_stream_t stream) {
    AMP_TRACE("fp4_dequant_mx");
    const char *fn = "fp4_dequant_mx";
    if (bad_shape(rows, cols)) return fail(AMP_EINVAL, kShape, fn);
    const int oc = elem_code(out_dtype);
    if (oc < 0) return fail(AMP_EDTYPE, kType, fn);
    if (rows * cols == 0) return AMP_OK;
    if (!q || !scales || !out) return fail(AMP_EINVAL, kNull, fn);
    if (misaligned(q, 16) || misaligned(scales, 16))
        return fail(AMP_EINVAL, "%s: q and scales must be 16-byte aligned", fn);
    if (off_type(oc, out)) return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_fp4_dequant(u8(q), u8(scales), rows, cols, out, oc, dev, cu(stream)), fn);
}

static amp_status product(const char *fn, const void *a, const void *a_scales, const void *b, const void *b_scales,
                          int64_t m, int64_t n, int64_t k, void *out, amp_dtype out_dtype, amp_stream_t stream,
                          amp::Fp4Limits limits) {
    // k: one tile's products have to end well within the second that a wait may take
    if (bad_shape(m, n) || bad_shape(m, k) || bad_shape(n, k) || k > (int64_t(1) << 27))
        return fail(AMP_EINVAL, kShape, fn);
    const int oc = elem_code(out_dtype);
    if (oc < 0) return fail(AMP_EDTYPE, kType, fn);
    if (m * n == 0) return AMP_OK;
    if (!out || (k > 0 && (!a || !a_scales || !b || !b_scales))) return fail(AMP_EINVAL, kNull, fn);
    if (misaligned(a, 16) || misaligned(a_scales, 16) || misaligned(b, 16) || misaligned(b_scales, 16))
        return fail(AMP_EINVAL, "%s: operands must be 16-byte aligned", fn);
    if (off_type(oc, out)) return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(
        amp::launch_fp4_product(a, u8(a_scales), b, u8(b_scales), m, n, k, out, oc, dev, cu(stream), limits), fn);
}

amp_status fp4_product_mx(const void *a, const void *a_scales, const void *b, const void *b_scales,
                          int64_t m, int64_t n, int64_t k, void *out, amp_dtype out_dtype,
                          amp_stream_t stream) {
    AMP_TRACE("fp4_product_mx");
    return product("fp4_product_mx", a, a_scales, b, b_scales, m, n, k, out, out_dtype, stream, {30, 3, 0});
}

amp_status fp4_product_mx_selftest(const void *a, const void *a_scales, const void *b, const void *b_scales,
                                   int64_t m, int64_t n, int64_t k, void *out, amp_dtype out_dtype, int32_t role,
                                   int32_t stages, int32_t limit_log2_ns, amp_stream_t stream) {
    AMP_TRACE("fp4_product_mx_selftest");
    const char *fn = "fp4_product_mx_selftest";
    if (role < 0 || role > 2 || stages < 0) return fail(AMP_EINVAL, "%s: role not in [0, 2] or stages < 0", fn);
    if (limit_log2_ns < 0 || limit_log2_ns > 30) return fail(AMP_EINVAL, "%s: limit above 2^30 ns", fn);
    return product(fn, a, a_scales, b, b_scales, m, n, k, out, out_dtype, stream,
                   {uint8_t(limit_log2_ns), uint8_t(role), uint32_t(stages)});
}

amp_status fp4_mx_check(amp_stream_t stream) {
    AMP_TRACE("fp4_mx_check");
    int32_t v = 0;
    const cudaError_t e = amp::fp4_error_take(&v, cu(stream));
    if (e != cudaSuccess) return finish(e, "fp4_mx_check");
    return v == 0 ? AMP_OK : fail(AMP_ETIMEOUT, "fp4_mx_check: a bounded wait of fp4_product_mx or fp4_linear_mx gave up; "
                                                "the output of that call is unspecified");
}

amp_status amp_layer_norm_forward(const void *x, amp_dtype x_dtype, int64_t rows, int64_t cols,
                                  const void *weight, const void *bias, amp_dtype w_dtype, double eps,
                                  void *y, float *mean, float *rstd, void *ckpt, void *ckpt_scales,
                                  amp_stream_t stream) {
    AMP_TRACE("amp_layer_norm_forward");
    const char *fn = "amp_layer_norm_forward";
    if (bad_shape(rows, cols)) return fail(AMP_EINVAL, kShape, fn);
    const int xc = elem_code(x_dtype), wc = elem_code(w_dtype);
    if (xc < 0 || wc < 0 || (wc != amp::kF32 && wc != xc)) return fail(AMP_EDTYPE, kType, fn);
    if (!(eps >= 0.0) || std::isinf(eps)) return fail(AMP_EINVAL, "%s: eps must be finite and >= 0", fn);
    if ((ckpt == nullptr) != (ckpt_scales == nullptr))
        return fail(AMP_EINVAL, "%s: ckpt and ckpt_scales go together", fn);
    if (rows * cols == 0) return AMP_OK;
    if (!x || !y) return fail(AMP_EINVAL, kNull, fn);
    if (off_type(xc, x, y) || off_type(wc, weight, bias) || off_type(amp::kF32, mean, rstd))
        return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_norm_fwd(x, xc, rows, cols, weight, bias, wc, float(eps), y, mean, rstd, u8(ckpt),
                                       u8(ckpt_scales), dev, cu(stream)),
                  fn);
}

int64_t amp_layer_norm_workspace_bytes(int64_t rows, int64_t cols) {
    int dev = 0;
    if (bad_shape(rows, cols) || cudaGetDevice(&dev) != cudaSuccess) return -1;
    return amp::norm_parts(rows, cols, dev) * 2 * cols * int64_t(sizeof(float));
}

amp_status amp_layer_norm_backward(const void *dy, const void *x, amp_dtype dtype, const void *ckpt,
                                   const void *ckpt_scales, int64_t rows, int64_t cols,
                                   const void *weight, amp_dtype w_dtype, const float *mean,
                                   const float *rstd, void *dx, void *dweight, void *dbias,
                                   void *workspace, int64_t workspace_bytes, amp_stream_t stream) {
    AMP_TRACE("amp_layer_norm_backward");
    const char *fn = "amp_layer_norm_backward";
    if (bad_shape(rows, cols)) return fail(AMP_EINVAL, kShape, fn);
    const int xc = elem_code(dtype), wc = elem_code(w_dtype);
    if (xc < 0 || wc < 0 || (wc != amp::kF32 && wc != xc)) return fail(AMP_EDTYPE, kType, fn);
    if ((ckpt == nullptr) != (ckpt_scales == nullptr))
        return fail(AMP_EINVAL, "%s: ckpt and ckpt_scales go together", fn);
    if (x && ckpt) return fail(AMP_EINVAL, "%s: x or its checkpoint, not both", fn);
    const bool params = dweight || dbias;
    if (cols == 0 || (rows == 0 && !params)) return AMP_OK;
    if (rows > 0 && (!dy || (!x && !ckpt) || !mean || !rstd)) return fail(AMP_EINVAL, kNull, fn);
    if (!dx && !params) return AMP_OK;
    if (off_type(xc, dy, x, dx) || off_type(wc, weight, dweight, dbias) || off_type(amp::kF32, mean, rstd))
        return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    if (params) {
        const int64_t need = amp::norm_parts(rows, cols, dev) * 2 * cols * int64_t(sizeof(float));
        if (!workspace || workspace_bytes < need || misaligned(workspace, 16))
            return fail(AMP_EINVAL, "%s: the workspace needs %lld bytes, 16-byte aligned", fn, (long long)need);
    }
    return finish(amp::launch_norm_bwd(dy, x, xc, u8(ckpt), u8(ckpt_scales), rows, cols, weight, wc, mean, rstd, dx,
                                       dweight, dbias, static_cast<float *>(workspace), dev, cu(stream)),
                  fn);
}

// Checks shared by the four entries of the 8-bit checkpoints; act < 0: none.
static amp_status act_args(const char *fn, int act, bool any_act, amp_dtype dtype, int64_t rows, int64_t cols) {
    if (bad_shape(rows, cols)) return fail(AMP_EINVAL, kShape, fn);
    if (elem_code(dtype) < 0) return fail(AMP_EDTYPE, kType, fn);
    if (any_act && (act < AMP_ACT_GELU || act > AMP_ACT_SILU)) return fail(AMP_EINVAL, "%s: unknown act", fn);
    return AMP_OK;
}

amp_status amp_act_forward_mx8(amp_act act, const void *x, const void *up, amp_dtype dtype, int64_t rows,
                               int64_t cols, void *y, void *q, void *scales, void *q_up, void *scales_up,
                               amp_stream_t stream) {
    AMP_TRACE("amp_act_forward_mx8");
    const char *fn = "amp_act_forward_mx8";
    const amp_status st = act_args(fn, int(act), true, dtype, rows, cols);
    if (st != AMP_OK) return st;
    if ((q == nullptr) != (scales == nullptr) || (q_up == nullptr) != (scales_up == nullptr))
        return fail(AMP_EINVAL, "%s: a checkpoint and its scales go together", fn);
    if ((q_up != nullptr) != (up != nullptr && q != nullptr))
        return fail(AMP_EINVAL, "%s: with up, both checkpoints or none", fn);
    if (rows * cols == 0) return AMP_OK;
    if (!x || !y) return fail(AMP_EINVAL, kNull, fn);
    if (off_type(elem_code(dtype), x, up, y)) return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_act_fwd(int(act), x, up, elem_code(dtype), rows, cols, y, u8(q), u8(scales), u8(q_up),
                                      u8(scales_up), dev, cu(stream)),
                  fn);
}

amp_status amp_act_backward_mx8(amp_act act, const void *dy, amp_dtype dtype, int64_t rows, int64_t cols,
                                const void *q, const void *scales, const void *q_up, const void *scales_up,
                                void *dx, void *dup, amp_stream_t stream) {
    AMP_TRACE("amp_act_backward_mx8");
    const char *fn = "amp_act_backward_mx8";
    const amp_status st = act_args(fn, int(act), true, dtype, rows, cols);
    if (st != AMP_OK) return st;
    if ((q_up == nullptr) != (scales_up == nullptr) || (q_up == nullptr) != (dup == nullptr))
        return fail(AMP_EINVAL, "%s: q_up, scales_up and dup go together", fn);
    if (rows * cols == 0) return AMP_OK;
    if (!dy || !q || !scales || !dx) return fail(AMP_EINVAL, kNull, fn);
    if (off_type(elem_code(dtype), dy, dx, dup)) return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_act_bwd(int(act), dy, elem_code(dtype), rows, cols, u8(q), u8(scales), u8(q_up),
                                      u8(scales_up), dx, dup, dev, cu(stream)),
                  fn);
}

amp_status amp_ckpt8_save(const void *x, amp_dtype x_dtype, int64_t rows, int64_t cols, void *q, void *scales,
                          amp_stream_t stream) {
    AMP_TRACE("amp_ckpt8_save");
    const char *fn = "amp_ckpt8_save";
    const amp_status st = act_args(fn, 0, false, x_dtype, rows, cols);
    if (st != AMP_OK || rows * cols == 0) return st;
    if (!x || !q || !scales) return fail(AMP_EINVAL, kNull, fn);
    if (off_type(elem_code(x_dtype), x)) return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_act_fwd(-1, x, nullptr, elem_code(x_dtype), rows, cols, nullptr, u8(q), u8(scales),
                                      nullptr, nullptr, dev, cu(stream)),
                  fn);
}

amp_status amp_ckpt8_restore(const void *q, const void *scales, int64_t rows, int64_t cols, void *out,
                             amp_dtype out_dtype, amp_stream_t stream) {
    AMP_TRACE("amp_ckpt8_restore");
    const char *fn = "amp_ckpt8_restore";
    const amp_status st = act_args(fn, 0, false, out_dtype, rows, cols);
    if (st != AMP_OK || rows * cols == 0) return st;
    if (!q || !scales || !out) return fail(AMP_EINVAL, kNull, fn);
    if (off_type(elem_code(out_dtype), out)) return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_act_bwd(-1, nullptr, elem_code(out_dtype), rows, cols, u8(q), u8(scales), nullptr,
                                      nullptr, out, nullptr, dev, cu(stream)),
                  fn);
}

static bool known_act(int32_t act) { return act == AMP_ACT_NONE || (act >= AMP_ACT_GELU && act <= AMP_ACT_SILU); }

static amp_status linear(const char *fn, const void *a, const void *a_scales, const void *b, const void *b_scales,
                         int64_t m, int64_t n, int64_t k, const void *bias, amp_dtype bias_dtype, int32_t act,
                         const void *residual, void *out, amp_dtype out_dtype, void *q, void *scales,
                         amp_stream_t stream, amp::Fp4Limits limits) {
    if (bad_shape(m, n) || bad_shape(m, k) || bad_shape(n, k) || k > (int64_t(1) << 27))
        return fail(AMP_EINVAL, kShape, fn);
    const int oc = elem_code(out_dtype), bc = bias ? elem_code(bias_dtype) : int(amp::kF32);
    if (oc < 0 || bc < 0 || (bc != amp::kF32 && bc != oc)) return fail(AMP_EDTYPE, kType, fn);
    if (!known_act(act)) return fail(AMP_EINVAL, "%s: unknown act", fn);
    if ((q == nullptr) != (scales == nullptr)) return fail(AMP_EINVAL, "%s: q and scales go together", fn);
    if (m * n == 0) return AMP_OK;
    if (!out || (k > 0 && (!a || !a_scales || !b || !b_scales))) return fail(AMP_EINVAL, kNull, fn);
    if (misaligned(a, 16) || misaligned(a_scales, 16) || misaligned(b, 16) || misaligned(b_scales, 16))
        return fail(AMP_EINVAL, "%s: operands must be 16-byte aligned", fn);
    if (off_type(oc, out, residual) || off_type(bc, bias)) return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_fp4_linear(a, u8(a_scales), b, u8(b_scales), m, n, k, bias, bc, act, residual, out, oc,
                                         u8(q), u8(scales), dev, cu(stream), limits),
                  fn);
}

amp_status fp4_linear_mx(const void *a, const void *a_scales, const void *b, const void *b_scales, int64_t m,
                         int64_t n, int64_t k, const void *bias, amp_dtype bias_dtype, int32_t act,
                         const void *residual, void *out, amp_dtype out_dtype, void *q, void *scales,
                         amp_stream_t stream) {
    AMP_TRACE("fp4_linear_mx");
    return linear("fp4_linear_mx", a, a_scales, b, b_scales, m, n, k, bias, bias_dtype, act, residual, out, out_dtype,
                  q, scales, stream, {30, 3, 0});
}

amp_status fp4_linear_mx_selftest(const void *a, const void *a_scales, const void *b, const void *b_scales, int64_t m,
                                  int64_t n, int64_t k, const void *bias, amp_dtype bias_dtype, int32_t act,
                                  const void *residual, void *out, amp_dtype out_dtype, void *q, void *scales,
                                  int32_t role, int32_t stages, int32_t limit_log2_ns, amp_stream_t stream) {
    AMP_TRACE("fp4_linear_mx_selftest");
    const char *fn = "fp4_linear_mx_selftest";
    if (role < 0 || role > 2 || stages < 0) return fail(AMP_EINVAL, "%s: role not in [0, 2] or stages < 0", fn);
    if (limit_log2_ns < 0 || limit_log2_ns > 30) return fail(AMP_EINVAL, "%s: limit above 2^30 ns", fn);
    return linear(fn, a, a_scales, b, b_scales, m, n, k, bias, bias_dtype, act, residual, out, out_dtype, q, scales,
                  stream, {uint8_t(limit_log2_ns), uint8_t(role), uint32_t(stages)});
}

// The element codes of a tensor and of a bias gradient next to it (f32, or the tensor's).
static bool bias_types(amp_dtype dtype, amp_dtype bias_dtype, bool bias, int &ec, int &bc) {
    ec = elem_code(dtype);
    bc = bias ? elem_code(bias_dtype) : int(amp::kF32);
    return ec >= 0 && bc >= 0 && (bc == amp::kF32 || bc == ec);
}
// Zeros for a bias gradient over no rows.
static amp_status no_rows(const char *fn, void *dbias, int bc, int64_t cols, cudaStream_t s) {
    if (!dbias || cols == 0) return AMP_OK;
    return finish(cudaMemsetAsync(dbias, 0, size_t(cols) * (bc == amp::kF32 ? 4 : 2), s), fn);
}

amp_status amp_bias_act_backward_mx8(int32_t act, const void *dy, amp_dtype dtype, int64_t rows, int64_t cols,
                                     const void *q, const void *scales, void *dz, void *dbias, amp_dtype bias_dtype,
                                     amp_stream_t stream) {
    AMP_TRACE("amp_bias_act_backward_mx8");
    const char *fn = "amp_bias_act_backward_mx8";
    if (bad_shape(rows, cols)) return fail(AMP_EINVAL, kShape, fn);
    int ec, bc;
    if (!bias_types(dtype, bias_dtype, true, ec, bc)) return fail(AMP_EDTYPE, kType, fn);
    if (!known_act(act)) return fail(AMP_EINVAL, "%s: unknown act", fn);
    const bool none = act == AMP_ACT_NONE;
    if (none ? (q || scales || dz) : ((q == nullptr) != (scales == nullptr)))
        return fail(AMP_EINVAL, "%s: q, scales and dz go with an activation", fn);
    if (cols == 0) return AMP_OK;
    if (!dbias) return fail(AMP_EINVAL, kNull, fn);
    if (off_type(ec, dy, dz) || off_type(bc, dbias)) return fail(AMP_EINVAL, kOff, fn);
    if (rows == 0) return no_rows(fn, dbias, bc, cols, cu(stream));
    if (!dy || (!none && (!q || !dz))) return fail(AMP_EINVAL, kNull, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_bias_bwd(act, dy, ec, rows, cols, u8(q), u8(scales), dz, dbias, bc, dev, cu(stream)),
                  fn);
}

// p as the number of 65536 that drops, or -1.
static int64_t drop_of(double p) { return p >= 0.0 && p <= 1.0 ? int64_t(std::nearbyint(p * 65536.0)) : -1; }
static amp_status dropout_args(const char *fn, int64_t rows, int64_t cols, double p, int32_t site) {
    if (bad_shape(rows, cols)) return fail(AMP_EINVAL, kShape, fn);
    if (drop_of(p) < 0) return fail(AMP_EINVAL, "%s: p must be in [0, 1]", fn);
    if (site < 0 || site >= (1 << 30)) return fail(AMP_EINVAL, "%s: site must be in [0, 2^30)", fn);
    return AMP_OK;
}

amp_status amp_dropout_forward(const void *x, amp_dtype dtype, int64_t rows, int64_t cols, double p, uint64_t seed,
                               const int32_t *step_dev, int32_t site, const void *residual, void *y,
                               amp_stream_t stream) {
    AMP_TRACE("amp_dropout_forward");
    const char *fn = "amp_dropout_forward";
    const amp_status st = dropout_args(fn, rows, cols, p, site);
    if (st != AMP_OK) return st;
    const int ec = elem_code(dtype);
    if (ec < 0) return fail(AMP_EDTYPE, kType, fn);
    if (rows * cols == 0) return AMP_OK;
    if (!x || !y) return fail(AMP_EINVAL, kNull, fn);
    if (off_type(ec, x, residual, y) || off_type(amp::kF32, step_dev)) return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_dropout(x, residual, ec, rows, cols, uint32_t(drop_of(p)), seed, step_dev,
                                      (1u << 30) + uint32_t(site), y, nullptr, amp::kF32, dev, cu(stream)),
                  fn);
}

amp_status amp_dropout_backward(const void *dy, amp_dtype dtype, int64_t rows, int64_t cols, double p, uint64_t seed,
                                const int32_t *step_dev, int32_t site, void *dx, void *dbias, amp_dtype bias_dtype,
                                amp_stream_t stream) {
    AMP_TRACE("amp_dropout_backward");
    const char *fn = "amp_dropout_backward";
    const amp_status st = dropout_args(fn, rows, cols, p, site);
    if (st != AMP_OK) return st;
    int ec, bc;
    if (!bias_types(dtype, bias_dtype, dbias != nullptr, ec, bc)) return fail(AMP_EDTYPE, kType, fn);
    if (off_type(ec, dy, dx) || off_type(amp::kF32, step_dev) || off_type(bc, dbias)) return fail(AMP_EINVAL, kOff, fn);
    if (rows * cols == 0) return no_rows(fn, dbias, bc, cols, cu(stream));
    if (!dy || !dx) return fail(AMP_EINVAL, kNull, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_dropout(dy, nullptr, ec, rows, cols, uint32_t(drop_of(p)), seed, step_dev,
                                      (1u << 30) + uint32_t(site), dx, dbias, bc, dev, cu(stream)),
                  fn);
}

// A matrix whose rows lie ld elements apart; a row's 16-byte pieces are counted in 32 bits,
// with a batch of loads behind the last one.
static bool bad_rows(int64_t rows, int64_t cols, int64_t ld) {
    return bad_shape(rows, cols) || ld < cols || bad_shape(rows, ld) || cols > (int64_t(1) << 30);
}

amp_status amp_token_logprobs_forward(const void *z, amp_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                                      const int64_t *targets, float *logp, float *entropy, float *stats,
                                      int64_t *top_ids, float *top_logp, int32_t top_n, amp_stream_t stream) {
    AMP_TRACE("amp_token_logprobs_forward");
    const char *fn = "amp_token_logprobs_forward";
    if (bad_rows(rows, cols, ld)) return fail(AMP_EINVAL, kShape, fn);
    const int ec = elem_code(dtype);
    if (ec < 0) return fail(AMP_EDTYPE, kType, fn);
    if (top_n < 0 || top_n > 32) return fail(AMP_EINVAL, "%s: top_n must be in [0, 32]", fn);
    if ((top_ids == nullptr) != (top_logp == nullptr) || (top_n == 0 && top_ids))
        return fail(AMP_EINVAL, "%s: top_ids, top_logp and top_n go together", fn);
    if (rows == 0) return AMP_OK;
    if (cols == 0) return fail(AMP_EINVAL, "%s: a row needs a logit", fn);
    if (logp && !targets) return fail(AMP_EINVAL, "%s: logp needs targets", fn);
    if (!z || (top_n > 0 && !top_ids)) return fail(AMP_EINVAL, kNull, fn);
    if (off_type(ec, z) || off_type(amp::kF32, logp, entropy, stats, top_logp) || misaligned(targets, 8) ||
        misaligned(stats, 8) || misaligned(top_ids, 8))
        return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_logprobs_fwd(z, ec, rows, cols, ld, targets, logp, entropy, stats, top_ids, top_logp,
                                           top_n, dev, cu(stream)),
                  fn);
}

// Whether two matrices of this shape and element size share an element without being one
// and the same.  Rows of one stride may lie between each other's (column slices of one
// buffer); of two strides, the ranges they span have to be apart.
static bool overlap_partly(const void *a, int64_t lda, const void *b, int64_t ldb, int64_t rows, int64_t cols,
                           int64_t esz) {
    if (a == b && (rows == 1 || lda == ldb)) return false;
    const char *lo = static_cast<const char *>(a), *hi = static_cast<const char *>(b);
    if (hi < lo) {
        std::swap(lo, hi);
        std::swap(lda, ldb);
    }
    const int64_t d = hi - lo;  // bytes; the lower one spans ((rows - 1) lda + cols) elements
    if (d >= ((rows - 1) * lda + cols) * esz) return false;
    if (rows == 1 || lda != ldb) return true;
    // a row of the upper one starts `in` bytes behind the start of a row of the lower one
    const int64_t in = d % (lda * esz), past = d / (lda * esz);
    return in < cols * esz || (past + 1 < rows && in > (lda - cols) * esz);
}

amp_status amp_token_logprobs_backward(const float *dlogp, const void *z, amp_dtype dtype, int64_t rows, int64_t cols,
                                       int64_t ld, const int64_t *targets, const float *stats, const float *entropy,
                                       const float *dentropy, const float *scale_dev, void *dz, int64_t dld,
                                       amp_stream_t stream) {
    AMP_TRACE("amp_token_logprobs_backward");
    const char *fn = "amp_token_logprobs_backward";
    if (bad_rows(rows, cols, ld) || bad_rows(rows, cols, dld)) return fail(AMP_EINVAL, kShape, fn);
    const int ec = elem_code(dtype);
    if (ec < 0) return fail(AMP_EDTYPE, kType, fn);
    if (rows * cols == 0) return AMP_OK;
    if (dlogp && !targets) return fail(AMP_EINVAL, "%s: dlogp needs targets", fn);
    if (dentropy && !entropy) return fail(AMP_EINVAL, "%s: dentropy needs the entropy", fn);
    if (!z || !stats || !dz) return fail(AMP_EINVAL, kNull, fn);
    if (dz == z && dld != ld) return fail(AMP_EINVAL, "%s: in place, the rows need one stride", fn);
    if (overlap_partly(z, ld, dz, dld, rows, cols, ec == amp::kF32 ? 4 : 2))
        return fail(AMP_EINVAL, "%s: dz overlaps z without being z", fn);
    if (off_type(ec, z, dz) || off_type(amp::kF32, dlogp, entropy, dentropy, scale_dev) || misaligned(targets, 8) ||
        misaligned(stats, 8))
        return fail(AMP_EINVAL, kOff, fn);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return finish(e, fn);
    return finish(amp::launch_logprobs_bwd(z, ec, rows, cols, ld, targets, stats, dlogp, entropy, dentropy, scale_dev,
                                           dz, dld, dev, cu(stream)),
                  fn);
}

}  // extern "C"
