"""The forward/backward operators (declared in include/ampops.h): microscaled
4-bit quantisation and products, layer norm, and activations whose inputs are
kept in 8 bits.

As in ``_lib``: argument marshalling only, here by ``csrc/ops_bind.cpp`` (built
into ``_ops_bind.so``), because the smallest of these calls take microseconds.
Each function checks its tensors (contiguous, on one GPU, of the right type and
size: ``ValueError``), passes pointers, sizes and the stream (None: that GPU's
current one) to the C entry point of the same name, with the tensors' GPU made
current, and raises ``AmpError`` on a non-OK status.  Outputs are the caller's
tensors; nothing is allocated except by the two ``*_buffers`` helpers and
``amp_layer_norm_workspace``, which a program calls once.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib as A
from ._lib import P, _check, _stream

# every symbol include/ampops.h declares
EXPORTS = ("fp4_mx_bytes", "fp4_mx_scale_bytes", "fp4_quant_mx", "fp4_dequant_mx",
           "fp4_product_mx", "fp4_mx_check", "fp4_product_mx_selftest", "amp_layer_norm_forward",
           "amp_layer_norm_workspace_bytes", "amp_layer_norm_backward", "amp_act_forward_mx8",
           "amp_act_backward_mx8", "amp_ckpt8_save", "amp_ckpt8_restore")
# those that _ops_bind calls, in the order it takes their addresses
_BOUND = ("fp4_quant_mx", "fp4_dequant_mx", "fp4_product_mx", "amp_layer_norm_forward",
          "amp_layer_norm_backward", "amp_act_forward_mx8", "amp_act_backward_mx8",
          "amp_ckpt8_save", "amp_ckpt8_restore")

_library = None
_native = None


def _load():
    """The shared library with the prototypes of these functions declared."""
    global _library
    if _library is not None:
        return _library
    L = A.load()
    i32, i64, dbl = ctypes.c_int, ctypes.c_int64, ctypes.c_double
    L.fp4_mx_bytes.argtypes = [i64, i64]
    L.fp4_mx_scale_bytes.argtypes = [i64, i64]
    L.fp4_quant_mx.argtypes = [P, i32, i64, i64, P, P, P, P, P, P]
    L.fp4_dequant_mx.argtypes = [P, P, i64, i64, P, i32, P]
    L.fp4_product_mx.argtypes = [P, P, P, P, i64, i64, i64, P, i32, P]
    L.fp4_mx_check.argtypes = [P]
    L.fp4_product_mx_selftest.argtypes = [P, P, P, P, i64, i64, i64, P, i32, i32, i32, i32, P]
    L.amp_layer_norm_forward.argtypes = [P, i32, i64, i64, P, P, i32, dbl, P, P, P, P, P, P]
    L.amp_layer_norm_workspace_bytes.argtypes = [i64, i64]
    L.amp_layer_norm_backward.argtypes = [P, P, i32, P, P, i64, i64, P, i32] + [P] * 6 + [i64, P]
    L.amp_act_forward_mx8.argtypes = [i32, P, P, i32, i64, i64, P, P, P, P, P, P]
    L.amp_act_backward_mx8.argtypes = [i32, P, i32, i64, i64, P, P, P, P, P, P, P]
    L.amp_ckpt8_save.argtypes = [P, i32, i64, i64, P, P, P]
    L.amp_ckpt8_restore.argtypes = [P, P, i64, i64, P, i32, P]
    for name in EXPORTS:
        getattr(L, name).restype = i64 if name.endswith("_bytes") else ctypes.c_int
    _library = L
    return L


def _bound():
    """The marshalling module, bound to the loaded library (raises if not built)."""
    global _native
    if _native is None:
        L = _load()
        try:
            from . import _ops_bind
        except ImportError as e:
            raise RuntimeError("_ops_bind.so is missing or was built for another torch: build it "
                               "with `python -c 'import __graft_entry__ as g; g.build()'`") from e
        _ops_bind.bind(*[ctypes.cast(getattr(L, n), P).value for n in _BOUND])
        _native = _ops_bind
    return _native


def fp4_mx_buffers(rows: int, cols: int, device="cuda"):
    """(q, scales) for a [rows, cols] matrix: uint8 [rows, 16 ceil(cols/32)], the tiled scales."""
    nq, ns = _load().fp4_mx_bytes(rows, cols), _load().fp4_mx_scale_bytes(rows, cols)
    if nq < 0 or ns < 0:
        raise ValueError(f"[{rows}, {cols}]: negative or too large")
    return (torch.empty((rows, -(-cols // 32) * 16), dtype=torch.uint8, device=device),
            torch.empty(ns, dtype=torch.uint8, device=device))


def ckpt8_buffers(rows: int, cols: int, device="cuda"):
    """(q, scales) of a checkpoint: float8_e4m3fn [rows, cols], uint8 [rows, ceil(cols/32)]."""
    return (torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((rows, -(-cols // 32)), dtype=torch.uint8, device=device))


def amp_layer_norm_workspace(x):
    """Scratch for amp_layer_norm_backward on tensors of x's shape (allocates: keep it)."""
    cols = x.shape[-1]
    rows = x.shape[:-1].numel()
    with torch.cuda.device(x.device):
        n = _load().amp_layer_norm_workspace_bytes(rows, cols)
    if n < 0:
        raise ValueError(f"[{rows}, {cols}]: negative or too large")
    return torch.empty(max(n, 16), dtype=torch.uint8, device=x.device)


def fp4_quant_mx(x, q, scales, qt=None, scales_t=None, skip_if=None, stream=None):
    """x [rows, cols] -> 4-bit blocks along its rows (q, scales) and, with qt, of its transpose."""
    st = (_native or _bound()).quant(x, q, scales, qt, scales_t, skip_if, stream)
    if st:
        _check("fp4_quant_mx", st)


def fp4_dequant_mx(q, scales, out, stream=None):
    """out [rows, cols] = the values of the packed matrix of that shape."""
    st = (_native or _bound()).dequant(q, scales, out, stream)
    if st:
        _check("fp4_dequant_mx", st)


def fp4_product_mx(a, a_scales, b, b_scales, k: int, out, stream=None):
    """out [m, n] = A [m, k] times B [n, k] transposed, both packed in 4 bits."""
    st = (_native or _bound()).product(a, a_scales, b, b_scales, k, out, stream)
    if st:
        _check("fp4_product_mx", st)


def fp4_mx_check(stream=None):
    """Raise AmpError(AMP_ETIMEOUT) if a bounded wait of fp4_product_mx gave up on the current
    device (synchronises)."""
    _check("fp4_mx_check", _load().fp4_mx_check(_stream(stream)))


def amp_layer_norm_forward(x, weight, bias, eps: float, y, mean=None, rstd=None, saved=None,
                           stream=None):
    """Layer norm over the last dimension; saved: (q, scales) to keep x in 8 bits."""
    st = (_native or _bound()).norm_forward(x, weight, bias, eps, y, mean, rstd, saved, stream)
    if st:
        _check("amp_layer_norm_forward", st)


def amp_layer_norm_backward(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None,
                            workspace=None, saved=None, stream=None):
    """Gradients of the layer norm; x None: from the 8-bit checkpoint saved = (q, scales)."""
    st = (_native or _bound()).norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias,
                                             workspace, saved, stream)
    if st:
        _check("amp_layer_norm_backward", st)


def amp_act_forward_mx8(x, kind: str, y, saved=None, up=None, saved_up=None, stream=None):
    """y = f(x) [* up], kind "gelu", "gelu_tanh" or "silu"; saved / saved_up: (q, scales) that
    take x and up in 8 bits."""
    st = (_native or _bound()).act_forward(x, kind, y, saved, up, saved_up, stream)
    if st:
        _check("amp_act_forward_mx8", st)


def amp_act_backward_mx8(dy, kind: str, saved, dx, saved_up=None, dup=None, stream=None):
    """dx (and, gated, dup) from dy and the 8-bit checkpoints of the forward's inputs."""
    st = (_native or _bound()).act_backward(dy, kind, saved, dx, saved_up, dup, stream)
    if st:
        _check("amp_act_backward_mx8", st)


def amp_ckpt8_save(x, q, scales, stream=None):
    """The 8-bit checkpoint of x."""
    st = (_native or _bound()).save(x, q, scales, stream)
    if st:
        _check("amp_ckpt8_save", st)


def amp_ckpt8_restore(q, scales, out, stream=None):
    """out = the values of an 8-bit checkpoint."""
    st = (_native or _bound()).restore(q, scales, out, stream)
    if st:
        _check("amp_ckpt8_restore", st)
