"""ctypes binding of the forward/backward operators (declared in
include/ampops.h): microscaled 4-bit quantisation and products, layer norm,
and activations whose inputs are kept in 8 bits.

As in ``_lib``: argument marshalling only.  Each function checks its tensors
(contiguous, on the GPU, of the right type and size: ``ValueError``), passes
pointers, sizes and the stream to the C entry point of the same name and
raises ``AmpError`` on a non-OK status.  Outputs are the caller's tensors;
nothing is allocated except by the two ``*_buffers`` helpers and
``amp_layer_norm_workspace``, which a program calls once.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib as A
from ._lib import DT, P, _F32, _I32, _TORCH_DT, _buf, _check, _stream

# every symbol include/ampops.h declares
EXPORTS = ("fp4_mx_bytes", "fp4_mx_scale_bytes", "fp4_quant_mx", "fp4_dequant_mx",
           "fp4_product_mx", "fp4_mx_check", "amp_layer_norm_forward",
           "amp_layer_norm_workspace_bytes", "amp_layer_norm_backward", "amp_act_forward_mx8",
           "amp_act_backward_mx8", "amp_ckpt8_save", "amp_ckpt8_restore")
ACTS = {"gelu": 0, "gelu_tanh": 1, "silu": 2}

_ready = None


def _load():
    """The shared library with these prototypes declared."""
    global _ready
    if _ready is not None:
        return _ready
    L = A.load()
    i32, i64, dbl = ctypes.c_int, ctypes.c_int64, ctypes.c_double
    L.fp4_mx_bytes.argtypes = [i64, i64]
    L.fp4_mx_scale_bytes.argtypes = [i64, i64]
    L.fp4_quant_mx.argtypes = [P, i32, i64, i64, P, P, P, P, P, P]
    L.fp4_dequant_mx.argtypes = [P, P, i64, i64, P, i32, P]
    L.fp4_product_mx.argtypes = [P, P, P, P, i64, i64, i64, P, i32, P]
    L.fp4_mx_check.argtypes = [P]
    L.amp_layer_norm_forward.argtypes = [P, i32, i64, i64, P, P, i32, dbl, P, P, P, P, P, P]
    L.amp_layer_norm_workspace_bytes.argtypes = [i64, i64]
    L.amp_layer_norm_backward.argtypes = [P, P, i32, P, P, i64, i64, P, i32, P, P, P, P, P, P, i64, P]
    L.amp_act_forward_mx8.argtypes = [i32, P, P, i32, i64, i64, P, P, P, P, P, P]
    L.amp_act_backward_mx8.argtypes = [i32, P, i32, i64, i64, P, P, P, P, P, P, P]
    L.amp_ckpt8_save.argtypes = [P, i32, i64, i64, P, P, P]
    L.amp_ckpt8_restore.argtypes = [P, P, i64, i64, P, i32, P]
    for name in EXPORTS:
        getattr(L, name).restype = i64 if name.endswith("_bytes") else ctypes.c_int
    _ready = L
    return L


def _mat(t, what: str):
    """(rows, cols) of a matrix; a 1-D tensor is one row, leading dimensions are rows."""
    if t.dim() == 0:
        raise ValueError(f"{what}: needs at least one dimension")
    cols = t.shape[-1]
    rows = 1
    for s in t.shape[:-1]:
        rows *= s
    return rows, cols


def _code(t, what: str) -> int:
    name = _TORCH_DT.get(t.dtype)
    if name not in ("f32", "f16", "bf16"):
        raise ValueError(f"{what}: dtype {t.dtype}; f32, f16 or bf16 is needed")
    return DT[name]


def _fp4_sizes(rows: int, cols: int):
    """Bytes of the packed elements and of the scales of a [rows, cols] matrix."""
    return rows * (-(-cols // 32)) * 16, (-(-rows // 128)) * (-(-cols // 128)) * 512


def fp4_mx_buffers(rows: int, cols: int, device="cuda"):
    """(q, scales) for a [rows, cols] matrix: uint8 [rows, 16 ceil(cols/32)] and the tiled scales."""
    nq, ns = _load().fp4_mx_bytes(rows, cols), _load().fp4_mx_scale_bytes(rows, cols)
    if nq < 0 or ns < 0:
        raise ValueError(f"[{rows}, {cols}]: negative or too large")
    return (torch.empty((rows, -(-cols // 32) * 16), dtype=torch.uint8, device=device),
            torch.empty(ns, dtype=torch.uint8, device=device))


def ckpt8_buffers(rows: int, cols: int, device="cuda"):
    """(q, scales) of an 8-bit checkpoint: float8_e4m3fn [rows, cols], uint8 [rows, ceil(cols/32)]."""
    return (torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((rows, -(-cols // 32)), dtype=torch.uint8, device=device))


def fp4_quant_mx(x, q, scales, qt=None, scales_t=None, skip_if=None, stream=None):
    """x [rows, cols] -> 4-bit blocks along its rows (q, scales) and, with qt, of its transpose."""
    rows, cols = _mat(x, "x")
    nq, ns = _fp4_sizes(rows, cols)
    nqt, nst = _fp4_sizes(cols, rows) if qt is not None else (0, 0)
    _check("fp4_quant_mx",
           _load().fp4_quant_mx(_buf(x, "x", numel=0), _code(x, "x"), rows, cols,
                                _buf(q, "q", itemsize=1, numel=nq),
                                _buf(scales, "scales", itemsize=1, numel=ns),
                                _buf(qt, "qt", itemsize=1, numel=nqt),
                                _buf(scales_t, "scales_t", itemsize=1, numel=nst),
                                _buf(skip_if, "skip_if", _I32), _stream(stream)))


def fp4_dequant_mx(q, scales, out, stream=None):
    """out [rows, cols] = the values of the packed matrix of that shape."""
    rows, cols = _mat(out, "out")
    nq, ns = _fp4_sizes(rows, cols)
    _check("fp4_dequant_mx",
           _load().fp4_dequant_mx(_buf(q, "q", itemsize=1, numel=nq),
                                  _buf(scales, "scales", itemsize=1, numel=ns), rows, cols,
                                  _buf(out, "out", numel=0), _code(out, "out"), _stream(stream)))


def fp4_product_mx(a, a_scales, b, b_scales, k: int, out, stream=None):
    """out [m, n] = A [m, k] times B [n, k] transposed, both packed in 4 bits."""
    m, n = _mat(out, "out")
    k = int(k)
    if k < 0:
        raise ValueError(f"k = {k}")
    na, nas = _fp4_sizes(m, k)
    nb, nbs = _fp4_sizes(n, k)
    _check("fp4_product_mx",
           _load().fp4_product_mx(_buf(a, "a", itemsize=1, numel=na),
                                  _buf(a_scales, "a_scales", itemsize=1, numel=nas),
                                  _buf(b, "b", itemsize=1, numel=nb),
                                  _buf(b_scales, "b_scales", itemsize=1, numel=nbs), m, n, k,
                                  _buf(out, "out", numel=0), _code(out, "out"), _stream(stream)))


def fp4_mx_check(stream=None):
    """Raise AmpError(AMP_ETIMEOUT) if a bounded wait of fp4_product_mx gave up (synchronises)."""
    _check("fp4_mx_check", _load().fp4_mx_check(_stream(stream)))


def _pair(saved, what: str, rows: int, cols: int):
    """Pointers of an 8-bit checkpoint (q, scales), or (None, None)."""
    if saved is None:
        return None, None
    q, s = saved
    return (_buf(q, what, torch.float8_e4m3fn, rows * cols),
            _buf(s, what + " scales", torch.uint8, rows * -(-cols // 32)))


def _same(t, what: str, like):
    """Pointer of a tensor with the type and size of another."""
    return _buf(t, what, like.dtype, like.numel()) if t is not None else None


def _params(w, others, cols: int):
    """The parameters' element type: of the first that is given (f32 if none is)."""
    given = [t for t in (w, *others) if t is not None]
    if any(t.dtype != given[0].dtype for t in given[1:]):
        raise ValueError("weight, bias and their gradients need one dtype")
    if any(t.numel() != cols for t in given):
        raise ValueError(f"weight, bias and their gradients need {cols} elements")
    return _code(given[0], "weight") if given else DT["f32"]


def amp_layer_norm_forward(x, weight, bias, eps: float, y, mean=None, rstd=None, saved=None,
                           stream=None):
    """Layer norm over the last dimension; saved: (q, scales) to keep x in 8 bits."""
    rows, cols = _mat(x, "x")
    wc = _params(weight, (bias,), cols)
    q, s = _pair(saved, "saved", rows, cols)
    _check("amp_layer_norm_forward",
           _load().amp_layer_norm_forward(_buf(x, "x", numel=0), _code(x, "x"), rows, cols,
                                          _buf(weight, "weight"), _buf(bias, "bias"), wc,
                                          float(eps), _same(y, "y", x),
                                          _buf(mean, "mean", _F32, rows),
                                          _buf(rstd, "rstd", _F32, rows), q, s, _stream(stream)))


def amp_layer_norm_workspace(x):
    """Scratch for amp_layer_norm_backward on tensors of x's shape (allocates: keep it)."""
    rows, cols = _mat(x, "x")
    with torch.cuda.device(x.device):
        n = _load().amp_layer_norm_workspace_bytes(rows, cols)
    if n < 0:
        raise ValueError(f"[{rows}, {cols}]: negative or too large")
    return torch.empty(max(n, 16), dtype=torch.uint8, device=x.device)


def amp_layer_norm_backward(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None,
                            workspace=None, saved=None, stream=None):
    """Gradients of the layer norm; x None: from the 8-bit checkpoint saved = (q, scales)."""
    rows, cols = _mat(dy, "dy")
    if (x is None) == (saved is None):
        raise ValueError("either x or saved")
    wc = _params(weight, (dweight, dbias), cols)
    q, s = _pair(saved, "saved", rows, cols)
    _check("amp_layer_norm_backward",
           _load().amp_layer_norm_backward(_buf(dy, "dy", numel=0), _same(x, "x", dy),
                                           _code(dy, "dy"), q, s, rows, cols,
                                           _buf(weight, "weight"), wc,
                                           _buf(mean, "mean", _F32, rows),
                                           _buf(rstd, "rstd", _F32, rows), _same(dx, "dx", dy),
                                           _buf(dweight, "dweight"), _buf(dbias, "dbias"),
                                           _buf(workspace, "workspace"),
                                           workspace.numel() * workspace.element_size()
                                           if workspace is not None else 0, _stream(stream)))


def _act(kind: str) -> int:
    if kind not in ACTS:
        raise ValueError(f"activation {kind!r}; one of {sorted(ACTS)}")
    return ACTS[kind]


def amp_act_forward_mx8(x, kind: str, y, saved=None, up=None, saved_up=None, stream=None):
    """y = f(x) [* up]; saved / saved_up: (q, scales) that take x and up in 8 bits."""
    rows, cols = _mat(x, "x")
    q, s = _pair(saved, "saved", rows, cols)
    qu, su = _pair(saved_up, "saved_up", rows, cols)
    _check("amp_act_forward_mx8",
           _load().amp_act_forward_mx8(_act(kind), _buf(x, "x", numel=0), _same(up, "up", x),
                                       _code(x, "x"), rows, cols, _same(y, "y", x), q, s, qu, su,
                                       _stream(stream)))


def amp_act_backward_mx8(dy, kind: str, saved, dx, saved_up=None, dup=None, stream=None):
    """dx (and, gated, dup) from dy and the 8-bit checkpoints of the forward's inputs."""
    rows, cols = _mat(dy, "dy")
    q, s = _pair(saved, "saved", rows, cols)
    qu, su = _pair(saved_up, "saved_up", rows, cols)
    _check("amp_act_backward_mx8",
           _load().amp_act_backward_mx8(_act(kind), _buf(dy, "dy", numel=0), _code(dy, "dy"), rows,
                                        cols, q, s, qu, su, _same(dx, "dx", dy),
                                        _same(dup, "dup", dy), _stream(stream)))


def amp_ckpt8_save(x, q, scales, stream=None):
    """The 8-bit checkpoint of x."""
    rows, cols = _mat(x, "x")
    _check("amp_ckpt8_save",
           _load().amp_ckpt8_save(_buf(x, "x", numel=0), _code(x, "x"), rows, cols,
                                  *_pair((q, scales), "q", rows, cols), _stream(stream)))


def amp_ckpt8_restore(q, scales, out, stream=None):
    """out = the values of an 8-bit checkpoint."""
    rows, cols = _mat(out, "out")
    _check("amp_ckpt8_restore",
           _load().amp_ckpt8_restore(*_pair((q, scales), "q", rows, cols), rows, cols,
                                     _buf(out, "out", numel=0), _code(out, "out"), _stream(stream)))
