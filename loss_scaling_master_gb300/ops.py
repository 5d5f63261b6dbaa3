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
from ._lib import P, _buf, _check

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
    L.amp_layer_norm_backward.argtypes = ([P, P, i32, P, P, i64, i64, P, i32] + [P] * 6 + [i64, P])
    L.amp_act_forward_mx8.argtypes = [i32, P, P, i32, i64, i64, P, P, P, P, P, P]
    L.amp_act_backward_mx8.argtypes = [i32, P, i32, i64, i64, P, P, P, P, P, P, P]
    L.amp_ckpt8_save.argtypes = [P, i32, i64, i64, P, P, P]
    L.amp_ckpt8_restore.argtypes = [P, P, i64, i64, P, i32, P]
    for name in EXPORTS:
        getattr(L, name).restype = i64 if name.endswith("_bytes") else ctypes.c_int
    _ready = L
    return L


# What follows runs once or more per argument of every call, next to 2.5 us for
# the call and launch themselves: the accepted case is tested in as few steps as
# there are conditions, and a refused tensor goes to _buf for its message.
_ELEM = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}
_F32, _I32, _U8, _E4M3 = torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn
_ONE_BYTE = frozenset((torch.uint8, torch.int8, torch.float8_e4m3fn, torch.float8_e5m2, torch.bool))
_raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _mat(t, what: str):
    """(rows, cols) of a matrix; a 1-D tensor is one row, leading dimensions are rows."""
    shape = t.shape
    if len(shape) == 2:
        return shape
    if len(shape) == 0:
        raise ValueError(f"{what}: needs at least one dimension")
    return shape[:-1].numel(), shape[-1]


def _code(t, what: str) -> int:
    code = _ELEM.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: dtype {t.dtype}; f32, f16 or bf16 is needed")
    return code


def _ptr(t, what: str, numel: int, dtype=None):
    """Address of a contiguous GPU tensor of the dtype with at least numel elements (None: none)."""
    if t is None:
        return None
    if t.is_cuda and t.is_contiguous() and t.numel() >= numel \
            and (dtype is None or t.dtype is dtype):
        return t.data_ptr()
    return _buf(t, what, dtype, numel)


def _bytes(t, what: str, nbytes: int):
    """Address of a contiguous GPU tensor of one-byte elements, at least nbytes of them."""
    if t is None:
        return None
    if t.is_cuda and t.is_contiguous() and t.numel() >= nbytes and t.dtype in _ONE_BYTE:
        return t.data_ptr()
    return _buf(t, what, numel=nbytes, itemsize=1)


def _stream(stream):
    """Handle of the stream: the current one of the current device for None."""
    if stream is None:
        return _raw_stream(_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _fp4_sizes(rows: int, cols: int):
    """Bytes of the packed elements and of the scales of a [rows, cols] matrix."""
    return rows * ((cols + 31) >> 5) * 16, ((rows + 127) >> 7) * ((cols + 127) >> 7) * 512


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


def fp4_quant_mx(x, q, scales, qt=None, scales_t=None, skip_if=None, stream=None):
    """x [rows, cols] -> 4-bit blocks along its rows (q, scales) and, with qt, of its transpose."""
    rows, cols = _mat(x, "x")
    nq, ns = _fp4_sizes(rows, cols)
    if qt is not None or scales_t is not None:
        nqt, nst = _fp4_sizes(cols, rows)
        qt, scales_t = _bytes(qt, "qt", nqt), _bytes(scales_t, "scales_t", nst)
    st = (_ready or _load()).fp4_quant_mx(
        _ptr(x, "x", 0), _code(x, "x"), rows, cols, _bytes(q, "q", nq),
        _bytes(scales, "scales", ns), qt, scales_t,
        None if skip_if is None else _ptr(skip_if, "skip_if", 1, _I32),
        _stream(stream))
    if st:
        _check("fp4_quant_mx", st)


def fp4_dequant_mx(q, scales, out, stream=None):
    """out [rows, cols] = the values of the packed matrix of that shape."""
    rows, cols = _mat(out, "out")
    nq, ns = _fp4_sizes(rows, cols)
    st = (_ready or _load()).fp4_dequant_mx(
        _bytes(q, "q", nq), _bytes(scales, "scales", ns), rows, cols, _ptr(out, "out", 0),
        _code(out, "out"), _stream(stream))
    if st:
        _check("fp4_dequant_mx", st)


def fp4_product_mx(a, a_scales, b, b_scales, k: int, out, stream=None):
    """out [m, n] = A [m, k] times B [n, k] transposed, both packed in 4 bits."""
    m, n = _mat(out, "out")
    if k < 0:
        raise ValueError(f"k = {k}")
    na, nas = _fp4_sizes(m, k)
    nb, nbs = _fp4_sizes(n, k)
    st = (_ready or _load()).fp4_product_mx(
        _bytes(a, "a", na), _bytes(a_scales, "a_scales", nas), _bytes(b, "b", nb),
        _bytes(b_scales, "b_scales", nbs), m, n, k, _ptr(out, "out", 0), _code(out, "out"),
        _stream(stream))
    if st:
        _check("fp4_product_mx", st)


def fp4_mx_check(stream=None):
    """Raise AmpError(AMP_ETIMEOUT) if a bounded wait of fp4_product_mx gave up (synchronises)."""
    _check("fp4_mx_check", _load().fp4_mx_check(_stream(stream)))


def _pair(saved, what: str, rows: int, cols: int):
    """Addresses of an 8-bit checkpoint (q, scales), or (None, None)."""
    if saved is None:
        return None, None
    q, s = saved
    return _ptr(q, what, rows * cols, _E4M3), _ptr(s, what, rows * ((cols + 31) >> 5), _U8)


def _same(t, what: str, like):
    """Address of a tensor with the type and size of another."""
    return None if t is None else _ptr(t, what, like.numel(), like.dtype)


def _params(cols: int, *given):
    """The element type of the parameters and their gradients (f32 if none is given)."""
    dtype = None
    for t in given:
        if t is None:
            continue
        if dtype is None:
            dtype = t.dtype
        elif t.dtype is not dtype:
            raise ValueError("weight, bias and their gradients need one dtype")
        if t.numel() != cols:
            raise ValueError(f"weight, bias and their gradients need {cols} elements")
    if dtype is None:
        return 1
    if dtype not in _ELEM:
        raise ValueError(f"weight: dtype {dtype}; f32, f16 or bf16 is needed")
    return _ELEM[dtype]


def amp_layer_norm_forward(x, weight, bias, eps: float, y, mean=None, rstd=None, saved=None,
                           stream=None):
    """Layer norm over the last dimension; saved: (q, scales) to keep x in 8 bits."""
    rows, cols = _mat(x, "x")
    wc = _params(cols, weight, bias)
    q, s = _pair(saved, "saved", rows, cols)
    st = (_ready or _load()).amp_layer_norm_forward(
        _ptr(x, "x", 0), _code(x, "x"), rows, cols, _ptr(weight, "weight", cols),
        _ptr(bias, "bias", cols), wc, eps, _same(y, "y", x), _ptr(mean, "mean", rows, _F32),
        _ptr(rstd, "rstd", rows, _F32), q, s, _stream(stream))
    if st:
        _check("amp_layer_norm_forward", st)


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
    wc = _params(cols, weight, dweight, dbias)
    q, s = _pair(saved, "saved", rows, cols)
    work = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = (_ready or _load()).amp_layer_norm_backward(
        _ptr(dy, "dy", 0), _same(x, "x", dy), _code(dy, "dy"), q, s, rows, cols,
        _ptr(weight, "weight", cols), wc, _ptr(mean, "mean", rows, _F32),
        _ptr(rstd, "rstd", rows, _F32), _same(dx, "dx", dy), _ptr(dweight, "dweight", cols),
        _ptr(dbias, "dbias", cols), _ptr(workspace, "workspace", 0), work, _stream(stream))
    if st:
        _check("amp_layer_norm_backward", st)


def _act(kind: str) -> int:
    act = ACTS.get(kind)
    if act is None:
        raise ValueError(f"activation {kind!r}; one of {sorted(ACTS)}")
    return act


def amp_act_forward_mx8(x, kind: str, y, saved=None, up=None, saved_up=None, stream=None):
    """y = f(x) [* up]; saved / saved_up: (q, scales) that take x and up in 8 bits."""
    rows, cols = _mat(x, "x")
    q, s = _pair(saved, "saved", rows, cols)
    qu, su = _pair(saved_up, "saved_up", rows, cols)
    st = (_ready or _load()).amp_act_forward_mx8(
        _act(kind), _ptr(x, "x", 0), _same(up, "up", x), _code(x, "x"), rows, cols,
        _same(y, "y", x), q, s, qu, su, _stream(stream))
    if st:
        _check("amp_act_forward_mx8", st)


def amp_act_backward_mx8(dy, kind: str, saved, dx, saved_up=None, dup=None, stream=None):
    """dx (and, gated, dup) from dy and the 8-bit checkpoints of the forward's inputs."""
    rows, cols = _mat(dy, "dy")
    q, s = _pair(saved, "saved", rows, cols)
    qu, su = _pair(saved_up, "saved_up", rows, cols)
    st = (_ready or _load()).amp_act_backward_mx8(
        _act(kind), _ptr(dy, "dy", 0), _code(dy, "dy"), rows, cols, q, s, qu, su,
        _same(dx, "dx", dy), _same(dup, "dup", dy), _stream(stream))
    if st:
        _check("amp_act_backward_mx8", st)


def amp_ckpt8_save(x, q, scales, stream=None):
    """The 8-bit checkpoint of x."""
    rows, cols = _mat(x, "x")
    st = (_ready or _load()).amp_ckpt8_save(_ptr(x, "x", 0), _code(x, "x"), rows, cols,
                                            *_pair((q, scales), "q", rows, cols), _stream(stream))
    if st:
        _check("amp_ckpt8_save", st)


def amp_ckpt8_restore(q, scales, out, stream=None):
    """out = the values of an 8-bit checkpoint."""
    rows, cols = _mat(out, "out")
    st = (_ready or _load()).amp_ckpt8_restore(*_pair((q, scales), "q", rows, cols), rows, cols,
                                               _ptr(out, "out", 0), _code(out, "out"),
                                               _stream(stream))
    if st:
        _check("amp_ckpt8_restore", st)
