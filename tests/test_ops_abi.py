"""include/ampops.h: every symbol is exported, and wrong arguments are refused
with a status and a message before anything reaches the GPU; and the plain
64-bit reference that the GPU tests use agrees with what it is made from."""
import ctypes
import math
import os
import re

import pytest
import torch

import ops_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EDTYPE, OK = -1, -2, 0
BF16, F16, F32, E4M3 = 3, 2, 1, 4
D = ctypes.c_void_p(4096)     # never dereferenced: every call here is refused or empty
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def lib():
    from loss_scaling_master_gb300 import build as B
    B.build()
    from loss_scaling_master_gb300 import ops
    return ops._load()


def test_every_declared_symbol_is_exported(lib):
    src = open(os.path.join(ROOT, "include", "ampops.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:amp_status|int64_t)\s+(\w+)\s*\(", src, flags=re.M)))
    from loss_scaling_master_gb300.ops import EXPORTS
    assert names == sorted(EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_sizes(lib):
    assert lib.fp4_mx_bytes(3, 33) == 3 * 32 and lib.fp4_mx_bytes(0, 5) == 0
    assert lib.fp4_mx_scale_bytes(129, 129) == 4 * 512 and lib.fp4_mx_scale_bytes(1, 1) == 512
    for r, c in ((-1, 4), (4, -1), (1 << 31, 4), (1 << 30, 1 << 31)):
        assert lib.fp4_mx_bytes(r, c) == -1 and lib.fp4_mx_scale_bytes(r, c) == -1
        assert lib.amp_layer_norm_workspace_bytes(r, c) == -1


@pytest.mark.parametrize("args,want", [
    ((D, BF16, -1, 4, D, D, None, None), EINVAL),
    ((D, BF16, 1 << 31, 4, D, D, None, None), EINVAL),
    ((D, E4M3, 4, 4, D, D, None, None), EDTYPE),
    ((D, 77, 4, 4, D, D, None, None), EDTYPE),
    ((None, BF16, 4, 4, D, D, None, None), EINVAL),
    ((D, BF16, 4, 4, None, D, None, None), EINVAL),
    ((D, BF16, 4, 4, D, None, None, None), EINVAL),
    ((D, BF16, 4, 4, D, D, D, None), EINVAL),
    ((D, BF16, 4, 4, D, D, None, D), EINVAL),
    ((D, BF16, 4, 4, ODD, D, None, None), EINVAL),
    ((D, BF16, 4, 4, D, ODD, None, None), EINVAL),
    ((None, BF16, 0, 4, None, None, None, None), OK),
    ((None, BF16, 4, 0, None, None, None, None), OK),
])
def test_fp4_quant_refusals(lib, args, want):
    assert lib.fp4_quant_mx(*args, None, None) == want
    if want != OK:
        assert lib.amp_last_error().startswith(b"fp4_quant_mx")


@pytest.mark.parametrize("args,want", [
    ((D, D, -1, 4, D, BF16), EINVAL), ((D, D, 4, 4, D, E4M3), EDTYPE), ((None, D, 4, 4, D, F32), EINVAL),
    ((D, None, 4, 4, D, F32), EINVAL), ((D, D, 4, 4, None, F32), EINVAL), ((ODD, D, 4, 4, D, F32), EINVAL),
    ((None, None, 4, 0, None, F16), OK),
])
def test_fp4_dequant_refusals(lib, args, want):
    assert lib.fp4_dequant_mx(*args, None) == want


@pytest.mark.parametrize("args,want", [
    ((D, D, D, D, -1, 4, 4, D, BF16), EINVAL), ((D, D, D, D, 4, -1, 4, D, BF16), EINVAL),
    ((D, D, D, D, 4, 4, -1, D, BF16), EINVAL), ((D, D, D, D, 4, 4, (1 << 27) + 1, D, BF16), EINVAL),
    ((D, D, D, D, 1 << 31, 4, 4, D, BF16), EINVAL),
    ((D, D, D, D, 4, 4, 4, D, E4M3), EDTYPE), ((None, D, D, D, 4, 4, 4, D, BF16), EINVAL),
    ((D, None, D, D, 4, 4, 4, D, BF16), EINVAL), ((D, D, None, D, 4, 4, 4, D, BF16), EINVAL),
    ((D, D, D, None, 4, 4, 4, D, BF16), EINVAL), ((D, D, D, D, 4, 4, 4, None, BF16), EINVAL),
    ((ODD, D, D, D, 4, 4, 4, D, BF16), EINVAL), ((D, D, ODD, D, 4, 4, 4, D, BF16), EINVAL),
    ((D, D, D, D, 4, 4, 4, ODD, BF16), EINVAL), ((D, D, D, D, 4, 4, 4, ctypes.c_void_p(4098), F32), EINVAL),
    ((None, None, None, None, 0, 4, 4, None, BF16), OK), ((None, None, None, None, 4, 0, 4, None, F32), OK),
])
def test_fp4_product_refusals(lib, args, want):
    assert lib.fp4_product_mx(*args, None) == want


@pytest.mark.parametrize("args,want", [
    ((D, BF16, -1, 4, D, D, F32, 1e-5, D, D, D, None, None), EINVAL),
    ((D, E4M3, 4, 4, D, D, F32, 1e-5, D, D, D, None, None), EDTYPE),
    ((D, BF16, 4, 4, D, D, F16, 1e-5, D, D, D, None, None), EDTYPE),
    ((D, BF16, 4, 4, D, D, F32, -1.0, D, D, D, None, None), EINVAL),
    ((D, BF16, 4, 4, D, D, F32, math.nan, D, D, D, None, None), EINVAL),
    ((D, BF16, 4, 4, D, D, F32, math.inf, D, D, D, None, None), EINVAL),
    ((D, BF16, 4, 4, D, D, F32, 1e-5, D, D, D, D, None), EINVAL),
    ((D, BF16, 4, 4, D, D, F32, 1e-5, D, D, D, None, D), EINVAL),
    ((None, BF16, 4, 4, D, D, F32, 1e-5, D, D, D, None, None), EINVAL),
    ((D, BF16, 4, 4, D, D, F32, 1e-5, None, D, D, None, None), EINVAL),
    ((None, BF16, 0, 4, None, None, F32, 1e-5, None, None, None, None, None), OK),
])
def test_layer_norm_forward_refusals(lib, args, want):
    assert lib.amp_layer_norm_forward(*args, None) == want


@pytest.mark.parametrize("args,want", [
    ((D, D, BF16, None, None, -1, 4, D, F32, D, D, D, None, None, None, 0), EINVAL),
    ((D, D, E4M3, None, None, 4, 4, D, F32, D, D, D, None, None, None, 0), EDTYPE),
    ((D, D, F32, None, None, 4, 4, D, BF16, D, D, D, None, None, None, 0), EDTYPE),
    ((D, D, BF16, D, None, 4, 4, D, F32, D, D, D, None, None, None, 0), EINVAL),
    ((D, D, BF16, D, D, 4, 4, D, F32, D, D, D, None, None, None, 0), EINVAL),
    ((D, None, BF16, None, None, 4, 4, D, F32, D, D, D, None, None, None, 0), EINVAL),
    ((None, D, BF16, None, None, 4, 4, D, F32, D, D, D, None, None, None, 0), EINVAL),
    ((D, D, BF16, None, None, 4, 4, D, F32, None, D, D, None, None, None, 0), EINVAL),
    ((D, D, BF16, None, None, 4, 4, D, F32, D, None, D, None, None, None, 0), EINVAL),
    ((None, None, BF16, None, None, 0, 4, None, F32, None, None, None, None, None, None, 0), OK),
    ((D, D, BF16, None, None, 4, 0, None, F32, D, D, D, D, D, None, 0), OK),
    ((D, D, BF16, None, None, 4, 4, None, F32, D, D, None, None, None, None, 0), OK),
])
def test_layer_norm_backward_refusals(lib, args, want):
    assert lib.amp_layer_norm_backward(*args, None) == want


@pytest.mark.parametrize("args,want", [
    ((3, D, None, BF16, 4, 4, D, None, None, None, None), EINVAL),
    ((-1, D, None, BF16, 4, 4, D, None, None, None, None), EINVAL),
    ((0, D, None, E4M3, 4, 4, D, None, None, None, None), EDTYPE),
    ((0, D, None, BF16, 4, -4, D, None, None, None, None), EINVAL),
    ((0, D, None, BF16, 4, 4, D, D, None, None, None), EINVAL),
    ((0, D, D, BF16, 4, 4, D, D, D, None, None), EINVAL),
    ((0, D, D, BF16, 4, 4, D, D, D, D, None), EINVAL),
    ((0, D, None, BF16, 4, 4, D, D, D, D, D), EINVAL),
    ((0, D, None, BF16, 4, 4, None, D, D, None, None), EINVAL),
    ((0, None, None, BF16, 4, 4, D, D, D, None, None), EINVAL),
    ((0, None, None, BF16, 0, 4, None, None, None, None, None), OK),
])
def test_act_forward_refusals(lib, args, want):
    assert lib.amp_act_forward_mx8(*args, None) == want


@pytest.mark.parametrize("args", [
    (3, D, BF16, 4, 4, D, D, None, None, D, None), (0, D, E4M3, 4, 4, D, D, None, None, D, None),
    (0, D, BF16, -4, 4, D, D, None, None, D, None), (0, D, BF16, 4, 4, D, D, D, None, D, D),
    (0, D, BF16, 4, 4, D, D, D, D, D, None), (0, D, BF16, 4, 4, D, D, None, None, D, D),
])
def test_act_backward_refusals(lib, args):
    assert lib.amp_act_backward_mx8(*args, None) in (EINVAL, EDTYPE)


# one tensor a call whose address is between two elements (last argument: the stream)
HALF = ctypes.c_void_p(4098)   # between two of four bytes


@pytest.mark.parametrize("name,args", [
    ("fp4_quant_mx", (ODD, BF16, 4, 4, D, D, None, None, None)),
    ("fp4_quant_mx", (HALF, F32, 4, 4, D, D, None, None, None)),
    ("fp4_quant_mx", (D, BF16, 4, 4, D, D, None, None, HALF)),
    ("fp4_dequant_mx", (D, D, 4, 4, ODD, F16)),
    ("fp4_dequant_mx", (D, D, 4, 4, HALF, F32)),
    ("amp_layer_norm_forward", (ODD, BF16, 4, 4, D, D, F32, 1e-5, D, D, D, None, None)),
    ("amp_layer_norm_forward", (D, BF16, 4, 4, HALF, D, F32, 1e-5, D, D, D, None, None)),
    ("amp_layer_norm_forward", (D, BF16, 4, 4, D, HALF, F32, 1e-5, D, D, D, None, None)),
    ("amp_layer_norm_forward", (D, BF16, 4, 4, D, D, F32, 1e-5, ODD, D, D, None, None)),
    ("amp_layer_norm_forward", (D, BF16, 4, 4, D, D, F32, 1e-5, D, HALF, D, None, None)),
    ("amp_layer_norm_forward", (D, BF16, 4, 4, D, D, F32, 1e-5, D, D, HALF, None, None)),
    ("amp_layer_norm_backward", (ODD, D, BF16, None, None, 4, 4, D, F32, D, D, D, None, None, None, 0)),
    ("amp_layer_norm_backward", (D, ODD, BF16, None, None, 4, 4, D, F32, D, D, D, None, None, None, 0)),
    ("amp_layer_norm_backward", (D, D, BF16, None, None, 4, 4, HALF, F32, D, D, D, None, None, None, 0)),
    ("amp_layer_norm_backward", (D, D, BF16, None, None, 4, 4, D, F32, HALF, D, D, None, None, None, 0)),
    ("amp_layer_norm_backward", (D, D, BF16, None, None, 4, 4, D, F32, D, HALF, D, None, None, None, 0)),
    ("amp_layer_norm_backward", (D, D, BF16, None, None, 4, 4, D, F32, D, D, ODD, None, None, None, 0)),
    ("amp_layer_norm_backward", (D, D, BF16, None, None, 4, 4, D, F32, D, D, D, HALF, None, D, 1 << 20)),
    ("amp_layer_norm_backward", (D, D, BF16, None, None, 4, 4, D, F32, D, D, D, None, HALF, D, 1 << 20)),
    ("amp_act_forward_mx8", (0, ODD, None, F16, 4, 4, D, D, D, None, None)),
    ("amp_act_forward_mx8", (0, D, HALF, F32, 4, 4, D, D, D, D, D)),
    ("amp_act_forward_mx8", (0, D, None, F16, 4, 4, ODD, D, D, None, None)),
    ("amp_act_backward_mx8", (0, ODD, F16, 4, 4, D, D, None, None, D, None)),
    ("amp_act_backward_mx8", (0, D, F32, 4, 4, D, D, None, None, HALF, None)),
    ("amp_act_backward_mx8", (0, D, F16, 4, 4, D, D, D, D, D, ODD)),
    ("amp_ckpt8_save", (ODD, BF16, 4, 4, D, D)),
    ("amp_ckpt8_restore", (D, D, 4, 4, HALF, F32)),
])
def test_addresses_between_elements_are_refused(lib, name, args):
    assert getattr(lib, name)(*args, None) == EINVAL
    assert b"not aligned to its type" in lib.amp_last_error()


def test_binding_refusals(lib):
    import loss_scaling_master_gb300 as G
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        G.fp4_quant_mx(x, q, s)
    with pytest.raises(ValueError, match="one dimension"):
        G.fp4_quant_mx(torch.tensor(1.0), q, s)
    with pytest.raises(ValueError, match="k = -1"):
        G.fp4_product_mx(q, s, q, s, -1, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="either x or saved"):
        G.amp_layer_norm_backward(x, None, None, x, x)
    with pytest.raises(ValueError, match="one dtype"):
        G.amp_layer_norm_forward(x, torch.zeros(64), torch.zeros(64, dtype=torch.float16), 1e-5, x)
    with pytest.raises(ValueError, match="64 elements"):
        G.amp_layer_norm_forward(x, torch.zeros(63), None, 1e-5, x)
    with pytest.raises(ValueError, match="activation 'relu'"):
        G.amp_act_forward_mx8(x, "relu", x)
    with pytest.raises(ValueError, match="negative or too large"):
        G.fp4_mx_buffers(-1, 4, device="cpu")


# ------------------------------------------------------------------ the reference itself
def test_reference_blocks_against_library_casts():
    """With a maximum of 448 * 2^k in every block the scale is 2^k, and the codes
    are the library's e4m3 conversion; e2m1's values round-trip."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(16, 64, generator=g)
    x[:, ::32] = 448.0
    v, e, _ = R.mx_blocks(x, "e4m3")
    assert (e == 127).all()
    assert torch.equal(v.float(), x.to(torch.float8_e4m3fn).float())
    grid = torch.cat([R.GRIDS["e2m1"], -R.GRIDS["e2m1"]]).repeat(2)[None] * 2.0 ** -5
    v, e, c = R.mx_blocks(grid, "e2m1")
    assert torch.equal(v, grid.double()) and (e == 122).all() and (c[0, :8] == torch.arange(8)).all()
    ties = torch.tensor([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]])
    v, _, _ = R.mx_blocks(ties, "e2m1")
    assert v.tolist() == [[0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]]


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_reference_gradients_against_differences(kind):
    x = torch.linspace(-6, 6, 241, dtype=torch.float64)
    h = 1e-5
    d = (R.act(x + h, kind)[0] - R.act(x - h, kind)[0]) / (2 * h)
    # central differences: h^2 / 6 times the third derivative (below 4), and rounding 1e-15 / h
    assert (d - R.act(x, kind)[1]).abs().max() < 4 * h * h / 6 + 1e-9


def test_reference_norm_gradients_against_differences():
    g = torch.Generator().manual_seed(5)
    x, dy = torch.randn(3, 17, generator=g).double(), torch.randn(3, 17, generator=g).double()
    w, b = torch.randn(17, generator=g).double(), torch.randn(17, generator=g).double()
    eps, h = 1e-3, 1e-5
    _, mean, rstd = R.layer_norm(x, w, b, eps)
    dx, dw, db = R.layer_norm_grads(dy, x, w, mean, rstd)
    for t, d in ((x, dx), (w, dw), (b, db)):
        flat, got = t.view(-1), d.reshape(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = (R.layer_norm(x, w, b, eps)[0] * dy).sum()
            flat[i] = keep - h
            dn = (R.layer_norm(x, w, b, eps)[0] * dy).sum()
            flat[i] = keep
            assert abs((up - dn) / (2 * h) - got[i]) < 1e-6
