"""The linear layer, dropout and token log probabilities of include/ampops.h without a GPU: wrong
arguments are refused with a status and a message, the Python calls refuse tensors of two GPUs by
name, and the 64-bit reference of the GPU tests agrees with what it is made from."""
import ctypes
import math

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import more_ops_reference as M
import ops_reference as R

EINVAL, EDTYPE, OK = -1, -2, 0
BF16, F16, F32, E4M3 = 3, 2, 1, 4
NONE, GELU = -1, 0
D = ctypes.c_void_p(4096)     # never dereferenced: every call here is refused or empty
ODD, HALF = ctypes.c_void_p(4097), ctypes.c_void_p(4098)
N = None


@pytest.fixture(scope="module")
def lib():
    from loss_scaling_master_gb300 import build as B
    B.build()
    from loss_scaling_master_gb300 import ops
    return ops._load()


def linear(a=D, sa=D, b=D, sb=D, m=4, n=4, k=4, bias=N, bt=F32, act=NONE, res=N, out=D, ot=BF16, q=N, s=N):
    return (a, sa, b, sb, m, n, k, bias, bt, act, res, out, ot, q, s)


@pytest.mark.parametrize("args,want", [
    (linear(m=-1), EINVAL), (linear(n=-1), EINVAL), (linear(k=-1), EINVAL), (linear(k=(1 << 27) + 1), EINVAL),
    (linear(m=1 << 31), EINVAL), (linear(ot=E4M3), EDTYPE), (linear(bias=D, bt=F16), EDTYPE),
    (linear(bias=D, bt=E4M3), EDTYPE), (linear(bias=D, bt=BF16, ot=F32), EDTYPE), (linear(act=3), EINVAL),
    (linear(act=-2), EINVAL), (linear(q=D), EINVAL), (linear(s=D), EINVAL), (linear(a=N), EINVAL),
    (linear(sa=N), EINVAL), (linear(b=N), EINVAL), (linear(sb=N), EINVAL), (linear(out=N), EINVAL),
    (linear(a=ODD), EINVAL), (linear(sb=ODD), EINVAL), (linear(out=ODD), EINVAL), (linear(res=ODD), EINVAL),
    (linear(out=HALF, ot=F32), EINVAL), (linear(bias=HALF), EINVAL), (linear(bias=ODD, bt=BF16), EINVAL),
    (linear(m=0, a=N, out=N), OK), (linear(n=0, b=N, out=N), OK),
])
def test_linear_refusals(lib, args, want):
    assert lib.fp4_linear_mx(*args, None) == want
    if want != OK:
        assert lib.amp_last_error().startswith(b"fp4_linear_mx")


def test_linear_selftest_refusals(lib):
    for role, stages, limit in ((-1, 0, 22), (3, 0, 22), (0, -1, 22), (0, 0, -1), (0, 0, 31)):
        assert lib.fp4_linear_mx_selftest(*linear(), role, stages, limit, None) == EINVAL
    assert lib.fp4_linear_mx_selftest(*linear(a=N), 0, 0, 22, None) == EINVAL


@pytest.mark.parametrize("args,want", [
    ((3, D, BF16, 4, 4, D, D, D, D, F32), EINVAL), ((-2, D, BF16, 4, 4, N, N, N, D, F32), EINVAL),
    ((GELU, D, E4M3, 4, 4, D, D, D, D, F32), EDTYPE), ((GELU, D, BF16, 4, 4, D, D, D, D, F16), EDTYPE),
    ((GELU, D, F32, 4, 4, D, D, D, D, BF16), EDTYPE), ((GELU, D, BF16, -1, 4, D, D, D, D, F32), EINVAL),
    ((GELU, D, BF16, 4, 1 << 31, D, D, D, D, F32), EINVAL), ((GELU, N, BF16, 4, 4, D, D, D, D, F32), EINVAL),
    ((GELU, D, BF16, 4, 4, N, N, D, D, F32), EINVAL), ((GELU, D, BF16, 4, 4, D, N, D, D, F32), EINVAL),
    ((GELU, D, BF16, 4, 4, N, D, D, D, F32), EINVAL), ((GELU, D, BF16, 4, 4, D, D, N, D, F32), EINVAL),
    ((GELU, D, BF16, 4, 4, D, D, D, N, F32), EINVAL), ((NONE, D, BF16, 4, 4, N, N, N, N, F32), EINVAL),
    ((NONE, D, BF16, 4, 4, D, D, N, D, F32), EINVAL), ((NONE, D, BF16, 4, 4, N, N, D, D, F32), EINVAL),
    ((NONE, N, BF16, 4, 4, N, N, N, D, F32), EINVAL), ((GELU, ODD, BF16, 4, 4, D, D, D, D, F32), EINVAL),
    ((GELU, D, BF16, 4, 4, D, D, ODD, D, F32), EINVAL), ((GELU, D, BF16, 4, 4, D, D, D, HALF, F32), EINVAL),
    ((GELU, N, BF16, 4, 0, N, N, N, N, F32), OK), ((NONE, N, BF16, 0, 0, N, N, N, N, F32), OK),
])
def test_bias_act_backward_refusals(lib, args, want):
    assert lib.amp_bias_act_backward_mx8(*args, None) == want


def dropout(x=D, dt=BF16, r=4, c=4, p=0.5, seed=7, step=N, site=0, res=N, y=D):
    return (x, dt, r, c, p, seed, step, site, res, y)


@pytest.mark.parametrize("args,want", [
    (dropout(r=-1), EINVAL), (dropout(c=1 << 31), EINVAL), (dropout(p=-0.1), EINVAL), (dropout(p=1.1), EINVAL),
    (dropout(p=math.nan), EINVAL), (dropout(p=math.inf), EINVAL), (dropout(site=-1), EINVAL),
    (dropout(site=1 << 30), EINVAL), (dropout(dt=E4M3), EDTYPE), (dropout(x=N), EINVAL), (dropout(y=N), EINVAL),
    (dropout(x=ODD), EINVAL), (dropout(res=ODD), EINVAL), (dropout(y=HALF, dt=F32), EINVAL),
    (dropout(step=HALF), EINVAL), (dropout(r=0, x=N, y=N), OK),
])
def test_dropout_forward_refusals(lib, args, want):
    assert lib.amp_dropout_forward(*args, None) == want


@pytest.mark.parametrize("args,want", [
    ((D, BF16, 4, 4, 2.0, 7, N, 0, D, N, F32), EINVAL), ((D, BF16, 4, 4, 0.5, 7, N, -1, D, N, F32), EINVAL),
    ((D, E4M3, 4, 4, 0.5, 7, N, 0, D, N, F32), EDTYPE), ((D, BF16, 4, 4, 0.5, 7, N, 0, D, D, F16), EDTYPE),
    ((D, F32, 4, 4, 0.5, 7, N, 0, D, D, BF16), EDTYPE), ((N, BF16, 4, 4, 0.5, 7, N, 0, D, N, F32), EINVAL),
    ((D, BF16, 4, 4, 0.5, 7, N, 0, N, N, F32), EINVAL), ((D, BF16, 4, 4, 0.5, 7, N, 0, D, HALF, F32), EINVAL),
    ((D, BF16, 4, 4, 0.5, 7, ODD, 0, D, N, F32), EINVAL), ((N, BF16, 0, 4, 0.5, 7, N, 0, N, N, F32), OK),
])
def test_dropout_backward_refusals(lib, args, want):
    assert lib.amp_dropout_backward(*args, None) == want


def forward(z=D, dt=BF16, r=4, c=8, ld=8, t=D, logp=D, ent=D, stats=D, ids=N, lp=N, k=0):
    return (z, dt, r, c, ld, t, logp, ent, stats, ids, lp, k)


@pytest.mark.parametrize("args,want", [
    (forward(r=-1), EINVAL), (forward(ld=7), EINVAL), (forward(c=-1), EINVAL), (forward(ld=1 << 31), EINVAL),
    (forward(dt=E4M3), EDTYPE), (forward(k=33, ids=D, lp=D), EINVAL), (forward(k=-1), EINVAL),
    (forward(k=3, ids=D), EINVAL), (forward(k=3, lp=D), EINVAL), (forward(k=3), EINVAL),
    (forward(ids=D, lp=D), EINVAL), (forward(t=N), EINVAL), (forward(z=N), EINVAL), (forward(c=0), EINVAL),
    (forward(z=ODD), EINVAL), (forward(z=HALF, dt=F32), EINVAL), (forward(t=ctypes.c_void_p(4100)), EINVAL),
    (forward(logp=HALF), EINVAL), (forward(ent=HALF), EINVAL), (forward(stats=ctypes.c_void_p(4100)), EINVAL),
    (forward(k=2, ids=ctypes.c_void_p(4100), lp=D), EINVAL), (forward(k=2, ids=D, lp=HALF), EINVAL),
    (forward(c=(1 << 30) + 1, ld=(1 << 30) + 1), EINVAL), (forward(r=0, z=N, logp=N), OK),
])
def test_logprobs_forward_refusals(lib, args, want):
    assert lib.amp_token_logprobs_forward(*args, None) == want


def backward(dlogp=D, z=D, dt=BF16, r=4, c=8, ld=8, t=D, stats=D, ent=D, dent=D, scale=D, dz=ctypes.c_void_p(1 << 20),
             dld=8):
    return (dlogp, z, dt, r, c, ld, t, stats, ent, dent, scale, dz, dld)


@pytest.mark.parametrize("args,want", [
    (backward(r=-1), EINVAL), (backward(ld=7), EINVAL), (backward(dld=7), EINVAL), (backward(dt=E4M3), EDTYPE),
    (backward(t=N), EINVAL), (backward(ent=N), EINVAL), (backward(z=N), EINVAL), (backward(stats=N), EINVAL),
    (backward(dz=N), EINVAL), (backward(dz=D, dld=9), EINVAL), (backward(z=ODD), EINVAL),
    (backward(dz=ODD), EINVAL), (backward(dlogp=HALF), EINVAL), (backward(scale=HALF), EINVAL),
    (backward(stats=ctypes.c_void_p(4100)), EINVAL), (backward(r=0, z=N, dz=N), OK), (backward(c=0, dz=N), OK),
])
def test_logprobs_backward_refusals(lib, args, want):
    assert lib.amp_token_logprobs_backward(*args, None) == want


# ------------------------------------------------------------------ the Python calls
def test_binding_refusals(lib):
    import loss_scaling_master_gb300 as G
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    for match, f in (
            ("CUDA", lambda: G.fp4_linear_mx(q, s, q, s, 64, torch.zeros(4, 4))),
            ("k = -1", lambda: G.fp4_linear_mx(q, s, q, s, -1, torch.zeros(4, 4))),
            ("activation 'relu'", lambda: G.fp4_linear_mx(q, s, q, s, 64, torch.zeros(4, 4), kind="relu")),
            ("activation 'relu'", lambda: G.amp_bias_act_backward_mx8(x, x[0], kind="relu")),
            ("CUDA", lambda: G.amp_bias_act_backward_mx8(x, x[0])),
            ("p: needs a number", lambda: G.amp_dropout_forward(x, "a", 1, 0, x)),
            ("seed", lambda: G.amp_dropout_forward(x, 0.5, -1, 0, x)),
            ("seed", lambda: G.amp_dropout_forward(x, 0.5, 1 << 64, 0, x)),
            ("seed", lambda: G.amp_dropout_backward(x, 0.5, 1.5, 0, x)),
            ("site", lambda: G.amp_dropout_forward(x, 0.5, 1, -1, x)),
            ("site", lambda: G.amp_dropout_backward(x, 0.5, 1, 1 << 30, x)),
            ("CUDA", lambda: G.amp_dropout_forward(x, 0.5, (1 << 64) - 1, 0, x)),
            ("logits: needs a CUDA", lambda: G.amp_token_logprobs_forward(x, None, None)),
            ("one dimension", lambda: G.amp_token_logprobs_forward(torch.tensor(1.0), None, None))):
        with pytest.raises(ValueError, match=match):
            f()


R_, C = 4, 64
BF, U8, F8, FL, I32, I64 = torch.bfloat16, torch.uint8, torch.float8_e4m3fn, torch.float32, torch.int32, torch.int64
SAVED = [("saved", (R_, C), F8), ("saved", (R_, 2), U8)]
# name -> (arguments in order, keyword arguments); (name, shape, type) stands for a tensor, a list for a pair
CALLS = {
    "fp4_linear_mx": ([("a", (R_, 32), U8), ("a_scales", (512,), U8), ("b", (C, 32), U8), ("b_scales", (512,), U8), 64,
                       ("out", (R_, C), BF), ("bias", (C,), FL), "silu", ("residual", (R_, C), BF), SAVED], "out"),
    "amp_bias_act_backward_mx8": ([("dy", (R_, C), BF), ("dbias", (C,), FL), "silu", SAVED, ("dx", (R_, C), BF)], "dy"),
    "amp_dropout_forward": ([("x", (R_, C), BF), 0.5, 1, 2, ("y", (R_, C), BF), ("residual", (R_, C), BF),
                             ("step", (1,), I32)], "x"),
    "amp_dropout_backward": ([("dy", (R_, C), BF), 0.5, 1, 2, ("dx", (R_, C), BF), ("step", (1,), I32),
                              ("dbias", (C,), FL)], "dy"),
    "amp_token_logprobs_forward": ([("logits", (R_, C), BF), ("targets", (R_,), I64), ("logp", (R_,), FL),
                                    ("entropy", (R_,), FL), ("stats", (R_, 2), FL), ("top_ids", (R_, 3), I64),
                                    ("top_logp", (R_, 3), FL)], "logits"),
    "amp_token_logprobs_backward": ([("dlogp", (R_,), FL), ("logits", (R_, C), BF), ("targets", (R_,), I64),
                                     ("stats", (R_, 2), FL), ("dlogits", (R_, C), BF), ("entropy", (R_,), FL),
                                     ("dentropy", (R_,), FL), ("scale", (1,), FL)], "logits"),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_on_another_gpu_is_refused(lib, name):
    import loss_scaling_master_gb300 as G
    args, main = CALLS[name]
    tensors = [t for a in args for t in (a if isinstance(a, list) else [a]) if isinstance(t, tuple)]
    for odd in range(len(tensors)):
        place = iter(range(len(tensors)))
        with FakeTensorMode():
            def make(a):
                if isinstance(a, list):
                    return tuple(make(t) for t in a)
                if not isinstance(a, tuple):
                    return a
                return torch.empty(a[1], dtype=a[2], device="cuda:1" if next(place) == odd else "cuda:0")
            call = [make(a) for a in args]
            who = tensors[odd][0]
            match = "on cuda:0, the call is on cuda:1" if who == main else f"{who}: on cuda:1, the call is on cuda:0"
            with pytest.raises(ValueError, match=match):
                getattr(G, name)(*call)


# ------------------------------------------------------------------ the reference itself
def test_philox_known_answers():
    """The published test vectors of Philox4x32-10."""
    f = 0xFFFFFFFF
    pi = (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344)
    for c, k, want in (((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
                       ((f, f, f, f), (f, f), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
                       (pi, (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(v) for v in M.philox(np.array([c]), k)[0]) == want


def test_kept_share_and_factor():
    for p in (0.0, 0.1, 0.5, 0.9, 1.0):
        k, by = M.keep(0, 1 << 16, p, 12345, 6, 7)
        t = round(p * 65536) / 65536
        # five standard deviations of a binomial share
        assert abs(k.double().mean() - (1 - t)) <= 5 * math.sqrt(t * (1 - t) / 2 ** 16)
        assert by * (1 - t) == pytest.approx(0.0 if t == 1 else 1.0)
    a, _ = M.keep(0, 100, 0.5, 1, 2, 3)
    b, _ = M.keep(37, 50, 0.5, 1, 2, 3)
    assert torch.equal(a[37:87], b)


def test_logprobs_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    z = torch.randn(4, 9, generator=g).double()
    z[1, 3] = -math.inf
    t = torch.tensor([2, 0, -1, 8])
    dl, de = torch.randn(4, generator=g).double(), torch.randn(4, generator=g).double()
    got, h = M.logprobs_grad(z, t, dl, de, 3.0), 1e-5

    def f(z):
        _, lp, ent = M.logprobs(z, t)
        return 3.0 * ((lp * dl).sum() + (ent * de).sum())
    for i in range(z.numel()):
        flat = z.view(-1)
        keep = flat[i].item()
        if keep == -math.inf:
            assert got.view(-1)[i] == 0
            continue
        flat[i] = keep + h
        up = f(z)
        flat[i] = keep - h
        dn = f(z)
        flat[i] = keep
        # h^2 / 6 of a third derivative below 100, and roundings of 1e-15 / h
        assert abs((up - dn) / (2 * h) - got.view(-1)[i]) < 100 * h * h + 1e-8


def test_reference_alternatives():
    z = torch.tensor([[1.0, 3.0, 3.0, -math.inf, 2.0], [-math.inf] * 5])
    assert M.top(z, 7).tolist() == [[1, 2, 4, 0, -1, -1, -1], [-1] * 7]
    assert M.top(z, 2).tolist() == [[1, 2], [-1, -1]]


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_no_activation_is_steeper_than_the_bound_says(kind):
    assert R.act(torch.linspace(-10, 10, 200001, dtype=torch.float64), kind)[1].abs().max() < 1.13
