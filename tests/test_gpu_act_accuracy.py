"""How far the activations and their derivatives are from 64 bits, over every
finite value of the 16-bit types and over fp32's range: relative bounds, so that
the tails count as much as the middle.

16 bits (ampops.h: 2^-14 of f, or of the derivative's parts, before the rounding to
the type).  GELU: the fit 2^-18.8; the exponent u = -x^2 log2(e) / 2 with two
roundings and a rounded constant, 2.5 U |u| ln 2 = 2^-16.3 at the last exponential
(|u| = 126); a lookup each 2^-22.  gelu_tanh: sigma's argument is good to 4 U and
scaled by a rounded constant and rounded, 5.5 U |t| = 2^-15 at |t| = 94, where bf16
ends; silu less.  What e flushes below 2^-126 is 2^-122 of f.

fp32 (U = 2^-24, half an ulp; a lookup is good to 2 ulp, 4 U).  v = Phi(-|x|): an
exponential 4 U and its argument 1.25 U x^2 (two roundings and the constant), fit and
polynomial 5 U, a product 1 U: 10 U + 1.25 U x^2.  v = sigma(-|t|): an exponential 4 U
and its argument (silu's rounding is made good; gelu_tanh 5.5 U |t| as above), a
reciprocal 2 U, a sum and a product: 8 U + 5.5 U |t|.  f has two roundings more.  The
derivative's parts: s (1 - v or v) one rounding more than v; k is x phi, or x v (1 - v) t'
with twice v's errors and six roundings; their sum one more."""
import math

import pytest
import torch

import ops_reference as R
from test_gpu_ops import G, close, dev  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
U = R.U


def parts(x, kind):
    """f, and the derivative as s + k, in 64 bits; |t|, what gelu_tanh's argument is scaled by."""
    x = x.double()
    f, d = R.act(x, kind)
    if kind == "gelu":
        s, t = 0.5 * torch.erfc(-x / math.sqrt(2)), torch.zeros_like(x)
    elif kind == "silu":
        s, t = torch.sigmoid(x), torch.zeros_like(x)
    else:
        t = 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
        s, t = torch.sigmoid(t), t.abs().clamp(max=200)
    return f, s, d - s, t


def bounds(x, kind, dtype):
    f, s, k, t = parts(x, kind)
    if dtype == torch.float32:
        v = 10 + 1.25 * x.double() ** 2 if kind == "gelu" else 8 + 5.5 * t
        return (v + 2) * U * f.abs() + 2.0 ** -122, ((v + 2) * s + (2 * v + 8) * k.abs()) * U + 2.0 ** -122
    return 2.0 ** -14 * f.abs() + 2.0 ** -122, 2.0 ** -14 * (s + k.abs()) + 2.0 ** -122


def inputs(dtype):
    if dtype != torch.float32:
        x = torch.arange(-32768, 32768).to(torch.int16).view(dtype)
        return x[x.isfinite()]
    g = torch.Generator().manual_seed(11)
    return torch.cat([torch.linspace(-15, 15, 300001), torch.linspace(-110, 110, 100001),
                      1.5 * torch.randn(200000, generator=g),
                      torch.exp2(torch.empty(50000).uniform_(-149, 127, generator=g))
                      * torch.sign(torch.randn(50000, generator=g))])


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_values(G, dev, dt, kind):
    x = inputs(dt)
    for cols in (64, 61):        # 16-byte pieces, and single elements
        v = x[:x.numel() // cols * cols].view(-1, cols)
        y = torch.empty_like(v, device=dev)
        G.amp_act_forward_mx8(v.to(dev), kind, y)
        f = R.act(v, kind)[0]
        off = bounds(v, kind, dt)[0]
        close(y, f, off + R.half_ulp(f.abs() + off, dt))


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_derivatives(G, dev, dt, kind):
    """dy = 1 at every code of the checkpoint under scales of 2^-25 to 2^15."""
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    for cols in (64, 61):
        rows, kb = 41 * 8, 2
        pick = codes[torch.arange(rows * cols) * 7 % codes.numel()].view(rows, cols)
        e = (127 - 25 + torch.arange(rows)[:, None] // 8 - torch.arange(kb)[None] % 2).to(torch.uint8)
        q, s = pick.view(torch.float8_e4m3fn).to(dev), e.to(dev)
        x = torch.empty(rows, cols, device=dev)
        G.amp_ckpt8_restore(q, s, x)
        x = x.cpu()
        want = torch.ldexp(pick.view(torch.float8_e4m3fn).double(),
                           (e.int() - 127).repeat_interleave(32, 1)[:, :cols])
        assert torch.equal(x.double(), want) and (x.abs() > 1).any() and (x.abs() < 1e-9).any()
        dy, dx = torch.ones(rows, cols, dtype=dt, device=dev), torch.empty(rows, cols, dtype=dt, device=dev)
        G.amp_act_backward_mx8(dy, kind, (q, s), dx)
        d = R.act(x, kind)[1]
        off = bounds(x, kind, dt)[1]
        close(dx, d, off + R.half_ulp(d.abs() + off, dt))


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_infinite_inputs(G, dev, kind):
    """+infinity is infinity; -infinity is infinity times zero, NaN."""
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        x = torch.tensor([[math.inf, -math.inf, 1.0, 0.0, -0.0, 2.0, 3.0, 65504.0]], dtype=dt, device=dev)
        y = torch.empty_like(x)
        G.amp_act_forward_mx8(x, kind, y)
        assert y[0, 0] == math.inf and y[0, 1].isnan() and y[0, 2:].isfinite().all() and (y[0, 3:5] == 0).all()


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_fp32_is_no_worse_than_the_elementary_forms(G, dev, kind):
    """Relative norm of the error over N(0, 1.5), against erf, tanh and exp in fp32."""
    g = torch.Generator().manual_seed(5)
    x = (1.5 * torch.randn(4096, 256, generator=g)).to(dev)
    y = torch.empty_like(x)
    G.amp_act_forward_mx8(x, kind, y)
    q, s = G.ckpt8_buffers(4096, 256)
    G.amp_ckpt8_save(x, q, s)
    xh, dx = torch.empty_like(x), torch.empty_like(x)
    G.amp_ckpt8_restore(q, s, xh)
    G.amp_act_backward_mx8(torch.ones_like(x), kind, (q, s), dx)

    def plain(x):
        if kind == "silu":
            s = 1.0 / (1.0 + torch.exp(-x))
            return x * s, s * (1.0 + x * (1.0 - s))
        if kind == "gelu":
            p = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
            return x * p, p + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
        a, b = math.sqrt(2.0 / math.pi), 0.044715
        t = torch.tanh(a * (x + b * x * x * x))
        return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * a * (1.0 + 3.0 * b * x * x)
    for got, at, i in ((y, x, 0), (dx, xh, 1)):
        want = R.act(at.cpu(), kind)[i].to(dev)
        far = lambda v: ((v.double() - want).norm() / want.norm()).item()
        assert far(got) <= far(plain(at)[i])
