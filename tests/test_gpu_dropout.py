"""amp_dropout_forward and _backward: the mask is the one that the definition gives, element for
element, and the values are fp32's; every type, odd sizes, misaligned tensors, in place, past 32-bit
offsets, with a step on the device in a captured graph."""
import math

import pytest
import torch

import more_ops_reference as M
import ops_reference as R
from test_gpu_bounds import Guarded
from test_gpu_linear import bias_bound
from test_gpu_ops import G, close, dev, place, same, values  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SEED = 0x9E3779B97F4A7C15
SIZES = [(1, 1), (1, 7), (1, 8), (3, 3), (5, 129), (64, 64), (65, 72), (130, 1000), (1024, 768), (513, 1111),
         (37, 20001), (3000, 33)]


def expected(x, res, p, seed, step, site):
    """In fp32 as the kernels compute: one rounding of the product, one of the sum, one to the type."""
    k, by = M.keep(0, x.numel(), p, seed, step, site)
    y = torch.where(k.view(x.shape), x.float() * torch.tensor(by, dtype=torch.float32), 0.0)
    return (y if res is None else res.float() + y).to(x.dtype)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(G, dev, dt, lead, size):
    r, c = size
    t = TYPES[dt]
    x, res = values(r, c, t, r + c), values(r, c, t, 2 * r + c)
    step = torch.tensor([77], dtype=torch.int32, device=dev)
    for i, p in enumerate((0.1, 0.5, 0.0, 1.0)):
        xd, rd = place(x, dev, lead), place(res, dev, lead) if i % 2 == 0 else None
        y = Guarded(r * c, t, dev, lead, shape=(r, c))
        G.amp_dropout_forward(xd, p, SEED + i, 5, y.view, residual=rd, step=step)
        want = expected(x, res if i % 2 == 0 else None, p, SEED + i, 77, 5)
        assert y.intact() and same(y.view, want) and same(xd, x)
        dx = Guarded(r * c, t, dev, lead, shape=(r, c))
        G.amp_dropout_backward(xd, p, SEED + i, 5, dx.view, step=step)
        grad = expected(x, None, p, SEED + i, 77, 5)
        assert dx.intact() and same(dx.view, grad)
        for bt in {t, torch.float32}:
            db, dx2 = Guarded(c, bt, dev, lead), Guarded(r * c, t, dev, lead, shape=(r, c))
            G.amp_dropout_backward(xd, p, SEED + i, 5, dx2.view, step=step, dbias=db.view)
            assert db.intact() and dx2.intact() and same(dx2.view, grad)
            k, by = M.keep(0, r * c, p, SEED + i, 77, 5)
            exact = torch.where(k.view(r, c), x.double() * by, 0.0)
            # the factor's rounding and the product's
            close(db.view, exact.sum(0), bias_bound(exact, 2 * R.U * exact.abs(), bt))
            again, mine = db.view.clone(), xd.clone()
            G.amp_dropout_backward(xd, p, SEED + i, 5, dx2.view, step=step, dbias=db.view)
            assert same(again, db.view)     # equal calls, equal bits
            G.amp_dropout_backward(mine, p, SEED + i, 5, mine, step=step, dbias=again)   # in place, aligned
            assert same(mine, grad)
            close(again, exact.sum(0), bias_bound(exact, 2 * R.U * exact.abs(), bt))
        if rd is not None:
            G.amp_dropout_forward(xd, p, SEED + i, 5, rd, residual=rd, step=step)   # onto the residual
            assert same(rd, want)
        G.amp_dropout_forward(xd, p, SEED + i, 5, xd, step=step)                    # onto x
        assert same(xd, grad)


@pytest.mark.parametrize("dt", TYPES)
def test_mixed_alignments(G, dev, dt):
    """One tensor off a 16-byte boundary takes the other kernels, with the same mask."""
    t = TYPES[dt]
    x, res = values(40, 72, t, 1), values(40, 72, t, 2)
    want, grad = expected(x, res, 0.3, 9, 0, 1), expected(x, None, 0.3, 9, 0, 1)
    for lx, lr, ly in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (2, 3, 1)):
        y = Guarded(40 * 72, t, dev, ly, shape=(40, 72))
        G.amp_dropout_forward(place(x, dev, lx), 0.3, 9, 1, y.view, residual=place(res, dev, lr))
        assert y.intact() and same(y.view, want)
        db = torch.empty(72, device=dev)
        G.amp_dropout_backward(place(x, dev, lx), 0.3, 9, 1, y.view, dbias=db)
        assert y.intact() and same(y.view, grad)


def test_what_is_dropped_leaves_nothing(G, dev):
    """NaN and infinities where the mask drops are gone; where it keeps they stay."""
    for t in TYPES.values():
        x = torch.full((50, 40), math.nan, dtype=t, device=dev)
        x[::2] = math.inf
        y, db = torch.empty_like(x), torch.empty(40, device=dev)
        k, _ = M.keep(0, 2000, 0.5, 3, 0, 0)
        k = k.view(50, 40)
        for call in (lambda: G.amp_dropout_forward(x, 0.5, 3, 0, y), lambda: G.amp_dropout_backward(x, 0.5, 3, 0, y),
                     lambda: G.amp_dropout_backward(x, 0.5, 3, 0, y, dbias=db)):
            y.fill_(7.0)
            call()
            assert (y.cpu()[~k] == 0).all() and same(y.cpu()[k], x.cpu()[k])
        assert not db.isfinite().any()
        G.amp_dropout_backward(x, 1.0, 3, 0, y, dbias=db)
        assert not y.any() and not db.any()


def test_streams_differ(G, dev):
    """Seeds, steps and sites give other masks; the step is the device's value; the whole seed counts."""
    x, step = torch.ones(64, 64, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)

    def mask(seed, site, s):
        step.fill_(s)
        y = torch.empty_like(x)
        G.amp_dropout_forward(x, 0.5, seed, site, y, step=step)
        want = expected(x.cpu(), None, 0.5, seed, s, site)
        assert same(y, want)
        return y
    base = mask(1, 0, 0)
    for other in ((2, 0, 0), (1 + (1 << 32), 0, 0), (1, 1, 0), (1, 0, 1), (1, 0, -1), ((1 << 64) - 1, (1 << 30) - 1, 0)):
        got = mask(*other)
        # 4096 fair coins agree in half, up to five standard deviations
        assert abs((got == base).float().mean() - 0.5) < 5 * 0.5 / 64
    y = torch.empty_like(x)
    G.amp_dropout_forward(x, 0.5, 1, 0, y)
    assert torch.equal(y, base)


@pytest.mark.parametrize("lead", [0, 1])
def test_offsets_past_32_bits(G, dev, lead):
    """More than 2^31 elements, and groups past 2^28: the last ones have their own mask."""
    r, c = 131073, 32800
    buf = torch.zeros(lead + r * c, dtype=torch.bfloat16, device=dev)
    x = buf[lead:].view(r, c)
    x[-2:] = 1.0
    x[0] = 1.0
    k, by = M.keep((r - 2) * c, 2 * c, 0.25, 11, 0, 2)
    k0, _ = M.keep(0, c, 0.25, 11, 0, 2)
    want = torch.where(k, torch.tensor(by), 0.0).to(torch.bfloat16).view(2, c)
    db = torch.empty(c, device=dev)
    y = torch.empty_like(buf)[lead:].view(r, c) if lead == 0 else x
    G.amp_dropout_backward(x, 0.25, 11, 2, y, dbias=db)
    assert same(y[-2:], want) and not y[1:1000].any()
    one = torch.tensor(by, dtype=torch.float32).double()
    exact = (k.view(2, c).double().sum(0) + k0.double()) * one
    close(db, exact, 2 * R.U * exact)      # at most two additions that round (3 factors are not a float)
    if lead == 0:
        G.amp_dropout_forward(x, 0.25, 11, 2, x)
        assert same(x[-2:], want)


def test_graph_takes_the_step_from_the_device(G, dev):
    """A captured pair of calls draws the mask of the step's value at each replay."""
    x = torch.ones(33, 100, dtype=torch.bfloat16, device=dev)
    step = torch.zeros(1, dtype=torch.int32, device=dev)
    y, dx, db = torch.empty_like(x), torch.empty_like(x), torch.empty(100, device=dev)

    def calls(stream=None):
        G.amp_dropout_forward(x, 0.4, 5, 6, y, step=step, stream=stream)
        G.amp_dropout_backward(x, 0.4, 5, 6, dx, step=step, dbias=db, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        calls(s)
    for v in (3, 4):
        step.fill_(v)
        g.replay()
        torch.cuda.synchronize()
        want = expected(x.cpu(), None, 0.4, 5, v, 6)
        assert same(y, want) and same(dx, want)


def test_empty(G, dev):
    for r, c in ((0, 5), (5, 0), (0, 0)):
        x, db = torch.empty(r, c, device=dev), torch.full((c,), 2.0, device=dev)
        G.amp_dropout_forward(x, 0.5, 1, 0, x, residual=x)
        G.amp_dropout_backward(x, 0.5, 1, 0, x, dbias=db)
        assert not db.any()


def test_refusals(G, dev):
    x, f = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev), torch.zeros(4, 64, device=dev)
    i = torch.zeros(1, dtype=torch.int32, device=dev)
    for match, call in (
            ("y: dtype Float, expected BFloat16", lambda: G.amp_dropout_forward(x, 0.5, 1, 0, f)),
            ("residual: dtype Float", lambda: G.amp_dropout_forward(x, 0.5, 1, 0, x, residual=f)),
            ("step: dtype Float", lambda: G.amp_dropout_forward(x, 0.5, 1, 0, x, step=f)),
            ("y: 192 elements", lambda: G.amp_dropout_forward(x, 0.5, 1, 0, x[:3])),
            ("x: needs a contiguous", lambda: G.amp_dropout_forward(x.t(), 0.5, 1, 0, x)),
            ("dbias: 63 elements, 64 needed", lambda: G.amp_dropout_backward(x, 0.5, 1, 0, x, dbias=f[0, :63])),
            ("dbias: dtype Int", lambda: G.amp_dropout_backward(x, 0.5, 1, 0, x, dbias=i.expand(64)))):
        with pytest.raises(ValueError, match=match):
            call()
    for p in (-0.1, 1.5, math.nan):
        with pytest.raises(G.AmpError, match="p must be"):
            G.amp_dropout_forward(x, p, 1, 0, x, step=i)
    with pytest.raises(G.AmpError, match="dtype"):
        G.amp_dropout_backward(f, 0.5, 1, 0, f, dbias=x[0])
