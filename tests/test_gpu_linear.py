"""fp4_linear_mx and amp_bias_act_backward_mx8 against the 64-bit reference: each width of the
product, cut reductions and pairs of CTAs, ragged sizes, every combination of bias, activation,
residual and checkpoint, misaligned tensors, non-finite values, in place, in graphs."""
import ctypes
import math

import pytest
import torch

import more_ops_reference as M
import ops_reference as R
from test_gpu_bounds import Guarded, _INT
from test_gpu_fp4_product import bound, operand
from test_gpu_ops import G, close, dev, place, same, values  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DT = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}
KINDS = (None, "gelu", "gelu_tanh", "silu")
_INT.setdefault(torch.float8_e4m3fn, (torch.uint8, 0xA5))


def guarded_ckpt(m, n, dev, lead=0):
    return (Guarded(m * n, torch.float8_e4m3fn, dev, lead, shape=(m, n)),
            Guarded(m * -(-n // 32), torch.uint8, dev, lead, shape=(m, -(-n // 32))))


def saved_values(G, q, s):
    v = torch.empty(q.shape, device="cuda")
    G.amp_ckpt8_restore(q, s, v)
    return v.double().cpu()


def check(G, dev, shape, t, bias, kind, residual, keep, seed, lead=0):
    m, n, k = shape
    a, sa, av = operand(G, m, k, seed)
    b, sb, bv = operand(G, n, k, seed + 1, 0.3 / math.sqrt(k))
    z0, off = (av @ bv.t()).cpu(), bound(av, bv, k).cpu()
    bt = place(torch.randn(n, generator=torch.Generator().manual_seed(seed)).to(bias), dev, lead) if bias else None
    res = place(values(m, n, t, seed + 2), dev, lead) if residual else None
    z, want = M.linear(z0, bt.cpu() if bias else None, kind, res.cpu() if residual else None)
    tol, ez = M.linear_bound(z, off, kind, res, want, t)
    out = Guarded(m * n, t, dev, lead, shape=(m, n))
    ck = guarded_ckpt(m, n, dev, lead) if keep else None
    args = dict(bias=bt, kind=kind, residual=res, saved=tuple(c.view for c in ck) if keep else None)
    G.fp4_linear_mx(a, sa, b, sb, k, out.view, **args)
    G.fp4_mx_check()
    assert out.intact()
    close(out.view, want, tol)
    if keep:
        assert ck[0].intact() and ck[1].intact()
        close(saved_values(G, ck[0].view, ck[1].view), z, M.saved_bound(z, ez))
        # the blocks are those of z as fp32 holds it
        z32 = torch.empty(m, n, device=dev)
        G.fp4_linear_mx(a, sa, b, sb, k, z32, bias=bt.float() if bias else None)
        q, s = G.ckpt8_buffers(m, n)
        G.amp_ckpt8_save(z32, q, s)
        assert torch.equal(q.view(torch.uint8), ck[0].view.view(torch.uint8)) and torch.equal(s, ck[1].view)
    again = torch.empty_like(out.view)
    G.fp4_linear_mx(a, sa, b, sb, k, again, **args)
    assert torch.equal(again, out.view)
    if residual:  # onto the residual itself
        G.fp4_linear_mx(a, sa, b, sb, k, res, **args)
        assert torch.equal(res, out.view)


# every width of one CTA's tile, cut and whole reductions, pairs; odd and even rows
SHAPES = [(1, 1, 1), (1, 128, 32), (1, 4096, 3000), (3, 7, 33), (16, 128, 64), (17, 200, 96), (33, 130, 129),
          (48, 1024, 4096), (64, 64, 1000), (65, 129, 257), (129, 1000, 777), (300, 300, 300), (128, 6401, 700),
          (4096, 4099, 160), (2049, 5122, 288), (1000, 20000, 65)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dt", TYPES)
def test_linear(G, dev, shape, dt):
    t = TYPES[dt]
    big = shape[0] * shape[1] > 1 << 20
    for i, kind in enumerate(KINDS):
        check(G, dev, shape, t, torch.float32 if i % 2 else t, kind, i % 2 == 0, True, 10 * i, lead=0)
        if not big:
            check(G, dev, shape, t, None if i % 2 else torch.float32, kind, i % 2 == 1, i < 2, 10 * i + 5, lead=1)


@pytest.mark.parametrize("dt", TYPES)
def test_linear_is_the_product(G, dev, dt):
    """With nothing in its epilogue it gives the product's bits."""
    for m, n, k in ((1, 300, 2600), (40, 129, 257), (300, 1000, 700), (2049, 5121, 288)):
        a, sa, _ = operand(G, m, k, 1)
        b, sb, _ = operand(G, n, k, 2, 0.02)
        x, y = torch.empty(m, n, dtype=TYPES[dt], device=dev), torch.empty(m, n, dtype=TYPES[dt], device=dev)
        G.fp4_product_mx(a, sa, b, sb, k, x)
        G.fp4_linear_mx(a, sa, b, sb, k, y)
        assert torch.equal(x, y)


def test_empty(G, dev):
    """No rows, no columns, and an empty reduction: z = bias."""
    q, s = G.fp4_mx_buffers(300, 0)
    for m, n in ((0, 4), (4, 0)):
        G.fp4_linear_mx(q, s, q, s, 0, torch.empty(m, n, device=dev), bias=torch.empty(n, device=dev))
    for t in TYPES.values():
        for m, n in ((1, 1), (37, 101), (200, 96)):
            bias, res = torch.randn(n, device=dev).to(t), torch.randn(m, n, device=dev).to(t)
            out, ck = torch.empty(m, n, dtype=t, device=dev), G.ckpt8_buffers(m, n)
            G.fp4_linear_mx(q, s, q, s, 0, out, bias=bias, kind="silu", residual=res, saved=ck)
            z = torch.zeros(m, n, dtype=torch.float64)
            zz, want = M.linear(z, bias.cpu(), "silu", res.cpu())
            tol, ez = M.linear_bound(zz, z, "silu", res, want, t)
            close(out, want, tol)
            close(saved_values(G, *ck), zz, M.saved_bound(zz, ez))
            G.fp4_linear_mx(q, s, q, s, 0, out)
            assert not out.any()


@pytest.mark.parametrize("shape", [(5, 70, 100), (300, 260, 300), (2049, 5121, 96)], ids=str)
def test_non_finite(G, dev, shape):
    """A NaN block of a token reaches that token's outputs and blocks alone; infinities of the
    bias and the residual reach theirs."""
    m, n, k = shape
    x = torch.randn(m, k, device=dev)
    x[m // 2, k // 2] = math.nan
    a, sa = G.fp4_mx_buffers(m, k)
    G.fp4_quant_mx(x, a, sa)
    b, sb, _ = operand(G, n, k, 2, 0.02)
    bias, res = torch.zeros(n, device=dev), torch.zeros(m, n, dtype=torch.bfloat16, device=dev)
    bias[n - 1], res[0, 1] = math.inf, -math.inf
    out, ck = torch.empty_like(res), G.ckpt8_buffers(m, n)
    G.fp4_linear_mx(a, sa, b, sb, k, out, bias=bias, kind="silu", residual=res, saved=ck)
    nan, inf = out.isnan().cpu(), out.isinf().cpu()
    want = torch.zeros(m, n, dtype=torch.bool)
    want[m // 2] = True
    assert torch.equal(nan, want)
    want = torch.zeros(m, n, dtype=torch.bool)
    want[:, n - 1] = True
    want[m // 2] = False
    want[0, 1] = True
    assert torch.equal(inf, want)
    bad = ck[1].cpu() == 255
    want = torch.zeros_like(bad)
    want[m // 2], want[:, -1] = True, True
    assert torch.equal(bad, want)


# one CTA a tile (whole and cut reductions) and pairs
GIVE_UP = [(1, 128, 4096), (50, 301, 8192), (128, 25600, 700), (2049, 5121, 600)]


@pytest.mark.parametrize("shape", GIVE_UP, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("role", [0, 1, 2])
@pytest.mark.parametrize("stages", [0, 3])
def test_a_wait_that_gives_up(G, dev, shape, role, stages):
    """What was not finished is NaN in the output and in the checkpoint's scales, the rest is
    right, and the next call is."""
    m, n, k = shape
    if role == 1 and m < 1000:
        return  # one CTA a tile has no second CTA's loads
    a, sa, _ = operand(G, m, k, 1)
    b, sb, _ = operand(G, n, k, 2, 0.02)
    for t in DT:
        bias, res = torch.randn(n, device=dev), torch.randn(m, n, device=dev).to(t)
        want, wq = torch.empty_like(res), G.ckpt8_buffers(m, n)
        G.fp4_linear_mx(a, sa, b, sb, k, want, bias=bias, kind="gelu", residual=res, saved=wq)
        out, ck = torch.full_like(res, 7.0), G.ckpt8_buffers(m, n)
        ck[0].view(torch.uint8).fill_(9)
        ck[1].fill_(9)
        st = G.ops._load().fp4_linear_mx_selftest(
            *[x.data_ptr() for x in (a, sa, b, sb)], m, n, k, bias.data_ptr(), 1, 0, res.data_ptr(), out.data_ptr(),
            DT[t], ck[0].data_ptr(), ck[1].data_ptr(), role, stages, 22,
            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        with pytest.raises(G.AmpError) as e:
            G.fp4_mx_check()
        assert e.value.status == -6
        G.fp4_mx_check()
        bad = out.isnan()
        assert bad.all() if stages == 0 else bad.any() or role != 2
        assert torch.equal(torch.where(bad, want, out), want)
        blocks = bad.view(m, n)[:, ::32]            # a block is finished or not as a whole
        assert (ck[1][blocks] == 255).all() and torch.equal(ck[1][~blocks], wq[1][~blocks])
        cols = blocks.repeat_interleave(32, 1)[:, :n]
        assert torch.equal(ck[0].view(torch.uint8)[~cols], wq[0].view(torch.uint8)[~cols])
        G.fp4_linear_mx(a, sa, b, sb, k, out, bias=bias, kind="gelu", residual=res, saved=ck)
        G.fp4_mx_check()
        assert torch.equal(out, want) and torch.equal(ck[1], wq[1])


# ------------------------------------------------------------------ the backward pass
BSIZES = [(1, 1), (1, 33), (3, 8), (5, 129), (64, 64), (65, 72), (513, 40), (1000, 2304), (2047, 1111), (37, 20001),
          (4096, 768), (20011, 64)]


def bias_bound(dz, e, t):
    """Sums over rows of terms each off by e, added in fp32 in any order: U a level of the sum on
    what it holds, at most 40 levels (a thread's own additions are a share of the rows over 64)."""
    rows = dz.shape[0]
    total = dz.abs().sum(0) + e.sum(0)
    off = e.sum(0) + U * (40 + rows / 8) * total
    return off + R.half_ulp(dz.sum(0).abs() + off, t)


U = R.U


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("size", BSIZES, ids=lambda s: "x".join(map(str, s)))
def test_bias_act_backward(G, dev, dt, lead, size):
    r, c = size
    t = TYPES[dt]
    x, dy = values(r, c, t, 3 * r + c), place(values(r, c, t, r + 7 * c), dev, lead)
    q, s = guarded_ckpt(r, c, dev, lead)
    G.amp_ckpt8_save(x.to(dev), q.view, s.view)
    zh = saved_values(G, q.view, s.view)
    dyd = dy.cpu().double()
    for i, kind in enumerate(KINDS):
        bt = torch.float32 if i % 2 else t
        db = Guarded(c, bt, dev, lead)
        if kind is None:
            G.amp_bias_act_backward_mx8(dy, db.view)
            assert db.intact()
            close(db.view, dyd.sum(0), bias_bound(dyd, torch.zeros_like(dyd), bt))
            continue
        dx, same_as = Guarded(r * c, t, dev, lead, shape=(r, c)), torch.empty(r, c, dtype=t, device=dev)
        G.amp_bias_act_backward_mx8(dy, db.view, kind, (q.view, s.view), dx.view)
        assert db.intact() and dx.intact()
        G.amp_act_backward_mx8(dy, kind, (q.view, s.view), same_as)
        assert same(dx.view, same_as)
        dz = dyd * R.act(zh, kind)[1]
        e = dyd.abs() * R.act_bounds(zh, kind)[1] + 2.0 ** -126
        if t != torch.float32:  # the 16-bit forms' derivative is good to 2^-14 (1 + |x|)
            e = dyd.abs() * (1 + zh.abs()) * 2.0 ** -14 + 2.0 ** -126
        close(db.view, dz.sum(0), bias_bound(dz, e, bt))
        again, mine = db.view.clone(), dy.clone()
        G.amp_bias_act_backward_mx8(dy, db.view, kind, (q.view, s.view), dx.view)
        assert same(again, db.view)         # equal calls, equal bits
        G.amp_bias_act_backward_mx8(mine, again, kind, (q.view, s.view), mine)   # in place, dy aligned
        assert same(mine, dx.view)
        close(again, dz.sum(0), bias_bound(dz, e, bt))


def test_bias_gradient_of_no_rows_and_of_bad_values(G, dev):
    for t in TYPES.values():
        db = torch.full((70,), 3.0, dtype=t, device=dev)
        G.amp_bias_act_backward_mx8(torch.empty(0, 70, dtype=t, device=dev), db)
        assert not db.any()
        dy = torch.ones(100, 70, dtype=t, device=dev)
        dy[50, 3], dy[60, 64] = math.nan, math.inf
        G.amp_bias_act_backward_mx8(dy, db)
        want = torch.full((70,), 100.0, dtype=torch.float64)
        want[3], want[64] = math.nan, math.inf
        assert same(db, want)


def test_bias_gradient_offsets_past_32_bits(G, dev):
    """More than 2^31 elements: the last rows count, and get their gradient."""
    r, c = 70001, 32768
    dy = torch.zeros(r, c, dtype=torch.bfloat16, device=dev)
    dy[-3:] = 0.5
    db = torch.empty(c, device=dev)
    G.amp_bias_act_backward_mx8(dy, db)
    assert (db == 1.5).all()


def test_bias_gradient_is_the_formulas(G, dev):
    """The chain forward, loss, backward against differences of the fp32 forward in the bias."""
    m, n, k = 200, 96, 128
    a, sa, _ = operand(G, m, k, 1)
    b, sb, _ = operand(G, n, k, 2, 0.1)
    g = torch.Generator().manual_seed(4)
    bias, w = torch.randn(n, generator=g).to(dev), torch.randn(m, n, generator=g).to(dev)
    for kind in KINDS[1:]:
        out, ck = torch.empty(m, n, device=dev), G.ckpt8_buffers(m, n)
        G.fp4_linear_mx(a, sa, b, sb, k, out, bias=bias, kind=kind, saved=ck)
        db, dz = torch.empty(n, device=dev), torch.empty(m, n, device=dev)
        G.amp_bias_act_backward_mx8(w, db, kind, ck, dz)
        h = 2.0 ** -5
        up, dn = torch.empty_like(out), torch.empty_like(out)
        G.fp4_linear_mx(a, sa, b, sb, k, up, bias=bias + h, kind=kind)
        G.fp4_linear_mx(a, sa, b, sb, k, dn, bias=bias - h, kind=kind)
        diff = ((up.double() - dn.double()) * w.double()).sum(0) / (2 * h)
        # z's 8-bit rounding moves f' by at most 1.2 (its slope's bound) * 2^-4 |z| an element, |z| f''
        # being below 0.8: 0.05 |w| a term; h^2 / 6 of a third derivative below 4; fp32's rounding over h
        z = torch.empty(m, n, device=dev)
        G.fp4_linear_mx(a, sa, b, sb, k, z, bias=bias)
        tol = (w.abs().double() * (0.05 + 4 * h * h / 6 + 2.0 ** -18 * (1 + z.abs().double()) / h)).sum(0)
        assert ((db.double() - diff).abs() <= tol).all()
