"""The operators of include/ampops.h on the GPU against the plain 64-bit
reference: every type, odd and ragged sizes, misaligned tensors, blocks of
zeros, of subnormals, with infinities and NaN; outputs inside canaries.  The
quantisers have to match exactly; the others within bounds derived from the
number of fp32 roundings on the way (ops_reference)."""
import math

import pytest
import torch

import ops_reference as R
from test_gpu_bounds import Guarded, _INT

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = R.U
_INT.setdefault(torch.float8_e4m3fn, (torch.uint8, 0xA5))


@pytest.fixture(scope="module")
def G():
    from loss_scaling_master_gb300 import build as B
    B.build()
    import loss_scaling_master_gb300 as pkg
    pkg.load()
    assert torch.cuda.is_available()
    return pkg


@pytest.fixture(scope="module")
def dev(G):
    return torch.device("cuda:0")


def values(rows, cols, dtype, seed, special=False):
    """N(0, 1) times a row's own power of two; with special, blocks of zeros, of
    the type's tiniest values, of large ones, and lone infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float())
    x = x.to(dtype)
    if special and rows * cols > 64:
        tiny = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}[dtype]
        x[0, :40] = 0.0
        x[rows // 3, :33] = tiny * 3
        x[rows // 2] = x[rows // 2] * torch.finfo(dtype).tiny
        x[(2 * rows) // 3, ::3] = torch.finfo(dtype).max
        x[rows - 1, cols // 2] = math.inf
        x[rows - 1, 0] = -math.inf
        x[rows // 4, cols - 1] = math.nan
    return x


def place(t, dev, lead=0):
    """t on the device, `lead` elements past a 16-byte boundary."""
    buf = torch.empty(lead + t.numel(), dtype=t.dtype, device=dev)
    v = buf[lead:].view(t.shape)
    v.copy_(t)
    return v


def same(a, b):
    """Equal as values, NaN with NaN."""
    a, b = a.detach().cpu().double(), b.detach().cpu().double()
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def close(got, want, bound):
    # what rounds past the largest f16 (65504, halfway to 65536) is an infinity there
    over = got.dtype == torch.float16
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= bound)
    if over:
        bad &= ~(got.isinf() & (want.sign() == got.sign()) & (want.abs() + bound >= 65520))
    bad &= ~(got.isnan() & want.isnan()) & ~(got == want)
    assert not bad.any(), (int(bad.sum()), float((got - want).abs()[bad].max()),
                           [int(i) for i in bad.nonzero()[0]])


SIZES = [(1, 1), (1, 31), (1, 32), (3, 33), (5, 129), (33, 40), (128, 128), (129, 257), (200, 1111),
         (31, 4096), (257, 96)]


# ------------------------------------------------------------------ 4-bit blocks
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("lead", [0, 1])
def test_fp4_quant(G, dev, dt, both, lead):
    for i, (r, c) in enumerate(SIZES):
        x = values(r, c, TYPES[dt], 100 * i + lead, special=True)
        xd = place(x, dev, lead)
        shapes = [(r, c)] + ([(c, r)] if both else [])
        outs = []
        for a, b in shapes:
            q, s = G.fp4_mx_buffers(a, b, device="meta")
            outs.append((Guarded(q.numel(), torch.uint8, dev, shape=q.shape), Guarded(s.numel(), torch.uint8, dev)))
        G.fp4_quant_mx(xd, *[g.view for pair in outs for g in pair])
        for (a, b), (q, s), m in zip(shapes, outs, (x, x.t())):
            v, e, code = R.mx_blocks(m, "e2m1")
            assert q.intact() and s.intact()
            assert torch.equal(s.view.cpu(), R.tiled_scales(e, a, b)), (r, c)
            good = (e != 255)[:, :, None].expand(-1, -1, 32).reshape(a, -1)[:, :b]
            want = R.packed_codes(torch.where(good, code, 0), torch.signbit(m) & good)
            ok = (e != 255).repeat_interleave(16, 1)
            assert torch.equal(q.view.cpu()[ok], want[ok]), (r, c)
            for od, t in TYPES.items():
                out = Guarded(a * b, t, dev, lead, shape=(a, b))
                G.fp4_dequant_mx(q.view, s.view, out.view)
                assert out.intact() and same(out.view, v.to(t)), (r, c, od)
        assert torch.equal(xd.view(torch.uint8).cpu(), x.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("r,c", [(130, 36), (129, 100), (5, 1028), (33, 1111), (5003, 1028), (2999, 1040), (20011, 301)])
def test_fp4_rows_of_fours_and_walks(G, dev, dt, r, c):
    """Rows that are whole 16-byte pieces in fp32 alone, and more rows than the
    kernels have places for at once."""
    x = values(r, c, TYPES[dt], r + c, special=True)
    q, s = G.fp4_mx_buffers(r, c)
    qt, st = G.fp4_mx_buffers(c, r)
    G.fp4_quant_mx(x.to(dev), q, s, qt, st)
    for a, b, codes, scales, m in ((r, c, q, s, x), (c, r, qt, st, x.t())):
        v, e, _ = R.mx_blocks(m, "e2m1")
        assert torch.equal(scales.cpu(), R.tiled_scales(e, a, b))
        for od, t in TYPES.items():
            out = Guarded(a * b, t, dev, shape=(a, b))
            G.fp4_dequant_mx(codes, scales, out.view)
            assert out.intact() and same(out.view, v.to(t)), (a, b, od)


def test_fp4_quant_skips(G, dev):
    x = torch.randn(40, 70, device=dev)
    q, s = G.fp4_mx_buffers(40, 70)
    q.fill_(7)
    s.fill_(9)
    G.fp4_quant_mx(x, q, s, skip_if=torch.ones(1, dtype=torch.int32, device=dev))
    assert (q == 7).all() and (s == 9).all()
    G.fp4_quant_mx(x, q, s, skip_if=torch.zeros(1, dtype=torch.int32, device=dev))
    assert not (q == 7).all()


# ------------------------------------------------------------------ layer norm
NORM_SIZES = [(1, 1), (3, 5), (7, 33), (9, 256), (5, 257), (17, 512), (6, 768), (6, 1000), (11, 1024), (5, 2040),
              (4, 4096), (3, 4100), (3, 8192), (2, 8200), (2, 16384), (2, 16385), (3, 20000), (700, 64)]
# more rows than the kernels have places for at once, whole and odd
NORM_WALKS = [(10007, 64), (5003, 768), (1501, 2048), (1001, 4095), (1003, 4096), (501, 8192), (331, 16384)]


def norm_inputs(r, c, dt, seed, shift=0.0):
    x = values(r, c, TYPES[dt], seed).float()
    x = (x / x.std(-1, keepdim=True, unbiased=False).clamp_min(1e-3) + shift).to(TYPES[dt])
    g = torch.Generator().manual_seed(seed + 1)
    return x, torch.randn(r, c, generator=g).to(TYPES[dt]), 1 + 0.1 * torch.randn(c, generator=g), \
        0.1 * torch.randn(c, generator=g)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("own_type", [False, True])
@pytest.mark.parametrize("lead", [0, 1])
def test_layer_norm_forward(G, dev, dt, own_type, lead):
    t = TYPES[dt]
    for i, (r, c) in enumerate(NORM_SIZES + (NORM_WALKS if own_type and lead == 0 else [])):
        for shift in (0.0, 30.0) if r < 300 else (3.0,):
            x, _, w, b = norm_inputs(r, c, dt, i, shift)
            w, b = (w.to(t), b.to(t)) if own_type else (w, b)
            if i % 4 == 3:
                b = None
            if i % 5 == 4:
                w = None
            y = Guarded(r * c, t, dev, lead, shape=(r, c))
            mean, rstd = Guarded(r, torch.float32, dev), Guarded(r, torch.float32, dev)
            q = Guarded(r * c, torch.float8_e4m3fn, dev, lead, shape=(r, c))
            s = Guarded(r * -(-c // 32), torch.uint8, dev, shape=(r, -(-c // 32)))
            up = lambda p: None if p is None else place(p, dev, lead)
            G.amp_layer_norm_forward(place(x, dev, lead), up(w), up(b), 1e-5, y.view, mean.view, rstd.view,
                                     saved=(q.view, s.view))
            for g in (y, mean, rstd, q, s):
                assert g.intact()
            want, m, rs = R.layer_norm(x, w, b, 1e-5)
            xa = x.double().abs().mean(-1)
            # at most 64 roundings from x to each sum, and the mean's error seen through rstd
            close(mean.view, m, 64 * U * xa)
            dm = (64 * U * xa)[:, None]
            rel = 64 * U + (rs[:, None] * dm) ** 2 + 2 * U * (rs * xa)[:, None]
            close(rstd.view, rs, (rs[:, None] * rel)[:, 0])
            wa = w.double().abs() if w is not None else 1.0
            ba = b.double().abs() if b is not None else 0.0
            off = wa * rs[:, None] * (dm + 2 * U * x.double().abs()) + (want.abs() + ba) * (rel + 8 * U)
            close(y.view, want, off + R.half_ulp(want.abs() + off, t))
            v, e, _ = R.mx_blocks(x, "e4m3")
            assert torch.equal(s.view.cpu(), e.to(torch.uint8))
            out = torch.empty(r, c, device=dev)
            G.amp_ckpt8_restore(q.view, s.view, out)
            assert same(out, v)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("lead", [0, 1])
def test_layer_norm_backward(G, dev, dt, ckpt, lead):
    t = TYPES[dt]
    for i, (r, c) in enumerate(NORM_SIZES + (NORM_WALKS if lead == 0 else [])):
        x, dy, w, _ = norm_inputs(r, c, dt, 50 + i, 0.5)
        own_type = bool(i % 2)
        w = w.to(t) if own_type else w
        wt = w.dtype
        if i % 5 == 4:
            w = None
        _, mean, rstd = R.layer_norm(x, None, None, 1e-5)
        mean, rstd = mean.float(), rstd.float()
        saved, xs = None, x
        if ckpt:
            q, s = G.ckpt8_buffers(r, c)
            saved = (place(q.cpu(), dev, lead), s)
            G.amp_ckpt8_save(place(x, dev, lead), *saved)
            xs = R.mx_blocks(x, "e4m3")[0]
        dx = Guarded(r * c, t, dev, lead, shape=(r, c))
        dw, db = Guarded(c, wt, dev), Guarded(c, wt, dev)
        n = G.amp_layer_norm_workspace(dx.view).numel()
        work = Guarded(n, torch.uint8, dev)
        up = lambda p: None if p is None else place(p, dev, lead)
        args = (up(dy), None if ckpt else up(x), up(w), mean.to(dev), rstd.to(dev))
        G.amp_layer_norm_backward(*args, dx.view, dw.view, db.view, work.view, saved=saved)
        for g in (dx, dw, db, work):
            assert g.intact()
        wdx, wdw, wdb = R.layer_norm_grads(dy, xs, w, mean, rstd)
        # 64 roundings in each row sum; 128 in a column's (a share of the rows, then the shares)
        xh = ((xs.double() - mean.double()[:, None]) * rstd.double()[:, None]).abs()
        gw = (dy.double() * (w.double() if w is not None else 1.0)).abs()
        off = 64 * U * rstd.double()[:, None] * (gw + gw.mean(-1, keepdim=True)
                                                + xh * (gw * xh).mean(-1, keepdim=True))
        close(dx.view, wdx, off + R.half_ulp(wdx.abs() + off, t))
        ow, ob = 128 * U * (dy.double().abs() * xh).sum(0), 128 * U * dy.double().abs().sum(0)
        close(dw.view, wdw, ow + R.half_ulp(wdw.abs() + ow, wt))
        close(db.view, wdb, ob + R.half_ulp(wdb.abs() + ob, wt))
        # the same bits again; each output alone; in place
        again = torch.empty_like(dx.view)
        a, b = torch.empty(c, dtype=wt, device=dev), torch.empty(c, dtype=wt, device=dev)
        G.amp_layer_norm_backward(*args, None, a, None, work.view, saved=saved)
        G.amp_layer_norm_backward(*args, None, None, b, work.view, saved=saved)
        G.amp_layer_norm_backward(*args, again, saved=saved)
        assert torch.equal(again, dx.view) and torch.equal(a, dw.view) and torch.equal(b, db.view)
        G.amp_layer_norm_backward(*args, args[0], a, b, work.view, saved=saved)
        assert torch.equal(args[0], dx.view) and torch.equal(a, dw.view)


def test_layer_norm_gradient_against_differences(G, dev):
    """dx and dweight against central differences of the forward's own fp32 outputs."""
    r, c, h = 2, 48, 1e-2
    x, dy, w, b = norm_inputs(r, c, "f32", 9)
    x, dy, w, b = (t.to(dev) for t in (x, dy, w, b))
    y, mean, rstd = torch.empty_like(x), torch.empty(r, device=dev), torch.empty(r, device=dev)

    def loss():
        G.amp_layer_norm_forward(x, w, b, 1e-3, y, mean, rstd)
        return (y.double() * dy.double()).sum().item()
    loss()
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    G.amp_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, G.amp_layer_norm_workspace(x))
    for t, d in ((x, dx), (w, dw), (b, db)):
        flat = t.view(-1)
        for i in range(0, flat.numel(), 7):
            keep = flat[i].item()
            flat[i] = keep + h
            hi, up = flat[i].item(), loss()
            flat[i] = keep - h
            lo, dn = flat[i].item(), loss()
            flat[i] = keep
            # third derivatives of order 10 times h^2 / 6, and 96 outputs of order 1 good to 8 U each
            assert abs((up - dn) / (hi - lo) - d.view(-1)[i].item()) < 10 * h * h / 6 + 96 * 8 * U / h


def test_layer_norm_empty_and_nonfinite(G, dev):
    w = torch.ones(40, device=dev)
    e = torch.empty(0, 40, device=dev)
    z = torch.empty(0, device=dev)
    dw, db = torch.full_like(w, 5), torch.full_like(w, 5)
    G.amp_layer_norm_forward(e, w, w, 1e-5, e, z, z)
    G.amp_layer_norm_backward(e, e, w, z, z, e, dw, db, G.amp_layer_norm_workspace(e))
    assert (dw == 0).all() and (db == 0).all()
    x = torch.randn(4, 40, device=dev)
    x[1, 3], x[2, 5] = math.nan, math.inf
    y, m, r = torch.empty_like(x), torch.empty(4, device=dev), torch.empty(4, device=dev)
    G.amp_layer_norm_forward(x, w, None, 1e-5, y, m, r)
    assert y[1:3].isnan().all() and y[0].isfinite().all() and y[3].isfinite().all()
    c = torch.full((2, 40), 3.0, device=dev)      # no variance: rstd = 1 / sqrt(eps), y = bias
    G.amp_layer_norm_forward(c, w, w, 1e-5, y[:2], m[:2], r[:2])
    assert (y[:2] == 1).all() and torch.allclose(r[:2].double(), torch.full((2,), 1e-5 ** -0.5,
                                                 device=dev, dtype=torch.float64), rtol=8 * U)


# ------------------------------------------------------------------ activations
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_activations(G, dev, dt, kind, gated):
    t = TYPES[dt]
    for i, (r, c) in enumerate(SIZES):
        lead = i % 2
        x, u, dy = (values(r, c, t, 1000 + 10 * i + k) for k in range(3))
        mk = lambda: Guarded(r * c, t, dev, lead, shape=(r, c))
        q, qu = (Guarded(r * c, torch.float8_e4m3fn, dev, lead, shape=(r, c)) for _ in range(2))
        s, su = (Guarded(r * -(-c // 32), torch.uint8, dev, shape=(r, -(-c // 32))) for _ in range(2))
        y, dx, du, y2 = mk(), mk(), mk(), mk()
        up = dict(up=place(u, dev, lead), saved_up=(qu.view, su.view)) if gated else {}
        G.amp_act_forward_mx8(place(x, dev, lead), kind, y.view, (q.view, s.view), **up)
        G.amp_act_forward_mx8(place(x, dev, lead), kind, y2.view, up=up.get("up"))
        for g in (y, q, s, y2) + ((qu, su) if gated else ()):
            assert g.intact()
        assert torch.equal(y.view, y2.view)
        f, _ = R.act(x, kind)
        bf, _ = R.act_bounds(x, kind)
        m = u.double() if gated else torch.ones(1, dtype=torch.float64)
        off = bf * m.abs() + 2 * U * (f * m).abs()
        close(y.view, f * m, off + R.half_ulp((f * m).abs() + off, t))
        xv, e, _ = R.mx_blocks(x, "e4m3")
        assert torch.equal(s.view.cpu(), e.to(torch.uint8))
        back = torch.empty(r, c, device=dev)
        G.amp_ckpt8_restore(q.view, s.view, back)
        assert same(back, xv)
        q2, s2 = G.ckpt8_buffers(r, c)
        G.amp_ckpt8_save(place(x, dev, lead), q2, s2)
        assert torch.equal(q2.view(torch.uint8), q.view.view(torch.uint8)) and torch.equal(s2, s.view)
        dyd = place(dy, dev, lead)
        G.amp_act_backward_mx8(dyd, kind, (q.view, s.view), dx.view,
                               **(dict(saved_up=(qu.view, su.view), dup=du.view) if gated else {}))
        assert dx.intact() and du.intact()
        fh, dh = R.act(xv, kind)
        bf, bd = R.act_bounds(xv, kind)
        uv = R.mx_blocks(u, "e4m3")[0] if gated else torch.ones(1, dtype=torch.float64)
        g = dy.double()
        off = (g * uv).abs() * (bd + 4 * U * dh.abs())
        close(dx.view, g * uv * dh, off + R.half_ulp((g * uv * dh).abs() + off, t))
        if gated:
            off = g.abs() * (bf + 2 * U * fh.abs())
            close(du.view, g * fh, off + R.half_ulp((g * fh).abs() + off, t))
        G.amp_act_backward_mx8(dyd, kind, (q.view, s.view), dyd,      # in place
                               **(dict(saved_up=(qu.view, su.view), dup=du.view) if gated else {}))
        assert torch.equal(dyd, dx.view)


# rows of more than a thousand elements, as many as give every SM work, not whole groups of eight
LONG_SIZES = [(600, 1111), (301, 2999), (521, 1025)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("kind,gated", [("gelu", False), ("gelu_tanh", True), ("silu", True)])
def test_activations_of_long_odd_rows(G, dev, dt, kind, gated, monkeypatch):
    monkeypatch.setitem(globals(), "SIZES", LONG_SIZES)
    test_activations(G, dev, dt, kind, gated)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lead", [0, 1])
def test_ckpt8_of_long_odd_rows(G, dev, dt, lead, monkeypatch):
    monkeypatch.setitem(globals(), "SIZES", LONG_SIZES)
    test_ckpt8_special_values(G, dev, dt, lead)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lead", [0, 1])
def test_ckpt8_special_values(G, dev, dt, lead):
    for i, (r, c) in enumerate(SIZES):
        x = values(r, c, TYPES[dt], 300 + i, special=True)
        q = Guarded(r * c, torch.float8_e4m3fn, dev, lead, shape=(r, c))
        s = Guarded(r * -(-c // 32), torch.uint8, dev, shape=(r, -(-c // 32)))
        G.amp_ckpt8_save(place(x, dev, lead), q.view, s.view)
        assert q.intact() and s.intact()
        v, e, _ = R.mx_blocks(x, "e4m3")
        assert torch.equal(s.view.cpu(), e.to(torch.uint8))
        for t in TYPES.values():
            out = Guarded(r * c, t, dev, lead, shape=(r, c))
            G.amp_ckpt8_restore(q.view, s.view, out.view)
            assert out.intact() and same(out.view, v.to(t))


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_activation_extremes(G, dev, kind):
    """Large inputs reach the limits (0 and x), a NaN block's gradient is NaN."""
    x = torch.tensor([[-1e4, -100.0, -40.0, 0.0, 40.0, 100.0, 1e4, 3e4]], device=dev)
    y = torch.empty_like(x)
    q, s = G.ckpt8_buffers(1, 8)
    G.amp_act_forward_mx8(x, kind, y, (q, s))
    assert (y[0, :4].abs() < 1e-12).all() and torch.equal(y[0, 4:], x[0, 4:])
    dx, one = torch.empty_like(x), torch.ones_like(x)
    for v, want in ((-3e4, 0.0), (3e4, 1.0)):
        G.amp_ckpt8_save(torch.full_like(x, v), q, s)
        G.amp_act_backward_mx8(one, kind, (q, s), dx)
        assert (dx == want).all()
    x[0, 2] = math.nan
    G.amp_act_forward_mx8(x, kind, y, (q, s))
    G.amp_act_backward_mx8(one, kind, (q, s), dx)
    assert dx.isnan().all() and int(y.isnan().sum()) == 1


def test_empty_shapes(G, dev):
    for r, c in ((0, 40), (40, 0)):
        x = torch.empty(r, c, device=dev)
        q, s = G.fp4_mx_buffers(r, c)
        G.fp4_quant_mx(x, q, s)
        G.fp4_dequant_mx(q, s, x)
        q8, s8 = G.ckpt8_buffers(r, c)
        G.amp_ckpt8_save(x, q8, s8)
        G.amp_act_forward_mx8(x, "gelu", x, (q8, s8))
        G.amp_act_backward_mx8(x, "gelu", (q8, s8), x)


# ------------------------------------------------------------------ streams
def test_side_stream_and_graph(G, dev):
    """Calls on a stream of their own, and replayed from a CUDA graph, give the same bits."""
    x = torch.randn(130, 288, device=dev).to(torch.bfloat16)
    w = torch.randn(288, device=dev)
    want = None
    s = torch.cuda.Stream()
    y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    m, r, work = torch.empty(130, device=dev), torch.empty(130, device=dev), G.amp_layer_norm_workspace(x)
    q, sc = G.ckpt8_buffers(130, 288)
    p4, s4 = G.fp4_mx_buffers(130, 288)

    def calls(stream):
        G.amp_layer_norm_forward(x, w, None, 1e-5, y, m, r, saved=(q, sc), stream=stream)
        G.fp4_quant_mx(y, p4, s4, stream=stream)
        G.amp_layer_norm_backward(x, None, w, m, r, dx, dw, db, work, saved=(q, sc), stream=stream)
    calls(None)
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dx, dw, db, p4, s4)]
    for t in (y, dx, dw, db, p4, s4):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    calls(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, dw, db, p4, s4)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        calls(s)
    for t in (y, dx, dw, db, p4, s4):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, dw, db, p4, s4)))


def test_fp4_quant_offsets_past_32_bits(G, dev):
    """A matrix of more than 2^31 elements: its last rows."""
    r, c = 70001, 32768
    x = torch.zeros(r, c, dtype=torch.bfloat16, device=dev)
    x[-130:].normal_()
    q, s = G.fp4_mx_buffers(r, c)
    G.fp4_quant_mx(x, q, s)
    v, e, _ = R.mx_blocks(x[-2:], "e2m1")
    out = torch.empty(2, c, dtype=torch.bfloat16, device=dev)
    q2, s2 = G.fp4_mx_buffers(2, c)
    G.fp4_quant_mx(x[-2:], q2, s2)
    G.fp4_dequant_mx(q2, s2, out)
    assert same(out, v) and torch.equal(q[-2:], q2) and not q[:-130].any()
    full = torch.empty_like(x)
    G.fp4_dequant_mx(q, s, full)
    assert same(full[-2:], v) and not full[:1000].any()


# ------------------------------------------------------------------ refusals
def test_binding_refuses_what_would_not_fit(G, dev):
    """Wrong types, sizes and layouts are refused with their name before any call."""
    x = torch.zeros(40, 64, dtype=torch.bfloat16, device=dev)
    q, s = G.fp4_mx_buffers(40, 64)
    q8, s8 = G.ckpt8_buffers(40, 64)
    f, w = torch.zeros(40, device=dev), torch.zeros(64, device=dev)
    for match, call in (
            ("q: 1279 elements, at least 1280", lambda: G.fp4_quant_mx(x, q.view(-1)[:1279], s)),
            ("scales: 511 elements, at least 512", lambda: G.fp4_quant_mx(x, q, s[:511])),
            ("q: 2-byte elements", lambda: G.fp4_quant_mx(x, q.view(torch.int16), s)),
            ("x: dtype Int; f32, f16 or bf16", lambda: G.fp4_quant_mx(x.int(), q, s)),
            ("x: needs a contiguous CUDA", lambda: G.fp4_quant_mx(x.t(), q, s)),
            ("x: needs a tensor", lambda: G.fp4_quant_mx([1.0], q, s)),
            ("skip_if: dtype Float", lambda: G.fp4_quant_mx(x, q, s, skip_if=f)),
            ("stream: needs a stream", lambda: G.fp4_quant_mx(x, q, s, stream="s")),
            ("out: needs a contiguous", lambda: G.fp4_dequant_mx(q, s, torch.zeros(64, 40, device=dev).t())),
            ("b: 1280 elements, at least", lambda: G.fp4_product_mx(q, s, q, s, 64, torch.zeros(40, 41, device=dev))),
            ("k = 1.5", lambda: G.fp4_product_mx(q, s, q, s, 1.5, torch.zeros(40, 40, device=dev))),
            ("y: dtype Float, expected BFloat16", lambda: G.amp_layer_norm_forward(x, w, w, 1e-5, x.float())),
            ("mean: 39 elements", lambda: G.amp_layer_norm_forward(x, w, w, 1e-5, x, f[:39])),
            ("eps: needs a number", lambda: G.amp_layer_norm_forward(x, w, w, "e", x)),
            ("saved: needs", lambda: G.amp_layer_norm_forward(x, w, w, 1e-5, x, saved=q8)),
            ("saved: dtype Byte, expected Float8", lambda: G.amp_layer_norm_forward(x, w, w, 1e-5, x, saved=(q, s8))),
            ("saved: 79 elements", lambda: G.amp_ckpt8_save(x, q8, s8.view(-1)[:79]) or G.amp_act_forward_mx8(
                x, "silu", x, (q8, s8.view(-1)[:79]))),
            ("dx: 64 elements", lambda: G.amp_layer_norm_backward(x, x, w, f, f, x[0])),
            ("up: dtype Float", lambda: G.amp_act_forward_mx8(x, "silu", x, up=x.float())),
    ):
        if match.startswith("saved: 79"):
            with pytest.raises(ValueError, match="79 elements, at least 80"):
                call()
            continue
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(G.AmpError, match="workspace needs"):
        G.amp_layer_norm_backward(x, x, w, f, f, None, w, w, torch.zeros(16, dtype=torch.uint8, device=dev))
    with pytest.raises(G.AmpError, match="go together"):
        G.fp4_quant_mx(x, q, s, G.fp4_mx_buffers(64, 40)[0])
    with pytest.raises(G.AmpError, match="16-byte aligned"):
        G.fp4_dequant_mx(torch.zeros(2000, dtype=torch.uint8, device=dev)[1:], s, x)
    with pytest.raises(G.AmpError, match="both checkpoints or none"):
        G.amp_act_forward_mx8(x, "silu", x.clone(), (q8, s8), up=x)
    with pytest.raises(TypeError):
        G.fp4_quant_mx(x)
