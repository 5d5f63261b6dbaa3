"""The 4-bit product against the 64-bit product of the same codes' values: every
width of the instruction, cut reductions, ragged sizes, all output types."""
import math

import pytest
import torch

import ops_reference as R
from test_gpu_bounds import Guarded
from test_gpu_ops import G, close, dev, place, same, values  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def operand(G, rows, k, seed, sigma=1.0):
    x = (values(rows, k, torch.float32, seed) * sigma).to("cuda")
    q, s = G.fp4_mx_buffers(rows, k)
    G.fp4_quant_mx(x, q, s)
    v = torch.empty(rows, k, device="cuda")
    G.fp4_dequant_mx(q, s, v)
    return q, s, v.double()


def bound(a, b, k):
    """Each instruction sums 64 exact products and adds them to the accumulator:
    k/64 additions and at most 8 of partial sums, each wrong by at most 2^-23 of
    the largest magnitude on the way, which the sum of |a b| bounds."""
    return (math.ceil(k / 64) + 8) * 2.0 ** -23 * (a.abs() @ b.abs().t())


# m, n, k: each token width, one and several tiles, cut and whole reductions, ragged everything
SHAPES = [(1, 1, 1), (1, 128, 32), (1, 14336, 4096), (3, 7, 33), (16, 128, 64), (17, 200, 96), (33, 130, 129),
          (48, 4096, 4096), (64, 64, 1000), (65, 129, 257), (128, 128, 256), (129, 1000, 777), (256, 384, 512),
          (300, 300, 300), (1000, 2304, 768), (4096, 4099, 160), (2049, 5121, 288), (2000, 131, 2080),
          (128, 256, 20000), (3001, 3000, 1), (300, 20000, 64), (5000, 2600, 65)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_product(G, dev, shape):
    m, n, k = shape
    a, sa, av = operand(G, m, k, 7 * m + n)
    b, sb, bv = operand(G, n, k, 5 * n + k, 0.02)
    want, off = (av @ bv.t()).cpu(), bound(av, bv, k).cpu()
    for dt, t in TYPES.items():
        lead = 1 if dt != "bf16" else 0
        out = Guarded(m * n, t, dev, lead, shape=(m, n))
        G.fp4_product_mx(a, sa, b, sb, k, out.view)
        G.fp4_mx_check()
        assert out.intact()
        close(out.view, want, off + R.half_ulp(want.abs() + off, t))
        again = torch.empty_like(out.view)
        G.fp4_product_mx(a, sa, b, sb, k, again)
        assert torch.equal(again, out.view)


@pytest.mark.parametrize("shape", [(1, 300, 2600), (5, 130, 4001), (16, 1000, 5000), (20, 517, 3333), (32, 128, 7000),
                                   (50, 301, 4100), (100, 700, 8191), (7, 6401, 4100), (128, 6401, 7700)],
                         ids=lambda s: "x".join(map(str, s)))
def test_product_of_few_tiles_and_a_long_reduction(G, dev, shape):
    """Reductions that are cut in two or four, for each width of a tile."""
    test_product(G, dev, shape)


def test_product_is_exact_on_small_integers(G, dev):
    """Products and sums that fp32 holds exactly come out exactly."""
    g = torch.Generator().manual_seed(1)
    pick = torch.tensor([0.0, 0.5, 1.0, -1.5, 2.0, -3.0, 4.0, 6.0])
    for m, n, k in ((5, 260, 4096), (600, 700, 1056)):
        a, b = (pick[torch.randint(0, 8, (r, k), generator=g)].to(dev) for r in (m, n))
        ops = []
        for x in (a, b):
            q, s = G.fp4_mx_buffers(*x.shape)
            G.fp4_quant_mx(x, q, s)
            ops += [q, s]
        out = torch.empty(m, n, device=dev)
        G.fp4_product_mx(*ops, k, out)
        assert torch.equal(out.double(), a.double() @ b.double().t())


def test_product_scales_in_every_place(G, dev):
    """A distinct power of two in each block of both operands: any scale taken
    from the wrong row, block or half shows."""
    for m, n, k in ((40, 150, 640), (200, 300, 416), (700, 4200, 352)):
        kb = -(-k // 32)
        r, c = torch.arange(m)[:, None], torch.arange(kb)[None]
        ea = ((3 * r + 5 * c) % 13 - 6).repeat_interleave(32, 1)[:, :k].float()
        r = torch.arange(n)[:, None]
        eb = ((7 * r + 2 * c) % 11 - 5).repeat_interleave(32, 1)[:, :k].float()
        a, b = torch.exp2(ea).to(dev), torch.exp2(eb).to(dev)
        ops = []
        for x in (a, b):
            q, s = G.fp4_mx_buffers(*x.shape)
            G.fp4_quant_mx(x, q, s)
            ops += [q, s]
        out = torch.empty(m, n, device=dev)
        G.fp4_product_mx(*ops, k, out)
        want = a.double() @ b.double().t()
        assert ((out.double() - want).abs() <= bound(a.double(), b.double(), k)).all()


def test_product_nonfinite_and_padding(G, dev):
    """A NaN block makes its row (or column) NaN and nothing else; what lies
    behind the packed rows and in padding rows' scales is not used."""
    m, n, k = 130, 140, 300
    a, b = torch.randn(m, k, device=dev), torch.randn(n, k, device=dev)
    a[129, 299], b[3, 0] = math.nan, math.inf
    qa, sa = G.fp4_mx_buffers(m, k)
    qb, sb = G.fp4_mx_buffers(n, k)
    sa.fill_(255)
    sb.fill_(255)
    G.fp4_quant_mx(a, qa, sa)
    G.fp4_quant_mx(b, qb, sb)
    out = torch.empty(m, n, device=dev)
    G.fp4_product_mx(qa, sa, qb, sb, k, out)
    bad = out.isnan()
    assert bad[129].all() and bad[:, 3].all() and int(bad.sum()) == m + n - 1
    # padding rows of the scales hold anything
    ra = sa.clone()
    t = ra.view(2, 3, 32, 4, 4)
    t[1, :, 2:] = 255
    t[1, :, :2, 1:] = 255
    out2 = torch.empty_like(out)
    G.fp4_product_mx(qa, ra, qb, sb, k, out2)
    assert same(out, out2)


def test_product_empty(G, dev):
    z = torch.empty(0, dtype=torch.uint8, device=dev)
    out = torch.full((5, 7), 3.0, device=dev)
    G.fp4_product_mx(z, z, z, z, 0, out)
    assert (out == 0).all()
    G.fp4_product_mx(z, z, z, z, 0, torch.empty(0, 7, device=dev))
    q, s = G.fp4_mx_buffers(7, 64)
    G.fp4_product_mx(z, z, q, s, 64, torch.empty(0, 7, device=dev))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_linear_layer_gradients(G, dev, dt):
    """The three products of a linear layer, each over its own axis: y, dx and dW
    against 64-bit products of the blocks' values."""
    t = TYPES[dt]
    T, n, k = 200, 320, 416
    x, w, dy = (values(r, c, t, s).clamp(-50, 50) for r, c, s in ((T, k, 1), (n, k, 2), (T, n, 3)))
    packed = {}
    for name, m in (("x", x), ("w", w), ("dy", dy)):
        md = m.to(dev)
        q, qt = G.fp4_mx_buffers(*m.shape), G.fp4_mx_buffers(m.shape[1], m.shape[0])
        G.fp4_quant_mx(md, *q, *qt)
        packed[name], packed[name + "t"] = q, qt
    for left, right, red, lv, rv in (("x", "w", k, x, w), ("dy", "wt", n, dy, w.t()), ("dyt", "xt", T, dy.t(), x.t())):
        a, b = R.mx_blocks(lv, "e2m1")[0], R.mx_blocks(rv, "e2m1")[0]
        out = torch.empty(a.shape[0], b.shape[0], device=dev)
        G.fp4_product_mx(*packed[left], *packed[right], red, out)
        close(out, a @ b.t(), bound(a, b, red) + R.half_ulp(a @ b.t(), torch.float32))


def test_product_streams_and_graph(G, dev):
    a, sa, av = operand(G, 300, 512, 1)
    b, sb, _ = operand(G, 400, 512, 2)
    one, _s, _v = operand(G, 1, 512, 3)
    want, w1 = torch.empty(300, 400, device=dev), torch.empty(1, 400, device=dev)
    G.fp4_product_mx(a, sa, b, sb, 512, want)
    G.fp4_product_mx(one, _s, b, sb, 512, w1)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    o, o1 = torch.empty_like(want), torch.empty_like(w1)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        G.fp4_product_mx(a, sa, b, sb, 512, o, stream=s)
        G.fp4_product_mx(one, _s, b, sb, 512, o1, stream=s)
    for _ in range(3):
        o.zero_()
        o1.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(o1, w1)


def test_product_output_past_32_bits(G, dev):
    m, n, k = 70000, 32768, 64
    a, sa, av = operand(G, m, k, 1)
    b, sb, bv = operand(G, n, k, 2)
    out = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
    G.fp4_product_mx(a, sa, b, sb, k, out)
    for rows in (slice(0, 3), slice(40000, 40003), slice(m - 3, m)):
        want = (av[rows] @ bv.t()).cpu()
        off = bound(av[rows], bv, k).cpu()
        close(out[rows], want, off + R.half_ulp(want.abs() + off, torch.bfloat16))
