"""fp4_linear_mx on pairs of CTAs without a checkpoint, as a prompt and a forward pass without gradients
run it: a bias and a residual alone give, bit for bit, what fp32 additions make of fp4_product_mx's own
sums; every mixture of alignments, onto the residual, short and long reductions, several tiles a pair."""
import ctypes
import itertools

import pytest
import torch

import more_ops_reference as M
import ops_reference as R
from test_gpu_bounds import Guarded, _INT
from test_gpu_fp4_product import operand
from test_gpu_ops import G, dev, place, values  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DT = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}
_INT.setdefault(torch.float8_e4m3fn, (torch.uint8, 0xA5))
# rows of whole groups of eight, even and odd ones, a last tile of one row; k = 4096 is the longest
# reduction that stages a residual, 4160 the next one's
SHAPES = [(2049, 5120, 288), (2049, 5122, 288), (2049, 5121, 300), (2304, 5120, 4096), (2100, 5128, 4160)]
ids = lambda s: "x".join(map(str, s))


@pytest.fixture(scope="module")
def sums(G, dev):
    """Operands and their product in fp32, made once a shape."""
    made = {}

    def get(shape):
        if shape not in made:
            m, n, k = shape
            a, b = operand(G, m, k, 1)[:2], operand(G, n, k, 2, 0.02)[:2]
            z = torch.empty(m, n, device=dev)
            G.fp4_product_mx(*a, *b, k, z)
            G.fp4_mx_check()
            made[shape] = a, b, z
        return made[shape]
    return get


def inputs(m, n, t, dev, bias_lead, res_lead):
    g = torch.Generator().manual_seed(m + n)
    return place(torch.randn(n, generator=g), dev, bias_lead), place(values(m, n, t, 3), dev, res_lead)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_bias_and_residual(G, dev, sums, shape, dt):
    m, n, k = shape
    t = TYPES[dt]
    a, b, z32 = sums(shape)
    # leads of 1, 2 and 3 elements: off 16 bytes, and in 16-bit types off 4 bytes or not
    for bt, out_lead, res_lead in itertools.product((None, torch.float32, t), (0, 1, 2), (None, 0, 1, 2, 3)):
        bias, res = inputs(m, n, t, dev, 1 if out_lead else 0, res_lead or 0)
        bias = None if bt is None else place(bias.to(bt), dev, 1 if out_lead else 0)
        z = z32 if bias is None else z32 + bias.float()
        want = (z if res_lead is None else z + res.float()).to(t)
        out = Guarded(m * n, t, dev, out_lead, shape=(m, n))
        G.fp4_linear_mx(*a, *b, k, out.view, bias=bias, residual=None if res_lead is None else res)
        assert out.intact() and torch.equal(out.view, want), (bt, out_lead, res_lead)
        if res_lead is not None:        # onto the residual
            G.fp4_linear_mx(*a, *b, k, res, bias=bias, residual=res)
            assert torch.equal(res, want), (bt, out_lead, res_lead)
    G.fp4_mx_check()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shape", SHAPES[:3] + SHAPES[4:], ids=ids)
def test_activations_without_a_checkpoint(G, dev, sums, shape, dt):
    m, n, k = shape
    t = TYPES[dt]
    a, b, z32 = sums(shape)
    for kind, lead, with_res in itertools.product(("gelu", "gelu_tanh", "silu"), (0, 1), (False, True)):
        bias, res = inputs(m, n, t, dev, lead, lead)
        z = (z32 + bias).double()
        want = R.act(z, kind)[0]
        e = M.act_error(z, kind, t)
        if with_res:
            want = want + res.double()
            e = e + R.U * (want.abs() + e)
        e = e + R.half_ulp(want.abs() + e, t)
        out = Guarded(m * n, t, dev, lead, shape=(m, n))
        args = dict(bias=bias, kind=kind, residual=res if with_res else None)
        G.fp4_linear_mx(*a, *b, k, out.view, **args)
        off = (out.view.double() - want).abs()
        over = (t == torch.float16) & out.view.isinf() & (want.abs() + e >= 65520)
        assert out.intact() and ((off <= e) | over).all(), (kind, lead, with_res)
        if with_res:
            G.fp4_linear_mx(*a, *b, k, res, **args)
            assert torch.equal(res, out.view)


@pytest.mark.parametrize("dt", TYPES)
def test_the_checkpoint_of_tensors_off_16_bytes(G, dev, sums, dt):
    """Rows of whole groups of eight whose tensors start elsewhere: the blocks of z as fp32 holds it."""
    m, n, k = SHAPES[0]
    t = TYPES[dt]
    a, b, z32 = sums(SHAPES[0])
    for lead_out, lead_q, kind in ((1, 0, None), (0, 1, "gelu"), (2, 4, "silu")):
        bias, res = inputs(m, n, t, dev, 0, 0)
        q, s = G.ckpt8_buffers(m, n)
        G.amp_ckpt8_save(z32 + bias, q, s)
        ck = (Guarded(m * n, torch.float8_e4m3fn, dev, lead_q, shape=(m, n)),
              Guarded(m * n // 32, torch.uint8, dev, lead_q, shape=(m, n // 32)))
        out = Guarded(m * n, t, dev, lead_out, shape=(m, n))
        G.fp4_linear_mx(*a, *b, k, out.view, bias=bias, kind=kind, residual=res, saved=tuple(c.view for c in ck))
        assert out.intact() and all(c.intact() for c in ck)
        assert torch.equal(ck[0].view.view(torch.uint8), q.view(torch.uint8)) and torch.equal(ck[1].view, s)
        if kind is None:
            assert torch.equal(out.view, (z32 + bias + res.float()).to(t))


@pytest.mark.parametrize("role,stages", [(0, 0), (0, 3), (1, 3), (2, 3)])
@pytest.mark.parametrize("shape", [(2049, 5122, 600), (2049, 5120, 600), (2049, 5120, 4160)], ids=ids)
def test_a_wait_that_gives_up(G, dev, shape, role, stages):
    """A residual alone, and onto itself: what was not finished is NaN, the rest is right."""
    m, n, k = shape
    a, b = operand(G, m, k, 1)[:2], operand(G, n, k, 2, 0.02)[:2]
    for t, inplace in itertools.product(DT, (False, True)):
        res = values(m, n, t, 5).to(dev)
        want = torch.empty_like(res)
        G.fp4_linear_mx(*a, *b, k, want, residual=res)
        out = res if inplace else torch.full_like(res, 7.0)
        st = G.ops._load().fp4_linear_mx_selftest(
            *[x.data_ptr() for x in (*a, *b)], m, n, k, None, 1, -1, res.data_ptr(), out.data_ptr(), DT[t], None, None,
            role, stages, 22, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        with pytest.raises(G.AmpError) as e:
            G.fp4_mx_check()
        assert e.value.status == -6
        G.fp4_mx_check()
        bad = out.isnan()
        assert bad.all() if stages == 0 else bad.any() or role != 2
        assert torch.equal(torch.where(bad, want, out), want)
