"""What is left of a 4-bit product whose bounded waits gave up: an error status, NaN
in every element that was not finished and the right value in every other, and a GPU
that goes on working.  One of the kernel's roles is ended early, so that the others'
waits run out after a few milliseconds; no copy or product is lost."""
import ctypes

import pytest
import torch

from test_gpu_fp4_product import operand
from test_gpu_mlp_block import example  # noqa: F401  (fixture)
from test_gpu_ops import G, dev  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
ETIMEOUT = -6
DT = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}
LOADS, SECOND_LOADS, PRODUCTS = 0, 1, 2

# one CTA a tile: each width of the instruction, whole and cut reductions, more tiles than CTAs
SOLO = [(1, 128, 4096), (1, 14336, 1500), (20, 300, 1024), (50, 301, 8192), (100, 700, 8191), (128, 25600, 700)]
# pairs of CTAs: one tile and several a pair, reductions of one and of many stages
PAIR = [(2049, 5121, 600), (4096, 4099, 2600), (700, 20000, 4100)]


def give_up(G, a, sa, b, sb, k, out, role, stages):
    """The product with a role ended early and waits of 2^22 ns."""
    st = G.ops._load().fp4_product_mx_selftest(
        *[x.data_ptr() for x in (a, sa, b, sb)], *out.shape, k, out.data_ptr(), DT[out.dtype], role, stages, 22,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0


def run(G, dev, shape, role, stages, t):
    m, n, k = shape
    a, sa, _ = operand(G, m, k, 1)
    b, sb, _ = operand(G, n, k, 2, 0.02)
    want, out = torch.empty(m, n, dtype=t, device=dev), torch.full((m, n), 7.0, dtype=t, device=dev)
    G.fp4_product_mx(a, sa, b, sb, k, want)
    G.fp4_mx_check()
    assert not want.isnan().any()
    give_up(G, a, sa, b, sb, k, out, role, stages)
    with pytest.raises(G.AmpError) as e:
        G.fp4_mx_check()
    assert e.value.status == ETIMEOUT
    G.fp4_mx_check()                                   # the word is cleared
    bad = out.isnan()
    assert torch.equal(torch.where(bad, want, out), want)
    again = torch.empty_like(want)                     # and the next product is right
    G.fp4_product_mx(a, sa, b, sb, k, again)
    G.fp4_mx_check()
    assert torch.equal(again, want)
    return bad


@pytest.mark.parametrize("shape", SOLO, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("role", [LOADS, PRODUCTS])
@pytest.mark.parametrize("stages", [0, 1, 3])
def test_one_cta_a_tile(G, dev, shape, role, stages):
    for t in DT:
        bad = run(G, dev, shape, role, stages, t)
        if stages == 0:
            assert bad.all()
        else:
            assert bad.any()


@pytest.mark.parametrize("shape", PAIR, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("role", [LOADS, SECOND_LOADS, PRODUCTS])
@pytest.mark.parametrize("stages", [0, 1, 4, 7])
def test_pairs(G, dev, shape, role, stages):
    """Stages that both, the first or the second CTA alone have loaded when the
    products give up."""
    for t in DT:
        bad = run(G, dev, shape, role, stages, t)
        if stages == 0:
            assert bad.all()


def test_finished_tiles_stay(G, dev):
    """Roles that end after a whole tile leave it as it is."""
    assert not run(G, dev, (2049, 5121, 288), LOADS, 2, torch.float32).all()
    assert not run(G, dev, (128, 25600, 700), PRODUCTS, 4, torch.float32).all()


@pytest.mark.parametrize("which", range(6))
def test_a_training_step_is_skipped(G, example, which, monkeypatch):
    """Whichever of a step's six products gives up, the gradient check sees its NaN: the
    weights stay, the scale is halved, and the check of the product says why."""
    block = example.MlpBlock(300, 64, 96)
    x, target = example.task(300, 64)
    before = [t.clone() for t in block.step.master]
    product, calls = G.fp4_product_mx, iter(range(6))

    def one_gives_up(a, sa, b, sb, k, out):
        if next(calls) == which:
            return give_up(G, a, sa, b, sb, k, out, PRODUCTS, 0)
        product(a, sa, b, sb, k, out)
    monkeypatch.setattr(G, "fp4_product_mx", one_gives_up)
    block.train_step(x, target)
    assert next(calls, None) is None
    st = block.step.state()
    assert st["step"] == 0 and st["scale"] == 2.0 ** 11
    assert all(torch.equal(a, b) for a, b in zip(before, block.step.master))
    with pytest.raises(G.AmpError):
        G.fp4_mx_check()
    monkeypatch.undo()
    block.train_step(x, target)
    assert block.step.state()["step"] == 1
    G.fp4_mx_check()


def test_refusals(G, dev):
    f, q = G.ops._load().fp4_product_mx_selftest, torch.zeros(4096, dtype=torch.uint8, device=dev).data_ptr()
    for role, stages, limit in ((-1, 0, 22), (3, 0, 22), (0, -1, 22), (0, 0, -1), (0, 0, 31)):
        assert f(q, q, q, q, 4, 4, 4, q, 1, role, stages, limit, None) == -1
    assert f(None, q, q, q, 4, 4, 4, q, 1, 0, 0, 22, None) == -1
