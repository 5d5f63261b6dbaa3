"""Biases' gradients over many columns, where a CTA takes tiles of 64 of them, and over odd rows in
several steps: random values, so that no column can stand for another, in every type, with and without
an activation, and dropout's; on both sides of the width from which the tiles are wide."""
import itertools

import pytest
import torch

import ops_reference as R
from test_gpu_bounds import Guarded
from test_gpu_linear import bias_bound
from test_gpu_ops import G, close, dev, place  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# on 152 SMs tiles of 64 columns begin at 4864; 4099 and 2500 rows are several steps of a thread
SIZES = [(700, 4856), (700, 4864), (4099, 5120), (33, 8192), (2500, 12288), (1000, 5121), (2500, 4869), (4099, 4868),
         (129, 20003)]


def matrix(r, c, t, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    # a column's size is its own, so a sum that lands elsewhere shows
    return (torch.randn(r, c, generator=g, device=dev) * (0.5 + torch.rand(c, generator=g, device=dev))).to(t)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_bias_and_activation(G, dev, size, dt):
    r, c = size
    t = TYPES[dt]
    x, dy = matrix(r, c, t, 1, dev), matrix(r, c, t, 2, dev)
    q, s = G.ckpt8_buffers(r, c)
    G.amp_ckpt8_save(x, q, s)
    zh = torch.empty(r, c, device=dev)
    G.amp_ckpt8_restore(q, s, zh)
    zh, d = zh.double(), dy.double()
    for kind, bt in itertools.product((None, "gelu", "gelu_tanh", "silu"), {t, torch.float32}):
        db = Guarded(c, bt, dev)
        if kind is None:
            G.amp_bias_act_backward_mx8(dy, db.view)
            dz, e = d, torch.zeros_like(d)
        else:
            dx, want = torch.empty_like(dy), torch.empty_like(dy)
            G.amp_bias_act_backward_mx8(dy, db.view, kind, (q, s), dx)
            G.amp_act_backward_mx8(dy, kind, (q, s), want)
            assert torch.equal(dx, want)
            dz = d * R.act(zh, kind)[1]
            e = d.abs() * R.act_bounds(zh, kind)[1] + 2.0 ** -126
            if t != torch.float32:  # the 16-bit forms' derivative is good to 2^-14 (1 + |x|)
                e = d.abs() * (1 + zh.abs()) * 2.0 ** -14 + 2.0 ** -126
        assert db.intact()
        close(db.view, dz.sum(0).cpu(), bias_bound(dz, e, bt).cpu())
        first = db.view.clone()
        if kind is None:
            G.amp_bias_act_backward_mx8(dy, db.view)
        else:
            G.amp_bias_act_backward_mx8(dy, db.view, kind, (q, s), dx)
            mine = dy.clone()
            G.amp_bias_act_backward_mx8(mine, db.view, kind, (q, s), mine)      # in place
            assert torch.equal(mine, want)
        assert torch.equal(db.view, first)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_dropout(G, dev, size, dt):
    r, c = size
    t = TYPES[dt]
    dy, ones = matrix(r, c, t, 3, dev), torch.ones(r, c, dtype=t, device=dev)
    for p in (0.25, 0.0):
        keep = torch.empty_like(ones)
        G.amp_dropout_backward(ones, p, 77, 4, keep)            # the mask, as the definition's tests pin it
        want = torch.empty_like(dy)
        G.amp_dropout_backward(dy, p, 77, 4, want)
        exact = torch.where(keep != 0, dy.double() / (1 - p), 0.0)
        for bt in {t, torch.float32}:
            db, dx = Guarded(c, bt, dev), torch.empty_like(dy)
            G.amp_dropout_backward(dy, p, 77, 4, dx, dbias=db.view)
            assert db.intact() and torch.equal(dx, want)
            # the factor's rounding and the product's
            close(db.view, exact.sum(0).cpu(), bias_bound(exact, 2 * R.U * exact.abs(), bt).cpu())
            first, mine = db.view.clone(), dy.clone()
            G.amp_dropout_backward(mine, p, 77, 4, mine, dbias=db.view)         # in place
            assert torch.equal(mine, want) and torch.equal(db.view, first)
