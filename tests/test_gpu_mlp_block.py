"""examples/mlp_block_step.py: the operators together, as a training step uses them."""
import importlib.util
import os

import pytest
import torch

from test_gpu_ops import G, dev  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mlp_block_step.py")


@pytest.fixture(scope="module")
def example(G):
    spec = importlib.util.spec_from_file_location("mlp_block_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_follow_the_unquantised_block(example):
    """Each gradient points where the fp32 block's does.  Rounding to 4-bit blocks
    changes an operand by about 0.11 of its norm (e2m1 with a power-of-two scale), two
    operands a product and up to three products in a row: below 0.11 * sqrt(8) = 0.31 of
    a gradient's norm, a cosine above 0.95."""
    T, d, h = 1000, 192, 520
    b = example.MlpBlock(T, d, h)
    x, target = example.task(T, d)
    scale = b.step.scale.item()
    err = b.forward(x) - target
    dx = b.backward((err * (2 * scale / err.numel())).to(torch.bfloat16)).float() / scale
    got = [g.float() / scale for g in b.grads] + [dx.view(-1)]
    p = [t.float().clone().requires_grad_(True) for t in b.step.bf16]
    xf = x.float().requires_grad_(True)
    y = torch.nn.functional.layer_norm(xf, (d,), p[0], p[1], 1e-5)
    out = torch.nn.functional.gelu(y @ p[2].view(h, d).t()) @ p[3].view(d, h).t()
    # the same gradient at the output, so that only the backward's rounding shows
    grads = torch.autograd.grad(out, p + [xf], grad_outputs=err.detach() * (2 / err.numel()))
    for a, w in zip(got, grads):
        w = w.reshape(-1)
        assert torch.dot(a, w) / (a.norm() * w.norm()) > 0.95


def test_training_reduces_the_loss(example):
    losses = example.main(steps=60)
    assert losses[-1] < 0.5 * losses[0]


def test_inf_in_the_gradient_skips_the_step(example):
    """An infinite output gradient reaches every weight's gradient through the blocks as NaN,
    the check sees it, and the step is skipped with the scale halved."""
    b = example.MlpBlock(128, 64, 96)
    x, target = example.task(128, 64)
    before = [t.clone() for t in b.step.master]
    b.forward(x)
    do = torch.zeros(128, 64, dtype=torch.bfloat16, device="cuda")
    do[5, 7] = float("inf")
    b.backward(do)
    b.step.step()
    st = b.step.state()
    assert st["step"] == 0 and st["scale"] == 2.0 ** 11
    assert all(torch.equal(a, c) for a, c in zip(before, b.step.master))
