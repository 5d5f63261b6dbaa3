"""examples/token_step.py: linear layers, dropout and log probabilities together, as a training step
uses them."""
import importlib.util
import math
import os

import pytest
import torch

import more_ops_reference as M
from test_gpu_ops import G, dev  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "token_step.py")


@pytest.fixture(scope="module")
def example(G):
    spec = importlib.util.spec_from_file_location("token_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T,d,h,v", [(1000, 192, 520, 1003), (130, 64, 96, 257)])
def test_gradients_follow_the_unquantised_head(example, T, d, h, v):
    """Each gradient points where the fp32 head's does, with the mask of the definition.  Rounding to
    4-bit blocks changes an operand by about 0.11 of its norm, and up to four products in a row lie
    between the loss and a weight, two operands each: below 0.11 * sqrt(8) = 0.31 of a gradient's
    norm, a cosine above 0.95; the logits themselves move by 0.11 * sqrt(6), and with them the
    gradient that all of this starts from, so it starts from the example's own."""
    head = example.TokenHead(T, d, h, v, entropy=0.01)
    x, target = example.task(T, d, v)
    scale = head.step.scale.item()
    head.forward(x, target)
    logits = head.logits.float()
    dx = head.backward(target).float() / scale
    dlogits = head.logits.float() / scale
    got = [g.float() / scale for g in head.grads] + [dx.view(-1)]
    p = [t.float().clone().requires_grad_(True) for t in head.step.bf16]
    xf = x.float().requires_grad_(True)
    y = torch.nn.functional.layer_norm(xf, (d,), p[0], p[1], 1e-5)
    t = torch.nn.functional.gelu(y @ p[2].view(h, d).t() + p[3]) @ p[4].view(d, h).t() + p[5]
    keep, by = M.keep(0, T * d, head.p, head.SEED, 0, head.SITE)
    out = (xf + torch.where(keep.view(T, d).cuda(), t * by, 0.0)) @ p[6].view(v, d).t()
    for a, w in zip(got, torch.autograd.grad(out, p + [xf], grad_outputs=dlogits)):
        w = w.reshape(-1)
        assert torch.dot(a, w) / (a.norm() * w.norm()) > 0.95
    # and the start: what autograd gives for the same logits, up to bf16's rounding of an element
    lg = logits.clone().requires_grad_(True)
    lp = torch.log_softmax(lg, -1)
    used = target >= 0
    loss = -lp[used, target[used]].sum() / used.sum() + 0.01 / T * (lp.exp() * lp).sum(-1)[used].sum()
    w, = torch.autograd.grad(loss, lg)
    # half a step of bf16, and 2^-16 of the row's largest for fp32's sums on both sides
    assert ((dlogits - w).abs() <= w.abs() * 2.0 ** -8 + w.abs().amax(-1, keepdim=True) * 2.0 ** -16).all()


def test_it_runs(example):
    losses = example.main(steps=12, tokens=300, d=64, hidden=128, vocab=501)
    assert len(losses) == 3 and all(math.isfinite(l) for l in losses)


def test_an_infinite_gradient_skips_the_step(example):
    """A loss scale that the 16-bit gradient cannot hold reaches the weights' gradients as NaN, the
    step is skipped with the scale halved, and the next draws the same mask (the count stays)."""
    head = example.TokenHead(200, 64, 96, 300, scale=2.0 ** 127)
    x, target = example.task(200, 64, 300)
    before = [t.clone() for t in head.step.master]
    head.forward(x, target)
    head.logits[5, 7] = float("nan")
    r = head.r.clone()
    head.backward(target)
    head.step.step()
    st = head.step.state()
    assert st["step"] == 0 and st["scale"] == 2.0 ** 126
    assert all(torch.equal(a, b) for a, b in zip(before, head.step.master))
    head.forward(x, target)
    assert torch.equal(r, head.r)


def test_a_captured_step_is_the_eager_one(G, example):
    """Forward and backward captured into a graph and replayed give the same bits, with the step
    count, the scale and the tokens read from the device at each replay."""
    head = example.TokenHead(257, 72, 130, 777, entropy=0.02)
    x, target = example.task(257, 72, 777)
    other = example.task(257, 72, 777, seed=9)[1]

    def run():
        head.forward(x, target)
        head.backward(target)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run()
    for count, scale, tokens in ((0, 4096.0, target.clone()), (3, 1024.0, other)):
        head.step.step_count.fill_(count)
        head.step.scale.fill_(scale)
        target.copy_(tokens)
        run()
        torch.cuda.synchronize()
        want = [t.clone() for t in head.grads + [head.logp, head.ent, head.dx]]
        for t in head.grads + [head.logp, head.ent, head.dx]:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, head.grads + [head.logp, head.ent, head.dx]))
    G.fp4_mx_check()
