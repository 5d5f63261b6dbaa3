"""Training steps of one MLP block, norm -> linear -> GELU -> linear, in low precision:
the linear layers' three products each on 4-bit blocks, the norm's and the activation's
inputs kept in 8 bits for the backward pass, gradients scaled by the loss scale and taken
by AmpOptimizerStep, whose bf16 copies are quantised again after each step.

    python examples/mlp_block_step.py [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import loss_scaling_master_gb300 as G  # noqa: E402


class Packed:
    """A matrix [rows, cols] in 4 bits, along its rows and transposed."""

    def __init__(self, rows, cols):
        self.q, self.qt = G.fp4_mx_buffers(rows, cols), G.fp4_mx_buffers(cols, rows)

    def fill(self, x):
        G.fp4_quant_mx(x, *self.q, *self.qt)
        return self


class MlpBlock:
    EPS = 1e-5

    def __init__(self, tokens, d, hidden, seed=0, scale=2.0 ** 12, lr=3e-3):
        dev, bf16 = torch.device("cuda"), torch.bfloat16
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device=dev)
        e = lambda *s, dt=bf16: torch.empty(s, dtype=dt, device=dev)
        self.tokens, self.d, self.hidden = tokens, d, hidden
        # norm weight, norm bias, [hidden, d], [d, hidden]
        master = [torch.ones(d, device=dev), torch.zeros(d, device=dev),
                  (n(hidden, d) / d ** 0.5).view(-1), (n(d, hidden) / hidden ** 0.5).view(-1)]
        self.grads = [torch.empty(p.numel(), dtype=bf16, device=dev) for p in master]
        self.step = G.AmpOptimizerStep(master, self.grads, lr=lr, beta1=0.9, beta2=0.95, eps=1e-8,
                                       weight_decay=0.0, init_scale=scale, growth_interval=1000)
        self.w1, self.w2 = Packed(hidden, d), Packed(d, hidden)
        # activations in 4 bits, checkpoints in 8, and what passes between the calls
        self.y4, self.h4 = Packed(tokens, d), Packed(tokens, hidden)
        self.do4, self.da4 = Packed(tokens, d), Packed(tokens, hidden)
        self.x8, self.a8 = G.ckpt8_buffers(tokens, d), G.ckpt8_buffers(tokens, hidden)
        self.y, self.a, self.h = e(tokens, d), e(tokens, hidden), e(tokens, hidden)
        self.out = e(tokens, d, dt=torch.float32)
        self.mean, self.rstd = e(tokens, dt=torch.float32), e(tokens, dt=torch.float32)
        self.dh, self.da, self.dy = e(tokens, hidden), e(tokens, hidden), e(tokens, d)
        self.dx = e(tokens, d)
        self.work = G.amp_layer_norm_workspace(self.y)
        self.pack_weights()

    def pack_weights(self):
        _, _, w1, w2 = self.step.bf16
        self.w1.fill(w1.view(self.hidden, self.d))
        self.w2.fill(w2.view(self.d, self.hidden))

    def forward(self, x):
        lw, lb = self.step.bf16[:2]
        G.amp_layer_norm_forward(x, lw, lb, self.EPS, self.y, self.mean, self.rstd, saved=self.x8)
        G.fp4_product_mx(*self.y4.fill(self.y).q, *self.w1.q, self.d, self.a)
        G.amp_act_forward_mx8(self.a, "gelu", self.h, self.a8)
        G.fp4_product_mx(*self.h4.fill(self.h).q, *self.w2.q, self.hidden, self.out)
        return self.out

    def backward(self, dout):
        """Gradients of the scaled loss from its gradient [tokens, d] (bf16) at the output."""
        gw, gb, g1, g2 = self.grads
        do = self.do4.fill(dout)
        G.fp4_product_mx(*do.qt, *self.h4.qt, self.tokens, g2.view(self.d, self.hidden))
        G.fp4_product_mx(*do.q, *self.w2.qt, self.d, self.dh)
        G.amp_act_backward_mx8(self.dh, "gelu", self.a8, self.da)
        da = self.da4.fill(self.da)
        G.fp4_product_mx(*da.qt, *self.y4.qt, self.tokens, g1.view(self.hidden, self.d))
        G.fp4_product_mx(*da.q, *self.w1.qt, self.hidden, self.dy)
        G.amp_layer_norm_backward(self.dy, None, self.step.bf16[0], self.mean, self.rstd, self.dx,
                                  gw, gb, self.work, saved=self.x8)
        return self.dx

    def train_step(self, x, target):
        """One step on mean squared error; returns the loss (a device scalar)."""
        err = self.forward(x) - target
        self.backward((err * (self.step.scale * (2.0 / err.numel()))).to(torch.bfloat16))
        self.step.step()
        self.pack_weights()
        return err.square().mean()


def task(tokens, d, seed=1):
    """Inputs, and what another random block of the same form makes of them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = n(tokens, d).to(torch.bfloat16)
    h = torch.nn.functional.gelu(torch.nn.functional.layer_norm(x.float(), (d,)) @ n(d, 2 * d) / d ** 0.5)
    return x, h @ n(2 * d, d) / (2 * d) ** 0.5


def main(steps=60, tokens=1024, d=256, hidden=1024):
    block = MlpBlock(tokens, d, hidden)
    x, target = task(tokens, d)
    losses = []
    for k in range(steps):
        loss = block.train_step(x, target)
        if k % 10 == 0 or k == steps - 1:
            losses.append(loss.item())
            # a product whose wait gave up is NaN, so its step was skipped; this says why
            G.fp4_mx_check()
            print(f"step {k:4d}  loss {losses[-1]:.4f}")
    print(block.step.state())
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
