"""Training steps of a next-token head: norm -> linear with bias and GELU -> linear with bias ->
dropout onto the residual -> logits -> log probabilities of the next tokens.  The linear layers are
4-bit products with their biases and activation in the epilogue, the activation's and the norm's
inputs are kept in 8 bits, the dropout's mask is a function of the optimizer's step count, and the
loss scale multiplies the gradient where it begins, at the logits.

    python examples/token_step.py [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for p in (ROOT, os.path.join(ROOT, "examples")):
    if p not in sys.path:
        sys.path.insert(0, p)

import loss_scaling_master_gb300 as G  # noqa: E402
from mlp_block_step import Packed  # noqa: E402

PAD = -100  # a position without a next token


class TokenHead:
    # one dropout, one micro-batch a step, one rank (others take sites and seeds of their own)
    EPS, SEED, SITE = 1e-5, 0x5EED, 0

    def __init__(self, tokens, d, hidden, vocab, p=0.1, entropy=0.0, seed=0, scale=2.0 ** 12, lr=1e-3):
        dev, bf16, f32 = torch.device("cuda"), torch.bfloat16, torch.float32
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device=dev)
        e = lambda *s, dt=bf16: torch.empty(s, dtype=dt, device=dev)
        self.tokens, self.d, self.hidden, self.vocab, self.p = tokens, d, hidden, vocab, p
        # norm weight and bias, [hidden, d] and bias, [d, hidden] and bias, [vocab, d]
        master = [torch.ones(d, device=dev), torch.zeros(d, device=dev), (n(hidden, d) / d ** 0.5).view(-1),
                  torch.zeros(hidden, device=dev), (n(d, hidden) / hidden ** 0.5).view(-1), torch.zeros(d, device=dev),
                  (n(vocab, d) / d ** 0.5).view(-1)]
        self.grads = [torch.empty(m.numel(), dtype=bf16, device=dev) for m in master]
        self.step = G.AmpOptimizerStep(master, self.grads, lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0,
                                       init_scale=scale, growth_interval=1000)
        self.w1, self.w2, self.w3 = Packed(hidden, d), Packed(d, hidden), Packed(vocab, d)
        self.y4, self.h4, self.r4 = Packed(tokens, d), Packed(tokens, hidden), Packed(tokens, d)
        self.dz4, self.dt4, self.da4 = Packed(tokens, vocab), Packed(tokens, d), Packed(tokens, hidden)
        self.x8, self.a8 = G.ckpt8_buffers(tokens, d), G.ckpt8_buffers(tokens, hidden)
        self.y, self.h, self.t, self.r = e(tokens, d), e(tokens, hidden), e(tokens, d), e(tokens, d)
        self.mean, self.rstd = e(tokens, dt=f32), e(tokens, dt=f32)
        self.logits, self.logp, self.ent, self.stats = (e(tokens, vocab), e(tokens, dt=f32), e(tokens, dt=f32),
                                                        e(tokens, 2, dt=f32))
        self.dr, self.dt, self.dh, self.da, self.dy = (e(tokens, d), e(tokens, d), e(tokens, hidden),
                                                       e(tokens, hidden), e(tokens, d))
        self.dx = e(tokens, d)
        self.dlogp, self.dent = e(tokens, dt=f32), torch.full((tokens,), -entropy / tokens, device=dev)
        self.work = G.amp_layer_norm_workspace(self.y)
        self.pack_weights()

    def pack_weights(self):
        _, _, w1, _, w2, _, w3 = self.step.bf16
        self.w1.fill(w1.view(self.hidden, self.d))
        self.w2.fill(w2.view(self.d, self.hidden))
        self.w3.fill(w3.view(self.vocab, self.d))

    def forward(self, x, target):
        """Log probabilities of the target tokens [tokens] (0 where there is none)."""
        lw, lb, _, b1, _, b2, _ = self.step.bf16
        G.amp_layer_norm_forward(x, lw, lb, self.EPS, self.y, self.mean, self.rstd, saved=self.x8)
        G.fp4_linear_mx(*self.y4.fill(self.y).q, *self.w1.q, self.d, self.h, bias=b1, kind="gelu", saved=self.a8)
        G.fp4_linear_mx(*self.h4.fill(self.h).q, *self.w2.q, self.hidden, self.t, bias=b2)
        G.amp_dropout_forward(self.t, self.p, self.SEED, self.SITE, self.r, residual=x, step=self.step.step_count)
        G.fp4_product_mx(*self.r4.fill(self.r).q, *self.w3.q, self.d, self.logits)
        G.amp_token_logprobs_forward(self.logits, target, self.logp, self.ent, self.stats)
        return self.logp

    def backward(self, target):
        """Gradients of the scaled loss, minus the mean log probability (and the entropy's share)."""
        gw, gb, g1, gb1, g2, gb2, g3 = self.grads
        self.dlogp.copy_(-1.0 / (target >= 0).sum().float())
        # in place: the logits' gradient takes the logits' buffer
        G.amp_token_logprobs_backward(self.dlogp, self.logits, target, self.stats, self.logits, entropy=self.ent,
                                      dentropy=self.dent, scale=self.step.scale)
        dz = self.dz4.fill(self.logits)
        G.fp4_product_mx(*dz.qt, *self.r4.qt, self.tokens, g3.view(self.vocab, self.d))
        G.fp4_product_mx(*dz.q, *self.w3.qt, self.vocab, self.dr)
        G.amp_dropout_backward(self.dr, self.p, self.SEED, self.SITE, self.dt, step=self.step.step_count, dbias=gb2)
        dt = self.dt4.fill(self.dt)
        G.fp4_product_mx(*dt.qt, *self.h4.qt, self.tokens, g2.view(self.d, self.hidden))
        G.fp4_product_mx(*dt.q, *self.w2.qt, self.d, self.dh)
        G.amp_bias_act_backward_mx8(self.dh, gb1, kind="gelu", saved=self.a8, dx=self.da)
        da = self.da4.fill(self.da)
        G.fp4_product_mx(*da.qt, *self.y4.qt, self.tokens, g1.view(self.hidden, self.d))
        G.fp4_product_mx(*da.q, *self.w1.qt, self.hidden, self.dy)
        G.amp_layer_norm_backward(self.dy, None, self.step.bf16[0], self.mean, self.rstd, self.dx, gw, gb, self.work,
                                  saved=self.x8)
        self.dx += self.dr  # the residual's
        return self.dx

    def train_step(self, x, target):
        """One step; returns the loss (a device scalar)."""
        loss = -self.forward(x, target).sum() / (target >= 0).sum()
        self.backward(target)
        self.step.step()
        self.pack_weights()
        return loss


def task(tokens, d, vocab, seed=1):
    """Embeddings of a few tokens, and the token that follows each; some positions have none."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    table = torch.randn((512, d), generator=g, device="cuda")
    which = torch.randint(0, 512, (tokens,), generator=g, device="cuda")
    follows = torch.randint(0, vocab, (512,), generator=g, device="cuda")
    x = table[which] + torch.randn((tokens, d), generator=g, device="cuda")
    target = torch.where(torch.rand(tokens, generator=g, device="cuda") < 0.1, PAD, follows[which])
    return x.to(torch.bfloat16), target


def main(steps=60, tokens=1024, d=256, hidden=1024, vocab=5003):
    head = TokenHead(tokens, d, hidden, vocab)
    x, target = task(tokens, d, vocab)
    losses = []
    for k in range(steps):
        loss = head.train_step(x, target)
        if k % 10 == 0 or k == steps - 1:
            losses.append(loss.item())
            # a product whose wait gave up is NaN, so its step was skipped; this says why
            G.fp4_mx_check()
            print(f"step {k:4d}  loss {losses[-1]:.4f}")
    print(head.step.state())
    ids = torch.empty((4, 3), dtype=torch.int64, device="cuda")
    top = torch.empty((4, 3), device="cuda")
    head.forward(x, target)
    G.amp_token_logprobs_forward(head.logits[:4], None, None, top_ids=ids, top_logp=top)
    print("most probable", ids.tolist(), "expected", target[:4].tolist())
    return losses


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
