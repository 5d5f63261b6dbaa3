"""Plain 64-bit implementations of the linear layer's epilogue, dropout and the token log
probabilities of include/ampops.h, from their definitions, on CPU tensors; and error bounds of the
fp32 kernels against them."""
import math

import numpy as np
import torch

import ops_reference as R

U = R.U


# ------------------------------------------------------------------ dropout
def philox(c, k):
    """Philox4x32-10 of counters [n, 4] under the key (low, high), in numpy."""
    c = [np.asarray(c, dtype=np.uint64)[:, i] for i in range(4)]
    k = list(k)
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & low, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]),
             p & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, 1).astype(np.uint32)


def keep(first, n, p, seed, step, site):
    """Which of the elements first .. first + n - 1 stay, and their factor."""
    g = np.arange(first // 8, -(-(first + n) // 8), dtype=np.uint64)
    c = np.zeros((len(g), 4), dtype=np.uint64)
    c[:, 0], c[:, 1] = g & np.uint64(0xFFFFFFFF), g >> np.uint64(32)
    c[:, 2], c[:, 3] = step % 2 ** 32, 2 ** 30 + site
    w = philox(c, (seed % 2 ** 32, seed >> 32))
    bits = np.stack([w & 0xFFFF, w >> 16], -1).reshape(-1)[first % 8:][:n]
    t = round(p * 65536)
    return torch.from_numpy(bits >= t), (65536 / (65536 - t) if t < 65536 else 0.0)


# ------------------------------------------------------------------ the linear layer
def linear(z, bias, kind, residual):
    """(z + bias, out) in 64 bits."""
    z = z.double()
    if bias is not None:
        z = z + bias.double()
    y = R.act(z, kind)[0] if kind else z
    return z, y if residual is None else y + residual.double()


def act_error(z, kind, dtype):
    """How far the kernels' f may be from f(z) before its rounding (include/ampops.h)."""
    f = R.act(z, kind)[0].abs()
    if dtype != torch.float32:
        return f * 2.0 ** -14 + 2.0 ** -122
    c = {"gelu": 1.25 * z * z, "gelu_tanh": 5.5 * 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3).abs(),
         "silu": torch.zeros_like(z)}[kind]
    return (12 + c) * U * f + 2.0 ** -122


def linear_bound(z, off, kind, residual, want, dtype):
    """Of out, where z's sum is within off: the bias's addition rounds by U |z|, no f has a slope
    above 1.13, the residual's addition rounds by U |out|, and so does the type."""
    ez = off + U * (z.abs() + off)
    e = 1.13 * ez + act_error(z, kind, dtype) if kind else ez
    if residual is not None:
        e = e + U * (want.abs() + e)
    return e + R.half_ulp(want.abs() + e, dtype), ez


def saved_bound(z, ez):
    """Of the values of z's 8-bit blocks: ez, half a step of e4m3 (2^-4 of the value, or half its
    smallest step, 2^-10 of a scale that is below twice the block's maximum over 448)."""
    r, c = z.shape
    kb = -(-c // 32)
    a = torch.zeros(r, kb * 32, dtype=torch.float64)
    a[:, :c] = z.abs() + ez
    top = a.view(r, kb, 32).amax(-1).repeat_interleave(32, 1)[:, :c]
    return ez + (z.abs() + ez) * 2.0 ** -4 + top * (2 / 448) * 2.0 ** -10


# ------------------------------------------------------------------ log probabilities
def logprobs(z, t):
    """log p [rows, cols], log p of the targets and the entropy, in 64 bits, from the differences
    from the maximum (next to values of 1e38 a log of the sum would be lost even here)."""
    z = z.double() - z.double().amax(-1, keepdim=True)
    lp = z - torch.logsumexp(z, -1, keepdim=True)
    ent = -(lp.exp() * lp.clamp_min(-1e300)).sum(-1)
    if t is None:
        return lp, None, ent
    got = lp.gather(1, t.clamp(0, z.shape[1] - 1)[:, None])[:, 0]
    got = torch.where(t >= z.shape[1], torch.full_like(got, math.nan), got)
    return lp, torch.where(t < 0, torch.zeros_like(got), got), torch.where(t < 0, torch.zeros_like(ent), ent)


def logprobs_grad(z, t, dlogp, dent, scale):
    """The gradient at z by the formula."""
    lp, _, _ = logprobs(z, None)
    p = lp.exp()
    ent = -(p * lp.clamp_min(-1e300)).sum(-1, keepdim=True)
    g = torch.zeros_like(p)
    if dlogp is not None:
        hot = torch.zeros_like(p)
        hot.scatter_(1, t.clamp(0, z.shape[1] - 1)[:, None], 1.0)
        g += dlogp.double()[:, None] * (hot - p)
    if dent is not None:
        g -= dent.double()[:, None] * p * (lp.clamp_min(-1e300) + ent)
    if t is not None:
        g[t < 0] = 0.0
        g[t >= z.shape[1]] = math.nan
    return g * scale


def top(z, k):
    """The k largest of each row, equal ones by index; -1 where there are no more above -inf."""
    v, i = torch.sort(z.double(), dim=-1, descending=True, stable=True)
    ids = torch.full((z.shape[0], k), -1, dtype=torch.int64)
    m = min(k, z.shape[1])
    ids[:, :m] = torch.where(v[:, :m] > -math.inf, i[:, :m], -1)
    return ids


def logprobs_bounds(z):
    """(bound of log s and of a log probability less its own difference's rounding, of the entropy).

    A term exp(d) has its difference's, its product's and the constant's rounding, each U |d| in the
    exponent, and an exponential good to 2 ulp (4 U): 3 U |d| + 4 U relative, so the sum of terms is
    off by U (3 D + 4) s with D = sum p |d|.  A term's share of additions: at most cols / 128 on a
    thread and 32 levels of joins with a factor (4 U + its difference's) each, and the thread's
    maximum grows at most cols / 1024 times, a factor each."""
    lp, _, ent = logprobs(z, None)
    cols = z.shape[1]
    d = (z.double() - z.double().amax(-1, keepdim=True)).clamp_min(-1e4).abs()
    D = (lp.exp() * d).sum(-1)
    rel = U * (3 * D + 4 + cols / 128 + 32 * 12 + cols / 1024 * 12)
    logs = torch.logsumexp(z.double() - z.double().amax(-1, keepdim=True), -1)
    one = rel + 2 * U * logs.abs() + 2.0 ** -126
    # w = sum exp(d) d: each term as above and its product, so U (3 |d| + 5) e |d|: their sum over s
    # is below 3 U sum p d^2 + 5 U D; and the sums' own roundings on w
    D2 = (lp.exp() * d * d).sum(-1)
    e = one + U * (3 * D2 + 5 * D) + (rel + 4 * U) * D + 2 * U * ent.abs()
    return one, e
