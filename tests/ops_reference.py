"""Plain 64-bit implementations of the operators of include/ampops.h, from their
definitions, on CPU tensors; and error bounds of the fp32 kernels against them.

The block formats are rounded by searching the format's own list of values
(nearest, ties to the even code), so nothing is shared with the kernels' bit
arithmetic."""
import math

import torch

U = 2.0 ** -24  # half an ulp of fp32, relative


def _grid_e2m1():
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _grid_e4m3():
    v = []
    for code in range(127):  # 127 is NaN
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return torch.tensor(v, dtype=torch.float64)


GRIDS = {"e2m1": _grid_e2m1(), "e4m3": _grid_e4m3()}


def mx_blocks(x, fmt):
    """(values [rows, cols], scale bytes [rows, blocks], codes [rows, cols]) of x's block form."""
    grid = GRIDS[fmt]
    top = float(grid[-1])
    x = x.detach().cpu().double()
    rows, cols = x.shape
    kb = -(-cols // 32)
    b = torch.zeros(rows, kb * 32, dtype=torch.float64)
    b[:, :cols] = x
    b = b.view(rows, kb, 32)
    a = b.abs().amax(-1)
    e = torch.zeros(rows, kb, dtype=torch.int64)
    # the smallest e with a <= top * 2^(e - 127), by trying them all
    for p in range(254):
        e += (a > top * 2.0 ** (p - 127)).long()
    bad = ~torch.isfinite(a)
    e[bad] = 255
    scale = torch.where(bad, torch.full_like(a, math.nan), torch.ldexp(torch.ones_like(a), e - 127))
    y = b.abs() / scale[..., None]
    hi = torch.searchsorted(grid, y.nan_to_num(0.0).contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = y - grid[lo], grid[hi] - y
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = torch.where(up, hi, lo)
    v = torch.where(torch.signbit(b), -grid[code], grid[code]) * scale[..., None]
    return (v.view(rows, -1)[:, :cols], e, code.view(rows, -1)[:, :cols])


def tiled_scales(e, rows, cols):
    """Scale bytes [rows, blocks] in the 128 x 4 tile order of ampops.h, padded with zeros."""
    kb, tr, tc = -(-cols // 32), -(-rows // 128), -(-cols // 128)
    out = torch.zeros(tr * tc * 512, dtype=torch.uint8)
    r = torch.arange(rows)[:, None].expand(rows, kb)
    b = torch.arange(kb)[None, :].expand(rows, kb)
    at = ((r // 128) * tc + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    out[at.reshape(-1)] = e.reshape(-1).to(torch.uint8)
    return out


def packed_codes(code, sign):
    """Packed bytes [rows, 16 blocks] of 4-bit codes [rows, cols] with their signs."""
    rows, cols = code.shape
    kb = -(-cols // 32)
    c = torch.zeros(rows, kb * 32, dtype=torch.int64)
    c[:, :cols] = code + 8 * sign.long()
    return (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8)


def half_ulp(v, dtype):
    """The rounding of |v| to a type: at most this much (64-bit tensor)."""
    if dtype == torch.float32:
        return v.abs() * U + 2.0 ** -150
    if dtype == torch.bfloat16:
        return v.abs() * 2.0 ** -8 + 2.0 ** -134
    return v.abs() * 2.0 ** -11 + 2.0 ** -25


def layer_norm(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    y = (x - mean) * rstd
    y = y * w.double() if w is not None else y
    y = y + b.double() if b is not None else y
    return y, mean[:, 0], rstd[:, 0]


def layer_norm_grads(dy, x, w, mean, rstd):
    """dx, dweight, dbias by the formula, from a given mean and rstd [rows]."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    g = dy * w.double() if w is not None else dy
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def act(x, kind):
    """f(x) and f'(x) in 64 bits."""
    x = x.double()
    if kind == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    if kind == "gelu":
        p = 0.5 * torch.erfc(-x / math.sqrt(2))
        return x * p, p + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    # (1 + tanh z) / 2 = sigmoid(2 z): the same function, without the cancellation
    # that leaves the 64-bit 1 + tanh z at zero from z = -19 on
    c = 2 * math.sqrt(2 / math.pi)
    t = torch.sigmoid(c * (x + 0.044715 * x ** 3))
    return x * t, t + x * t * (1 - t) * c * (1 + 3 * 0.044715 * x * x)


def act_bounds(x, kind):
    """Absolute error bounds of the kernels' f and f': an exponential good to
    2 ulp plus the rounding of its argument, a division good to 2 ulp (silu,
    gelu_tanh), an error function good to 2 ulp (gelu)."""
    x = x.double()
    f, _ = act(x, kind)
    if kind == "gelu":
        return x.abs() * 2.0 ** -21 + f.abs() * 2.0 ** -22, (1 + x.abs()) * 2.0 ** -20
    t = x.abs() if kind == "silu" else 1.6 * x.abs() * (1 + 0.045 * x * x)
    return f.abs() * (t + 8) * 2.0 ** -22 + 2.0 ** -126, (1 + x.abs()) * 2.0 ** -19
