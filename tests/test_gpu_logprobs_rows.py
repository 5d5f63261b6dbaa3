"""Every element of a row counts once in amp_token_logprobs_forward, in each of its kernels: a logit
that dominates its row is moved over every 16-byte piece and over the ends, and sums over flat rows are
held to the additions that they really go through.  Alternatives of short rows with more equal logits
than a warp's queue holds."""
import math

import pytest
import torch

import more_ops_reference as M
from test_gpu_ops import G, close, dev, same  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def sum_bound(cols, dtype, D):
    """Relative, of the sum of exponentials, D = sum p |d| (d: differences from the maximum).

    A term exp(d) is off by U (3 |d| + 4): its difference's, its product's and the constant's rounding
    in the exponent, whichever way the difference is cut over the maxima on the way (they add up to d),
    and an exponential good to 2 ulp.  A thread adds a batch of eight loads of 16 bytes in two halves,
    so 32 elements one after another in 16-bit types and 16 in fp32, then the halves, then the batch to
    what it has: 34 additions, and one more a batch.  Each batch may raise the maximum, and each of at
    most 5 + 3 + 3 joins (lanes, warps, a cluster's CTAs) does: an exponential (4 U), its product (U)
    and the addition (U) each.  Batches: a row by at least 32 threads up to 520 pieces, else 128."""
    vn = 4 if dtype == torch.float32 else 8
    pieces = cols / vn + 2
    batches = math.ceil(pieces / (8 * (32 if pieces <= 522 else 128)))
    return U * (3 * D + 4 + 34 + 6 * batches + 6 * 11)


def matrix(rows, cols, ld, lead, dtype, dev, value):
    buf = torch.full((lead + rows * ld,), math.nan, dtype=dtype, device=dev)
    z = buf[lead:].view(rows, ld)[:, :cols]
    z.fill_(value)
    return z


# rows, cols, padding, lead: a warp a row, 128 threads, 256, and clusters of 2, 4 and 8 CTAs a row
PLACES = [(30, 2001, 0, 0), (31, 1003, 5, 3), (2432, 4001, 0, 1), (400, 8001, 3, 1), (1216, 20001, 0, 0),
          (153, 50257, 0, 0), (152, 50257, 0, 1), (76, 50257, 7, 0), (38, 50257, 0, 3), (38, 128256, 0, 0),
          (1, 16500, 0, 0), (3, 4100, 1, 2)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("place", PLACES, ids=lambda s: "x".join(map(str, s)))
def test_every_element_counts_once(G, dev, place, dt):
    """Lost, a dominant logit leaves the maximum at -8; taken twice, it makes log s log 2."""
    rows, cols, pad, lead = place
    t = TYPES[dt]
    vn = 4 if t == torch.float32 else 8
    at = torch.arange(0, cols, vn)
    at = torch.unique(torch.cat([(at + (at // vn) % vn).clamp(max=cols - 1), torch.arange(min(cols, 40)),
                                 torch.arange(max(0, cols - 40), cols)])).to(dev)
    at = torch.cat([at, at[:(-len(at)) % rows]]) if len(at) >= rows else at.repeat(-(-rows // len(at)))[:rows]
    z = matrix(rows, cols, cols + pad, lead, t, dev, -8.0)
    new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=dev)
    n, line = len(at), torch.arange(rows, device=dev)
    logp, ent, stats = new(n), new(n), new(n, 2)
    ids, top = new(n, 1, dt=torch.int64), new(n, 1)
    for i in range(0, n, rows):
        p, j = at[i:i + rows], slice(i, i + rows)
        z[line, p] = 8.0
        # with alternatives in every other call: they are another kernel
        more = dict(top_ids=ids[j], top_logp=top[j]) if i // rows % 2 == 0 or n == rows else {}
        G.amp_token_logprobs_forward(z, p, logp[j], ent[j], stats[j], **more)
        if not more:
            ids[j, 0], top[j, 0] = p, logp[j]
        z[line, p] = -8.0
    w = (cols - 1) * math.exp(-16.0)
    logs, D = math.log1p(w), 16.0 * w / (1 + w)
    one = sum_bound(cols, t, D) + 2 * U * logs
    assert (stats[:, 0] == 8.0).all() and torch.equal(ids[:, 0], at)
    for got in (stats[:, 1], -logp, -top[:, 0]):
        assert (got.double() - logs).abs().max() <= one
    # the entropy, log s + D: D's terms have the sum's error, their own |d| and two roundings more
    assert (ent.double() - (logs + D)).abs().max() <= one + (sum_bound(cols, t, 16.0) + 6 * U) * D + 2 * U * (logs + D)


FLAT = [(3, 33), (5, 2001), (2432, 4001), (400, 8001), (1216, 20001), (160, 50257), (40, 50257), (38, 70000),
        (1, 128256), (9, 128256), (200, 128256)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("size", FLAT, ids=lambda s: "x".join(map(str, s)))
def test_sums_of_flat_rows(G, dev, size, dt):
    """Rows without a peak: equal logits, N(0, 1/4), N(0, 4), and ones that rise all along.  Over 128256
    tokens the bound is 1.4e-5, two of the equal tokens."""
    rows, cols = size
    t = TYPES[dt]
    g = torch.Generator(device=dev).manual_seed(rows + cols)
    z = torch.randn(rows, cols, generator=g, device=dev)
    z[0::4] = 0.75
    z[1::4] *= 0.5
    z[2::4] *= 2.0
    z[3::4] = torch.linspace(-6, 6, cols, device=dev)
    z = z.to(t)
    logp, ent, stats = (torch.empty(rows, device=dev), torch.empty(rows, device=dev), torch.empty(rows, 2, device=dev))
    tok = torch.randint(0, cols, (rows,), generator=g, device=dev)
    G.amp_token_logprobs_forward(z, tok, logp, ent, stats)
    d = z.double() - z.double().amax(-1, keepdim=True)
    logs = torch.logsumexp(d, -1)
    p = (d - logs[:, None]).exp()
    D, D2 = (p * -d).sum(-1), (p * d * d).sum(-1)
    rel = sum_bound(cols, t, D)
    one = rel + 2 * U * logs.abs()
    assert torch.equal(stats[:, 0], z.float().amax(-1))
    assert ((stats[:, 1].double() - logs).abs() <= one).all()
    dt_ = d.gather(1, tok[:, None])[:, 0]
    assert ((logp.double() - (dt_ - logs)).abs() <= one + U * dt_.abs() + U * (dt_ - logs).abs()).all()
    # sum exp(d) d: a term has U (3 |d| + 5) e |d|, the sums' own roundings are those of s
    e = one + U * (3 * D2 + 5 * D) + (rel + 4 * U) * D + 2 * U * (logs + D)
    assert ((ent.double() - (logs + D)).abs() <= e).all()


def tied(cols, seed):
    """Rows with a few to all logits at or above the bound of the alternatives."""
    g = torch.Generator().manual_seed(seed)
    rows = [torch.full((cols,), 1.5), torch.arange(cols) % 3 * 1.0, torch.arange(cols) % 2 * -1.0,
            torch.linspace(9, -9, cols), torch.randint(0, 4, (cols,), generator=g).float()]
    half = torch.zeros(cols)
    half[::2] = -math.inf
    rows.append(half)
    lone = torch.full((cols,), -math.inf)
    lone[cols // 2] = 2.0
    rows.append(lone)
    for n in (7, 63, 64, 65, 66, 130):          # of equal largest ones, at random places; a warp's queue holds 64
        z = torch.randn(cols, generator=g).clamp(max=3.0)
        z[torch.randperm(cols, generator=g)[:n]] = 4.0
        rows.append(z)
    up = torch.full((cols,), -1.0)
    up[-70:], up[-1] = 2.0, 3.0                 # one above seventy equal ones
    rows.append(up)
    return torch.stack(rows)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("cols", [300, 1000, 1039, 2060])
@pytest.mark.parametrize("k", [1, 5, 8, 9, 32])
def test_ties_in_short_rows(G, dev, dt, cols, k):
    """Up to 8 alternatives a warp takes a row, beyond them 128 threads; the last CTA's rows are not
    four, an unused row lies between."""
    z = tied(cols, k).to(TYPES[dt])
    for rows in (len(z), len(z) - 1, len(z) - 3):
        x = z[:rows]
        t = torch.full((rows,), 3, dtype=torch.int64)
        t[4] = -1
        zd = x.to(dev)
        ids, top = torch.empty(rows, k, dtype=torch.int64, device=dev), torch.empty(rows, k, device=dev)
        logp, stats = torch.empty(rows, device=dev), torch.empty(rows, 2, device=dev)
        G.amp_token_logprobs_forward(zd, t.to(dev), logp, stats=stats, top_ids=ids, top_logp=top)
        want = M.top(x, k)
        want[4] = -1
        assert torch.equal(ids.cpu(), want)
        lp, _, _ = M.logprobs(x, t)
        w = torch.where(want < 0, torch.tensor(-math.inf, dtype=torch.float64), lp.gather(1, want.clamp_min(0)))
        d = (x.double() - x.double().amax(-1, keepdim=True)).clamp_min(-1e4)
        D = (lp.exp() * -d).sum(-1)
        one = torch.tensor([sum_bound(cols, x.dtype, v.item()) for v in D])[:, None]
        near = d.gather(1, want.clamp_min(0)).abs()
        close(top, w, (one + 2 * U * (lp.amax(-1, keepdim=True)).abs() + U * near + U * w.abs()).nan_to_num(0.0))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ties_in_many_rows_of_a_warp_each(G, dev, dt):
    """2437 rows of 510 pieces, which a warp takes where rows are that many."""
    cols = 510 * (4 if dt == "f32" else 8)
    z = tied(cols, 3).to(TYPES[dt])
    rows = 2437
    zd = z.to(dev).repeat(-(-rows // len(z)), 1)[:rows]
    ids, top = torch.empty(rows, 5, dtype=torch.int64, device=dev), torch.empty(rows, 5, device=dev)
    G.amp_token_logprobs_forward(zd, None, None, top_ids=ids, top_logp=top)
    assert torch.equal(ids.cpu(), M.top(z, 5).repeat(-(-rows // len(z)), 1)[:rows])
