"""amp_token_logprobs_forward and _backward against the 64-bit reference: every type, one logit a
row to a whole vocabulary, one row to many, rows that lie apart and start anywhere, masked tokens,
rows without a target or with nothing left, ties between alternatives, in place, in graphs."""
import math

import pytest
import torch

import more_ops_reference as M
import ops_reference as R
from test_gpu_bounds import Guarded, _INT
from test_gpu_ops import G, close, dev, same  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_INT.setdefault(torch.int64, (torch.int64, 0x7FA5A5A5A5A5A5A5))
U = R.U


def logits(rows, cols, dtype, seed, masked=0.0, peak=True):
    g = torch.Generator().manual_seed(seed)
    z = 2.0 * torch.randn(rows, cols, generator=g)
    if masked:
        z[torch.rand(rows, cols, generator=g) < masked] = -math.inf
    t = torch.randint(0, cols, (rows,), generator=g)
    if peak:
        z[torch.arange(rows), t] = 6.0 + 3.0 * torch.randn(rows, generator=g)
    return z.to(dtype), t


def lay_out(z, dev, ld, lead, fill=math.nan):
    """z on the device with rows ld apart, `lead` elements past a 16-byte boundary."""
    rows, cols = z.shape
    buf = torch.full((lead + rows * ld,), fill, dtype=z.dtype, device=dev)
    v = buf[lead:].view(rows, ld)[:, :cols]
    v.copy_(z)
    return v


def run(G, dev, z, t, ld, lead, k):
    rows, cols = z.shape
    zd, td = lay_out(z, dev, ld, lead), t.to(dev) if t is not None else None
    outs = {n: Guarded(rows * w, torch.float32, dev, shape=(rows, w) if w > 1 else (rows,))
            for n, w in (("logp", 1), ("entropy", 1), ("stats", 2))}
    args = {n: o.view for n, o in outs.items()}
    if td is None:
        args["logp"] = None
    if k:
        outs["ids"] = Guarded(rows * k, torch.int64, dev, shape=(rows, k))
        outs["top"] = Guarded(rows * k, torch.float32, dev, shape=(rows, k))
        args["top_ids"], args["top_logp"] = outs["ids"].view, outs["top"].view
    G.amp_token_logprobs_forward(zd, td, **args)
    assert all(o.intact() for o in outs.values())
    return zd, td, {n: o.view for n, o in outs.items()}


def held(want):
    """As fp32 holds it: a difference of two values near its largest is an infinity there."""
    return torch.where(want.abs() > 2.0 ** 128, want * math.inf, want)


def check(G, dev, z, t, ld, lead, k):
    rows, cols = z.shape
    zd, td, got = run(G, dev, z, t, ld, lead, k)
    lp, want, ent = M.logprobs(z, t)
    one, eb = M.logprobs_bounds(z)
    used = torch.ones(rows, dtype=torch.bool) if t is None else t >= 0
    top = z.double().amax(-1)
    if t is not None:
        # the difference from the maximum and the sum with log s round
        d = (z.double().gather(1, t.clamp(0, cols - 1)[:, None])[:, 0] - top).abs()
        close(got["logp"], held(want), torch.where(used, one + U * d + U * want.abs() + 2.0 ** -149, 0.0).nan_to_num(0.0))
    close(got["entropy"], ent, torch.where(used, eb, 0.0))
    close(got["stats"][:, 0], torch.where(used, top, 0.0), torch.zeros(rows))
    if k:
        ids = M.top(z, k)
        ids[~used] = -1
        assert torch.equal(got["ids"].cpu(), ids)
        w = torch.where(ids < 0, torch.tensor(-math.inf, dtype=torch.float64), lp.gather(1, ids.clamp_min(0)))
        d = torch.where(ids < 0, 0.0, top[:, None] - z.double().gather(1, ids.clamp_min(0)))
        close(got["top"], held(w), (one[:, None] + U * d + U * w.abs()).nan_to_num(0.0))
    _, _, again = run(G, dev, z, t, ld, lead, k)
    assert all(same(got[n], again[n]) for n in got if n != "logp" or t is not None)
    return zd, td, got


def check_grad(G, dev, z, t, zd, td, got, dld, lead, scale):
    rows, cols = z.shape
    g = torch.Generator().manual_seed(rows + cols)
    dl, de = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    lp, want, ent = M.logprobs(z, None)
    one, eb = M.logprobs_bounds(z)
    for use_l, use_e, s in ((True, True, scale), (True, False, None), (False, True, scale)):
        by = 1.0 if s is None else s
        w = M.logprobs_grad(z, t, dl if use_l else None, de if use_e else None, by)
        buf = Guarded(lead + rows * dld, z.dtype, dev)
        buf.view.fill_(5.0)
        out = buf.view[lead:].view(rows, dld)[:, :cols]
        G.amp_token_logprobs_backward(dl.to(dev) if use_l else None, zd, td, got["stats"], out,
                                      entropy=got["entropy"] if use_e else None,
                                      dentropy=de.to(dev) if use_e else None,
                                      scale=None if s is None else torch.tensor([s], device=dev))
        assert buf.intact()
        if dld > cols:
            assert (buf.view[lead:].view(rows, dld)[:, cols:] == 5.0).all() and (buf.view[:lead] == 5.0).all()
        # log p: off by `one`, its own two roundings and the statistics'; then p by as much
        # relatively and by its exponential (4 U and the argument's 3 U |log p|)
        l = lp.clamp_min(-1e4).abs()
        el = one[:, None] + 4 * U * (l + 20)
        p = lp.exp()
        ep = p * (el + 3 * U * l + 4 * U) + 2.0 ** -126
        a = (dl.double().abs() if use_l else torch.zeros(rows))[:, None]
        b = (de.double().abs() if use_e else torch.zeros(rows))[:, None]
        h = ent.abs()[:, None]
        e = by * (ep * (a + b * (l + h)) + b * p * (el + eb[:, None])
                  + 4 * U * (p * (a + b * (l + h)) + w.abs() / by) + 4 * U * a * (t.clamp(0)[:, None] ==
                                                                                 torch.arange(cols)))
        if t is not None:
            e[t < 0] = 0.0
        close(out, w, e + R.half_ulp(w.abs() + e, z.dtype))
        # in place
        mine = zd.clone() if zd.is_contiguous() else lay_out(z, dev, dld, lead)
        G.amp_token_logprobs_backward(dl.to(dev) if use_l else None, mine, td, got["stats"], mine,
                                      entropy=got["entropy"] if use_e else None,
                                      dentropy=de.to(dev) if use_e else None,
                                      scale=None if s is None else torch.tensor([s], device=dev))
        assert same(mine, out)


# rows, cols: one logit, less than a piece, whole pieces, odd; one row and few (cut over a
# cluster), many short rows, a vocabulary
SIZES = [(1, 1), (3, 2), (5, 7), (2, 8), (4, 33), (300, 65), (1, 4099), (7, 8192), (200, 1000), (1, 50257),
         (40, 50257), (100, 20001), (170, 9001), (330, 5000), (1300, 9001), (1, 128256), (9, 128256), (3000, 17)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_logprobs(G, dev, dt, size):
    r, c = size
    for i, (pad, lead, k) in enumerate(((0, 0, 0), (0, 0, 5), (3, 1, 32), (47, 3, 20), (8, 0, 1))):
        if r * c > 1 << 20 and i not in (0, 3):
            continue
        z, t = logits(r, c, TYPES[dt], 7 * r + c + i, masked=0.3 if i in (1, 3) else 0.0)
        t[torch.rand(r, generator=torch.Generator().manual_seed(i)) < 0.2] = -100
        zd, td, got = check(G, dev, z, t, c + pad, lead, k)
        check_grad(G, dev, z, t, zd, td, got, c + (5 if i % 2 else pad), (lead + i) % 4, 1024.0)


@pytest.mark.parametrize("dt", TYPES)
def test_no_targets(G, dev, dt):
    z, _ = logits(6, 3000, TYPES[dt], 1)
    zd, td, got = check(G, dev, z, None, 3000, 0, 4)
    de = torch.randn(6)
    out = torch.empty_like(zd)
    G.amp_token_logprobs_backward(None, zd, None, got["stats"], out, entropy=got["entropy"], dentropy=de.to(dev))
    w = M.logprobs_grad(z, None, None, de, 1.0)
    assert (out.double().cpu() - w).abs().max() < 0.01 * w.abs().max()
    G.amp_token_logprobs_backward(None, zd, None, got["stats"], out)
    assert not out.any()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("cols", [5, 300, 9000, 70000])
def test_hard_rows(G, dev, dt, cols):
    """A single token left, ties, constant rows, the type's largest and smallest values, a maximum
    that grows towards the end of the row."""
    t = TYPES[dt]
    big = torch.finfo(t).max
    z = torch.zeros(9, cols)
    z[0] = -math.inf
    z[0, cols // 2] = 3.0                                  # one token has all the probability
    z[1] = 1.5                                             # all equal
    z[2] = torch.linspace(-20, 20, cols)                   # rises
    z[3] = torch.linspace(20, -20, cols)                   # falls
    z[4], z[4, 1] = -big, big                              # as far apart as it gets
    z[5] = -big                                            # masked with the lowest value throughout
    z[6, :] = torch.arange(cols) % 3                       # ties
    z[7], z[7, -1] = -50.0, 4.0                            # log s = 0 but for nothing
    z[8, ::2] = -math.inf
    z = z.to(t)
    tg = torch.tensor([cols // 2, 0, cols - 1, 0, 1, cols - 1, 2, cols - 1, 1])
    for pad, lead in ((0, 0), (3, 1)):
        zd, td, got = check(G, dev, z, tg, cols + pad, lead, min(20, cols))
        check_grad(G, dev, z, tg, zd, td, got, cols + pad, lead, 2.0)
    assert got["logp"][0] == 0.0 and got["entropy"][0] == 0.0


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols", [(3, 40), (12, 5000), (2, 60000), (500, 700)])
def test_rows_without_an_answer(G, dev, dt, rows, cols):
    """Nothing but -inf, a NaN, +inf, a token outside the vocabulary: NaN in the row's own results;
    a row without a target is zero whatever its logits; the others are as alone."""
    t = TYPES[dt]
    z, tg = logits(rows, cols, t, 5)
    clean, ctg = z.clone(), tg.clone()
    for bad, ok_ids in ((-math.inf, False), (math.nan, True), (math.inf, True)):
        z, tg = clean.clone(), ctg.clone()
        if bad == -math.inf:
            z[1] = bad
        else:
            z[1, cols // 3] = bad
        _, _, base = run(G, dev, clean, ctg, cols, 0, 3)
        zd, td, got = run(G, dev, z, tg, cols, 0, 3)
        others = [r for r in range(rows) if r != 1]
        for n in got:
            assert same(got[n][others], base[n][others])
        assert got["logp"][1].isnan() and got["entropy"][1].isnan()
        assert ok_ids or (got["ids"][1] == -1).all()
        out = torch.empty_like(zd)
        dl = torch.ones(rows, device=dev)
        G.amp_token_logprobs_backward(dl, zd, td, got["stats"], out)
        assert out[1].isnan().all() and not out[others].isnan().any()
        tg[1] = -1                                         # not used: nothing of it shows
        zd, td, got = run(G, dev, z, tg, cols, 0, 3)
        assert got["logp"][1] == 0 and got["entropy"][1] == 0 and not got["stats"][1].any()
        assert (got["ids"][1] == -1).all() and (got["top"][1] == -math.inf).all()
        dl[1] = math.nan
        G.amp_token_logprobs_backward(dl, zd, td, got["stats"], out, entropy=got["entropy"], dentropy=dl)
        assert not out[1].any() and not out[others[2:] or others].isnan().any()
    tg = ctg.clone()
    tg[0], tg[rows - 1] = cols, 1 << 40                    # outside the vocabulary
    zd, td, got = run(G, dev, clean, tg, cols, 0, 3)
    out = torch.empty_like(zd)
    G.amp_token_logprobs_backward(torch.ones(rows, device=dev), zd, td, got["stats"], out)
    bad = torch.zeros(rows, dtype=torch.bool)
    bad[0] = bad[rows - 1] = True
    assert torch.equal(got["logp"].isnan().cpu(), bad) and torch.equal(out.isnan().any(1).cpu(), bad)
    assert out[0].isnan().all()


def test_overflow_of_the_scaled_gradient_is_seen(G, dev):
    """A loss scale too large for fp16 gives infinities, which the gradient check reports."""
    z, t = logits(4, 100, torch.float16, 3)
    zd, td, got = run(G, dev, z, t, 100, 0, 0)
    out = torch.empty_like(zd)
    G.amp_token_logprobs_backward(torch.full((4,), -1.0, device=dev), zd, td, got["stats"], out,
                                  scale=torch.tensor([2.0 ** 30], device=dev))
    assert out.isinf().any() and not out.isnan().any()


def test_gradient_against_differences(G, dev):
    """The gradient that the call gives against differences of what the forward call gives."""
    z, t = logits(3, 11, torch.float32, 9)
    zd, td, got = run(G, dev, z, t, 11, 0, 0)
    dl, de = torch.tensor([1.0, -2.0, 0.5], device=dev), torch.tensor([0.3, 1.0, -1.0], device=dev)
    out = torch.empty_like(zd)
    G.amp_token_logprobs_backward(dl, zd, td, got["stats"], out, entropy=got["entropy"], dentropy=de)
    h = 2.0 ** -6

    def f(x):
        _, _, o = run(G, dev, x, t, 11, 0, 0)
        return ((o["logp"] * dl).double() + (o["entropy"] * de).double()).cpu()
    for c in range(11):
        up, dn = z.clone(), z.clone()
        up[:, c] += h
        dn[:, c] -= h
        # h^2 / 6 of a third derivative below 60 (2 |dl| + |de| (2 + 6 log 11)); roundings of 1e-6 over h
        assert ((f(up) - f(dn)) / (2 * h) - out[:, c].double().cpu()).abs().max() < 60 * h * h / 6 + 1e-6 / h * 8


def test_offsets_past_32_bits(G, dev):
    """Logits of more than 2^31 elements: the last rows."""
    r, c = 17000, 128256
    z = torch.zeros(r, c, dtype=torch.bfloat16, device=dev)
    z[-2:].normal_()
    t = torch.full((r,), -1, dtype=torch.int64, device=dev)
    t[-2:] = torch.tensor([7, c - 1], device=dev)
    t[0] = 3
    logp, ent, stats = torch.empty(r, device=dev), torch.empty(r, device=dev), torch.empty(r, 2, device=dev)
    ids, top = torch.empty(r, 4, dtype=torch.int64, device=dev), torch.empty(r, 4, device=dev)
    G.amp_token_logprobs_forward(z, t, logp, ent, stats, ids, top)
    zc, tc = z[-2:].cpu(), t[-2:].cpu()
    lp, want, e = M.logprobs(zc, tc)
    assert (logp[-2:].cpu().double() - want).abs().max() < 1e-5 and torch.equal(ids[-2:].cpu(), M.top(zc, 4))
    assert abs(logp[0].item() + math.log(c)) < 1e-5 and ids[0].tolist() == [0, 1, 2, 3] and not logp[1:-2].any()
    G.amp_token_logprobs_backward(torch.ones(r, device=dev), z, t, stats, z)
    w = M.logprobs_grad(zc, tc, torch.ones(2), None, 1.0)
    assert (z[-2:].cpu().double() - w).abs().max() < 0.01 and not z[1:1000].any()


def test_strides(G, dev):
    """Leading dimensions of one stride are rows; others are refused."""
    buf = torch.randn(3, 4, 70, device=dev)
    z = buf[:, :, :50]
    t = torch.randint(0, 50, (3, 4), device=dev)
    logp, stats = torch.empty(3, 4, device=dev), torch.empty(3, 4, 2, device=dev)
    G.amp_token_logprobs_forward(z, t, logp, stats=stats)
    flat = torch.empty(12, device=dev)
    G.amp_token_logprobs_forward(z.reshape(12, 50).contiguous(), t.view(-1), flat)
    assert torch.equal(flat, logp.view(-1))
    one = torch.empty(1, device=dev)
    G.amp_token_logprobs_forward(z[1, 2], t[1, 2].view(1), one)
    assert one == logp[1, 2]
    wide = buf.transpose(0, 1)[:, :, :50]                   # rows of two strides
    odd = torch.empty(12, 50, device=dev)
    for match, call in (
            ("logits: needs", lambda: G.amp_token_logprobs_forward(wide, t, logp)),
            ("logits: needs", lambda: G.amp_token_logprobs_forward(buf.transpose(1, 2), t, logp)),
            ("logits: needs", lambda: G.amp_token_logprobs_forward(buf[0, :1].expand(4, 70), t[0], logp[0])),
            ("targets: dtype Int", lambda: G.amp_token_logprobs_forward(z, t.int(), logp)),
            ("targets: 4 elements", lambda: G.amp_token_logprobs_forward(z, t[0], logp)),
            ("logp: needs a contiguous", lambda: G.amp_token_logprobs_forward(z, t, logp.t())),
            ("stats: 12 elements, at least 24", lambda: G.amp_token_logprobs_forward(z, t, logp, stats=logp)),
            ("top_ids: 1 to 32", lambda: G.amp_token_logprobs_forward(z, t, logp, top_ids=torch.empty(
                12, 33, dtype=torch.int64, device=dev))),
            ("dlogits: needs the shape", lambda: G.amp_token_logprobs_backward(flat, z, t, stats, odd.bfloat16())),
            ("dlogits: needs the shape", lambda: G.amp_token_logprobs_backward(flat, z, t, stats, odd[:11])),
            ("scale: dtype Double", lambda: G.amp_token_logprobs_backward(flat, z, t, stats, odd, scale=one.double()))):
        with pytest.raises(ValueError, match=match):
            call()
    for match, call in (
            ("logp needs targets", lambda: G.amp_token_logprobs_forward(z, None, logp)),
            ("go together", lambda: G.amp_token_logprobs_forward(z, t, logp, top_ids=t.view(12, 1))),
            ("needs the entropy", lambda: G.amp_token_logprobs_backward(flat, z, t, stats, odd, dentropy=flat)),
            ("needs targets", lambda: G.amp_token_logprobs_backward(flat, z, None, stats, odd)),
            ("needs a logit", lambda: G.amp_token_logprobs_forward(z[:, :, :0], t, logp))):
        with pytest.raises(G.AmpError, match=match):
            call()
    G.amp_token_logprobs_forward(z[:0], t[:0], logp[:0])
    # rows of another stride in the gradient
    G.amp_token_logprobs_backward(flat, z, t, stats, odd)
    into = torch.zeros(3, 4, 70, device=dev)
    G.amp_token_logprobs_backward(flat, z, t, stats, into[:, :, :50])
    assert torch.equal(into[:, :, :50].reshape(12, 50), odd) and not into[:, :, 50:].any()


def test_side_stream_and_graph(G, dev):
    z, t = logits(20, 40000, torch.bfloat16, 2)
    zd, td, got = run(G, dev, z, t, 40000, 0, 6)
    dl, scale = torch.randn(20, device=dev), torch.ones(1, device=dev)
    logp, ent, stats = torch.empty(20, device=dev), torch.empty(20, device=dev), torch.empty(20, 2, device=dev)
    ids, top, out = torch.empty_like(got["ids"]), torch.empty_like(got["top"]), torch.empty_like(zd)

    def calls(s=None):
        G.amp_token_logprobs_forward(zd, td, logp, ent, stats, ids, top, stream=s)
        G.amp_token_logprobs_backward(dl, zd, td, stats, out, entropy=ent, dentropy=dl, scale=scale, stream=s)
    calls()
    torch.cuda.synchronize()
    want = [x.clone() for x in (logp, ent, stats, ids, top, out)]
    assert torch.equal(logp, got["logp"]) and torch.equal(ids, got["ids"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        calls(s)
    for x in (logp, ent, stats, ids, top, out):
        x.zero_()
    scale.fill_(2.0)                                        # read at each replay
    g.replay()
    torch.cuda.synchronize()
    got = (logp, ent, stats, ids, top, out)
    assert all(torch.equal(a, b) for a, b in zip(want[:5], got[:5])) and same(out, want[5].double() * 2)
