"""Cases of the operators that a training or sampling step needs around its 4-bit products: the
product with bias, activation and residual in its epilogue, dropout from a counter-based generator,
and the log probabilities of given tokens.

Three operators, named by a case's "op":

linear    fp4_linear_mx: residual + f(A B^T + bias) of two packed 4-bit matrices.  "train" keeps
          A B^T + bias in 8 bits and adds the backward pass from there, amp_bias_act_backward_mx8:
          the gradient at the product's output and the bias's
dropout   amp_dropout_forward (added to a residual) and amp_dropout_backward, with the gradient of
          the bias that was added before it ("bias")
logprobs  amp_token_logprobs_forward: the log probability of a token a row, the row's entropy, the
          most probable tokens.  "train" adds amp_token_logprobs_backward, with the loss scale

Packed 4-bit matrices: blocks of 32 consecutive elements of a row, e2m1 codes two a byte (the even
one in the low bits), one power-of-two scale a block (a byte e for 2^(e - 127)), scales in tiles of
128 rows x 4 blocks, 512 bytes each, byte (r % 32) * 16 + (r / 32) * 4 + b of a tile for its row r
and block b.  8 bits: e4m3 with the same scales.

Dropout: element k (row-major) takes 16 bits of Philox4x32-10 under the key `seed`, half (k % 8) % 2
(low first) of word (k % 8) / 2 for the counter {k / 8 low, k / 8 high, step, 2^30 + site}.  With T
the nearest whole number to 65536 p it is dropped where the bits are below T, and multiplied by
65536 / (65536 - T) otherwise.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_SITE = 3
_IGNORED = -100


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token through the 8B set's down projection, onto the residual stream
        {"name": "linear_one_token", "op": "linear", "tokens": 1, "n": 4096, "k": 14336, "dtype": "bf16",
         "bias": "", "kind": "", "residual": True, "train": False},
        # a decoding batch through a projection with a bias and SiLU
        {"name": "linear_decode_batch", "op": "linear", "tokens": 48, "n": 4096, "k": 4096, "dtype": "bf16",
         "bias": "bf16", "kind": "silu", "residual": False, "train": False},
        # a prompt of 8192 tokens through the 8B set's down projection, onto the residual stream
        {"name": "linear_prompt", "op": "linear", "tokens": 8192, "n": 4096, "k": 14336, "dtype": "bf16",
         "bias": "", "kind": "", "residual": True, "train": False},
        # a ragged fp16 batch through a layer of GPT-2's width, trained with its bias
        {"name": "linear_train_ragged", "op": "linear", "tokens": 1000, "n": 2304, "k": 768, "dtype": "f16",
         "bias": "f16", "kind": "gelu_tanh", "residual": False, "train": True},
        # the 1B set's up projection with a bias and GELU, trained
        {"name": "linear_train_1b", "op": "linear", "tokens": 4096, "n": 8192, "k": 2048, "dtype": "bf16",
         "bias": "bf16", "kind": "gelu", "residual": False, "train": True},
        # GPT-2's dropout over a micro-batch, onto the residual stream
        {"name": "dropout_gpt2", "op": "dropout", "rows": 1024, "cols": 768, "dtype": "f16", "p": 0.1,
         "residual": True, "bias": "f32"},
        # an fp32 batch whose sides divide nothing, no residual
        {"name": "dropout_odd_f32", "op": "dropout", "rows": 2047, "cols": 1111, "dtype": "f32", "p": 0.25,
         "residual": False, "bias": "f32"},
        # a wide training batch
        {"name": "dropout_wide", "op": "dropout", "rows": 16384, "cols": 5120, "dtype": "bf16", "p": 0.1,
         "residual": True, "bias": "bf16"},
        # the logits of one sampled token over Llama 3's vocabulary, with alternatives
        {"name": "logprobs_one_token", "op": "logprobs", "rows": 1, "cols": 128256, "pad": 0,
         "dtype": "bf16", "top": 20, "masked": 0.0, "train": False},
        # a batch of sampled tokens over GPT-2's vocabulary, a part of it masked by a grammar
        {"name": "logprobs_batch", "op": "logprobs", "rows": 64, "cols": 50257, "pad": 0, "dtype": "f32",
         "top": 5, "masked": 0.3, "train": False},
        # the loss of GPT-2's micro-batch in fp16, logits padded to whole tiles, gradient scaled
        {"name": "logprobs_train_gpt2", "op": "logprobs", "rows": 1023, "cols": 50257, "pad": 47,
         "dtype": "f16", "top": 0, "masked": 0.0, "train": True},
        # the loss of a training batch over Llama 3's vocabulary
        {"name": "logprobs_train_8b", "op": "logprobs", "rows": 4096, "cols": 128256, "pad": 0,
         "dtype": "bf16", "top": 0, "masked": 0.0, "train": True},
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def _side(rng, lo, hi):
    """A size over the logarithm of the range: a multiple of 128, of 8, or anything."""
    v = _log(rng, lo, hi)
    step = rng.choice((128, 8, 1, 1))
    return min(hi, max(lo, (v + step - 1) // step * step))


def draw(rng):
    op = rng.choice(("linear", "dropout", "logprobs"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "linear":
        train = rng.random() < 0.5
        while True:
            t, n, k = _side(rng, 1, 8192), _side(rng, 64, 14336), _side(rng, 64, 14336)
            if t * n * k <= 8192 * 4096 * 14336 // 2:
                break
        if train and dtype == "f32":  # 32 bits of an 8-bit checkpoint's gradient would hang on its borders
            dtype = "f16"
        kind = rng.choice(("gelu", "gelu_tanh", "silu")) if train else rng.choice(("", "gelu", "gelu_tanh", "silu"))
        return {"op": op, "tokens": t, "n": n, "k": k, "dtype": dtype,
                "bias": dtype if train else rng.choice(("", "f32", dtype)), "kind": kind, "residual": rng.random() < 0.5, "train": train}
    if op == "dropout":
        while True:
            r, c = _side(rng, 1, 16384), _side(rng, 33, 16384)
            if r * c * _SIZE[dtype] <= 16384 * 5120 * 2:
                break
        return {"op": op, "rows": r, "cols": c, "dtype": dtype, "p": rng.choice((0.05, 0.1, 0.25, 0.5)),
                "residual": rng.random() < 0.6, "bias": rng.choice(("", "f32", dtype))}
    train = rng.random() < 0.5
    while True:
        r, c = _log(rng, 1, 8192), _side(rng, 1000, 131072)
        if r * c * _SIZE[dtype] <= 4096 * 128256:
            break
    return {"op": op, "rows": r, "cols": c, "pad": rng.choice((0, 0, 47, 64)), "dtype": dtype,
            "top": 0 if train else rng.choice((0, 1, 5, 20)), "masked": rng.choice((0.0, 0.0, 0.3)), "train": train}


# ------------------------------------------------------------------ the formats
def _up(v, step):
    return -(-v // step) * step


def _blocks(x):
    """[rows, blocks, 32], the rows padded with zeros."""
    r, c = x.shape
    p = _up(c, 32)
    if p != c:
        x = torch.nn.functional.pad(x, (0, p - c))
    return x.reshape(r, p // 32, 32)


def _scale_code(b, over, low):
    """The scale byte of each block of b (fp32): the bits of the largest magnitude, rounded up to
    a power of two over the format's largest value (its mantissa gives `over`, its exponent `low`)."""
    bits = b.abs().amax(-1).view(torch.int32)
    return (((bits + over) >> 23) - low).clamp_min(0)


def _scale(e):
    """2^(e - 127) in 32 bits (2^-127 is subnormal)."""
    return torch.where(e == 0, torch.full_like(e, 0x400000), e << 23).view(torch.float32)


def _unscale(e):
    """2^(127 - e) for e of at most 253."""
    return ((254 - e).clamp_min(1) << 23).view(torch.float32)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _pack(x):
    """Packed rows and tiled scales of x (fp32), nearest codes, ties to the even one."""
    b = _blocks(x)
    e = _scale_code(b, 0x3FFFFF, 2)
    y = b * _unscale(e)[..., None]
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int()) + 8 * torch.signbit(y).int()
    r, kb, _ = code.shape
    c = code.reshape(r, kb * 16, 2).to(torch.uint8)
    s = torch.nn.functional.pad(e.to(torch.uint8), (0, _up(kb, 4) - kb, 0, _up(r, 128) - r))
    s = s.reshape(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return (c[..., 0] | (c[..., 1] << 4)).contiguous(), s.reshape(-1).contiguous()


def _unpack(q, s, rows, cols, table):
    """The values of a packed matrix, in 32 bits."""
    kb = q.shape[1] // 16
    code = torch.stack((q & 15, q >> 4), -1).reshape(rows, kb, 32)
    t = s.reshape(-1, _up(kb, 4) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    e = t.reshape(_up(rows, 128), _up(kb, 4))[:rows, :kb].int()
    return (table[code.long()] * _scale(e)[..., None]).reshape(rows, kb * 32)[:, :cols]


def _mx8_round(x):
    """What the 8-bit form (e4m3) of x (fp32) stands for."""
    b = _blocks(x)
    e = _scale_code(b, 0x1FFFFF, 8)
    y = b * _unscale(e)[..., None]
    q = y.to(torch.float8_e4m3fn).float() * _scale(e)[..., None]
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 29)
    dt = _DT[case["dtype"]]

    def n(*shape):
        return torch.randn(shape, generator=g, device=dev)

    st = {"case": dict(case)}
    if case["op"] == "linear":
        t, m, k = case["tokens"], case["n"], case["k"]
        # activations with a scale of each row's own, and a weight
        st["x"] = _pack(n(t, k) * torch.exp(0.3 * n(t, 1)))
        st["w"] = _pack((n(m, k) * 0.02).to(torch.bfloat16).float())
        st["table"] = torch.tensor(_E2M1, dtype=torch.float32, device=dev)
        st["bias"] = (0.1 * n(m)).to(_DT[case["bias"]]) if case["bias"] else None
        st["res"] = n(t, m).to(dt) if case["residual"] else None
        st["y"] = torch.empty((t, m), dtype=dt, device=dev)
        if case["train"]:
            st["dy"] = (0.1 * n(t, m)).to(dt)
            st["saved"] = (torch.empty((t, m), dtype=torch.float8_e4m3fn, device=dev),
                           torch.empty((t, _up(m, 32) // 32), dtype=torch.uint8, device=dev))
            st["dz"], st["db"] = torch.empty_like(st["dy"]), torch.empty_like(st["bias"])
    elif case["op"] == "dropout":
        r, c = case["rows"], case["cols"]
        st["x"], st["dy"] = n(r, c).to(dt), (0.1 * n(r, c)).to(dt)
        st["res"] = n(r, c).to(dt) if case["residual"] else None
        st["seed"] = (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 63)
        st["step"] = torch.tensor([1000 + seed % 1000], dtype=torch.int32, device=dev)
        st["y"], st["dx"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        st["db"] = torch.empty(c, dtype=_DT[case["bias"]], device=dev) if case["bias"] else None
    else:
        r, c = case["rows"], case["cols"]
        t = torch.randint(0, c, (r,), generator=g, device=dev)
        # a trained model's logits: a spread, a few likely tokens, and mostly the right one among them
        z = torch.empty((r, c + case["pad"]), dtype=dt, device=dev)
        for i in range(0, r, 512):  # in parts, so that the 32-bit numbers stay small beside the logits
            part = 2.0 * n(min(512, r - i), c + case["pad"])
            if case["masked"]:
                hide = torch.rand(part.shape, generator=g, device=dev) < case["masked"]
                part = torch.where(hide, torch.full_like(part, -math.inf), part)
            rows = torch.arange(part.shape[0], device=dev)
            for _ in range(4):
                part[rows, torch.randint(0, c, rows.shape, generator=g, device=dev)] = 8.0 + 2.0 * n(rows.shape[0])
            part[rows, t[i:i + 512]] = 9.0 + 3.0 * n(rows.shape[0])
            z[i:i + 512] = part.to(dt)
        st["z"] = z[:, :c]
        if case["train"]:  # a tenth of the positions is padding
            t = torch.where(torch.rand(r, generator=g, device=dev) < 0.1, torch.full_like(t, _IGNORED), t)
            st["dlogp"] = -(0.5 + torch.rand(r, generator=g, device=dev)) / r
            st["dent"] = 0.01 * n(r) / r
            st["scale"] = torch.tensor([4096.0], device=dev)
            st["dz"] = torch.empty_like(z)[:, :c]
        st["t"] = t
        st["logp"], st["ent"] = torch.empty(r, device=dev), torch.empty(r, device=dev)
        st["stats"] = torch.empty((r, 2), device=dev)
        if case["top"]:
            st["ids"] = torch.empty((r, case["top"]), dtype=torch.int64, device=dev)
            st["top"] = torch.empty((r, case["top"]), device=dev)
    return st


# ------------------------------------------------------------------ one pass, in plain form
def _act(x, kind):
    """f(x) and f'(x)."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return x * s, s * (1.0 + x * (1.0 - s))
    if kind == "gelu":
        p = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * p, p + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    a, b = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(a * (x + b * x * x * x))
    return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * a * (1.0 + 3.0 * b * x * x)


_LOW = 0xFFFFFFFF


def _philox(c0, c1, c2, c3, seed):
    """The four words of Philox4x32-10 (int64 tensors of 32-bit values)."""
    k0, k1 = seed & _LOW, seed >> 32
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # modulo 2^64
        c0, c1, c2, c3 = (((q >> 32) & _LOW) ^ c1 ^ k0, q & _LOW, ((p >> 32) & _LOW) ^ c3 ^ k1, p & _LOW)
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return c0, c1, c2, c3


def _keep(shape, p, seed, step):
    """Where an element stays, and what it is multiplied by."""
    n = shape[0] * shape[1]
    group = torch.arange(_up(n, 8) // 8, device=step.device)
    w = torch.stack(_philox(group & _LOW, group >> 32, (step.long() & _LOW).expand_as(group),
                            torch.full_like(group, (1 << 30) + _SITE), seed), -1)
    bits = torch.stack((w & 0xFFFF, w >> 16), -1).reshape(-1)[:n].reshape(shape)
    drop = round(p * 65536)
    return bits >= drop, 65536.0 / (65536 - drop)


def _plain(st):
    case = st["case"]
    dt = _DT[case["dtype"]]
    if case["op"] == "linear":
        t, m, k = case["tokens"], case["n"], case["k"]
        z = _unpack(*st["x"], t, k, st["table"]) @ _unpack(*st["w"], m, k, st["table"]).t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        y = _act(z, case["kind"])[0] if case["kind"] else z
        if st["res"] is not None:
            y = y + st["res"].float()
        got = {"y": y.to(dt)}
        if case["train"]:
            dz = st["dy"].float() * _act(_mx8_round(z), case["kind"])[1]
            got["dz"], got["db"] = dz.to(dt), dz.sum(0).to(st["bias"].dtype)
        return got
    if case["op"] == "dropout":
        keep, by = _keep(st["x"].shape, case["p"], st["seed"], st["step"])
        y = torch.where(keep, st["x"].float() * by, 0.0)
        if st["res"] is not None:
            y = st["res"].float() + y
        dx = torch.where(keep, st["dy"].float() * by, 0.0)
        got = {"y": y.to(dt), "dx": dx.to(dt)}
        if case["bias"]:
            got["db"] = dx.sum(0).to(_DT[case["bias"]])
        return got
    z, t = st["z"].float(), st["t"]
    top = z.amax(-1, keepdim=True)
    d = z - top
    e = torch.exp(d)
    s = e.sum(-1, keepdim=True)
    logs = torch.log(s)
    used = t >= 0
    at = t.clamp_min(0)[:, None]
    logp = torch.where(used, (d.gather(1, at) - logs)[:, 0], 0.0)
    pd = torch.where(e == 0, 0.0, e * d).sum(-1, keepdim=True) / s
    ent = (logs - pd)[:, 0]
    got = {"logp": logp, "ent": torch.where(used, ent, 0.0)}
    if case["top"]:
        col, left, ids, lp = torch.arange(z.shape[1], device=z.device), d.clone(), [], []
        for _ in range(case["top"]):  # the lowest index among the largest
            best = left.amax(-1, keepdim=True)
            i = torch.where(left == best, col, z.shape[1]).amin(-1, keepdim=True)
            ids.append(i)
            lp.append(best - logs)
            left.scatter_(1, i, -math.inf)
        got["ids"], got["top"] = torch.cat(ids, 1), torch.cat(lp, 1)
    if case["train"]:
        p = e / s
        g = -st["dlogp"][:, None] * p
        g.scatter_add_(1, at, st["dlogp"][:, None])
        g -= st["dent"][:, None] * torch.where(p == 0, 0.0, p * (d - logs + ent[:, None]))
        got["dz"] = torch.where(used[:, None], g * st["scale"], 0.0).to(dt)
    return got


# ------------------------------------------------------------------ one pass, by the framework
def _kernels(st):
    import loss_scaling_master_gb300 as G
    case = st["case"]
    if case["op"] == "linear":
        kind = case["kind"] or None
        saved = st.get("saved")
        G.fp4_linear_mx(*st["x"], *st["w"], case["k"], st["y"], bias=st["bias"], kind=kind, residual=st["res"],
                        saved=saved)
        if not case["train"]:
            return {"y": st["y"]}
        G.amp_bias_act_backward_mx8(st["dy"], st["db"], kind=kind, saved=saved, dx=st["dz"])
        return {"y": st["y"], "dz": st["dz"], "db": st["db"]}
    if case["op"] == "dropout":
        G.amp_dropout_forward(st["x"], case["p"], st["seed"], _SITE, st["y"], residual=st["res"], step=st["step"])
        G.amp_dropout_backward(st["dy"], case["p"], st["seed"], _SITE, st["dx"], step=st["step"], dbias=st["db"])
        got = {"y": st["y"], "dx": st["dx"]}
        if case["bias"]:
            got["db"] = st["db"]
        return got
    G.amp_token_logprobs_forward(st["z"], st["t"], st["logp"], entropy=st["ent"], stats=st["stats"],
                                 top_ids=st.get("ids"), top_logp=st.get("top"))
    got = {"logp": st["logp"], "ent": st["ent"]}
    if case["top"]:
        got["ids"], got["top"] = st["ids"], st["top"]
    if case["train"]:
        G.amp_token_logprobs_backward(st["dlogp"], st["z"], st["t"], st["stats"], st["dz"], entropy=st["ent"],
                                      dentropy=st["dent"], scale=st["scale"])
        got["dz"] = st["dz"]
    return got


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    b = _SIZE[case["dtype"]]
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        moved = (t + n) * k * (0.5 + 1 / 32) + t * n * b * (2 if case["residual"] else 1)
        moved += n * _SIZE[case["bias"]] if case["bias"] else 0
        if not case["train"]:
            return {"bytes": moved, "flops": 2 * t * n * k + 20 * t * n}
        # the 8-bit copy is written and read, the gradient read and written
        return {"bytes": moved + t * n * (2 * (1 + 1 / 32) + 2 * b) + n * _SIZE[case["bias"]],
                "flops": 2 * t * n * k + 60 * t * n}
    n = case["rows"] * case["cols"]
    if case["op"] == "dropout":
        return {"bytes": n * b * (5 if case["residual"] else 4)
                + (case["cols"] * _SIZE[case["bias"]] if case["bias"] else 0), "flops": 30 * n}
    rows = case["rows"] * 16 + case["rows"] * case["top"] * 12
    return {"bytes": n * b * (3 if case["train"] else 1) + rows, "flops": n * (16 if case["train"] else 6)}


# ------------------------------------------------------------------ in 64 bits
def _two(p):
    """2^p in 64 bits, from its exponent field."""
    return ((p.long() + 1023) << 52).view(torch.float64)


def _dense(packed, rows, cols):
    """The values of a packed matrix in 64 bits, a byte's halves and a scale's place at a time."""
    q, s = packed
    kb = q.shape[1] // 16
    v = torch.empty((rows, kb * 32), dtype=torch.float64, device=q.device)
    for half in (0, 1):
        c = ((q >> (4 * half)) & 15).long()
        m, ex = c & 1, (c >> 1) & 3
        a = torch.where(ex == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * _two(ex - 1))
        v[:, half::2] = torch.where(c >= 8, -a, a)
    row = torch.arange(rows, device=q.device)[:, None]
    blk = torch.arange(kb, device=q.device)[None, :]
    tile = (row // 128) * (_up(kb, 4) // 4) + blk // 4
    e = s[tile * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + blk % 4].int()
    return (v.view(rows, kb, 32) * _two(e - 127)[..., None]).view(rows, -1)[:, :cols]


def _mx8_exact(x):
    """The 8-bit block form: magnitudes at most 448, quanta 2^(exponent - 3) down to the exponent
    -6, a block's scale the smallest power of two that fits."""
    r, c = x.shape
    b = torch.zeros((r, _up(c, 32)), dtype=torch.float64, device=x.device)
    b[:, :c] = x
    b = b.unflatten(1, (-1, 32))
    a = b.abs().max(-1, keepdim=True).values
    m, p = torch.frexp(a)                       # a = m 2^p, 0.5 <= m < 1
    s = torch.where(a == 0, torch.full_like(p, -127), (p - 9 + (m > 0.875).int()).clamp_min(-127))
    y = b * _two(-s)
    _, q = torch.frexp(y)
    step = _two((q - 1).clamp_min(-6) - 3)
    y = torch.where(y == 0, y, torch.round(y / step) * step)
    return (y * _two(s)).flatten(1)[:, :c]


def _act_exact(x, kind):
    if kind == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * (1 - s)
    if kind == "gelu":
        p = torch.special.ndtr(x)
        return x * p, p + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(8 / math.pi)                  # 0.5 (1 + tanh(z / 2)) = sigmoid(z)
    s = torch.sigmoid(c * (x + 0.044715 * x ** 3))
    return x * s, s + x * s * (1 - s) * c * (1 + 3 * 0.044715 * x ** 2)


def _bits_exact(n, seed, step, dev):
    """16 bits an element, the generator's products formed from 16-bit halves."""
    def product(a, m):
        lo, hi = (a & 0xFFFF) * m, (a >> 16) * m   # each below 2^48
        low = lo + ((hi & 0xFFFF) << 16)           # below 2^49
        return (hi >> 16) + (low >> 32), low & _LOW

    g = torch.arange(-(-n // 8), device=dev)
    x = [g % (1 << 32), g // (1 << 32), torch.full_like(g, step % (1 << 32)), torch.full_like(g, (1 << 30) + _SITE)]
    for i in range(10):
        key = ((seed % (1 << 32) + i * 0x9E3779B9) % (1 << 32), (seed // (1 << 32) + i * 0xBB67AE85) % (1 << 32))
        (h0, l0), (h1, l1) = product(x[0], 0xD2511F53), product(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
    out = torch.empty((g.numel(), 8), dtype=torch.int64, device=dev)
    for j in range(8):
        out[:, j] = x[j // 2] // (1 << 16) if j % 2 else x[j // 2] % (1 << 16)
    return out.flatten()[:n]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        z = _dense(st["x"], t, k) @ _dense(st["w"], n, k).t()
        if st["bias"] is not None:
            z += st["bias"].double()
        y = _act_exact(z, case["kind"])[0] if case["kind"] else z
        got = {"y": y + st["res"].double() if st["res"] is not None else y}
        if case["train"]:
            got["dz"] = _act_exact(_mx8_exact(z), case["kind"])[1].mul_(st["dy"].double())
            got["db"] = got["dz"].sum(0)
        return got
    if case["op"] == "dropout":
        r, c = case["rows"], case["cols"]
        drop = round(case["p"] * 65536)
        by = (_bits_exact(r * c, st["seed"], int(st["step"]), st["x"].device) >= drop).view(r, c).double()
        by *= 65536 / (65536 - drop)
        y, dx = st["x"].double() * by, st["dy"].double() * by
        if st["res"] is not None:
            y += st["res"].double()
        got = {"y": y, "dx": dx}
        if case["bias"]:
            got["db"] = dx.sum(0)
        return got
    z, t = st["z"].double(), st["t"]
    lse = torch.logsumexp(z, -1, keepdim=True)
    lp = z - lse
    pl = torch.special.entr(lp.exp())           # -p log p, 0 for p = 0
    ent = pl.sum(-1)
    used = t >= 0
    rows = torch.arange(t.numel(), device=t.device)
    got = {"logp": torch.where(used, lp[rows, t.clamp_min(0)], 0.0), "ent": torch.where(used, ent, 0.0)}
    if case["top"]:
        v, i = torch.sort(z, dim=-1, descending=True, stable=True)
        got["ids"], got["top"] = i[:, :case["top"]].contiguous(), v[:, :case["top"]] - lse
    if case["train"]:
        p = lp.exp_()
        g = pl.addcmul_(p, ent[:, None], value=-1.0).mul_(st["dent"].double()[:, None])
        g.addcmul_(p, st["dlogp"].double()[:, None], value=-1.0)
        g[rows[used], t[used]] += st["dlogp"].double()[used]
        got["dz"] = g.mul_(float(st["scale"]) * used[:, None].double())
    return got
