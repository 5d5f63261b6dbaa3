"""Cases of the forward/backward operators around the optimizer step: microscaled 4-bit
quantisation and products, layer norm, and activations whose inputs are kept in 8 bits.

Four operators, named by a case's "op":

quant   fp4_quant_mx of a matrix (rows, and with "both" the transposed copy too), returned as the
        values the 4-bit codes stand for (fp4_dequant_mx)
linear  a linear layer on 4-bit operands: the activations are quantised in the call, the weight is
        held packed.  "train" adds the input's and the weight's gradient (three products)
norm    layer norm, forward and backward; with "ckpt" the backward reads the input from the 8-bit
        checkpoint that the forward made
act     GELU / SiLU, plain or gated, forward and backward from 8-bit checkpoints of its inputs

Blocks are 32 consecutive elements of a row with one power-of-two scale (a byte e for 2^(e - 127)):
the smallest that brings the block's largest magnitude to at most 6 (e2m1) or 448 (e4m3); a block
that holds a NaN or an infinity gets e = 255 and decodes to NaN.  Packed 4-bit rows hold two
elements a byte, the even one in the low bits, padded with zeros to whole blocks; their scales lie
in tiles of 128 rows x 4 blocks, 512 bytes each, byte (r % 32) * 16 + (r / 32) * 4 + b of a tile
for its row r and block b.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decoding batch's activations before a product: latency
        {"name": "quant_batch_of_tokens", "op": "quant", "rows": 32, "cols": 4096, "dtype": "bf16",
         "both": False},
        # a weight's two copies, at the largest matrix of the quantisation sweep
        {"name": "quant_weight", "op": "quant", "rows": 16384, "cols": 5120, "dtype": "bf16",
         "both": True},
        # an fp32 matrix whose sides divide nothing
        {"name": "quant_odd_f32", "op": "quant", "rows": 1537, "cols": 1111, "dtype": "f32",
         "both": True},
        # one new token through the 8B set's up projection
        {"name": "linear_one_token", "op": "linear", "tokens": 1, "n": 14336, "k": 4096,
         "dtype": "bf16", "grad": "bf16", "train": False},
        # a small decoding batch through its attention output projection
        {"name": "linear_decode_batch", "op": "linear", "tokens": 48, "n": 4096, "k": 4096,
         "dtype": "bf16", "grad": "bf16", "train": False},
        # a prompt of 8192 tokens through its up projection
        {"name": "linear_prompt", "op": "linear", "tokens": 8192, "n": 14336, "k": 4096,
         "dtype": "bf16", "grad": "bf16", "train": False},
        # a ragged fp16 batch through GPT-2's attention projection, forward and backward
        {"name": "linear_train_ragged", "op": "linear", "tokens": 1000, "n": 2304, "k": 768,
         "dtype": "f16", "grad": "f16", "train": True},
        # the 1B set's up projection, forward and backward, weight gradient kept in fp32
        {"name": "linear_train_1b", "op": "linear", "tokens": 4096, "n": 8192, "k": 2048,
         "dtype": "bf16", "grad": "f32", "train": True},
        # GPT-2's norm over a micro-batch, fp16 activations and fp32 parameters
        {"name": "norm_gpt2", "op": "norm", "rows": 1024, "cols": 768, "dtype": "f16",
         "param": "f32", "ckpt": False},
        # a wide norm over a training batch, its input kept in 8 bits
        {"name": "norm_wide_ckpt", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "param": "bf16", "ckpt": True},
        # a GELU whose rows end inside a block
        {"name": "act_gelu_odd", "op": "act", "rows": 2047, "cols": 1111, "dtype": "f16",
         "kind": "gelu", "gated": False},
        # the 8B set's gated SiLU over a training batch
        {"name": "act_swiglu", "op": "act", "rows": 8192, "cols": 14336, "dtype": "bf16",
         "kind": "silu", "gated": True},
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def _side(rng, lo, hi):
    """A size over the logarithm of the range: a multiple of 128, of 8, or anything."""
    v = _log(rng, lo, hi)
    step = rng.choice((128, 8, 1, 1))
    v = min(hi, max(lo, (v + step - 1) // step * step))
    return v - 8 if v == 3072 else v


def draw(rng):
    op = rng.choice(("quant", "linear", "norm", "act"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    most = {"quant": 16384 * 5120, "norm": 16384 * 4096, "act": 8192 * 14336 // 2}.get(op, 0)
    while True:
        r, c = _side(rng, 1, 16384), _side(rng, 33, 16384)
        if r * c <= most or not most:
            break
    if op == "quant":
        return {"op": op, "rows": r, "cols": c, "dtype": dtype, "both": rng.random() < 0.6}
    if op == "linear":
        train = rng.random() < 0.4
        while True:
            t, n, k = _side(rng, 1, 8192), _side(rng, 64, 14336), _side(rng, 64, 14336)
            if (3 if train else 1) * t * n * k <= 8192 * 14336 * 4096:
                break
        return {"op": op, "tokens": t, "n": n, "k": k, "dtype": dtype,
                "grad": rng.choice((dtype, "f32")), "train": train}
    if op == "norm":
        return {"op": op, "rows": r, "cols": c, "dtype": dtype, "param": rng.choice(("f32", dtype)),
                "ckpt": rng.random() < 0.5}
    return {"op": op, "rows": r, "cols": c, "dtype": dtype,
            "kind": rng.choice(("gelu", "gelu_tanh", "silu")), "gated": rng.random() < 0.5}


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
    e = (((bits + over) >> 23) - low).clamp_min(0)
    return torch.where(bits >= 0x7F800000, torch.full_like(e, 255), e)


def _scale(e):
    """2^(e - 127) in 32 bits (2^-127 is subnormal); NaN where e is 255."""
    v = torch.where(e == 0, torch.full_like(e, 0x400000), e << 23).view(torch.float32)
    return torch.where(e == 255, torch.full_like(v, math.nan), v)


def _unscale(e):
    """2^(127 - e) for e of at most 253; NaN where e is 255."""
    v = ((254 - e).clamp_min(1) << 23).view(torch.float32)
    return torch.where(e == 255, torch.full_like(v, math.nan), v)


def _e2m1_code(y):
    """Round to nearest, ties to the even code, of |y| <= 6: the magnitude's code and the sign bit."""
    a = y.abs()
    n = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
         + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    return n + 8 * torch.signbit(y).int()


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _fp4_codes(x):
    b = _blocks(x.float())
    e = _scale_code(b, 0x3FFFFF, 2)
    y = b * _unscale(e)[..., None]
    return _e2m1_code(torch.where(torch.isnan(y), torch.zeros_like(y), y)), e


def _fp4_round(x, table):
    """What x's 4-bit form stands for, in 32 bits."""
    code, e = _fp4_codes(x)
    return (table[code.long()] * _scale(e)[..., None]).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _mx8_round(x):
    """What x's 8-bit form (e4m3) stands for, in 32 bits."""
    b = _blocks(x.float())
    e = _scale_code(b, 0x1FFFFF, 8)
    y = b * _unscale(e)[..., None]
    q = y.to(torch.float8_e4m3fn).float() * _scale(e)[..., None]
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]]


def _pack(code, e):
    """Packed rows and tiled scales of codes [rows, blocks, 32] and scale bytes [rows, blocks]."""
    r, kb, _ = code.shape
    c = code.reshape(r, kb * 16, 2).to(torch.uint8)
    q = c[..., 0] | (c[..., 1] << 4)
    s = torch.nn.functional.pad(e.to(torch.uint8), (0, _up(kb, 4) - kb, 0, _up(r, 128) - r))
    s = s.reshape(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return q.contiguous(), s.reshape(-1).contiguous()


def _unpack(q, s, rows, cols, table):
    """The values of a packed matrix, in 32 bits."""
    kb = q.shape[1] // 16
    code = torch.stack((q & 15, q >> 4), -1).reshape(rows, kb, 32)
    t = s.reshape(-1, _up(kb, 4) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    e = t.reshape(_up(rows, 128), _up(kb, 4))[:rows, :kb].int()
    return (table[code.long()] * _scale(e)[..., None]).reshape(rows, kb * 32)[:, :cols]


def _fp4_buffers(rows, cols, dev):
    kb = _up(cols, 32) // 32
    return (torch.empty((rows, kb * 16), dtype=torch.uint8, device=dev),
            torch.empty(_up(rows, 128) * _up(kb, 4), dtype=torch.uint8, device=dev))


def _mx8_buffers(rows, cols, dev):
    return (torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=dev),
            torch.empty((rows, _up(cols, 32) // 32), dtype=torch.uint8, device=dev))


# ------------------------------------------------------------------ inputs
def _normal(g, rows, cols, dtype, sigma=1.0, spread=0.0):
    """N(0, sigma), a row's own scale exp(spread * N(0, 1)), one element in a thousand 20 times that."""
    x = torch.randn((rows, cols), generator=g, device=g.device) * sigma
    if spread:
        x *= torch.exp(spread * torch.randn((rows, 1), generator=g, device=g.device))
        x *= 1.0 + 19.0 * (torch.rand((rows, cols), generator=g, device=g.device) < 1e-3).float()
    return x.to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 17)
    dt = _DT[case["dtype"]]
    st = {"case": dict(case), "table": torch.tensor(_E2M1, dtype=torch.float32, device=dev)}
    if case["op"] == "quant":
        r, c = case["rows"], case["cols"]
        st["x"] = _normal(g, r, c, dt, 1.0, 0.5)
        st["q"], st["out"] = _fp4_buffers(r, c, dev), torch.empty((r, c), dtype=dt, device=dev)
        if case["both"]:
            st["qt"], st["out_t"] = _fp4_buffers(c, r, dev), torch.empty((c, r), dtype=dt, device=dev)
    elif case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        st["x"] = _normal(g, t, k, dt, 1.0, 0.3)
        w = _normal(g, n, k, torch.bfloat16, 0.02)
        st["w"] = _pack(*_fp4_codes(w))
        st["xq"], st["y"] = _fp4_buffers(t, k, dev), torch.empty((t, n), dtype=dt, device=dev)
        if case["train"]:
            st["dy"] = _normal(g, t, n, dt, 0.1, 0.3)
            st["wt"] = _pack(*_fp4_codes(w.t()))
            st["xtq"], st["dyq"] = _fp4_buffers(k, t, dev), _fp4_buffers(t, n, dev)
            st["dytq"] = _fp4_buffers(n, t, dev)
            st["dx"] = torch.empty((t, k), dtype=dt, device=dev)
            st["dw"] = torch.empty((n, k), dtype=_DT[case["grad"]], device=dev)
    elif case["op"] == "norm":
        r, c, pt = case["rows"], case["cols"], _DT[case["param"]]
        st["x"] = _normal(g, r, c, dt, 1.0, 0.3) + 0.25
        st["dy"] = _normal(g, r, c, dt, 0.1)
        st["w"] = (1.0 + 0.1 * torch.randn(c, generator=g, device=dev)).to(pt)
        st["b"] = (0.1 * torch.randn(c, generator=g, device=dev)).to(pt)
        st["y"], st["dx"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        st["mean"], st["rstd"] = torch.empty(r, device=dev), torch.empty(r, device=dev)
        st["dw"], st["db"] = torch.empty_like(st["w"]), torch.empty_like(st["b"])
        st["saved"] = _mx8_buffers(r, c, dev) if case["ckpt"] else None
    else:
        r, c = case["rows"], case["cols"]
        st["x"], st["dy"] = _normal(g, r, c, dt, 1.5, 0.2), _normal(g, r, c, dt, 0.1)
        st["saved"] = _mx8_buffers(r, c, dev)
        st["y"], st["dx"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        if case["gated"]:
            st["u"] = _normal(g, r, c, dt, 1.0, 0.2)
            st["saved_u"], st["du"] = _mx8_buffers(r, c, dev), torch.empty_like(st["x"])
    return st


# ------------------------------------------------------------------ one pass
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


def _plain(st):
    case = st["case"]
    dt, table = _DT[case["dtype"]], st["table"]
    if case["op"] == "quant":
        x = st["x"]
        got = {"out": _fp4_round(x, table).to(dt)}
        if case["both"]:
            got["out_t"] = _fp4_round(x.t(), table).to(dt)
        return got
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        w = _unpack(*st["w"], n, k, table)
        got = {"y": (_fp4_round(st["x"], table) @ w.t()).to(dt)}
        if case["train"]:
            wt = _unpack(*st["wt"], k, n, table)
            got["dx"] = (_fp4_round(st["dy"], table) @ wt.t()).to(dt)
            dyt, xt = _fp4_round(st["dy"].t(), table), _fp4_round(st["x"].t(), table)
            got["dw"] = (dyt @ xt.t()).to(_DT[case["grad"]])
        return got
    if case["op"] == "norm":
        x, dy, w, b = st["x"].float(), st["dy"].float(), st["w"].float(), st["b"].float()
        mean = x.mean(-1, keepdim=True)
        rstd = 1.0 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + _EPS)
        y = (x - mean) * rstd * w + b
        xh = ((_mx8_round(st["x"]) if case["ckpt"] else x) - mean) * rstd
        gw = dy * w
        dx = rstd * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
        pt = _DT[case["param"]]
        return {"y": y.to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0], "dx": dx.to(dt),
                "dw": (dy * xh).sum(0).to(pt), "db": dy.sum(0).to(pt)}
    kind = case["kind"]
    f, _ = _act(st["x"].float(), kind)
    fh, dfh = _act(_mx8_round(st["x"]), kind)
    dy = st["dy"].float()
    if not case["gated"]:
        return {"y": f.to(dt), "dx": (dy * dfh).to(dt)}
    return {"y": (f * st["u"].float()).to(dt), "dx": (dy * _mx8_round(st["u"]) * dfh).to(dt),
            "du": (dy * fh).to(dt)}


def _kernels(st):
    import loss_scaling_master_gb300 as G
    case = st["case"]
    if case["op"] == "quant":
        q, qt = st["q"], st.get("qt", (None, None))
        G.fp4_quant_mx(st["x"], *q, *qt)
        G.fp4_dequant_mx(*q, st["out"])
        if not case["both"]:
            return {"out": st["out"]}
        G.fp4_dequant_mx(*qt, st["out_t"])
        return {"out": st["out"], "out_t": st["out_t"]}
    if case["op"] == "linear":
        k = case["k"]
        if not case["train"]:
            G.fp4_quant_mx(st["x"], *st["xq"])
            G.fp4_product_mx(*st["xq"], *st["w"], k, st["y"])
            return {"y": st["y"]}
        G.fp4_quant_mx(st["x"], *st["xq"], *st["xtq"])
        G.fp4_product_mx(*st["xq"], *st["w"], k, st["y"])
        G.fp4_quant_mx(st["dy"], *st["dyq"], *st["dytq"])
        G.fp4_product_mx(*st["dyq"], *st["wt"], case["n"], st["dx"])
        G.fp4_product_mx(*st["dytq"], *st["xtq"], case["tokens"], st["dw"])
        return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}
    if case["op"] == "norm":
        saved = st["saved"]
        if "work" not in st:  # a training loop keeps this with its buffers
            st["work"] = G.amp_layer_norm_workspace(st["x"])
        G.amp_layer_norm_forward(st["x"], st["w"], st["b"], _EPS, st["y"], st["mean"], st["rstd"],
                                 saved=saved)
        G.amp_layer_norm_backward(st["dy"], None if saved else st["x"], st["w"], st["mean"],
                                  st["rstd"], st["dx"], st["dw"], st["db"], st["work"], saved=saved)
        return {k: st[k] for k in ("y", "mean", "rstd", "dx", "dw", "db")}
    if not case["gated"]:
        G.amp_act_forward_mx8(st["x"], case["kind"], st["y"], st["saved"])
        G.amp_act_backward_mx8(st["dy"], case["kind"], st["saved"], st["dx"])
        return {"y": st["y"], "dx": st["dx"]}
    G.amp_act_forward_mx8(st["x"], case["kind"], st["y"], st["saved"], up=st["u"],
                          saved_up=st["saved_u"])
    G.amp_act_backward_mx8(st["dy"], case["kind"], st["saved"], st["dx"], saved_up=st["saved_u"],
                           dup=st["du"])
    return {"y": st["y"], "dx": st["dx"], "du": st["du"]}


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    b = _SIZE[case["dtype"]]
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        copies = 2 if case["both"] else 1
        return {"bytes": n * b + copies * n * b, "flops": 6 * n * copies}
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]
        packed = n * k * (0.5 + 1 / 32)
        if not case["train"]:
            return {"bytes": t * k * b + packed + t * n * b, "flops": 2 * t * n * k}
        return {"bytes": 2 * (t * k + t * n) * b + 2 * packed + n * k * _SIZE[case["grad"]],
                "flops": 6 * t * n * k}
    n = case["rows"] * case["cols"]
    if case["op"] == "norm":
        return {"bytes": 4 * n * b + 16 * case["rows"] + 4 * case["cols"] * _SIZE[case["param"]],
                "flops": 20 * n}
    return {"bytes": n * b * (6 if case["gated"] else 4), "flops": 40 * n}


# ------------------------------------------------------------------ in 64 bits
def _two(p):
    """2^p in 64 bits, from its exponent field."""
    return ((p.long() + 1023) << 52).view(torch.float64)


def _mx_exact(x, top, least, bits):
    """The values of a block format in 64 bits: magnitudes at most `top`, quanta 2^(exponent - bits)
    down to the exponent `least`, a block's scale the smallest power of two that fits."""
    r, c = x.shape
    x = x.double()
    b = torch.zeros((r, _up(c, 32)), dtype=torch.float64, device=x.device)
    b[:, :c] = x
    b = b.unflatten(1, (-1, 32))
    a = b.abs().max(-1, keepdim=True).values
    m, p = torch.frexp(a)                       # a = m 2^p, 0.5 <= m < 1
    tm, tp = math.frexp(top)
    s = (p - tp + (m > tm).int()).clamp_min(-127)
    s = torch.where(a == 0, torch.full_like(s, -127), s)
    y = b * _two(-s)
    _, q = torch.frexp(y)
    step = _two((q - 1).clamp_min(least) - bits)
    y = torch.where(y == 0, y, torch.round(y / step) * step)
    y = y * _two(s)
    y = torch.where(torch.isfinite(a), y, torch.full_like(y, math.nan))
    return y.flatten(1)[:, :c]


def _fp4_exact(x):
    return _mx_exact(x, 6.0, 0, 1)


def _mx8_exact(x):
    return _mx_exact(x, 448.0, -6, 3)


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


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        got = {"out": _fp4_exact(st["x"])}
        if case["both"]:
            got["out_t"] = _fp4_exact(st["x"].t())
        return got
    if case["op"] == "linear":
        t, n, k = case["tokens"], case["n"], case["k"]

        def dense(packed, rows, cols):
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

        got = {"y": _fp4_exact(st["x"]) @ dense(st["w"], n, k).t()}
        if case["train"]:
            got["dx"] = _fp4_exact(st["dy"]) @ dense(st["wt"], k, n).t()
            got["dw"] = _fp4_exact(st["dy"].t()) @ _fp4_exact(st["x"].t()).t()
        return got
    if case["op"] == "norm":
        x, dy, w, b = (st[k].double() for k in ("x", "dy", "w", "b"))
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        rstd = (var + _EPS).rsqrt()
        xs = _mx8_exact(st["x"]) if case["ckpt"] else x
        xh, gw = (xs - mean) * rstd, dy * w
        c = x.shape[1]
        dx = rstd / c * (c * gw - gw.sum(-1, keepdim=True) - xh * (gw * xh).sum(-1, keepdim=True))
        return {"y": torch.addcmul(b, (x - mean) * rstd, w), "mean": mean.flatten(),
                "rstd": rstd.flatten(), "dx": dx, "dw": torch.einsum("rc,rc->c", dy, xh),
                "db": dy.sum(0)}
    f, _ = _act_exact(st["x"].double(), case["kind"])
    fh, dfh = _act_exact(_mx8_exact(st["x"]), case["kind"])
    dy = st["dy"].double()
    if not case["gated"]:
        return {"y": f, "dx": dy * dfh}
    return {"y": f * st["u"].double(), "dx": dy * _mx8_exact(st["u"]) * dfh, "du": dy * fh}
