"""Cases of the operators at the ends of a melded layer's step: operands in
microscaled FP4 (quantisation, and the product with its epilogue), activations
kept in 8 bits between forward and backward (saved, and read by the backward of
an activation and of layer norm), and softmax cross entropy over the vocabulary
of an FP8 output layer with its gradient, the logits never kept.

listed() names the cases, draw() gives more of the same ranges, prepare() makes
the inputs of one, run() is one pass and exact() its result in 64 bits.  With
`own` false run() computes the plain form from elementary torch operations;
with `own` true it calls this package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
LN_EPS = 1e-5
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
IGNORE = -100

# the largest work of a drawn case: the listed ones' largest
MOST_PRODUCT = 8192 * 4096 * 11008        # T * d_in * d_out of the FP4 product
MOST_LOSS = 4096 * 4096 * 32000           # T * d * V
MOST_ROWS = 8192 * 11008                  # elements of the row-wise operators


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one token's activations through FP4 and back: latency
        dict(name="fp4_token", op="fp4", rows=1, K=4096, x="bf16", out="f32"),
        # a 7B MLP weight rounded to FP4, as a check of what the format does to it
        dict(name="fp4_weight_7b", op="fp4", rows=11008, K=4096, x="f32", out="bf16"),
        # one token through the attention output projection, onto the residual stream
        dict(name="product_token", op="product", T=1, d_in=4096, d_out=4096, act="none",
             bias=False, residual=True, z=False),
        # a few sequences served together, an inner dimension that ends inside a step
        dict(name="product_few", op="product", T=37, d_in=4064, d_out=11008, act="silu",
             bias=False, residual=False, z=False),
        # the 7B MLP's up projection in training: the pre-activation is kept
        dict(name="product_up_7b", op="product", T=8192, d_in=4096, d_out=11008, act="gelu",
             bias=True, residual=False, z=True),
        # the pre-activation of that projection kept in 8 bits, and the activation's backward
        dict(name="keep_act_7b", op="keep_act", T=8192, d=11008, act="gelu", dy="f32", z="bf16"),
        # a short ragged batch of it, an odd width
        dict(name="keep_act_odd", op="keep_act", T=131, d=1027, act="silu", dy="bf16", z="bf16"),
        # the input of a 7B layer's norm kept in 8 bits, and the norm's backward
        dict(name="keep_norm_7b", op="keep_norm", T=8192, d=4096, x="bf16", dy="f32"),
        # few rows, a width that is a multiple of 8 only
        dict(name="keep_norm_few", op="keep_norm", T=200, d=1000, x="f32", dy="f32"),
        # one position scored against a vocabulary of 32000: the output layer is read once
        dict(name="loss_token", op="loss", T=1, d=4096, V=32000, grad=False),
        # a training batch: loss and gradient
        dict(name="loss_train", op="loss", T=4096, d=4096, V=32000, grad=True),
        # a short ragged batch, an odd large vocabulary
        dict(name="loss_odd", op="loss", T=333, d=1040, V=131071, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fp4", "product", "product", "keep_act", "keep_norm", "loss", "loss"))
    two = ("f32", "bf16")
    if op == "fp4":
        K = _log(rng, 1, 432) * 32
        rows = _log(rng, 1, max(1, min(16384, MOST_ROWS // K)))
        return dict(op=op, rows=rows, K=K, x=rng.choice(two), out=rng.choice(two))
    if op == "product":
        d_in = _log(rng, 2, 432) * 32
        d_out = _log(rng, 4, 864) * 16
        T = _log(rng, 1, max(1, min(8192, MOST_PRODUCT // (d_in * d_out))))
        act = rng.choice(ACTS)
        return dict(op=op, T=T, d_in=d_in, d_out=d_out, act=act, bias=rng.random() < 0.7,
                    residual=rng.random() < 0.4, z=act != "none" and rng.random() < 0.5)
    if op == "loss":
        d = _log(rng, 4, 512) * 16
        V = _log(rng, 1000, 131072)
        T = _log(rng, 1, max(1, min(8192, MOST_LOSS // (d * V))))
        return dict(op=op, T=T, d=d, V=V, grad=rng.random() < 0.7)
    d = _log(rng, 16, 13824)
    if rng.random() < 0.5:
        d = max(16, d // 16 * 16)
    T = _log(rng, 1, max(1, min(16384, MOST_ROWS // d)))
    if op == "keep_act":
        return dict(op=op, T=T, d=d, act=rng.choice(ACTS[1:]), dy=rng.choice(two),
                    z=rng.choice(two))
    return dict(op=op, T=T, d=d, x=rng.choice(two), dy=rng.choice(two))


# --------------------------------------------------------------------------
# the formats: blocks of 32 along a row, one power of two each
# --------------------------------------------------------------------------
def _blocks(x):
    """x [rows x n] as float32 [rows x blocks x 32], the last block filled up."""
    rows, n = x.shape
    nb = (n + 31) // 32
    v = torch.zeros((rows, nb * 32), dtype=torch.float32, device=x.device)
    v[:, :n] = x
    return v.view(rows, nb, 32)


def _fp4_exponent(amax):
    """floor(log2(amax)) - 2, so that the largest element lies in [4, 8); 0 for zeros."""
    e = torch.frexp(amax).exponent.to(torch.int32) - 3
    return torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))


def _fp8_exponent(amax):
    """the smallest e with amax <= 448 * 2^e; 0 for zeros"""
    m, E = torch.frexp(amax)
    e = E.to(torch.int32) - torch.where(m <= 0.875, 9, 8).to(torch.int32)
    return torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))


def _round_fp4(a):
    """|values| up to 6 to the nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code"""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(a / step) * step


def _fp4_codes(x):
    """Codes [rows x K / 2] (two a byte, the lower index in the low half) and
    exponents [rows x K / 32] of x."""
    v = _blocks(x)
    e = _fp4_exponent(v.abs().amax(2))
    v = torch.ldexp(v, -e[:, :, None])
    a = _round_fp4(v.abs().clamp(max=6.0))
    c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = (c | (torch.signbit(v).to(torch.uint8) << 3)).view(x.shape[0], -1)
    return c[:, 0::2] | (c[:, 1::2] << 4), e


def _fp4_values(q, e):
    """float32 values of codes and exponents."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=torch.float32, device=q.device)
    c = torch.stack((q & 15, q >> 4), 2).view(q.shape[0], -1)
    v = table[c.long()].view(q.shape[0], -1, 32)
    return torch.ldexp(v, e[:, :, None]).view(q.shape[0], -1)


def _packed(e):
    """Exponents [rows x blocks] as the product takes them: bytes e + 127 in
    [steps x rows16 x 8], a step of eight blocks, block b of a step at
    2 (b % 4) + b // 4; rows16 is rows rounded up to a multiple of 16."""
    rows, nb = e.shape
    steps, rows16 = (nb + 7) // 8, (rows + 15) // 16 * 16
    s = torch.full((rows16, steps * 8), 127, dtype=torch.uint8, device=e.device)
    s[:rows, :nb] = (e + 127).to(torch.uint8)
    return s.view(rows16, steps, 2, 4).permute(1, 0, 3, 2).reshape(steps, rows16, 8).contiguous()


def _unpacked(s, rows, nb):
    steps, rows16 = s.shape[:2]
    b = s.view(steps, rows16, 4, 2).permute(1, 0, 3, 2).reshape(rows16, steps * 8)
    return b[:rows, :nb].to(torch.int32) - 127


def _kept(x):
    """x as 8 bits keep it: E4M3 under a power of two for each block of 32."""
    v = _blocks(x)
    e = _fp8_exponent(v.abs().amax(2))[:, :, None]
    c = torch.ldexp(v, -e).to(torch.float8_e4m3fn)
    return torch.ldexp(c.float(), e).view(x.shape[0], -1)[:, : x.shape[1]]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _f8(codes):
    return codes.view(torch.float8_e4m3fn)


def _quantized(x):
    """E4M3 codes of x under the per-tensor scale 448 / max|x|."""
    s = (448.0 / x.abs().max()).reshape(1)
    return (x * s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), s


def _stream_like(g, T, d):
    """Rows as a residual stream has them: an offset, a hundredth of the
    channels twenty times the others."""
    x = torch.randn((T, d), generator=g, device="cuda")
    gain = torch.ones(d, device="cuda")
    gain[torch.randperm(d, generator=g, device="cuda")[: d // 100]] = 20.0
    return x.mul_(gain).add_(0.1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    op, s = case["op"], {"case": case}
    if op == "fp4":
        s["x"] = _stream_like(g, case["rows"], case["K"]).to(DTYPES[case["x"]])
    elif op == "product":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        s["x"] = _stream_like(g, T, d_in).bfloat16()
        s["wq"], e = _fp4_codes(randn(d_out, d_in) * 0.02)       # the weight, laid out once
        s["we"] = _packed(e)
        s["bias"] = 0.1 * randn(d_out) if case["bias"] else None
        s["residual"] = randn(T, d_out).bfloat16() if case["residual"] else None
    elif op == "keep_act":
        T, d = case["T"], case["d"]
        s["dy"] = (randn(T, d) * 1e-3).to(DTYPES[case["dy"]])
        s["z"] = (randn(T, d) * 1.5).to(DTYPES[case["z"]])
    elif op == "keep_norm":
        T, d = case["T"], case["d"]
        s["x"] = _stream_like(g, T, d).to(DTYPES[case["x"]])
        s["weight"] = 1.0 + 0.1 * randn(d)
        s["dy"] = (randn(T, d) * 1e-3).to(DTYPES[case["dy"]])
        x = s["x"].float()
        s["mean"] = x.mean(1)
        s["rstd"] = 1.0 / ((x - s["mean"][:, None]).square().mean(1) + LN_EPS).sqrt()
    else:
        T, d, V = case["T"], case["d"], case["V"]
        # normalised rows, some tokens far surer of their next one than others
        x = _stream_like(g, T, d)
        x = x / x.square().mean(1, keepdim=True).sqrt()
        x = x * torch.exp(1.5 * torch.rand((T, 1), generator=g, device="cuda"))
        s["xq"], s["s_x"] = _quantized(x)
        s["wq"], s["s_w"] = _quantized(randn(V, d) * (1.5 / math.sqrt(d)))
        t = torch.randint(0, V, (T,), generator=g, device="cuda")
        # a tenth is padding, which counts for nothing; the others weigh the same
        keep = torch.rand(T, generator=g, device="cuda") >= 0.1
        keep[0] = True
        s["target"] = torch.where(keep, t, torch.full_like(t, IGNORE))
        s["dloss"] = keep.float() / keep.sum()
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 + z * (1.0 - p))


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "fp4":
        return {"values": _fp4_values(*_fp4_codes(s["x"])).to(DTYPES[case["out"]])}
    if op == "product":
        x = _fp4_values(*_fp4_codes(s["x"]))
        w = _fp4_values(s["wq"], _unpacked(s["we"], case["d_out"], case["d_in"] // 32))
        z = x @ w.T
        if case["bias"]:
            z = z + s["bias"]
        y = _act(z, case["act"])
        if case["residual"]:
            y = y + s["residual"].float()
        return {"y": y.bfloat16(), **({"z": z.bfloat16()} if case["z"] else {})}
    if op == "keep_act":
        dz = s["dy"].float() * _act_slope(_kept(s["z"]), case["act"])
        return {"dz": dz.to(DTYPES[case["dy"]]), "dbias": dz.sum(0)}
    if op == "keep_norm":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (_kept(s["x"]) - s["mean"][:, None]) * rstd
        g = dy * s["weight"]
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return {"dx": dx.to(DTYPES[case["dy"]]), "dweight": (dy * xh).sum(0),
                "dbias": dy.sum(0)}
    w = _f8(s["wq"]).float() / s["s_w"]
    logits = (_f8(s["xq"]).float() / s["s_x"]) @ w.T
    m = logits.amax(1, keepdim=True)
    p = torch.exp(logits - m)
    total = p.sum(1, keepdim=True)
    lse = (m + total.log())[:, 0]
    keep = s["target"] >= 0
    at = s["target"].clamp(min=0)[:, None]
    loss = torch.where(keep, lse - logits.gather(1, at)[:, 0], torch.zeros_like(lse))
    if not case["grad"]:
        return {"loss": loss, "lse": lse}
    g = p / total
    g.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
    g *= torch.where(keep, s["dloss"], torch.zeros_like(lse))[:, None]
    return {"loss": loss, "lse": lse, "dx": (g @ w).bfloat16()}


def _own(s):
    import fp8_quantized_lora_amd as fq

    case, op = s["case"], s["case"]["op"]
    new = lambda *shape, dtype=torch.float32: torch.empty(  # noqa: E731
        shape, dtype=dtype, device="cuda")
    u8 = torch.uint8
    if op in ("fp4", "product"):
        x = s["x"]
        rows, K = x.shape
        q, e = new(rows, K // 2, dtype=u8), new(*fq.mxfp4_scales_shape(rows, K), dtype=u8)
        fq.mxfp4_quantize(x, q, e)
        if op == "fp4":
            out = new(rows, K, dtype=DTYPES[case["out"]])
            fq.mxfp4_dequantize(q, e, out)
            return {"values": out}
        y = new(rows, case["d_out"], dtype=torch.bfloat16)
        z = torch.empty_like(y) if case["z"] else None
        fq.melded_linear_fwd_mxfp4(q, e, s["wq"], s["we"], y, bias=s["bias"], act=case["act"],
                                   residual=s["residual"], z=z)
        return {"y": y, **({"z": z} if case["z"] else {})}
    if op in ("keep_act", "keep_norm"):
        x = s["z"] if op == "keep_act" else s["x"]
        T, d = x.shape
        codes, scales = new(T, d, dtype=u8), new(T, (d + 31) // 32, dtype=u8)
        fq.checkpoint_save(x, codes, scales)
        out, db = new(T, d, dtype=DTYPES[case["dy"]]), new(d)
        if op == "keep_act":
            fq.linear_act_bwd_ckpt(s["dy"], codes, scales, out, dbias=db, act=case["act"])
            return {"dz": out, "dbias": db}
        dw = new(d)
        fq.layer_norm_bwd_ckpt(s["dy"], codes, scales, s["weight"], s["mean"], s["rstd"], out, dw,
                               db)
        return {"dx": out, "dweight": dw, "dbias": db}
    T, d = s["xq"].shape
    loss, lse = new(T), new(T)
    fq.linear_cross_entropy_fwd(s["xq"], s["s_x"], s["wq"], s["s_w"], s["target"], loss, lse)
    if not case["grad"]:
        return {"loss": loss, "lse": lse}
    dx = new(T, d, dtype=torch.bfloat16)
    fq.linear_cross_entropy_bwd(s["xq"], s["s_x"], s["wq"], s["s_w"], s["target"], lse,
                                s["dloss"], dx)
    return {"loss": loss, "lse": lse, "dx": dx}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def _nearest(v, mags):
    """|v| to the nearest of the sorted magnitudes, a tie to the even index, by
    search among the midpoints; signs kept, larger ones to the last."""
    t = torch.tensor(mags, dtype=torch.float64, device=v.device)
    mid = (t[1:] + t[:-1]) / 2
    a = v.abs()
    up = torch.searchsorted(mid, a, right=True)                   # a tie goes up
    down = torch.searchsorted(mid, a, right=False)                # a tie goes down
    return torch.copysign(t[torch.where(up % 2 == 0, up, down)], v)


def _e4m3_magnitudes():
    return [m * 2.0 ** -9 for m in range(8)] + [
        (8 + m) * 2.0 ** (E - 10) for E in range(1, 16) for m in range(8) if (E, m) != (15, 7)]


def _exact_blocks(x, mags, exponent):
    """x rounded to magnitudes times a power of two per block of 32, in float64."""
    rows, n = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -n % 32)).view(rows, -1, 32)
    amax = v.abs().amax(2)
    e = exponent(torch.where(amax > 0, amax, torch.ones_like(amax))).clamp(-127, 127)
    s = torch.exp2(torch.where(amax > 0, e, torch.zeros_like(e)))[:, :, None]
    return (_nearest(v / s, mags) * s).view(rows, -1)[:, :n]


def _floor_log2(a):
    """floor(log2 a) from the bits of a float64"""
    return ((a.view(torch.int64) >> 52) & 2047).double() - 1023


def _exact_fp4(x):
    return _exact_blocks(x, [0, .5, 1, 1.5, 2, 3, 4, 6], lambda a: _floor_log2(a) - 2)


def _exact_kept(x):
    def exponent(a):
        e = _floor_log2(a) - 8                                    # a / 2^e in [256, 512)
        return e + (a / torch.exp2(e) > 448).double()
    return _exact_blocks(x, _e4m3_magnitudes(), exponent)


def _exact_act(z, act, slope=False):
    """act(z), or its derivative, from erfc and the logistic function."""
    if act == "none":
        return torch.ones_like(z) if slope else z
    if act == "relu":
        return (z > 0).double() if slope else z.clamp(min=0)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi) if slope else z * cdf
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * torch.sigmoid(-z) if slope else z * p
    # (1 + tanh u) / 2 is the logistic function of 2u
    u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(u2)
    if not slope:
        return z * p
    return p + z * p * torch.sigmoid(-u2) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fp4":
        return {"values": _exact_fp4(s["x"])}
    if op == "product":
        nb = case["d_in"] // 32
        codes = torch.stack((s["wq"] & 15, s["wq"] >> 4), 2).flatten(1)
        mags = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        w = mags[(codes & 7).long()] * (1 - 2 * (codes >> 3).double())
        at = torch.arange(nb, device="cuda")
        scale = s["we"][at // 8, :, 2 * (at % 4) + at % 8 // 4].T[: case["d_out"]]
        w = w * torch.exp2(scale.double() - 127).repeat_interleave(32, 1)
        z = torch.mm(_exact_fp4(s["x"]), w.t())
        if case["bias"]:
            z += s["bias"].double()
        y = _exact_act(z, case["act"])
        if case["residual"]:
            y = y + s["residual"].double()
        return {"y": y, **({"z": z} if case["z"] else {})}
    if op == "keep_act":
        dz = s["dy"].double() * _exact_act(_exact_kept(s["z"]), case["act"], slope=True)
        return {"dz": dz, "dbias": dz.sum(0)}
    if op == "keep_norm":
        dy, r, d = s["dy"].double(), s["rstd"].double()[:, None], case["d"]
        xh = (_exact_kept(s["x"]) - s["mean"].double()[:, None]) * r
        g = dy * s["weight"].double()
        dx = r / d * (d * g - g.sum(1, True) - xh * (g * xh).sum(1, True))
        return {"dx": dx, "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}
    # a strip of rows at a time: float64 logits of all of them would be large
    T = case["T"]
    w = _f8(s["wq"]).double() / s["s_w"].double()
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    dx = torch.zeros((T, case["d"]), dtype=torch.float64, device="cuda") if case["grad"] else None
    for a in range(0, T, 1024):
        r = slice(a, min(T, a + 1024))
        z = torch.mm(_f8(s["xq"][r]).double() / s["s_x"].double(), w.t())
        lse[r] = torch.logsumexp(z, 1)
        rows = torch.nonzero(s["target"][r] >= 0)[:, 0]
        cols = s["target"][r][rows]
        loss[a + rows] = lse[r][rows] - z[rows, cols]
        if dx is not None:
            z -= lse[r][:, None]
            z.exp_()
            z[rows, cols] -= 1.0
            dx[a + rows] = torch.mm(z[rows], w) * s["dloss"][r][rows].double()[:, None]
    return {"loss": loss, "lse": lse, **({"dx": dx} if case["grad"] else {})}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "fp4":
        n = case["rows"] * case["K"]
        # read, the codes and exponents written and read, the values written
        return {"bytes": n * (BYTES[case["x"]] + BYTES[case["out"]]) + 2 * (n // 2 + n // 32),
                "flops": 4 * n}
    if op == "product":
        T, i, o = case["T"], case["d_in"], case["d_out"]
        return {"bytes": 2 * T * i + (i // 2 + i // 32) * o + 4 * o * case["bias"]
                + 2 * T * o * (1 + case["residual"] + case["z"]), "flops": 2 * T * i * o}
    if op in ("keep_act", "keep_norm"):
        T, d = case["T"], case["d"]
        n, nb = T * d, T * ((d + 31) // 32)
        kept = case["z"] if op == "keep_act" else case["x"]
        small = 4 * d if op == "keep_act" else 12 * d + 8 * T
        return {"bytes": n * (BYTES[kept] + 2 * BYTES[case["dy"]]) + 2 * (n + nb) + small,
                "flops": 20 * n}
    T, d, V = case["T"], case["d"], case["V"]
    return {"bytes": T * d + V * d + 16 * T + (4 * T + 2 * T * d) * case["grad"],
            "flops": 2 * T * d * V * (1 + case["grad"])}
