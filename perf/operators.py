"""Cases of the operators around a melded FP8 linear layer: layer norm (both
directions), the FP8 product with bias, activation and residual in its
epilogue, the backward of that epilogue, and the clipping of many gradients by
their global norm.

listed() names the cases, draw() gives more of the same ranges, prepare() makes
the inputs of one, run() is one pass and exact() its result in 64 bits.  With
`own` false run() computes the plain form from elementary torch operations;
with `own` true it calls this package.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
LN_EPS = 1e-5
CLIP_EPS = 1e-6
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")

# the largest work of a drawn case: the listed ones' largest
MOST_PRODUCT = 8192 * 4096 * 11008        # T * d_in * d_out
MOST_ROWS = 8192 * 11008                  # T * d of the row-wise operators
MOST_GRADS = 32 * 7 * 64 * 11000          # gradient elements


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one token through a 7B model's norm: latency
        dict(name="ln_fwd_token", op="ln_fwd", T=1, d=4096, x="bf16", y="bf16", affine=True),
        # the norm before a 13B layer's projections, fp32 residual stream, bf16 activations
        dict(name="ln_fwd_13b", op="ln_fwd", T=4096, d=5120, x="f32", y="bf16", affine=True),
        # the 7B MLP's norm in training: dX of the product arrives in fp32
        dict(name="ln_bwd_7b", op="ln_bwd", T=8192, d=4096, x="bf16", dy="f32", affine=True),
        # odd rows and an odd width
        dict(name="ln_bwd_odd", op="ln_bwd", T=1003, d=1027, x="f32", dy="f32", affine=True),
        # one token through the attention output projection: the weight is read once
        dict(name="linear_token", op="linear", T=1, d_in=4096, d_out=4096, act="none", bias=True,
             residual=True, z=False),
        # a few sequences served together through the up projection
        dict(name="linear_few", op="linear", T=37, d_in=4096, d_out=11008, act="gelu_tanh",
             bias=True, residual=False, z=False),
        # the 7B MLP's up projection in training: the pre-activation is kept
        dict(name="linear_up_7b", op="linear", T=8192, d_in=4096, d_out=11008, act="gelu",
             bias=True, residual=False, z=True),
        # the 13B layer's down projection, added onto the residual stream
        dict(name="linear_down_13b", op="linear", T=4096, d_in=13824, d_out=5120, act="none",
             bias=True, residual=True, z=False),
        # the activation's backward behind the up projection
        dict(name="act_bwd_7b", op="act_bwd", T=8192, d=11008, act="gelu", dy="f32", z="bf16"),
        # a short ragged batch of it
        dict(name="act_bwd_ragged", op="act_bwd", T=130, d=400, act="silu", dy="bf16", z="bf16"),
        # one attention projection's dA and dB at rank 64
        dict(name="clip_layer", op="clip", layers=0, count=2, total=2 * 64 * 4096, sizes=0,
             dtype="f32", max_norm=1.0),
        # every projection of a 32-layer 7B model at rank 64: 448 tensors
        dict(name="clip_7b", op="clip", layers=32, rank=64, d=4096, ff=11008, dtype="f32",
             max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("ln_fwd", "ln_bwd", "linear", "linear", "act_bwd", "clip"))
    two = ("f32", "bf16")
    if op in ("ln_fwd", "ln_bwd", "act_bwd"):
        d = _log(rng, 16, 13824)
        if rng.random() < 0.5:
            d = max(16, d // 16 * 16)
        T = _log(rng, 1, max(1, min(16384, MOST_ROWS // d)))
        if op == "ln_fwd":
            return dict(op=op, T=T, d=d, x=rng.choice(two), y=rng.choice(two),
                        affine=rng.random() < 0.8)
        if op == "ln_bwd":
            return dict(op=op, T=T, d=d, x=rng.choice(two), dy=rng.choice(two),
                        affine=rng.random() < 0.8)
        return dict(op=op, T=T, d=d, act=rng.choice(ACTS[1:]), dy=rng.choice(two),
                    z=rng.choice(two))
    if op == "linear":
        d_in = _log(rng, 4, 864) * 16
        d_out = _log(rng, 4, 864) * 16
        T = _log(rng, 1, max(1, min(8192, MOST_PRODUCT // (d_in * d_out))))
        act = rng.choice(ACTS)
        return dict(op=op, T=T, d_in=d_in, d_out=d_out, act=act, bias=rng.random() < 0.7,
                    residual=rng.random() < 0.4, z=act != "none" and rng.random() < 0.5)
    count = _log(rng, 1, 448)
    total = max(count, _log(rng, 1000, MOST_GRADS))
    return dict(op="clip", layers=0, count=count, total=total, sizes=rng.randrange(1 << 20),
                dtype=rng.choice(("f32", "bf16", "mixed")), max_norm=rng.choice((0.5, 1.0, 1e6)))


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


def _grad_shapes(case):
    """Numbers of elements of the gradients, in order, with their types."""
    if case["layers"]:
        r, d, ff = case["rank"], case["d"], case["ff"]
        pairs = [(r * d, d * r)] * 4 + [(r * d, ff * r)] * 2 + [(r * ff, d * r)]
        sizes = [n for _ in range(case["layers"]) for pair in pairs for n in pair]
    else:
        n = case["count"]
        sizes = [case["total"] // n] * n
        if case["sizes"]:
            rng = random.Random(case["sizes"])
            share = [math.exp(rng.uniform(0.0, 5.0)) for _ in range(n)]
            sizes = [max(1, int(case["total"] * s / sum(share))) for s in share]
    kinds = [case["dtype"] if case["dtype"] != "mixed" else ("f32", "bf16")[i % 2]
             for i in range(len(sizes))]
    return sizes, kinds


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    op, s = case["op"], {"case": case}
    if op in ("ln_fwd", "ln_bwd"):
        T, d = case["T"], case["d"]
        s["x"] = _stream_like(g, T, d).to(DTYPES[case["x"]])
        s["weight"] = 1.0 + 0.1 * randn(d) if case["affine"] else None
        s["bias"] = 0.1 * randn(d) if case["affine"] else None
        if op == "ln_bwd":
            s["dy"] = (randn(T, d) * 1e-3).to(DTYPES[case["dy"]])
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = 1.0 / ((x - s["mean"][:, None]).square().mean(1) + LN_EPS).sqrt()
    elif op == "linear":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        s["xq"], s["s_x"] = _quantized(_stream_like(g, T, d_in))
        s["wq"], s["s_w"] = _quantized(randn(d_out, d_in) * 0.02)
        s["bias"] = 0.1 * randn(d_out) if case["bias"] else None
        s["residual"] = randn(T, d_out).bfloat16() if case["residual"] else None
    elif op == "act_bwd":
        T, d = case["T"], case["d"]
        s["dy"] = (randn(T, d) * 1e-3).to(DTYPES[case["dy"]])
        s["z"] = (randn(T, d) * 1.5).to(DTYPES[case["z"]])
    else:
        # the gradients lie in one bucket for each type, as a data-parallel program has them
        sizes, kinds = _grad_shapes(case)
        s["buckets"] = {}
        for k in sorted(set(kinds)):
            n = sum(m for m, kk in zip(sizes, kinds) if kk == k)
            s["buckets"][k] = (randn(n) * 1e-2).to(DTYPES[k])
        s["clipped"] = {k: torch.zeros_like(b) for k, b in s["buckets"].items()}
        at = dict.fromkeys(s["buckets"], 0)
        s["grads"], s["out"] = [], []
        for n, k in zip(sizes, kinds):
            s["grads"].append(s["buckets"][k][at[k]: at[k] + n])
            s["out"].append(s["clipped"][k][at[k]: at[k] + n])
            at[k] += n
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
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        xc = x - mean[:, None]
        rstd = 1.0 / (xc.square().mean(1) + LN_EPS).sqrt()
        y = xc * rstd[:, None]
        if case["affine"]:
            y = y * s["weight"] + s["bias"]
        return {"y": y.to(DTYPES[case["y"]]), "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"] if case["affine"] else dy
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        out = {"dx": dx.to(DTYPES[case["dy"]])}
        if case["affine"]:
            out["dweight"], out["dbias"] = (dy * xh).sum(0), dy.sum(0)
        return out
    if op == "linear":
        z = (_f8(s["xq"]).float() @ _f8(s["wq"]).float().T) * (1.0 / (s["s_x"] * s["s_w"]))
        if case["bias"]:
            z = z + s["bias"]
        y = _act(z, case["act"])
        if case["residual"]:
            y = y + s["residual"].float()
        return {"y": y.bfloat16(), **({"z": z.bfloat16()} if case["z"] else {})}
    if op == "act_bwd":
        dz = s["dy"].float() * _act_slope(s["z"].float(), case["act"])
        return {"dz": dz.to(DTYPES[case["dy"]]), "dbias": dz.sum(0)}
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    coef = (case["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["out"])]
    return {"norm": norm.reshape(1), "clipped": s["clipped"]}


def _own(s):
    import fp8_quantized_lora_amd as fq

    case, op = s["case"], s["case"]["op"]
    new = lambda *shape, dtype=torch.float32: torch.empty(  # noqa: E731
        shape, dtype=dtype, device="cuda")
    if op == "ln_fwd":
        T, d = case["T"], case["d"]
        y, mean, rstd = new(T, d, dtype=DTYPES[case["y"]]), new(T), new(T)
        fq.layer_norm_fwd(s["x"], s["weight"], s["bias"], y, mean, rstd, eps=LN_EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        T, d = case["T"], case["d"]
        dx = new(T, d, dtype=DTYPES[case["dy"]])
        dw, db = (new(d), new(d)) if case["affine"] else (None, None)
        fq.layer_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dx, dw, db)
        return {"dx": dx, **({"dweight": dw, "dbias": db} if case["affine"] else {})}
    if op == "linear":
        T, n = case["T"], case["d_out"]
        y = new(T, n, dtype=torch.bfloat16)
        z = new(T, n, dtype=torch.bfloat16) if case["z"] else None
        fq.melded_linear_fwd_act(s["xq"], s["s_x"], s["wq"], s["s_w"], y, bias=s["bias"],
                                 act=case["act"], residual=s["residual"], z=z)
        return {"y": y, **({"z": z} if case["z"] else {})}
    if op == "act_bwd":
        dz, db = new(case["T"], case["d"], dtype=DTYPES[case["dy"]]), new(case["d"])
        fq.linear_act_bwd(s["dy"], s["z"], dz, dbias=db, act=case["act"])
        return {"dz": dz, "dbias": db}
    norm = new(1)
    fq.grad_clip(s["grads"], case["max_norm"], norm, out=s["out"], eps=CLIP_EPS)
    return {"norm": norm, "clipped": s["clipped"]}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
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
    if op in ("ln_fwd", "ln_bwd"):
        x = s["x"].double()
        w = s["weight"].double() if case["affine"] else 1.0
        if op == "ln_fwd":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + LN_EPS) ** -0.5
            y = (x - mean[:, None]) * rstd[:, None] * w
            return {"y": y + s["bias"].double() if case["affine"] else y, "mean": mean,
                    "rstd": rstd}
        dy, r = s["dy"].double(), s["rstd"].double()[:, None]
        xh = (x - s["mean"].double()[:, None]) * r
        g, d = dy * w, case["d"]
        dx = r / d * (d * g - g.sum(1, True) - xh * (g * xh).sum(1, True))
        if not case["affine"]:
            return {"dx": dx}
        return {"dx": dx, "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}
    if op == "linear":
        z = torch.mm(_f8(s["xq"]).double(), _f8(s["wq"]).double().t())
        z /= s["s_x"].double() * s["s_w"].double()
        if case["bias"]:
            z += s["bias"].double()
        y = _exact_act(z, case["act"])
        if case["residual"]:
            y = y + s["residual"].double()
        return {"y": y, **({"z": z} if case["z"] else {})}
    if op == "act_bwd":
        dz = s["dy"].double() * _exact_act(s["z"].double(), case["act"], slope=True)
        return {"dz": dz, "dbias": dz.sum(0)}
    norm = math.sqrt(sum(float(b.double().square().sum()) for b in s["buckets"].values()))
    coef = min(1.0, case["max_norm"] / (norm + CLIP_EPS))
    return {"norm": torch.tensor([norm], dtype=torch.float64),
            "clipped": {k: b.double() * coef for k, b in s["buckets"].items()}}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "ln_fwd":
        n, d = case["T"] * case["d"], case["d"]
        return {"bytes": n * (BYTES[case["x"]] + BYTES[case["y"]]) + 8 * case["T"]
                + 8 * d * case["affine"], "flops": 7 * n}
    if op == "ln_bwd":
        n, d = case["T"] * case["d"], case["d"]
        return {"bytes": n * (BYTES[case["x"]] + 2 * BYTES[case["dy"]]) + 8 * case["T"]
                + 12 * d * case["affine"], "flops": 14 * n}
    if op == "linear":
        T, i, o = case["T"], case["d_in"], case["d_out"]
        return {"bytes": T * i + i * o + 4 * o * case["bias"]
                + 2 * T * o * (1 + case["residual"] + case["z"]), "flops": 2 * T * i * o}
    if op == "act_bwd":
        n = case["T"] * case["d"]
        return {"bytes": n * (2 * BYTES[case["dy"]] + BYTES[case["z"]]) + 4 * case["d"],
                "flops": 15 * n}
    sizes, kinds = _grad_shapes(case)
    return {"bytes": 2 * sum(n * BYTES[k] for n, k in zip(sizes, kinds)) + 4,
            "flops": 3 * sum(sizes)}
