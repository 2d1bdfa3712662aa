"""Timed cases of the channel operators: RMS norm with the residual's addition,
the linear layer with its epilogue, and the gated feed-forward projections.

Every tensor is rows (pixels or tokens) by channels, channels innermost.  With
``own`` false ``run`` computes a case in elementary torch operations in FP32;
with ``own`` true it calls this package's operators.  ``exact`` is the
definition in FP64, written apart from the plain form.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}

# the largest listed case's operations; drawn cases stay below them
MOST_FLOPS = 4 * 16384 * 4096 * 8192


def listed():
    return [
        # one token of a serving step: latency
        dict(name="norm_token_e4m3", op="norm", rows=1, c=4096, dtype="bf16", out="e4m3", pad=0),
        # the residual stream of an image batch, 128 images of 28 x 28 pixels
        dict(name="norm_pixels", op="norm", rows=100352, c=512, dtype="bf16", out="bf16", pad=0),
        # odd channels in FP32, rows with a pitch of their own
        dict(name="norm_odd_f32", op="norm", rows=2401, c=333, dtype="f32", out="f32", pad=3),
        # training, 128 images of 14 x 14 pixels
        dict(name="norm_backward", op="norm_bwd", rows=25088, c=1024, dtype="bf16", pad=0),
        # a classifier's logits for a handful of images
        dict(name="linear_logits", op="linear", rows=4, c=4096, k=1000, dtype="bf16", out="f32",
             act="identity", bias=True, residual=False),
        # a classifier's hidden layer for one batch
        dict(name="linear_batch", op="linear", rows=128, c=4096, k=4096, dtype="bf16", out="bf16",
             act="relu", bias=True, residual=False),
        # sizes that no alignment rule likes
        dict(name="linear_odd", op="linear", rows=785, c=147, k=1001, dtype="bf16", out="bf16",
             act="gelu", bias=True, residual=True),
        # the down projection of a training step: bias, residual, and its gradients
        dict(name="linear_train", op="linear_train", rows=8192, c=4096, k=2048, act="identity",
             bias=True),
        # one token's up projections
        dict(name="gated_token", op="gated", rows=1, c=2048, f=8192, dtype="bf16", act="silu"),
        # a batch of decoding sequences, 8-bit operands
        dict(name="gated_decode_e4m3", op="gated", rows=64, c=4096, f=8192, dtype="e4m3", act="silu"),
        # prompt tokens or a whole image batch, 8-bit operands
        dict(name="gated_prompt_e4m3", op="gated", rows=16384, c=4096, f=8192, dtype="e4m3",
             act="silu"),
        # a training step of the block
        dict(name="gated_train", op="gated_train", rows=8192, c=2048, f=5632, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _channels(rng, lo, hi):
    c = _log(rng, lo, hi)
    return c if rng.random() < 0.25 else max(16, c // 16 * 16)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "linear", "linear", "linear_train", "gated", "gated",
                     "gated_train"])
    if op == "norm" or op == "norm_bwd":
        c = _channels(rng, 64, 8192)
        rows = _log(rng, 1, min(100352, 100352 * 512 // c))
        case = dict(op=op, rows=rows, c=c, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    pad=rng.choice([0, 0, 8, 5]))
        if op == "norm":
            case["out"] = rng.choice(["bf16", "e4m3", "e4m3", "f32"])
        return case
    train = op.endswith("train")
    n = "k" if op.startswith("linear") else "f"
    case = dict(op=op, c=_channels(rng, 64, 4096))
    case[n] = _channels(rng, 64, 8192)
    per_row = (6 if train else 2) * (1 if n == "k" else 2) * case["c"] * case[n]
    case["rows"] = _log(rng, 1, max(1, min(16384, MOST_FLOPS // per_row)))
    case["act"] = rng.choice(["silu", "gelu"]) if n == "f" else rng.choice(
        ["identity", "identity", "relu", "gelu", "silu"])
    if train:
        if n == "k":
            case["act"] = rng.choice(["identity", "gelu", "silu"])
            case["bias"] = rng.random() < 0.5
        return case
    case["dtype"] = rng.choice(["bf16", "bf16", "e4m3"])
    if n == "k":
        case["out"] = rng.choice(["bf16", "f32"]) if case["dtype"] == "bf16" else "bf16"
        case["bias"] = rng.random() < 0.5
        case["residual"] = rng.random() < 0.5
    return case


def work(case):
    rows, c, op = case["rows"], case["c"], case["op"]
    if op == "norm":
        e = SIZE[case["dtype"]]
        # read x and the residual, write their sum and the normed rows (and scales)
        scale = 4 * rows if case["out"] == "e4m3" else 0
        return {"bytes": rows * c * (3 * e + SIZE[case["out"]]) + 4 * c + scale, "flops": 6 * rows * c}
    if op == "norm_bwd":
        e = SIZE[case["dtype"]]
        return {"bytes": rows * c * 4 * e + 8 * c, "flops": 12 * rows * c}
    k = case["k"] if op.startswith("linear") else case["f"]
    nw = 1 if op.startswith("linear") else 2
    if op in ("linear", "gated"):
        e = SIZE[case["dtype"]]
        out = SIZE[case.get("out", "bf16")]
        b = e * (rows * c + nw * k * c) + out * rows * k
        if case["dtype"] == "e4m3":
            b += 4 * (rows + nw * k)
        if case.get("bias"):
            b += 4 * k
        if case.get("residual"):
            b += 2 * rows * k
        return {"bytes": b, "flops": 2 * nw * rows * c * k}
    # training: x, w and dy read, y, dx and dw written (and the residual, the biases)
    b = 2 * (2 * rows * c + 2 * nw * k * c + 2 * rows * k)
    if op == "linear_train":
        b += 2 * rows * k + (8 * k if case["bias"] else 0)
    return {"bytes": b, "flops": 6 * nw * rows * c * k}


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    t = torch.randn(*shape, generator=g, device=DEV)
    return (t * std if std != 1.0 else t).to(dtype)


def _rows(g, rows, c, pad, std, dtype):
    """rows x c values inside rows of c + pad elements."""
    if not pad:
        return _randn(g, rows, c, std=std, dtype=dtype)
    t = torch.empty(rows, c + pad, dtype=dtype, device=DEV)[:, :c]
    t.copy_(_randn(g, rows, c, std=std))
    return t


def _quantized(t):
    """E4M3 values and one scale for each row."""
    scale = t.abs().amax(1, keepdim=True).clamp_min(1e-30) / E4M3_MAX
    return (t / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale[:, 0].contiguous()


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rows, c, op = case["rows"], case["c"], case["op"]
    s = {}
    if op.startswith("norm"):
        dt, pad = TYPES[case["dtype"]], case["pad"]
        s["gamma"] = 1.0 + 0.2 * _randn(g, c)
        if op == "norm":
            s["x"] = _rows(g, rows, c, pad, 1.0, dt)
            s["residual"] = _rows(g, rows, c, pad, 2.0, dt)
        else:
            s["dy"] = _rows(g, rows, c, pad, 1.0, dt)
            s["total"] = _rows(g, rows, c, pad, 2.0, dt)
            s["dtotal"] = _rows(g, rows, c, pad, 1.0, dt)
        return s
    bf = torch.bfloat16
    n = case["k"] if op.startswith("linear") else 2 * case["f"]  # gate filters, then up filters
    x, w = _randn(g, rows, c), _randn(g, n, c, std=c ** -0.5)
    if case.get("dtype") == "e4m3":
        s["x"], s["x_scale"] = _quantized(x)
        s["w"], s["w_scale"] = _quantized(w)
    else:
        s["x"], s["w"] = x.to(bf), w.to(bf)
    if case.get("bias"):
        s["bias"] = _randn(g, n, std=0.3)
    if case.get("residual") or op == "linear_train":
        s["residual"] = _randn(g, rows, n, std=2.0, dtype=bf)
    if op.endswith("train"):
        s["dy"] = _randn(g, rows, n if op == "linear_train" else case["f"], dtype=bf)
    return s


_handle = None


def _plan(case, s):
    """The operators a program keeps for these shapes, and its output buffers."""
    global _handle
    from deep_learning_convolution_gb300 import api
    if _handle is None:
        _handle = api.Handle()
    h, op, rows, c = _handle, case["op"], case["rows"], case["c"]

    def new(*shape, like=None, dtype=torch.bfloat16):
        if like is not None:
            return torch.empty_strided(like.shape, like.stride(), dtype=like.dtype, device=DEV)
        return torch.empty(*shape, dtype=dtype, device=DEV)

    if op == "norm":
        s["total"] = new(like=s["x"])
        s["y"] = new(rows, c, dtype=TYPES[case["out"]])
        s["scale"] = new(rows, dtype=torch.float32) if case["out"] == "e4m3" else None
        s["op"] = api.RmsNormForward(h, s["x"], s["y"], residual=s["residual"], total=s["total"],
                                     eps=EPS)
    elif op == "norm_bwd":
        s["dx"] = new(like=s["total"])
        s["dgamma"] = new(c, dtype=torch.float32)
        s["op"] = api.RmsNormBackward(h, s["dy"], s["total"], s["dx"], dtotal=s["dtotal"], eps=EPS)
    elif op == "linear":
        s["y"] = new(rows, case["k"], dtype=TYPES[case["out"]])
        s["op"] = api.LinearForward(h, s["x"], s["w"], s["y"], act=case["act"],
                                    residual=s.get("residual"))
    elif op == "gated":
        s["y"] = new(rows, case["f"])
        s["op"] = api.GatedForward(h, s["x"], s["w"], s["y"], act=case["act"])
    else:
        linear = op == "linear_train"
        n = s["w"].shape[0]
        s["y"] = new(rows, case["k"] if linear else case["f"])
        s["z"] = None
        if case["act"] != "identity":
            # what the backward pass reads; in FP32 where a bias gradient is summed from it
            s["z"] = new(rows, n, dtype=torch.float32 if case.get("bias") else torch.bfloat16)
        s["dx"], s["dw"] = new(like=s["x"]), new(like=s["w"])
        s["dbias"] = new(n, dtype=torch.float32) if case.get("bias") else None
        if linear:
            s["op"] = api.LinearForward(h, s["x"], s["w"], s["y"], act=case["act"],
                                        residual=s["residual"], z=s["z"])
            s["back"] = api.LinearBackward(h, s["x"], s["w"], s["dy"], s["dx"], s["dw"], z=s["z"],
                                           act=case["act"])
        else:
            s["op"] = api.GatedForward(h, s["x"], s["w"], s["y"], act=case["act"], z=s["z"])
            s["back"] = api.GatedBackward(h, s["x"], s["w"], s["dy"], s["dx"], s["dw"], z=s["z"],
                                          act=case["act"])


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _plan(case, s)
    return s


def _run_own(s):
    op = s["case"]["op"]
    if op == "norm":
        s["op"](s["x"], s["gamma"], s["y"], residual=s["residual"], total=s["total"],
                scale=s["scale"])
        return [s["total"], s["y"]] + ([s["scale"]] if s["scale"] is not None else [])
    if op == "norm_bwd":
        s["op"](s["dy"], s["total"], s["gamma"], s["dx"], dgamma=s["dgamma"], dtotal=s["dtotal"])
        return [s["dx"], s["dgamma"]]
    if op == "linear":
        s["op"](s["x"], s["w"], s["y"], bias=s.get("bias"), residual=s.get("residual"),
                x_scale=s.get("x_scale"), w_scale=s.get("w_scale"))
        return [s["y"]]
    if op == "gated":
        s["op"](s["x"], s["w"], s["y"], x_scale=s.get("x_scale"), w_scale=s.get("w_scale"))
        return [s["y"]]
    if op == "linear_train":
        s["op"](s["x"], s["w"], s["y"], bias=s.get("bias"), residual=s["residual"], z=s["z"])
    else:
        s["op"](s["x"], s["w"], s["y"], z=s["z"])
    s["back"](s["x"], s["w"], s["dy"], s["dx"], s["dw"], dbias=s["dbias"], z=s["z"])
    return [s["y"], s["dx"], s["dw"]] + ([s["dbias"]] if s["dbias"] is not None else [])


# ---- the plain form: elementary operations in FP32 -------------------------------

def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (
            1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _operands(s):
    x, w = s["x"].float(), s["w"].float()
    if "x_scale" in s:
        x, w = x * s["x_scale"][:, None], w * s["w_scale"][:, None]
    return x, w


def _run_plain(s):
    case, bf = s["case"], torch.bfloat16
    op = case["op"]
    if op == "norm":
        t = s["x"].float() + s["residual"].float()
        y = t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * s["gamma"]
        total = t.to(s["x"].dtype)
        if case["out"] != "e4m3":
            return [total, y.to(TYPES[case["out"]])]
        scale = y.abs().amax(1, keepdim=True).clamp_min(1e-30) / E4M3_MAX
        q = (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return [total, q, scale[:, 0]]
    if op == "norm_bwd":
        t, dy = s["total"].float(), s["dy"].float()
        r = torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
        n = t * r
        d = dy * s["gamma"]
        dx = r * (d - n * (d * n).mean(1, keepdim=True)) + s["dtotal"].float()
        return [dx.to(s["total"].dtype), (dy * n).sum(0)]
    x, w = _operands(s)
    z = x @ w.t()
    if "bias" in s:
        z = z + s["bias"]
    if op.startswith("linear"):
        y = _act(z, case["act"])
        if "residual" in s:
            y = y + s["residual"].float()
        y = y.to(TYPES[case.get("out", "bf16")])
        if op == "linear":
            return [y]
        dz = s["dy"].float()
        if case["act"] != "identity":
            dz = dz * _act_grad(z, case["act"])
        dbias = [dz.sum(0)] if "bias" in s else []
        return [y, (dz @ w).to(bf), (dz.t() @ x).to(bf)] + dbias
    f = case["f"]
    gate, up = z[:, :f], z[:, f:]
    a = _act(gate, case["act"])
    y = (a * up).to(bf)
    if op == "gated":
        return [y]
    dy = s["dy"].float()
    dz = torch.cat([dy * up * _act_grad(gate, case["act"]), dy * a], 1)
    return [y, (dz @ w).to(bf), (dz.t() @ x).to(bf)]


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---- the definition in FP64 -------------------------------------------------------

def _phi(v):
    """The standard normal distribution function."""
    return 0.5 * torch.erfc(v * -(0.5 ** 0.5))


def _act64(v, act):
    """(f(v), f'(v))"""
    if act == "identity":
        return v, torch.ones_like(v)
    if act == "relu":
        return torch.where(v > 0, v, 0.0), torch.where(v > 0, 1.0, 0.0)
    if act == "silu":
        sg = torch.sigmoid(v)
        return v * sg, sg + v * sg * torch.sigmoid(-v)
    p = _phi(v)
    return v * p, p + v * torch.exp(-v.square() / 2) / (2 * math.pi) ** 0.5


def exact(case, seed):
    if work(case)["flops"] > MOST_FLOPS:
        return None
    s = {k: v.double() for k, v in _inputs(case, seed).items()}
    op = case["op"]
    if op == "norm":
        total = s["x"] + s["residual"]
        rms = (total.square().sum(1) / case["c"] + EPS).sqrt()
        y = torch.einsum("rc,r,c->rc", total, 1 / rms, s["gamma"])
        if case["out"] == "e4m3":  # the 8-bit values depend on ties of the rounding
            return [total, None, y.abs().amax(1) / E4M3_MAX]
        return [total, y]
    if op == "norm_bwd":
        t, dy = s["total"], s["dy"]
        rms = (t.square().sum(1) / case["c"] + EPS).sqrt()
        dgamma = torch.einsum("rc,rc,r->c", dy, t, 1 / rms)
        dot = torch.einsum("rc,rc,c->r", dy, t, s["gamma"])
        dx = dy * s["gamma"] / rms[:, None] - t * (dot / (case["c"] * rms ** 3))[:, None]
        return [dx + s["dtotal"], dgamma]
    x, w = s["x"], s["w"]
    if "x_scale" in s:
        x = torch.einsum("rc,r->rc", x, s["x_scale"])
        w = torch.einsum("kc,k->kc", w, s["w_scale"])
    z = torch.einsum("rc,kc->rk", x, w)
    if "bias" in s:
        z = z + s["bias"][None]
    if op.startswith("linear"):
        y, slope = _act64(z, case["act"])
        if "residual" in s:
            y = s["residual"] + y
        if op == "linear":
            return [y]
        dz = slope * s["dy"]
    else:
        gate, up = z.chunk(2, 1)
        a, slope = _act64(gate, case["act"])
        y = a * up
        if op == "gated":
            return [y]
        dz = torch.hstack([slope * up, a]) * s["dy"].repeat(1, 2)
    out = [y, torch.einsum("rk,kc->rc", dz, w), torch.einsum("rk,rc->kc", dz, x)]
    return out + ([dz.sum(0)] if "bias" in s else [])
