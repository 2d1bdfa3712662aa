"""Timed cases of the channel operators at the ends of a trained network and
between its layers: layer norm with the residual's addition, dropout from a
counter-based generator, the embedding of tokens, and softmax cross entropy on
top of a linear layer, with their gradients.

Every tensor is rows (pixels or tokens) by channels, channels innermost.  With
``own`` false ``run`` computes a case in elementary torch operations in FP32;
with ``own`` true it calls this package's operators.  ``exact`` is the
definition in FP64, written apart from the plain form.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}

# the largest listed case's operations; drawn cases stay below them
MOST_FLOPS = 6 * 4096 * 2048 * 131072


def listed():
    return [
        # one token of a serving step: latency
        dict(name="layer_token", op="layer", rows=1, c=4096, dtype="bf16", out="bf16", pad=0),
        # the residual stream of an image batch before a projection in 8 bits
        dict(name="layer_pixels_e4m3", op="layer", rows=65536, c=768, dtype="bf16", out="e4m3", pad=0),
        # training, the tokens of a few long sequences
        dict(name="layer_backward", op="layer_bwd", rows=16384, c=2048, dtype="bf16", pad=0),
        # training in FP32, odd channels, rows with a pitch of their own
        dict(name="layer_backward_odd", op="layer_bwd", rows=4001, c=333, dtype="f32", pad=3),
        # a block's output dropped on its way into the residual stream
        dict(name="dropout_stream", op="dropout", rows=16384, c=4096, dtype="bf16", p=0.1, residual=True,
             pad=0),
        # the gradient of a classifier's hidden layer, sizes that no vector likes
        dict(name="dropout_backward_odd", op="dropout_bwd", rows=777, c=1001, dtype="f32", p=0.5, pad=0),
        # the tokens of one decoding step
        dict(name="embedding_decode", op="embed", rows=64, c=4096, v=131072, dtype="bf16", out="bf16",
             scale=64.0, pad=0),
        # a training step's tokens: the whole table's gradient
        dict(name="embedding_backward", op="embed_bwd", rows=16384, c=2048, v=65536, dtype="bf16",
             out="bf16", scale=1.0, accumulate=False, pad=0),
        # a small FP32 table shared with another layer, whose gradient is there already
        dict(name="embedding_accumulate", op="embed_bwd", rows=5000, c=300, v=1003, dtype="f32",
             out="f32", scale=17.3, accumulate=True, pad=0),
        # a classifier's training step on one batch of images
        dict(name="entropy_classifier_step", op="entropy_train", rows=256, c=2048, v=1000, bias=True),
        # how likely the tokens of a few sequences are
        dict(name="entropy_score", op="entropy", rows=32, c=4096, v=131072, bias=False),
        # a training step over a large vocabulary
        dict(name="entropy_vocabulary_step", op="entropy_train", rows=4096, c=2048, v=131072, bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _channels(rng, lo, hi):
    c = _log(rng, lo, hi)
    return c if rng.random() < 0.25 else max(16, c // 16 * 16)


def draw(rng):
    op = rng.choice(["layer", "layer_bwd", "dropout", "dropout_bwd", "embed", "embed_bwd", "entropy",
                     "entropy", "entropy_train", "entropy_train"])
    pad = rng.choice([0, 0, 8, 5])
    if op.startswith("layer"):
        c = _channels(rng, 64, 8192)
        case = dict(op=op, rows=_log(rng, 1, 65536 * 768 // c), c=c, pad=pad,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "layer":
            case["out"] = rng.choice(["bf16", "bf16", "e4m3", "f32"])
        return case
    if op.startswith("dropout"):
        c = _channels(rng, 16, 8192)
        case = dict(op=op, rows=_log(rng, 1, 16384 * 4096 // c), c=c, pad=pad,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), p=rng.choice([0.0, 0.05, 0.1, 0.2, 0.5, 0.9]))
        if op == "dropout":
            case["residual"] = rng.random() < 0.5
        return case
    if op.startswith("embed"):
        c = _channels(rng, 32, 4096)
        case = dict(op=op, rows=_log(rng, 1, 16384), c=c, v=_log(rng, 100, min(131072, 65536 * 2048 // c)),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32"]),
                    scale=rng.choice([1.0, math.sqrt(c)]), pad=pad)
        if op == "embed_bwd":
            case["accumulate"] = rng.random() < 0.3
        return case
    c, v = _channels(rng, 32, 4096), _log(rng, 10, 131072)
    if rng.random() < 0.5:
        v = max(16, v // 16 * 16)
    per_row = (6 if op == "entropy_train" else 2) * c * v
    return dict(op=op, c=c, v=v, rows=_log(rng, 1, max(1, min(8192, MOST_FLOPS // per_row))),
                bias=rng.random() < 0.4)


def work(case):
    rows, c, op = case["rows"], case["c"], case["op"]
    n = rows * c
    if op == "layer":
        e = SIZE[case["dtype"]]
        # read x and the residual, write their sum and the normed rows (and scales)
        scale = 4 * rows if case["out"] == "e4m3" else 0
        return {"bytes": n * (3 * e + SIZE[case["out"]]) + 8 * c + scale, "flops": 9 * n}
    if op == "layer_bwd":
        return {"bytes": n * 4 * SIZE[case["dtype"]] + 12 * c, "flops": 16 * n}
    if op.startswith("dropout"):
        streams = 3 if case.get("residual") else 2
        return {"bytes": n * streams * SIZE[case["dtype"]] + 16, "flops": 2 * n}
    if op == "embed":
        return {"bytes": n * (SIZE[case["dtype"]] + SIZE[case["out"]]) + 8 * rows, "flops": n}
    if op == "embed_bwd":
        # every row of the table's gradient is written; where it accumulates, the tokens'
        # rows are read and written (as many of them as tokens, or the whole table)
        touched = 2 * min(rows, case["v"]) if case["accumulate"] else case["v"]
        return {"bytes": n * SIZE[case["dtype"]] + touched * c * SIZE[case["out"]] + 8 * rows, "flops": 2 * n}
    v = case["v"]
    b = 2 * (n + v * c) + 16 * rows + (4 * v if case["bias"] else 0)
    if op == "entropy":
        return {"bytes": b, "flops": 2 * n * v}
    return {"bytes": 2 * b, "flops": 6 * n * v}


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


def _indices(g, rows, n):
    """rows numbers below n, as frequent as words are (the i-th of them with probability
    about 1 / i), in no order of size; a few rows are padding, -1."""
    rank = torch.exp(torch.rand(rows, generator=g, device=DEV, dtype=torch.float64) * math.log(n))
    step = 1 + 2 * (n // 5)
    while math.gcd(step, n) != 1:
        step += 1
    index = (rank.long().clamp(max=n) - 1).clamp_min(0) * step % n
    return torch.where(torch.rand(rows, generator=g, device=DEV) < 0.03, -1, index)


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rows, c, op, pad = case["rows"], case["c"], case["op"], case.get("pad", 0)
    s = {}
    if op.startswith("layer"):
        dt = TYPES[case["dtype"]]
        s["gamma"] = 1.0 + 0.2 * _randn(g, c)
        if op == "layer":
            s["beta"] = 0.2 * _randn(g, c)
            s["x"] = _rows(g, rows, c, pad, 1.0, dt)
            s["residual"] = _rows(g, rows, c, pad, 2.0, dt)
        else:
            s["dy"] = _rows(g, rows, c, pad, 1.0, dt)
            s["total"] = _rows(g, rows, c, pad, 2.0, dt)
            s["dtotal"] = _rows(g, rows, c, pad, 1.0, dt)
        return s
    if op.startswith("dropout"):
        dt = TYPES[case["dtype"]]
        s["x" if op == "dropout" else "dy"] = _rows(g, rows, c, pad, 1.0, dt)
        if case.get("residual"):
            s["residual"] = _rows(g, rows, c, pad, 2.0, dt)
        # the generator's seed, and a number for this layer and step
        s["random"] = torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=g, device=DEV)
        return s
    if op.startswith("embed"):
        v = case["v"]
        s["tokens"] = _indices(g, rows, v)
        if op == "embed":
            s["table"] = _randn(g, v, c, std=c ** -0.5, dtype=TYPES[case["dtype"]])
        else:
            s["dy"] = _rows(g, rows, c, pad, 1.0, TYPES[case["dtype"]])
            if case["accumulate"]:
                s["before"] = _randn(g, v, c, dtype=TYPES[case["out"]])
        return s
    v, bf = case["v"], torch.bfloat16
    s["target"] = _indices(g, rows, v)
    w = _randn(g, v, c, std=c ** -0.5)
    # rows that know something about their class, as they do in training
    x = _randn(g, rows, c) + w[s["target"].clamp_min(0)] * (3.0 * torch.rand(rows, 1, generator=g, device=DEV))
    s["x"], s["w"] = x.to(bf), w.to(bf)
    if case["bias"]:
        s["bias"] = _randn(g, v, std=0.5)
    if op == "entropy_train":  # the mean over the rows, each with a weight
        s["dloss"] = (0.5 + torch.rand(rows, generator=g, device=DEV)) / rows
    return s


_handle = None


def _plan(case, s):
    """The operators a program keeps for these shapes, and its output buffers."""
    global _handle
    from deep_learning_convolution_gb300 import api
    if _handle is None:
        _handle = api.Handle()
    h, op, rows, c = _handle, case["op"], case["rows"], case["c"]

    def new(*shape, like=None, dtype=torch.float32):
        if like is not None:
            return torch.empty_strided(like.shape, like.stride(), dtype=like.dtype, device=DEV)
        return torch.empty(*shape, dtype=dtype, device=DEV)

    if op == "layer":
        s["total"] = new(like=s["x"])
        s["y"] = new(rows, c, dtype=TYPES[case["out"]])
        s["scale"] = new(rows) if case["out"] == "e4m3" else None
        s["op"] = api.LayerNormForward(h, s["x"], s["y"], residual=s["residual"], total=s["total"], eps=EPS)
    elif op == "layer_bwd":
        s["dx"], s["dgamma"], s["dbeta"] = new(like=s["total"]), new(c), new(c)
        s["op"] = api.LayerNormBackward(h, s["dy"], s["total"], s["dx"], dtotal=s["dtotal"], eps=EPS)
    elif op == "dropout":
        s["y"] = new(like=s["x"])
        s["op"] = api.DropoutForward(h, s["x"], s["y"], p=case["p"], residual=s.get("residual"))
    elif op == "dropout_bwd":
        s["dx"] = new(like=s["dy"])
        s["op"] = api.DropoutBackward(h, s["dy"], s["dx"], p=case["p"])
    elif op == "embed":
        s["y"] = new(rows, c + case["pad"], dtype=TYPES[case["out"]])[:, :c]
        s["op"] = api.EmbeddingForward(h, s["tokens"], s["table"], s["y"], scale=case["scale"])
    elif op == "embed_bwd":
        s["dtable"] = new(case["v"], c, dtype=TYPES[case["out"]])
        s["op"] = api.EmbeddingBackward(h, s["tokens"], s["dy"], s["dtable"], scale=case["scale"],
                                        accumulate=case["accumulate"])
    else:
        s["loss"], s["lse"] = new(rows), new(rows)
        s["op"] = api.CrossEntropyForward(h, s["x"], s["w"], s["target"])
        if op == "entropy_train":
            s["dx"], s["dw"] = new(like=s["x"]), new(like=s["w"])
            s["dbias"] = new(case["v"]) if case["bias"] else None
            s["back"] = api.CrossEntropyBackward(h, s["x"], s["w"], s["target"], s["dx"], s["dw"])


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _plan(case, s)
    return s


def _run_own(s):
    case = s["case"]
    op = case["op"]
    if op == "layer":
        s["op"](s["x"], s["gamma"], s["y"], beta=s["beta"], residual=s["residual"], total=s["total"],
                scale=s["scale"])
        return [s["total"], s["y"]] + ([s["scale"]] if s["scale"] is not None else [])
    if op == "layer_bwd":
        s["op"](s["dy"], s["total"], s["gamma"], s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"],
                dtotal=s["dtotal"])
        return [s["dx"], s["dgamma"], s["dbeta"]]
    if op == "dropout":
        s["op"](s["x"], s["random"], s["y"], residual=s.get("residual"))
        return [s["y"]]
    if op == "dropout_bwd":
        s["op"](s["dy"], s["random"], s["dx"])
        return [s["dx"]]
    if op == "embed":
        s["op"](s["tokens"], s["table"], s["y"])
        return [s["y"]]
    if op == "embed_bwd":
        if case["accumulate"]:
            s["dtable"].copy_(s["before"])  # what the other layer left there
        s["op"](s["tokens"], s["dy"], s["dtable"])
        return [s["dtable"]]
    s["op"](s["x"], s["w"], s["target"], s["loss"], s["lse"], bias=s.get("bias"))
    if op == "entropy":
        return [s["loss"], s["lse"]]
    s["back"](s["x"], s["w"], s["target"], s["lse"], s["dloss"], s["dx"], s["dw"], bias=s.get("bias"),
              dbias=s["dbias"])
    return [s["loss"], s["lse"], s["dx"], s["dw"]] + ([s["dbias"]] if s["dbias"] is not None else [])


# ---- the plain form: elementary operations in FP32 -------------------------------

_WORD = 0xFFFFFFFF


def _philox_words(random, rows, c):
    """The generator's words of rows x c elements: Philox 4x32 with ten rounds (Salmon et
    al., 2011), the key being the seed, the counter (c / 4, row, step's low and high
    word); element c takes word c mod 4."""
    groups = (c + 3) // 4
    shape = (rows, groups)
    x0 = torch.arange(groups, device=DEV).expand(shape)
    x1 = torch.arange(rows, device=DEV)[:, None].expand(shape)
    k0, k1 = random[0] & _WORD, (random[0] >> 32) & _WORD
    x2, x3 = (random[1] & _WORD).expand(shape), ((random[1] >> 32) & _WORD).expand(shape)
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = ((b >> 32) & _WORD) ^ x1 ^ k0, b & _WORD, ((a >> 32) & _WORD) ^ x3 ^ k1, a & _WORD
        k0, k1 = (k0 + 0x9E3779B9) & _WORD, (k1 + 0xBB67AE85) & _WORD
    return torch.stack([x0, x1, x2, x3], 2).view(rows, 4 * groups)[:, :c]


def _run_plain(s):
    case, bf = s["case"], torch.bfloat16
    op, rows, c = case["op"], case["rows"], case["c"]
    if op == "layer":
        t = s["x"].float() + s["residual"].float()
        d = t - t.mean(1, keepdim=True)
        y = d * torch.rsqrt((d * d).mean(1, keepdim=True) + EPS) * s["gamma"] + s["beta"]
        total = t.to(s["x"].dtype)
        if case["out"] != "e4m3":
            return [total, y.to(TYPES[case["out"]])]
        scale = y.abs().amax(1, keepdim=True).clamp_min(1e-30) / E4M3_MAX
        q = (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return [total, q, scale[:, 0]]
    if op == "layer_bwd":
        t, dy = s["total"].float(), s["dy"].float()
        n = t - t.mean(1, keepdim=True)
        r = torch.rsqrt((n * n).mean(1, keepdim=True) + EPS)
        n = n * r
        d = dy * s["gamma"]
        dx = r * (d - d.mean(1, keepdim=True) - n * (d * n).mean(1, keepdim=True)) + s["dtotal"].float()
        return [dx.to(s["total"].dtype), (dy * n).sum(0), dy.sum(0)]
    if op.startswith("dropout"):
        x = s["x" if op == "dropout" else "dy"]
        border = math.floor(case["p"] * 2 ** 32)
        keep = _philox_words(s["random"], rows, c) >= border
        y = torch.where(keep, x.float() * (2 ** 32 / (2 ** 32 - border)), 0.0)
        if "residual" in s:
            y = y + s["residual"].float()
        return [y.to(x.dtype)]
    if op == "embed":
        y = s["table"][s["tokens"].clamp_min(0)].float() * case["scale"]
        return [torch.where((s["tokens"] >= 0)[:, None], y, 0.0).to(TYPES[case["out"]])]
    if op == "embed_bwd":
        dt, there = torch.zeros(case["v"], c, device=DEV), (s["tokens"] >= 0)[:, None]
        dt.index_add_(0, s["tokens"].clamp_min(0), torch.where(there, s["dy"].float(), 0.0))
        dt = dt * case["scale"]
        if case["accumulate"]:
            dt = dt + s["before"].float()
        return [dt.to(TYPES[case["out"]])]
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if "bias" in s:
        z = z + s["bias"]
    counted, target = (s["target"] >= 0)[:, None], s["target"].clamp_min(0)[:, None]
    top = z.amax(1, keepdim=True)
    chosen = z.gather(1, target)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    loss = torch.where(counted, lse - chosen, 0.0)[:, 0]
    if op == "entropy":
        return [loss, lse[:, 0]]
    dz = e / total
    dz.scatter_add_(1, target, torch.full_like(chosen, -1.0))
    dz = dz * torch.where(counted, s["dloss"][:, None], 0.0)
    dbias = [dz.sum(0)] if "bias" in s else []
    return [loss, lse[:, 0], (dz @ w).to(bf), (dz.t() @ x).to(bf)] + dbias


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---- the definition in FP64 -------------------------------------------------------

def _kept(case, random):
    """Which elements dropout keeps, by the generator's definition on 64-bit unsigned numbers."""
    rows, c = case["rows"], case["c"]
    seed, step = (int(r) % 2 ** 64 for r in random.cpu())
    word, shift = np.uint64(2 ** 32 - 1), np.uint64(32)
    border = np.uint64(int(case["p"] * 2 ** 32))
    keep = np.empty((rows, (c + 3) // 4, 4), dtype=bool)
    column = np.arange(keep.shape[1], dtype=np.uint64)[None, :]
    most = max(1, 2 ** 20 // keep.shape[1])
    for r0 in range(0, rows, most):
        row = np.arange(r0, min(rows, r0 + most), dtype=np.uint64)[:, None]
        counter = [column + 0 * row, row + 0 * column, np.uint64(step % 2 ** 32), np.uint64(step >> 32)]
        for i in range(10):
            key = [np.uint64((seed + i * 0x9E3779B9) % 2 ** 32),
                   np.uint64(((seed >> 32) + i * 0xBB67AE85) % 2 ** 32)]
            left, right = np.uint64(0xD2511F53) * counter[0], np.uint64(0xCD9E8D57) * counter[2]
            counter = [(right >> shift) ^ counter[1] ^ key[0], right & word,
                       (left >> shift) ^ counter[3] ^ key[1], left & word]
        for j in range(4):
            keep[r0:r0 + most, :, j] = counter[j] >= border
    return torch.from_numpy(keep.reshape(rows, -1)[:, :c].copy()).to(DEV)


def exact(case, seed):
    if work(case)["flops"] > MOST_FLOPS:
        return None
    op, rows, c = case["op"], case["rows"], case["c"]
    s = {k: v.double() if v.is_floating_point() else v for k, v in _inputs(case, seed).items()}
    if op == "layer":
        total = s["x"] + s["residual"]
        var, mean = torch.var_mean(total, 1, correction=0, keepdim=True)
        y = torch.addcmul(s["beta"], (total - mean) / (var + EPS).sqrt(), s["gamma"])
        if case["out"] == "e4m3":  # the 8-bit values depend on ties of the rounding
            return [total, None, y.abs().amax(1) / E4M3_MAX]
        return [total, y]
    if op == "layer_bwd":
        dy, gamma = s["dy"], s["gamma"]
        var, mean = torch.var_mean(s["total"], 1, correction=0, keepdim=True)
        sigma = (var + EPS).sqrt()
        n = (s["total"] - mean) / sigma
        dot = torch.einsum("rc,rc,c->r", dy, n, gamma)[:, None] / c
        level = (dy @ gamma)[:, None] / c
        dx = (dy * gamma - level - n * dot) / sigma
        return [dx + s["dtotal"], torch.einsum("rc,rc->c", dy, n), dy.sum(0)]
    if op.startswith("dropout"):
        border = int(case["p"] * 2 ** 32)
        x = s["x" if op == "dropout" else "dy"]
        y = x * _kept(case, s["random"]) / (1 - border / 2 ** 32)
        return [s["residual"] + y if "residual" in s else y]
    if op == "embed":
        y = torch.zeros(rows, c, dtype=torch.float64, device=DEV)
        there = s["tokens"] >= 0
        y[there] = case["scale"] * s["table"].index_select(0, s["tokens"][there])
        return [y]
    if op == "embed_bwd":
        there = s["tokens"] >= 0
        dt = torch.zeros(case["v"], c, dtype=torch.float64, device=DEV)
        dt.index_put_((s["tokens"][there],), s["dy"][there] * case["scale"], accumulate=True)
        return [dt + s["before"] if case["accumulate"] else dt]
    z = torch.einsum("rc,kc->rk", s["x"], s["w"])
    if "bias" in s:
        z += s["bias"]
    counted = torch.nonzero(s["target"] >= 0)[:, 0]
    target = s["target"][counted]
    lse = torch.logsumexp(z, 1)
    loss = torch.zeros_like(lse)
    loss[counted] = lse[counted] - z[counted, target]
    if op == "entropy":
        return [loss, lse]
    z.sub_(lse[:, None]).exp_()  # the probabilities, from here on
    z[counted, target] -= 1.0
    weight = torch.zeros_like(lse)
    weight[counted] = s["dloss"][counted]
    z *= weight[:, None]
    out = [loss, lse, torch.einsum("rk,kc->rc", z, s["w"]), torch.einsum("rk,rc->kc", z, s["x"])]
    return out + ([z.sum(0)] if "bias" in s else [])
