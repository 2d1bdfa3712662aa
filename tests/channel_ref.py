"""FP64 definitions of the channel operators on CPU tensors, with the sums of
absolute terms that the tests' error bounds are made of.

Error model (derived from the formats, not from runs):

* an FP32 sum of n terms by partial chains: relative to the sum of absolute
  terms at most 2^-24 * (length of the longest chain + tree levels + 2);
* products on the tensor cores: exact products, FP32 accumulation, 1e-5 of the
  sum of absolute terms (the bound the convolution tests use);
* storing BF16: half a unit in the last place, 2^-8 of the value at most;
  E4M3: 2^-4 of the value, or half the smallest step 2^-9 of the scale;
* activations in FP32: 4e-6 of their size, and slopes at most SLOPE.
"""
from __future__ import annotations

import math

import torch

BF16 = 2.0 ** -8
E4M3 = 2.0 ** -4
U32 = 2.0 ** -24
TC = 1e-5
ACT_REL = 4e-6
SLOPE = 1.13  # the largest |f'| of silu (1.0998) and gelu (1.1290)


def act(v, kind):
    """(f(v), f'(v)) in FP64."""
    if kind == "identity":
        return v, torch.ones_like(v)
    if kind == "relu":
        return v.clamp(min=0), (v > 0).double()
    if kind == "sigmoid":
        p = torch.sigmoid(v)
        return p, p * (1 - p)
    if kind == "tanh":
        t = torch.tanh(v)
        return t, 1 - t * t
    if kind == "silu":
        p = torch.sigmoid(v)
        return v * p, p * (1 + v * (1 - p))
    if kind == "gelu":
        p = 0.5 * torch.erfc(-v / math.sqrt(2))
        return v * p, p + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    raise ValueError(kind)


def stored(ref, dtype):
    """Rounding error of storing `ref` in `dtype`."""
    return {torch.float32: U32, torch.bfloat16: BF16}[dtype] * ref.abs() + 1e-30


def norm(x, r, gamma, eps):
    t = x if r is None else x + r
    rho = (t.square().mean(1, keepdim=True) + eps).rsqrt()
    return t, gamma * t * rho


def norm_rel(c):
    """Relative error of a norm of c channels before storing: the longest
    partial chain is c / 8 terms (at most 32 in registers), half of it in rho."""
    return U32 * (c / 8 + 64)


def norm_backward(dy, t, gamma, dt, eps):
    """dx, dgamma and the sums of absolute terms of each."""
    c = t.shape[1]
    rho = (t.square().mean(1, keepdim=True) + eps).rsqrt()
    d = dy * gamma
    dx = rho * d - t * rho ** 3 * (d * t).mean(1, keepdim=True)
    bx = rho * d.abs() + t.abs() * rho ** 3 * (d * t).abs().sum(1, keepdim=True) / c
    if dt is not None:
        dx, bx = dx + dt, bx + dt.abs()
    n = dy * t * rho
    return dx, n.sum(0), bx, n.abs().sum(0)


def product(x, w, bias=None, sx=None, sw=None):
    """z and the bound of its error."""
    if sx is not None:
        x, w = x * sx[:, None], w * sw[:, None]
    z, b = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, b = z + bias, b + bias.abs()
    return z, TC * b + 1e-6


def linear(z, ez, kind, r, dtype):
    f, _ = act(z, kind)
    y = f if r is None else f + r
    err = SLOPE * ez + ACT_REL * f.abs() + stored(y, dtype) + (U32 * r.abs() if r is not None else 0)
    return y, err


def gated(z, ez, kind, dtype):
    g, u = z.chunk(2, 1)
    eg, eu = ez.chunk(2, 1)
    f, _ = act(g, kind)
    y = f * u
    ef = SLOPE * eg + ACT_REL * f.abs()
    return y, ef * (u.abs() + eu) + f.abs() * eu + stored(y, dtype) + U32 * y.abs()


def act_grad(dy, z, kind, is_gated):
    """dz and the bound of its FP32 error (before it is rounded)."""
    if not is_gated:
        if kind == "identity":
            return dy, 0 * dy.abs()
        f, df = act(z, kind)
        # f' is a sum of terms of size 1 + |z| at most
        return dy * df, ACT_REL * dy.abs() * (1 + z.abs())
    g, u = z.chunk(2, 1)
    f, df = act(g, kind)
    e = ACT_REL * dy.abs() * (1 + g.abs())
    return torch.cat([dy * u * df, dy * f], 1), torch.cat([e * u.abs(), e], 1)


def backward(x, w, dz, edz, dx_dtype, dw_dtype):
    """dx, dw, dbias with error bounds; dz enters the products in BF16."""
    ez = edz + BF16 * dz.abs() + 1e-30
    dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    ex = ez @ w.abs() + TC * (dz.abs() @ w.abs()) + stored(dx, dx_dtype) + 1e-6
    ew = ez.t() @ x.abs() + TC * (dz.abs().t() @ x.abs()) + stored(dw, dw_dtype) + 1e-6
    eb = edz.sum(0) + TC * dz.abs().sum(0) + 1e-6
    return (dx, ex), (dw, ew), (db, eb)
