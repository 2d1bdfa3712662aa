"""FP64 definitions of layer norm, dropout, embedding and softmax cross entropy
(tensors of any device), with the bounds of the kernels' errors.

Error model, derived from the formats and the sums' lengths before any run
(channel_ref has the constants):

* FP32 sums of n terms: U32 times the chain's length times the sum of absolute
  terms; a row's chain is c / 8 + 64 terms, a column's as long as its rows;
* centred values carry the mean's error, so their bound is absolute: U32 * chain *
  mean |t|, however small the value;
* logits: TC of the sum of absolute products, as in the linear layer; log-sum-exp: the
  largest error of a logit that counts, and 4 U32 of its own size and of the
  rescaling's exponents; probabilities: the errors of z and lse as a factor, and 4e-6
  for the exponential of arguments up to 88 (2^-24 * 88 twice);
* dz enters the products rounded to BF16.
"""
from __future__ import annotations

import numpy as np
import torch

from tests.channel_ref import BF16, TC, U32, stored


def layer_norm(x, r, gamma, beta, eps):
    """t, y and the bound of y's FP32 error."""
    t = x if r is None else x + r
    c = t.shape[1]
    mean = t.mean(1, keepdim=True)
    d = t - mean
    var = d.square().mean(1, keepdim=True) + eps
    rho = var.rsqrt()
    y = gamma * d * rho + (0 if beta is None else beta)
    ed, rel = centring(t, d, var, c)
    err = gamma.abs() * rho * (ed + d.abs() * (rel + 4 * U32)) + 2 * U32 * y.abs()
    if beta is not None:
        err = err + U32 * beta.abs()
    return t, y, err


def centring(t, d, var, c):
    """Bounds of the centred values' absolute and of rho's relative error."""
    chain = c / 8 + 64
    ed = U32 * (chain * t.abs().mean(1, keepdim=True) + 2 * t.abs() + d.abs())
    return ed, U32 * chain + (d.abs() * ed).mean(1, keepdim=True) / var


def layer_norm_backward(dy, t, gamma, dt, eps):
    """(dx, error), (dgamma, error), (dbeta, error), without storing."""
    rows, c = t.shape
    v = t - t.mean(1, keepdim=True)
    var = v.square().mean(1, keepdim=True) + eps
    rho = var.rsqrt()
    n, d = v * rho, dy * gamma
    dx = rho * (d - d.mean(1, keepdim=True) - n * (d * n).mean(1, keepdim=True))
    ev, rel = centring(t, v, var, c)
    en = rho * ev + n.abs() * rel
    size = rho * (d.abs() + d.abs().mean(1, keepdim=True) + n.abs() * (d * n).abs().mean(1, keepdim=True))
    ex = (4 * U32 * (c / 8 + 64) + 2 * rel) * size
    ex = ex + rho * (en * (d * n).abs().mean(1, keepdim=True) + n.abs() * (d.abs() * en).mean(1, keepdim=True))
    if dt is not None:
        dx, ex = dx + dt, ex + 2 * U32 * dt.abs()
    chain = U32 * (rows + 64)
    eg = (dy.abs() * en).sum(0) + (chain + 4 * U32) * (dy * n).abs().sum(0)
    return (dx, ex), ((dy * n).sum(0), eg), (dy.sum(0), chain * dy.abs().sum(0))


def philox(seed: int, step: int, rows, c):
    """Words of the generator for the given rows (a sequence) and c channels: Philox 4x32
    with ten rounds, on Python's own integers vectorised as unsigned 64-bit numbers."""
    seed, step = seed % 2 ** 64, step % 2 ** 64
    rows = np.asarray(rows, dtype=np.uint64)[:, None]
    low, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    group = np.arange((c + 3) // 4, dtype=np.uint64)[None, :]
    x = [group + 0 * rows, rows + 0 * group, np.full_like(group + rows, step & 0xFFFFFFFF),
         np.full_like(group + rows, step >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> shift) ^ x[1] ^ np.uint64(k[0]), b & low, (a >> shift) ^ x[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(x, 2).reshape(rows.shape[0], -1)[:, :c]


def dropout(x, r, p, seed, step):
    border = int(p * 2 ** 32)
    keep = torch.from_numpy(philox(seed, step, range(x.shape[0]), x.shape[1]) >= np.uint64(border)).to(x.device)
    y = torch.where(keep, x * (2 ** 32 / (2 ** 32 - border)), 0.0)
    return (y if r is None else y + r), keep


def embedding(tokens, table, scale):
    there = (tokens >= 0) & (tokens < table.shape[0])
    return torch.where(there[:, None], scale * table[tokens.long().clamp(0, table.shape[0] - 1)], 0.0)


def embedding_backward(tokens, dy, v, scale, before=None):
    """dtable and the bound of its FP32 error: sums as long as a token's rows."""
    there = (tokens >= 0) & (tokens < v)
    at, rows = tokens[there].long(), dy[there]
    sums, size = (torch.zeros(v, dy.shape[1], dtype=torch.float64, device=dy.device).index_add_(0, at, q)
                  for q in (rows, rows.abs()))
    count = torch.zeros(v, dtype=torch.float64, device=dy.device).index_add_(0, at, torch.ones_like(rows[:, 0]))
    out, err = scale * sums, abs(scale) * size * U32 * (count[:, None] + 3)
    if before is not None:
        out, err = out + before, err + U32 * (before.abs() + out.abs())
    return out, err


def cross_entropy(x, w, target, bias=None, sx=None, sw=None):
    """dict of z, ez (logits and their bound), (loss, error), (lse, error)."""
    if sx is not None:
        x, w = x * sx[:, None], w * sw[:, None]
    z = x @ w.t()
    ez = TC * (x.abs() @ w.abs().t()) + 1e-6
    if bias is not None:
        z, ez = z + bias, ez + U32 * bias.abs().nan_to_num(posinf=0)
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    el = (p * ez).sum(1) * 1.1 + 8 * U32 * (lse.abs() + 20) + 2 * U32 * z.clamp(min=-1e4).abs().amax(1)
    there = (target >= 0) & (target < w.shape[0])
    at = target.long().clamp(0, w.shape[0] - 1)[:, None]
    loss = torch.where(there, lse - z.gather(1, at)[:, 0], 0.0)
    e = torch.where(there, el + ez.gather(1, at)[:, 0] + U32 * (loss.abs() + z.gather(1, at)[:, 0].abs()), 0.0)
    return dict(z=z, ez=ez, p=p, loss=(loss, e), lse=(lse, el))


def cross_entropy_backward(x, w, target, f, dloss, dx_dtype, dw_dtype):
    """(dx, error), (dw, error), (dbias, error) from cross_entropy's dict; the logits are worked
    out a second time, from the forward call's lse."""
    there = (target >= 0) & (target < w.shape[0])
    weight = torch.where(there, dloss, 0.0)[:, None]
    p = f["p"]
    one = torch.zeros_like(p).scatter_(1, target.long().clamp(0, w.shape[0] - 1)[:, None], 1.0)
    dz = weight * (p - one)
    edz = weight.abs() * p * (1.1 * (f["ez"] + f["lse"][1][:, None]) + 4e-6) + 2 * U32 * dz.abs()
    e = edz + BF16 * dz.abs() + 1e-30
    dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    ex = e @ w.abs() + TC * (dz.abs() @ w.abs()) + stored(dx, dx_dtype)
    ew = e.t() @ x.abs() + TC * (dz.abs().t() @ x.abs()) + stored(dw, dw_dtype)
    eb = edz.sum(0) + U32 * (x.shape[0] + 64) * dz.abs().sum(0) + 1e-30
    return (dx, ex), (dw, ew), (db, eb)
