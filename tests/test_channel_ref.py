"""The FP64 definitions of the channel operators against central differences
(CPU), so that the gradients the GPU tests compare with are gradients."""
import pytest
import torch

from tests import channel_ref as ref


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _difference(fn, v, direction, h=1e-5):
    return (fn(v + h * direction) - fn(v - h * direction)) / (2 * h)


# a central difference of step h is off by h^2 times the third derivative
# (h = 1e-5: about 1e-10 of sums of a few hundred terms) plus rounding 1e-16 / h
TOL = 1e-7


@pytest.mark.parametrize("with_dt", [False, True])
def test_norm_gradient(with_dt):
    t, dy, gamma = _rand(5, 12, seed=1), _rand(5, 12, seed=2), 1 + 0.3 * _rand(12, seed=3)
    dt = _rand(5, 12, seed=4) if with_dt else None
    dx, dgamma, _, _ = ref.norm_backward(dy, t, gamma, dt, 1e-3)

    def loss_t(v):
        return (dy * ref.norm(v, None, gamma, 1e-3)[1]).sum() + (0 if dt is None else (dt * v).sum())

    d = _rand(5, 12, seed=5)
    assert abs(_difference(loss_t, t, d) - (dx * d).sum()) < TOL * (dx * d).abs().sum()
    dg = _rand(12, seed=6)
    got = _difference(lambda v: (dy * ref.norm(t, None, v, 1e-3)[1]).sum(), gamma, dg)
    assert abs(got - (dgamma * dg).sum()) < TOL * (dgamma * dg).abs().sum()


@pytest.mark.parametrize("kind", ["identity", "relu", "sigmoid", "tanh", "silu", "gelu"])
@pytest.mark.parametrize("is_gated", [False, True])
def test_product_gradients(kind, is_gated):
    x, w, bias = _rand(7, 9, seed=1), _rand(10, 9, seed=2), _rand(10, seed=3)
    dy = _rand(7, 5 if is_gated else 10, seed=4)

    def out(x, w, bias):
        z = x @ w.t() + bias
        if is_gated:
            return (dy * ref.act(z[:, :5], kind)[0] * z[:, 5:]).sum()
        return (dy * ref.act(z, kind)[0]).sum()

    z = x @ w.t() + bias
    dz, e = ref.act_grad(dy, z, kind, is_gated)
    (dx, _), (dw, _), (db, _) = ref.backward(x, w, dz, e, torch.float32, torch.float32)
    for v, g, fn in ((x, dx, lambda v: out(v, w, bias)), (w, dw, lambda v: out(x, v, bias)),
                     (bias, db, lambda v: out(x, w, v))):
        d = _rand(*v.shape, seed=5)
        # relu's kink: no argument lies within the step of zero for these seeds
        assert abs(_difference(fn, v, d) - (g * d).sum()) < TOL * (g * d).abs().sum() + 1e-8
