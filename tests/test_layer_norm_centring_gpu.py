"""Layer norm of rows whose mean is all there is of them, or nearly: equal channels, and deviations a
millionth of the mean.  Their centred values must not be the mean's rounding."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from tests import channel_ref as cref
from tests import train_ref as ref
from tests.test_channel_ops_gpu import BF, F8, F32, laid_out, out_like, rand
from tests.test_train_ops_gpu import close, close_e4m3, d

pytestmark = pytest.mark.gpu
EPS = 1e-5
VALUES = [1.7, 1e5, -0.1, 3e7, 1e-3, 123456.7, -1e9]

# one thread, a warp's part, whole and partial vectors, several warps, one block a row, rows read again
SIZES = [(7, 3), (7, 48), (40, 96), (700, 130), (2000, 768), (300, 1001), (64, 2048), (9, 4097), (5, 8192), (4, 12288), (3, 16384),
         (3, 20000)]


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


def equal_rows(rows, c, dtype, layout):
    values = torch.tensor(VALUES, device="cuda").repeat(rows // len(VALUES) + 1)[:rows]
    return laid_out(values[:, None].expand(rows, c).to(dtype).contiguous(), layout)


@pytest.mark.parametrize("rows,c", SIZES)
@pytest.mark.parametrize("xdt,rdt,ydt", [(F32, None, F32), (BF, None, BF), (F32, F32, F8), (BF, F32, BF), (BF, BF, F32)])
@pytest.mark.parametrize("layout", ["dense", "odd", "columns"])
def test_rows_of_equal_channels_are_zeros(handle, rows, c, xdt, rdt, ydt, layout):
    x = equal_rows(rows, c, xdt, layout)
    r = None if rdt is None else laid_out(torch.full((rows, c), 0.3, device="cuda").to(rdt), layout)
    gamma, beta = 1 + 0.3 * rand(c, seed=3), rand(c, seed=4)
    y, scale = out_like(rows, c, ydt, layout), out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
    api.LayerNormForward(handle, x, y, residual=r, eps=EPS)(x, gamma, y, beta=beta, residual=r, scale=scale)
    want = beta.expand(rows, c)
    if ydt == F8:
        close_e4m3(y, scale, d(want), torch.zeros(rows, c, dtype=torch.float64, device="cuda"), "y")
    else:
        assert torch.equal(y, want.to(ydt))
    # without an epsilon 0 / 0
    api.LayerNormForward(handle, x, y, residual=r, eps=0.0)(x, gamma, y, beta=beta, residual=r, scale=scale)
    assert torch.isnan(y.float()).all()


@pytest.mark.parametrize("rows,c", SIZES)
@pytest.mark.parametrize("tdt,ddt", [(F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("layout", ["dense", "odd", "columns"])
def test_gradient_of_rows_of_equal_channels(handle, rows, c, tdt, ddt, layout):
    t, dy, dx = equal_rows(rows, c, tdt, layout), laid_out(rand(rows, c, seed=1, dtype=ddt), layout), out_like(rows, c, F32, layout)
    gamma = 1 + 0.3 * rand(c, seed=2)
    dgamma, dbeta = out_like(c, 1, F32)[:, 0], out_like(c, 1, F32)[:, 0]
    api.LayerNormBackward(handle, dy, t, dx, eps=EPS)(dy, t, gamma, dx, dgamma=dgamma, dbeta=dbeta)
    g = d(dy) * d(gamma)
    want = (g - g.mean(1, keepdim=True)) * EPS ** -0.5
    # the mean's chain and the roundings of rho (train_ref.layer_norm_backward where n is 0)
    err = 4 * cref.U32 * (c / 8 + 64) * EPS ** -0.5 * (g.abs() + g.abs().mean(1, keepdim=True))
    close(dx, want, err + cref.stored(want, F32), "dx")
    assert (dgamma == 0).all()
    close(dbeta, d(dy).sum(0), cref.U32 * (rows + 64) * d(dy).abs().sum(0) + 1e-30, "dbeta")


def precise(t, gamma, beta):
    """y and its bound where the mean's size does not count: values within a factor of two of their mean are
    subtracted exactly, and the rest of the mean is a mean of centred values."""
    c = t.shape[1]
    v = t - t.mean(1, keepdim=True)
    var = v.square().mean(1, keepdim=True) + EPS
    rho, chain = var.rsqrt(), c / 8 + 64
    ed = cref.U32 * (chain * v.abs().mean(1, keepdim=True) + 4 * v.abs())
    rel = cref.U32 * chain + (v.abs() * ed).mean(1, keepdim=True) / var
    y = gamma * v * rho + beta
    return y, gamma.abs() * rho * (ed + v.abs() * (rel + 4 * cref.U32)) + 2 * cref.U32 * (y.abs() + beta.abs()), (v, var, rho, ed, rel)


@pytest.mark.parametrize("rows,c", [(70, 96), (33, 333), (300, 768), (64, 1001), (40, 2048), (5, 8192), (3, 12288), (2, 20000)])
@pytest.mark.parametrize("level", [30.0, 1e3, 1e5, 3e6])
@pytest.mark.parametrize("layout", ["dense", "odd", "columns"])
def test_rows_far_from_zero_keep_their_digits(handle, rows, c, level, layout):
    x = laid_out(rand(rows, c, seed=1) + level, layout)
    gamma, beta, y = 1 + 0.3 * rand(c, seed=2), rand(c, seed=3), out_like(rows, c, F32, layout)
    api.LayerNormForward(handle, x, y, eps=EPS)(x, gamma, y, beta=beta)
    want, err, (v, var, rho, ed, rel) = precise(d(x), d(gamma), d(beta))
    close(y, want, err + cref.stored(want, F32), "y")
    dy, dx = laid_out(rand(rows, c, seed=4), layout), out_like(rows, c, F32, layout)
    dgamma, dbeta = out_like(c, 1, F32)[:, 0], out_like(c, 1, F32)[:, 0]
    api.LayerNormBackward(handle, dy, x, dx, eps=EPS)(dy, x, gamma, dx, dgamma=dgamma, dbeta=dbeta)
    # train_ref.layer_norm_backward with these bounds of the centred values and of rho
    n, g = v * rho, d(dy) * d(gamma)
    want = rho * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    en = rho * ed + n.abs() * rel
    size = rho * (g.abs() + g.abs().mean(1, keepdim=True) + n.abs() * (g * n).abs().mean(1, keepdim=True))
    ex = (4 * cref.U32 * (c / 8 + 64) + 2 * rel) * size
    ex = ex + rho * (en * (g * n).abs().mean(1, keepdim=True) + n.abs() * (g.abs() * en).mean(1, keepdim=True))
    close(dx, want, ex + cref.stored(want, F32), "dx")
    eg = (d(dy).abs() * en).sum(0) + cref.U32 * (rows + 68) * (d(dy) * n).abs().sum(0)
    close(dgamma, (d(dy) * n).sum(0), eg + 1e-30, "dgamma")


@pytest.mark.parametrize("c", [24, 96, 768, 3000])
@pytest.mark.parametrize("dtype,ydt", [(F32, F32), (BF, F8)])
@pytest.mark.parametrize("layout", ["dense", "odd", "columns"])
def test_a_row_does_not_depend_on_its_neighbours(handle, c, dtype, ydt, layout):
    """Rows that are centred again beside ordinary ones: the ordinary ones' bits stay."""
    rows = 61
    x = rand(rows, c, seed=1, dtype=dtype)
    mixed = x.clone()
    mixed[::3] = 1234.5
    x, mixed = laid_out(x, layout), laid_out(mixed, layout)
    gamma, dy = 1 + 0.3 * rand(c, seed=2), laid_out(rand(rows, c, seed=3, dtype=dtype), layout)
    outs = []
    for t in (x, mixed):
        y, dx = out_like(rows, c, ydt, layout), out_like(rows, c, dtype, layout)
        scale = out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
        api.LayerNormForward(handle, t, y, eps=EPS)(t, gamma, y, scale=scale)
        api.LayerNormBackward(handle, dy, t, dx, eps=EPS)(dy, t, gamma, dx)
        outs.append([y.float(), dx] + ([] if scale is None else [scale]))
    ordinary = [i for i in range(rows) if i % 3]
    for a, b in zip(*outs):
        assert torch.equal(a[ordinary], b[ordinary])
