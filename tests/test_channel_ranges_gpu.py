"""The channel operators at the ends of their ranges: zero rows beside a small
epsilon, rows of extreme size in the backward pass, long rows, and activations
far out by their relative error; against the FP64 definitions."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from tests import channel_ref as ref
from tests.test_channel_ops_gpu import BF, F8, F32, close, close_e4m3, f64, laid_out, out_like, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


# one for each way of reading rows: 16-byte vectors, single elements, rows too
# long for registers, channels apart
NORM_LAYOUTS = [(256, "dense"), (99, "odd"), (20000, "dense"), (256, "columns")]


@pytest.mark.parametrize("c,layout", NORM_LAYOUTS)
@pytest.mark.parametrize("eps", [0.0, 1e-12, 1e-8])
def test_e4m3_zero_rows_are_zeros_whatever_the_epsilon(handle, c, layout, eps):
    x = rand(40, c, seed=1)
    x[1] = 0
    x[39] = 0
    x[2] = 1e-37 * x[2].sign()  # |y| below the floor of the scale, if epsilon is not zero
    if eps == 0:
        x[2] = 1
    x = laid_out(x, layout)
    gamma = 1 + 0.3 * rand(c, seed=3)
    y, scale = out_like(40, c, F8, layout), out_like(40, 1, F32)[:, 0]
    api.RmsNormForward(handle, x, y, eps=eps)(x, gamma, y, scale=scale)
    for row in (1, 39):
        assert (y[row].float() == 0).all()
        assert abs(scale[row].item() - 1e-30 / 448) < 1e-36
    rest = [i for i in range(40) if i not in (1, 39)]
    _, want = ref.norm(f64(x)[rest], None, f64(gamma), eps)
    close_e4m3(y[rest], scale[rest], want, ref.norm_rel(c), "other rows")


@pytest.mark.parametrize("c,layout", NORM_LAYOUTS)
def test_e4m3_rows_under_a_zero_gamma_are_zeros(handle, c, layout):
    x = laid_out(1e-7 * rand(5, c, seed=1), layout)
    y, scale = out_like(5, c, F8, layout), out_like(5, 1, F32)[:, 0]
    api.RmsNormForward(handle, x, y, eps=1e-20)(x, torch.zeros(c, device="cuda"), y, scale=scale)
    assert (y.float() == 0).all() and torch.isfinite(scale).all()


@pytest.mark.parametrize("c,layout", NORM_LAYOUTS)
def test_norm_backward_of_tiny_and_large_rows(handle, c, layout):
    """Rows of size 1e-17 to 1e16 with no epsilon: rho^3 alone leaves FP32's
    range, the gradient does not."""
    sizes = [1.0, 1e-13, 1e-15, 1e-17, 1e13, 1e15, 1e16]
    t = rand(len(sizes), c, seed=1) * torch.tensor(sizes, device="cuda")[:, None]
    t, dy = laid_out(t, layout), laid_out(rand(len(sizes), c, seed=2), layout)
    gamma, dgamma = 1 + 0.3 * rand(c, seed=3), out_like(c, 1, F32)[:, 0]
    dx = out_like(len(sizes), c, F32, layout)
    api.RmsNormBackward(handle, dy, t, dx, eps=0.0)(dy, t, gamma, dx, dgamma=dgamma)
    want, wg, bx, bg = ref.norm_backward(f64(dy), f64(t), f64(gamma), None, 0.0)
    close(dx, want, 4 * ref.norm_rel(c) * bx + ref.stored(want, F32), "dx")
    close(dgamma, wg, (ref.norm_rel(c) + ref.U32 * (len(sizes) + 64)) * bg, "dgamma")


LONG = [8184, 8192, 8193, 8200, 12288, 16384, 16392]


@pytest.mark.parametrize("c", LONG)
@pytest.mark.parametrize("xdt,rdt,ydt", [(F32, F32, F32), (F32, None, F8), (BF, BF, BF), (BF, F32, F32)])
def test_norm_of_long_rows(handle, c, xdt, rdt, ydt):
    rows = 3
    x = rand(rows, c, seed=1, dtype=xdt)
    r = rand(rows, c, seed=2, dtype=rdt) if rdt else None
    gamma = 1 + 0.3 * rand(c, seed=3)
    total, y = out_like(rows, c, rdt or xdt), out_like(rows, c, ydt)
    scale = out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
    api.RmsNormForward(handle, x, y, residual=r, total=total)(x, gamma, y, residual=r, total=total, scale=scale)
    t, want = ref.norm(f64(x), f64(r), f64(gamma), 1e-6)
    close(total, t, ref.stored(t, rdt or xdt) + ref.U32 * t.abs(), "total")
    if ydt == F8:
        close_e4m3(y, scale, want, ref.norm_rel(c), "y")
    else:
        close(y, want, ref.norm_rel(c) * want.abs() + ref.stored(want, ydt), "y")


@pytest.mark.parametrize("c", LONG)
@pytest.mark.parametrize("dydt,tdt,dtdt", [(F32, F32, F32), (F32, F32, None), (BF, BF, BF), (BF, F32, F32)])
def test_norm_backward_of_long_rows(handle, c, dydt, tdt, dtdt):
    rows = 3
    dy, t = rand(rows, c, seed=1, dtype=dydt), rand(rows, c, seed=2, std=2.0, dtype=tdt)
    dt = rand(rows, c, seed=3, dtype=dtdt) if dtdt else None
    gamma, dgamma = 1 + 0.3 * rand(c, seed=4), out_like(c, 1, F32)[:, 0]
    dx = out_like(rows, c, tdt)
    api.RmsNormBackward(handle, dy, t, dx, dtotal=dt)(dy, t, gamma, dx, dgamma=dgamma, dtotal=dt)
    want, wg, bx, bg = ref.norm_backward(f64(dy), f64(t), f64(gamma), f64(dt), 1e-6)
    close(dx, want, 4 * ref.norm_rel(c) * bx + ref.stored(want, tdt), "dx")
    close(dgamma, wg, (ref.norm_rel(c) + ref.U32 * (rows + 64)) * bg, "dgamma")


def act_rel(v, kind):
    """Relative error of an activation in FP32, from its steps (U = 2^-24 each rounding):

    gelu: Phi by a quotient fitted to 2e-7, evaluated in some ten roundings (their
    sum at most four times the result's size): 40 U + 2e-7 < 4e-6; the exponent
    v^2/2, of three roundings, makes 3 U v^2/2 < 1e-7 v^2 of its exponential.
    silu, sigmoid: exponent v with two roundings, exponential 4 U, sum, reciprocal
    2 U and product: < 1e-6 + 2e-7 |v|."""
    return 4e-6 + 1e-7 * v * v if kind == "gelu" else 1e-6 + 2e-7 * v.abs()


# 1, 8 and 200 rows: a kernel each
@pytest.mark.parametrize("rows", [1, 8, 200])
@pytest.mark.parametrize("kind,lowest,step", [("gelu", -12.9375, 0.0625), ("silu", -79.5, 0.5), ("sigmoid", -79.5, 0.5)])
def test_activations_by_their_relative_error(handle, rows, kind, lowest, step):
    """Down to where FP32's normal range ends, which BF16 and FP32 outputs have."""
    v = torch.arange(lowest, -lowest, step, dtype=torch.float64)  # BF16 holds them exactly
    v = v[v != 0]
    assert torch.equal(v.to(BF).double(), v)
    n = v.numel()
    x, w = torch.ones(rows, 1, dtype=BF, device="cuda"), v.to(BF).cuda().view(-1, 1).contiguous()
    y, z = out_like(rows, n, F32), out_like(rows, n, F32)
    api.LinearForward(handle, x, w, y, act=kind, z=z)(x, w, y, z=z)
    assert torch.equal(f64(z), v.expand(rows, n))
    f, df = ref.act(v, kind)
    rel = act_rel(v, kind)
    close(y, f.expand(rows, n), (rel * f.abs()).expand(rows, n), kind)
    dy, db = torch.zeros(rows, n, device="cuda"), out_like(n, 1, F32)[:, 0]
    dy[rows - 1] = 1
    api.LinearBackward(handle, x, w, dy, z=z, act=kind)(x, w, dy, dbias=db, z=z)
    # the slope's terms: gelu Phi + v phi, silu p + v p (1 - p), sigmoid p (1 - p) from 1 - p of its own rounding
    if kind == "gelu":
        p = 0.5 * torch.erfc(-v / 2 ** 0.5)
        terms = p + (df - p).abs()
    elif kind == "silu":
        p = torch.sigmoid(v)
        terms = p * (1 + v.abs())
    else:
        terms = torch.sigmoid(v)
    close(db, df, rel * terms, kind + " slope")
