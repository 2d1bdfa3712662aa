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
