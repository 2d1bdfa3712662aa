"""Convolutions into the first channels of a wider tensor: the channels beside
them keep their values, whatever the number of filters."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from deep_learning_convolution_gb300 import binding as B

pytestmark = pytest.mark.gpu

BESIDE = 7.25


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


def rand(*shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def part(n, h, w, c, wider):
    """(an FP32 NHWC tensor of c channels, the rest of the wider one it lies in)"""
    big = torch.full((n, h, w, wider), BESIDE, device="cuda")
    return big[..., :c], big[..., c:]


def check(y, want, size, what):
    # (the tensor-core bound of the parity tests: 1e-5 of the sum of absolute products)
    assert ((y.double().cpu() - want).abs() <= 1e-5 * size + 1e-6).all(), what


def conv64(x, w, pad):
    """x NHWC, w KRSC -> the products and the sums of their absolute values, NHWC."""
    a, b = x.double().cpu().permute(0, 3, 1, 2), w.double().cpu().permute(0, 3, 1, 2)
    f = torch.nn.functional.conv2d
    return tuple(t.permute(0, 2, 3, 1) for t in (f(a, b, padding=pad), f(a.abs(), b.abs(), padding=pad)))


@pytest.mark.parametrize("k", [1, 30, 31, 32, 94, 130])
@pytest.mark.parametrize("c,n,side,kernel", [(64, 2, 13, "tc_im2col_pair"), (256, 20, 14, "tc_im2col_pair"), (3, 2, 32, "tc_window")])
def test_forward(handle, c, n, side, kernel, k):
    dtype = torch.bfloat16
    x, w = rand(n, side, side, c, seed=1, dtype=dtype), rand(k, 3, 3, c, seed=2, dtype=dtype)
    y, rest = part(n, side, side, k, (k + 15) // 16 * 16 + 16)
    op = api.Conv2dForward(handle, x, w, y, x_axes="NHWC", w_axes="KRSC", y_axes="NHWC", pads=(1, 1, 1, 1), math="bf16")
    if k > 1:
        assert op.kernel(x, w, y) == kernel
    op(x, w, y)
    want, size = conv64(x, w, 1)
    check(y, want, size, op.kernel(x, w, y))
    assert (rest == BESIDE).all()


@pytest.mark.parametrize("k", [30, 94])
@pytest.mark.parametrize("c", [3, 64])
def test_allocation_free_forward(handle, c, k):
    x, w = rand(2, 13, 13, c, seed=1, dtype=torch.bfloat16), rand(k, 3, 3, c, seed=2, dtype=torch.bfloat16)
    y, rest = part(2, 13, 13, k, (k + 15) // 16 * 16)
    op = api.Conv2dForward(handle, x, w, y, x_axes="NHWC", w_axes="KRSC", y_axes="NHWC", pads=(1, 1, 1, 1), math="bf16")
    status = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    B.dlcConvolutionForwardNoAlloc(torch.cuda.current_stream().cuda_stream, 1.0, op.x_desc, x.data_ptr(), op.w_desc, w.data_ptr(),
                                   op.conv, 0.0, op.y_desc, y.data_ptr(), status.data_ptr())
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0]
    want, size = conv64(x, w, 1)
    check(y, want, size, "allocation-free")
    assert (rest == BESIDE).all()


@pytest.mark.parametrize("c", [30, 72, 94, 104])
def test_data_gradient(handle, c):
    k, n, side = 64, 2, 13
    w, dy = rand(k, 3, 3, c, seed=1, dtype=torch.bfloat16), rand(n, side, side, k, seed=2, dtype=torch.bfloat16)
    dx, rest = part(n, side, side, c, (c + 15) // 16 * 16 + 16)
    op = api.Conv2dBackwardData(handle, w, dy, dx, w_axes="KRSC", dy_axes="NHWC", dx_axes="NHWC", pads=(1, 1, 1, 1), math="bf16")
    op(w, dy, dx)
    a, b = dy.double().cpu().permute(0, 3, 1, 2), w.double().cpu().permute(0, 3, 1, 2)
    f = torch.nn.functional.conv_transpose2d
    want, size = (t.permute(0, 2, 3, 1) for t in (f(a, b, padding=1), f(a.abs(), b.abs(), padding=1)))
    check(dx, want, size, op.kernel(w, dy, dx))
    assert (rest == BESIDE).all()
