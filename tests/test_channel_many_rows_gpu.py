"""Norms of images of more than 2^31 pixels whose rows no single pitch describes."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from deep_learning_convolution_gb300 import binding as B
from tests import channel_ref as ref
from tests.test_channel_ops_gpu import BF, close, f64

pytestmark = pytest.mark.gpu

SIDE = 46341  # 46341^2 = 2^31 + 4633 pixels


@pytest.fixture(scope="module")
def handle():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB free")
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()
    torch.cuda.empty_cache()


def image(n, pad_h, pad_w):
    return torch.zeros(n, SIDE + pad_h, SIDE + pad_w, 1, dtype=BF, device="cuda")[:, :SIDE, :SIDE]


def test_rows_past_32_bits(handle):
    x, y = image(1, 0, 3), image(1, 0, 5)
    # some lines with values, the rest zeros
    lines = [0, 1, SIDE // 2, SIDE - 2, SIDE - 1]
    g = torch.Generator().manual_seed(1)
    for i in lines:
        x[0, i] = torch.randn(SIDE, 1, generator=g).to(BF).cuda()
    gamma = torch.tensor([1.5], device="cuda")
    api.RmsNormForward(handle, x, y, eps=1.0)(x, gamma, y)
    _, want = ref.norm(f64(x[0, lines]).view(-1, 1), None, f64(gamma), 1.0)
    close(y[0, lines].reshape(-1, 1), want, ref.norm_rel(1) * want.abs() + ref.stored(want, BF), "y")
    assert y[0, 2:SIDE // 2].count_nonzero() == 0 and y[0, SIDE // 2 + 1:SIDE - 2].count_nonzero() == 0
    # backward: dy = 2 of the same lines, dx in the forward pass's place
    dy = x * 2
    dgamma = torch.empty(1, device="cuda")
    y.fill_(7)
    api.RmsNormBackward(handle, dy, x, y, eps=1.0)(dy, x, gamma, y, dgamma=dgamma)
    want, wg, bx, bg = ref.norm_backward(f64(dy[0, lines]).view(-1, 1), f64(x[0, lines]).view(-1, 1), f64(gamma), None, 1.0)
    close(y[0, lines].reshape(-1, 1), want, 4 * ref.norm_rel(1) * bx + ref.stored(want, BF), "dx")
    assert y[0, 2:SIDE // 2].count_nonzero() == 0 and y[0, SIDE // 2 + 1:SIDE - 2].count_nonzero() == 0
    # (a thread's chain of sums: 2^31 rows over thousands of threads, mostly zeros)
    close(dgamma, wg, (ref.norm_rel(1) + ref.U32 * (5 * SIDE + 64)) * bg, "dgamma")


def test_images_with_a_gap_between_them_are_refused(handle):
    x, y = image(2, 1, 3), image(2, 0, 3)
    gamma = torch.ones(1, device="cuda")
    for a, b in ((x, y), (y, x)):
        with pytest.raises(B.DlcError) as e:
            api.RmsNormForward(handle, a, b)(a, gamma, b)
        assert e.value.status == B.DLC_STATUS_NOT_SUPPORTED
        with pytest.raises(B.DlcError) as e:
            api.RmsNormBackward(handle, a, a, b)(a, a, gamma, b)
        assert e.value.status == B.DLC_STATUS_NOT_SUPPORTED
    assert handle.last_device_error() == (0, 0)
