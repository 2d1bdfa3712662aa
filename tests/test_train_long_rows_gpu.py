"""The layer norm of a row of more than 2^30 channels, whose two parameter gradients together have
more columns than 31 bits count."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from tests import channel_ref as cref
from tests.test_channel_ops_gpu import BF, F32

pytestmark = pytest.mark.gpu

CHANNELS = 2 ** 30 + 8


@pytest.fixture(scope="module")
def handle():
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GB free")
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()
    torch.cuda.empty_cache()


def periodic(base, dtype):
    """A row of `base` (4096 values) over and over."""
    out = torch.empty(1, CHANNELS, dtype=dtype, device="cuda")
    whole = CHANNELS // 4096 * 4096
    out[0, :whole].view(-1, 4096).copy_(base)
    out[0, whole:] = base[:CHANNELS - whole].to(dtype)
    return out


def test_layer_norm_of_more_than_2_30_channels(handle):
    """Values whose sums cancel group by group: mean 0, variance 1 and mean(d n) 0 in FP32 whatever the order, and
    mean(d) = 8 / 2^30, below half a step of BF16 beside 1."""
    c = torch.arange(4096, device="cuda")
    sign, dys, gammas = 1.0 - 2 * (c & 1), 1.0 - 2 * (c >> 9 & 1), 1.0 + (c >> 11 & 1)
    t, dy, gamma = periodic(sign, BF), periodic(dys, BF), periodic(gammas, F32)[0]
    y = torch.full_like(t, float("nan"))
    api.LayerNormForward(handle, t, y, eps=0.0)(t, gamma, y)
    assert torch.equal(y, periodic(sign * gammas, BF))
    dx = y.fill_(float("nan"))
    dgamma, dbeta = torch.full_like(gamma, float("nan")), torch.full_like(gamma, float("nan"))
    api.LayerNormBackward(handle, dy, t, dx, eps=0.0)(dy, t, gamma, dx, dgamma=dgamma, dbeta=dbeta)
    assert torch.equal(dx, periodic(dys * gammas, BF))
    assert torch.equal(dbeta, periodic(dys, F32)[0])
    # one product by a reciprocal root that is two steps off at most
    assert (dgamma.sub_(periodic(dys * sign, F32)[0]).abs_().max() <= 4 * cref.U32).item()
