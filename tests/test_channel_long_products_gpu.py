"""Products that run for longer than one pipeline wait may."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from tests.test_channel_ops_gpu import BF, rand

pytestmark = pytest.mark.gpu


def test_product_longer_than_a_wait_is_no_timeout(monkeypatch):
    """The limit of a wait is for one step of a pipeline, not for a whole product:
    here 1 ms, and a product of several."""
    monkeypatch.setenv("DLC_WAIT_TIMEOUT_US", "1000")
    rows, c, k = 131072, 4096, 8192
    x, w = torch.zeros(rows, c, dtype=BF, device="cuda"), rand(k, c, seed=2, dtype=BF)
    x[-1] = rand(c, seed=1, dtype=BF)
    y = torch.empty(rows, k, dtype=BF, device="cuda")
    with api.Handle() as h:
        op = api.LinearForward(h, x, w, y)
        assert op.kernel(x, w, y) == "gemm_pair"
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        op(x, w, y)
        end.record()
        h.synchronize()
        assert start.elapsed_time(end) > 2.0
        assert h.last_device_error() == (0, 0)
        op(x, w, y)
        h.synchronize()
        assert h.last_device_error() == (0, 0)
        # (products on the tensor core: 1e-5 of the sum of absolute terms, and y in BF16)
        want, size = x[-1].double() @ w.double().t(), x[-1].double().abs() @ w.double().abs().t()
        assert ((y[-1].double() - want).abs() <= 1e-5 * size + 2.0 ** -8 * want.abs()).all()
        assert not y[:-1].any()
