"""Tensors of a call that differ from the examples its operator was built from
are refused before anything is launched."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from deep_learning_convolution_gb300 import binding as B
from tests.test_channel_ops_gpu import BF, F32, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


def calls(handle):
    """(the operator, its right arguments by name) of every kind."""
    rows, c, k = 24, 64, 48
    x, w, y, z = rand(rows, c, seed=1, dtype=BF), rand(k, c, seed=2, dtype=BF), rand(rows, k, seed=3, dtype=BF), rand(rows, k, dtype=F32)
    wg, zg = rand(2 * k, c, seed=4, dtype=BF), rand(rows, 2 * k, dtype=F32)
    r, n, t = rand(rows, k, seed=5, dtype=BF), torch.empty_like(x), torch.empty_like(x)
    dx, dw, dwg, gamma = torch.empty_like(x), torch.empty_like(w), torch.empty_like(wg), torch.ones(c, device="cuda")
    return [
        (api.RmsNormForward(handle, x, n, residual=x, total=t), dict(x=x, gamma=gamma, y=n, residual=x, total=t)),
        (api.RmsNormBackward(handle, n, t, dx, dtotal=x), dict(dy=n, total=t, gamma=gamma, dx=dx, dtotal=x)),
        (api.LinearForward(handle, x, w, y, residual=r, z=z), dict(x=x, w=w, y=y, residual=r, z=z)),
        (api.GatedForward(handle, x, wg, y, z=zg), dict(x=x, w=wg, y=y, z=zg)),
        (api.LinearBackward(handle, x, w, y, dx, dw, z=z, act="silu"), dict(x=x, w=w, dy=y, dx=dx, dw=dw, z=z)),
        (api.GatedBackward(handle, x, wg, y, dx, dwg, z=zg), dict(x=x, w=wg, dy=y, dx=dx, dw=dwg, z=zg))]


def wrong(t):
    """Tensors that would be read or written outside, or as something else."""
    yield "fewer rows", t[:-1]
    yield "another type", t.to(F32 if t.dtype == BF else BF)
    yield "transposed", t.t().contiguous().t()
    yield "other strides", torch.cat([t, t], 1)[:, :t.shape[1]]
    yield "on the host", t.cpu()


def test_tensors_unlike_their_examples_are_refused(handle):
    for op, right in calls(handle):
        op(**right)
        before = handle.launches()
        for name, t in right.items():
            for what, bad in wrong(t) if t.dim() == 2 else [("shorter", t[1:]), ("on the host", t.cpu())]:
                with pytest.raises(ValueError, match=name):
                    op(**{**right, name: bad})
                    pytest.fail(f"{type(op).__name__} took {name} with {what}")
        assert handle.launches() == before
        op(**right)
    handle.synchronize()


def test_examples_on_the_host_are_refused(handle):
    x, w, y = rand(8, 64, dtype=BF), rand(32, 64, dtype=BF), torch.empty(8, 32, dtype=BF, device="cuda")
    for bad in ((x.cpu(), w, y), (x, w.cpu(), y), (x, w, y.cpu())):
        with pytest.raises(ValueError):
            api.LinearForward(handle, *bad)


def test_the_same_elements_in_other_dimensions_are_taken(handle):
    """What leaves every address where it was is no difference: dimensions of one
    element with other strides, filters with or without R = S = 1, images of the
    same rows."""
    x, w, y = rand(6, 64, seed=1, dtype=BF), rand(32, 64, seed=2, dtype=BF), torch.empty(6, 32, dtype=BF, device="cuda")
    op = api.LinearForward(handle, x, w, y)
    want = op(x, w, y).clone()
    y.zero_()
    op(x, w.view(32, 64, 1, 1), y)
    assert torch.equal(y, want)
    one, out = rand(12, 64, seed=3, dtype=BF), torch.empty(1, 32, dtype=BF, device="cuda")
    row = api.LinearForward(handle, one[:1], w, out)
    a = row(one[:1], w, out).clone()
    out.zero_()
    row(one.view(1, 12 * 64)[:, :64], w, out)  # a row of another pitch
    assert torch.equal(out, a)
    image = x.view(2, 3, 1, 64)
    over = api.LinearForward(handle, image, w, y.view(2, 3, 1, 32))
    y.zero_()
    over(image, w, y.view(2, 3, 1, 32))
    assert torch.equal(y, want)


def test_a_closed_operator_is_refused(handle):
    for op, right in calls(handle):
        op(**right)
        op.close()
        before = handle.launches()
        with pytest.raises(B.DlcError) as e:
            op(**right)
        assert e.value.status in (B.DLC_STATUS_BAD_PARAM, B.DLC_STATUS_NOT_INITIALIZED)
        if hasattr(op, "kernel"):
            with pytest.raises(B.DlcError):
                op.kernel()
        assert handle.launches() == before
        op.close()
