"""Forms of the layer norm's and dropout's calls: residuals of one row for all, and rows that begin
anywhere in a 16-byte piece without a residual."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from tests import channel_ref as cref
from tests import train_ref as ref
from tests.test_channel_ops_gpu import BF, F8, F32, out_like, rand
from tests.test_train_ops_gpu import close, close_e4m3, d, pitched, words

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


@pytest.mark.parametrize("rows,c,pad", [(70, 256, 0), (70, 1001, 7), (70, 1001, 0), (9, 130, 0), (300, 33, 2)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_residual_for_all_rows_is_taken(handle, rows, c, pad, dtype):
    x, one = pitched(rand(rows, c, seed=1, dtype=dtype), c + pad), rand(1, c, seed=2, dtype=dtype)
    y, total = (pitched(torch.zeros(rows, c, device="cuda").to(dtype), c + pad) for _ in range(2))
    many, gamma = one.expand(rows, c), 1 + 0.3 * rand(c, seed=3)
    api.LayerNormForward(handle, x, y, residual=many, total=total, eps=EPS)(x, gamma, y, residual=many, total=total)
    t, want, err = ref.layer_norm(d(x), d(many), d(gamma), None, EPS)
    close(total, t, cref.stored(t, dtype) + cref.U32 * t.abs(), "total")
    close(y, want, err + cref.stored(want, dtype), "y")
    api.DropoutForward(handle, x, y, p=0.5, residual=many)(x, words(1, 2), y, residual=many)
    want, _ = ref.dropout(d(x), d(many), 0.5, 1, 2)
    close(y, want, cref.stored(want, dtype) + 4 * cref.U32 * (want.abs() + d(many).abs()), "dropout")
    # one row of dtotal for all in the backward pass
    dy, dx = pitched(rand(rows, c, seed=4, dtype=dtype), c + pad), y
    (want, ex), _, _ = ref.layer_norm_backward(d(dy), d(x), d(gamma), d(many), EPS)
    api.LayerNormBackward(handle, dy, x, dx, dtotal=many, eps=EPS)(dy, x, gamma, dx, dtotal=many)
    close(dx, want, ex + cref.stored(want, dtype), "dx")


# as the same test with a residual: one thread's channels and a row's, first vectors of one channel, rows with blocks of
# their own, rows too long for shared memory
@pytest.mark.parametrize("rows,c", [(1, 5), (9, 8), (300, 1), (70, 57), (1000, 130), (41, 250), (33, 1024), (4001, 256), (700, 1001), (64, 2048),
                                    (19, 4033), (7, 4096), (11, 8185), (3, 16381)])
@pytest.mark.parametrize("pad,y_pad", [(0, 0), (5, 5), (3, 1), (1, 16), (0, 3)])
@pytest.mark.parametrize("dtype,ydt", [(BF, BF), (BF, F8), (BF, F32), (F32, F32), (F32, BF), (F32, F8)])
@pytest.mark.parametrize("total", [False, True])
def test_rows_that_begin_anywhere_without_a_residual(handle, rows, c, pad, y_pad, dtype, ydt, total):
    x = pitched(rand(rows, c, seed=1, std=2.0, dtype=dtype), c + pad)
    t = pitched(torch.zeros(rows, c, device="cuda").to(dtype), c + pad) if total else None
    gamma, beta = 1 + 0.3 * rand(c, seed=3), rand(c, seed=4) if total else None
    whole = torch.full((rows, c + y_pad), 7.0, device="cuda").to(ydt)
    y, scale = whole[:, :c], out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
    _, want, err = ref.layer_norm(d(x), None, d(gamma), d(beta), EPS)
    api.LayerNormForward(handle, x, y, total=t, eps=EPS)(x, gamma, y, beta=beta, total=t, scale=scale)
    if ydt == F8:
        close_e4m3(y, scale, want, err, "y")
    else:
        close(y, want, err + cref.stored(want, ydt), "y")
    assert (whole[:, c:].float() == 7).all()
    if total:
        assert torch.equal(t, x)
        assert torch.isnan(t.as_strided((rows - 1, pad), (c + pad, 1), c).float()).all()
