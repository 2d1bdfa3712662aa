"""Outputs that are parts of wider tensors: what lies beside them keeps its
bits, whatever their sizes, layouts and types; and what lies beside inputs is
not read."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from tests import channel_ref as ref
from tests.test_channel_ops_gpu import BF, F8, F32, close, f64, quantized, rand

pytestmark = pytest.mark.gpu

FILL = 0x7B


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


class Part:
    """A [rows, c] output at a pitch, 64 elements into a buffer of one byte value."""

    def __init__(self, rows, c, dtype, pitch=None):
        self.where = ((rows, c), (pitch or c, 1), 64)
        n = 64 + (rows - 1) * (pitch or c) + c + 64
        self.bytes = torch.full((n * dtype.itemsize,), FILL, dtype=torch.uint8, device="cuda")
        self.dtype = dtype
        self.t = self.bytes.view(dtype).as_strided(*self.where)

    def check(self, what):
        left = self.bytes.clone()
        same = torch.full_like(left, FILL).view(self.dtype).as_strided(*self.where)
        left.view(self.dtype).as_strided(*self.where).copy_(same)
        at = (left != FILL).nonzero().flatten()
        assert at.numel() == 0, f"{what}: {at.numel()} bytes beside it written, first {at[0].item()}"


def padded(t, pitch):
    """t's rows in a wider matrix whose other elements are NaN."""
    rows, c = t.shape
    big = torch.full((rows, pitch), float("nan"), device="cuda").to(t.dtype)
    big[:, :c] = t
    return big[:, :c]


# rows that end inside a piece of 16 bytes, and whole ones
@pytest.mark.parametrize("k", [1, 3, 30, 65, 130, 257, 1000])
@pytest.mark.parametrize("rows", [1, 5, 200, 3000])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gated", [False, True])
def test_forward_outputs(handle, rows, k, dtype, gated):
    c, n = 80, 2 * k if gated else k
    pitch, zpitch = (k + 15) // 16 * 16 + 16, (n + 15) // 16 * 16
    x, w = padded(rand(rows, c, seed=1, dtype=BF), c + 16), rand(n, c, seed=2, std=c ** -0.5, dtype=BF)
    y, z = Part(rows, k, dtype, pitch), Part(rows, n, dtype, zpitch)
    (api.GatedForward if gated else api.LinearForward)(handle, x, w, y.t, act="silu", z=z.t)(x, w, y.t, z=z.t)
    zw, ez = ref.product(f64(x), f64(w))
    want, err = ref.gated(zw, ez, "silu", dtype) if gated else ref.linear(zw, ez, "silu", None, dtype)
    close(y.t, want, err, "y")
    close(z.t, zw, ez + ref.stored(zw, dtype), "z")
    y.check("y")
    z.check("z")


@pytest.mark.parametrize("c", [1, 3, 9, 100, 257, 447, 1398])
@pytest.mark.parametrize("rows,k", [(1, 1), (2, 1), (1, 40), (300, 24), (2052, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients(handle, rows, c, k, dtype):
    x, w = padded(rand(rows, c, seed=1, dtype=BF), (c + 7) // 8 * 8 + 8), rand(k, c, seed=2, std=c ** -0.5, dtype=BF)
    dy = padded(rand(rows, k, seed=3, dtype=BF), (k + 7) // 8 * 8)
    dx, dw, db = Part(rows, c, dtype, (c + 15) // 16 * 16), Part(k, c, dtype), Part(1, k, F32)
    op = api.LinearBackward(handle, x, w, dy, dx.t, dw.t)
    if op.workspace is not None:
        op.workspace.fill_(255)
    op(x, w, dy, dx.t, dw.t, dbias=db.t[0])
    (dxw, ex), (dww, ew), (dbw, eb) = ref.backward(f64(x), f64(w), f64(dy), 0 * f64(dy), dtype, dtype)
    for part, want, err, what in ((dx, dxw, ex, "dx"), (dw, dww, ew, "dw"), (db, dbw[None], eb[None], "dbias")):
        close(part.t, want, err, what)
        part.check(what)


@pytest.mark.parametrize("c", [1, 30, 257, 1398, 9001])
@pytest.mark.parametrize("pitched", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32, F8])
def test_norm_outputs(handle, c, pitched, dtype):
    rows = 50
    pitch = (c + 15) // 16 * 16 + 16 if pitched else None
    x = padded(rand(rows, c, seed=1, dtype=BF), pitch or c)
    gamma = 1 + 0.3 * rand(c, seed=3)
    t, y, s = Part(rows, c, BF, pitch), Part(rows, c, dtype, pitch), Part(1, rows, F32)
    api.RmsNormForward(handle, x, y.t, total=t.t)(x, gamma, y.t, total=t.t, scale=s.t[0] if dtype == F8 else None)
    for part, what in ((t, "total"), (y, "y"), (s, "scale")):
        part.check(what)
    assert torch.equal(t.t, x) and torch.isfinite(y.t.float()).all()
    if dtype == F8:
        return
    dy, dx, dg = x, Part(rows, c, dtype, pitch), Part(1, c, F32)
    api.RmsNormBackward(handle, dy, x, dx.t)(dy, x, gamma, dx.t, dgamma=dg.t[0])
    dx.check("dx")
    dg.check("dgamma")
    assert torch.isfinite(dx.t.float()).all() and torch.isfinite(dg.t).all()


@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("c", [33, 100, 130])
def test_e4m3_operands_beside_nan(handle, rows, c):
    (x, sx), (w, sw) = quantized(rand(rows, c, seed=1)), quantized(rand(56, c, seed=2))
    x = padded(x, (c + 15) // 16 * 16)
    y = Part(rows, 56, F32, 60)
    api.LinearForward(handle, x, w, y.t)(x, w, y.t, x_scale=sx, w_scale=sw)
    z, ez = ref.product(f64(x), f64(w), None, f64(sx), f64(sw))
    close(y.t, z, ez + ref.stored(z, F32), "y")
    y.check("y")
