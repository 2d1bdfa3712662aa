"""Products whose outputs need different ways of writing side by side, the
few-row kernel's tile widths and splits, copies shared by a backward pass's two
products, and an operator released while its kernels run; against FP64 under
channel_ref's bounds."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from tests.test_channel_ops_gpu import BF, F8, F32, rand, run_backward, run_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


# rows: several tiles for every pair of SMs, and fewer tiles than pairs
@pytest.mark.parametrize("rows,c,k", [(20001, 40, 200), (2500, 136, 333), (700, 64, 1000)])
@pytest.mark.parametrize("layout,zr_layout", [("pitch", "odd"), ("odd", "pitch"), ("pitch", "columns")])
@pytest.mark.parametrize("ydt,zdt", [(BF, BF), (F32, F32), (BF, F32)])
def test_outputs_of_different_layouts(handle, rows, c, k, layout, zr_layout, ydt, zdt):
    lay = dict(layout=layout, zr_layout=zr_layout)
    run_forward(handle, rows, c, k, gated=False, ydt=ydt, kind="gelu", bias=True, z=zdt, **lay)
    run_forward(handle, rows, c, k, gated=False, ydt=ydt, residual=zdt, **lay)
    run_forward(handle, rows, c, k // 2, gated=True, ydt=ydt, kind="silu", bias=True, z=zdt, **lay)


# row pitches of 8 and 4 bytes' alignment: dense rows of k elements
@pytest.mark.parametrize("k", [196, 198, 452, 454])
@pytest.mark.parametrize("dt", [BF, F32])
def test_outputs_at_narrow_pitches(handle, k, dt):
    run_forward(handle, 3000, 72, k, gated=False, ydt=dt, kind="relu", residual=dt, z=dt)
    run_forward(handle, 3000, 72, k, gated=True, ydt=dt, kind="silu", z=dt)
    run_backward(handle, 260, k, 96, gated=False, dxdt=dt, dwdt=dt)


@pytest.mark.parametrize("rows", [5, 16, 33, 64, 100, 128, 130])
@pytest.mark.parametrize("c,k", [(64, 17), (600, 48), (600, 136), (4096, 16), (4096, 1000), (1024, 4100)])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_few_row_tiles(handle, rows, c, k, dtype):
    run_forward(handle, rows, c, k, gated=False, dtype=dtype, kind="silu", bias=True, residual=BF)
    run_forward(handle, rows, c, k, gated=True, dtype=dtype, z=F32, bias=True)


@pytest.mark.parametrize("rows,c,k", [(203, 61, 35), (1000, 147, 333), (65, 1109, 260), (1, 77, 13)])
@pytest.mark.parametrize("want", [("dx", "dw"), ("dx",), ("dw",)])
def test_backward_with_copied_operands(handle, rows, c, k, want):
    for kind, dydt in (("identity", BF), ("identity", F32), ("gelu", BF)):
        run_backward(handle, rows, c, k, gated=False, kind=kind, dydt=dydt, want=want)
        run_backward(handle, rows, c, k, gated=False, kind=kind, dydt=dydt, want=want, layout="odd", bias=False)
    run_backward(handle, rows, c, k, gated=True, want=want, layout="columns")


def test_released_while_its_kernels_run():
    """The workspace of an operator on a stream of its own outlives the operator
    until the kernels that use it are done."""
    x, w = rand(4000, 1000, seed=1, dtype=BF)[:, :999], rand(1024, 999, seed=2, dtype=BF)
    dy = rand(4000, 1024, seed=3, dtype=BF)
    want, got = torch.empty(1024, 999, dtype=BF, device="cuda"), torch.empty(1024, 999, dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with api.Handle(s) as h:
        op = api.LinearBackward(h, x, w, dy, dw=want)
        size = op.workspace.numel()
        op(x, w, dy, dw=want)
        torch.cuda.synchronize()
        for _ in range(20):
            op(x, w, dy, dw=got)
        del op
        other = torch.empty(size, dtype=torch.uint8, device="cuda")
        for _ in range(200):
            other.fill_(255)  # NaN, as BF16 and as FP32
        torch.cuda.synchronize()
    assert torch.equal(want, got)
