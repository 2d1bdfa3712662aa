"""The ways of the cross entropy's forward call: the product's own epilogue, or FP32 logits in memory from a
product in parts or of few rows, on both sides of each border, with operands of any address, masks and
E4M3; and E4M3 operands in pieces of the classes."""
import math

import pytest
import torch

from deep_learning_convolution_gb300 import api
from deep_learning_convolution_gb300 import binding as B
from tests import train_ref as ref
from tests.test_channel_ops_gpu import BF, F8, F32, laid_out, out_like, rand
from tests.test_train_ops_gpu import check_entropy, classes_of, close, d, entropy_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


def shifted(t, by):
    """The same values, beginning `by` elements behind a vector's address, between values that are none."""
    out = torch.full((t.numel() + 16,), float("nan"), device="cuda").to(t.dtype)[by:by + t.numel()].view(t.shape)
    out.copy_(t)
    return out


# rows around 64 and 128, channels around 1024 and 2560, classes around 4096; few tiles and many; odd sizes
WAYS = [(64, 1024, 12), (65, 1024, 12), (65, 1016, 12), (65, 1023, 40), (65, 1025, 1), (128, 4096, 1000), (128, 1024, 500), (129, 2560, 300),
        (129, 2552, 300), (129, 2559, 300), (130, 1024, 300), (197, 2992, 232), (90, 2001, 333), (70, 1100, 4096), (70, 1100, 4097), (2000, 4000, 64),
        (512, 4096, 2048), (300, 2563, 77), (1000, 2600, 3)]


@pytest.mark.parametrize("rows,c,v", WAYS)
@pytest.mark.parametrize("bias", [False, True])
def test_either_way_of_few_classes(handle, rows, c, v, bias):
    check_entropy(handle, *entropy_case(rows, c, v, bias))


@pytest.mark.parametrize("rows,c,v", [(65, 1024, 12), (100, 2001, 333), (129, 2560, 300), (197, 2993, 232)])
@pytest.mark.parametrize("layout,by", [("odd", 1), ("columns", 3), ("pitch", 0), ("dense", 5)])
def test_few_classes_of_operands_at_any_address(handle, rows, c, v, layout, by):
    x, w, b, target, dloss = entropy_case(rows, c, v, True)
    check_entropy(handle, laid_out(x, layout), shifted(w, by), b, target.to(torch.int32), dloss, layout=layout)


@pytest.mark.parametrize("rows,c,v", [(100, 1024, 1000), (197, 2992, 232), (65, 4096, 9)])
def test_few_classes_that_are_masked(handle, rows, c, v):
    x, w, b, target, dloss = entropy_case(rows, c, v, True)
    b[::3] = float("-inf")
    b[1::3] = torch.finfo(F32).min
    target = torch.where(target < 3, -1, target // 3 * 3 - 1)
    loss, lse, dx, dw, db = check_entropy(handle, x, w, b, target, dloss)
    assert (db[::3] == 0).all() and (db[1::3] == 0).all() and (dw[::3] == 0).all()
    op = api.CrossEntropyForward(handle, x, w, target)
    target[0] = 3  # a target that is masked: an infinite loss
    op(x, w, target, loss, lse, bias=b)
    assert loss[0] == float("inf") and torch.isfinite(lse).all()
    b[:] = float("-inf")  # nothing is left
    op(x, w, target, loss, lse, bias=b)
    assert (lse == float("-inf")).all() and torch.isnan(loss[target >= 0]).all() and (loss[target < 0] == 0).all()


@pytest.mark.parametrize("rows,c,v", [(349, 3536, 3003), (686, 2560, 1634), (3129, 2784, 329), (622, 2720, 1985), (1400, 2944, 809)])
def test_logits_in_memory_only_where_the_product_is_dealt_out(handle, rows, c, v):
    """A few-row product of whole rows is neither more exact nor faster than the one with the loss's epilogue, whose
    workspace has no logits."""
    x, w, b, target, dloss = entropy_case(rows, c, v, True)
    assert api.CrossEntropyForward(handle, x, w, target)._ws_bytes < 4 * rows * v
    check_entropy(handle, x, w, b, target, dloss)


def e4m3_case(rows, c, v, seed=0):
    """Quantised rows and filters with their scales, a bias, targets; values as a model's logits have them."""
    x, w, b, target, _ = entropy_case(rows, c, v, True, seed)
    sx, sw = (t.float().abs().amax(1) / 448 for t in (x, w))
    return (x.float() / sx[:, None]).to(F8), (w.float() / sw[:, None]).to(F8), sx, sw, b, target


def check_e4m3(handle, qx, qw, sx, sw, b, target, rows_at_once=1 << 30):
    rows = qx.shape[0]
    loss, lse = out_like(rows, 1, F32)[:, 0], out_like(rows, 1, F32)[:, 0]
    op = api.CrossEntropyForward(handle, qx, qw, target)
    op(qx, qw, target, loss, lse, bias=b, x_scale=sx, w_scale=sw)
    for r in range(0, rows, rows_at_once):
        at = slice(r, r + rows_at_once)
        f = ref.cross_entropy(d(qx[at]), d(qw), target[at], d(b), d(sx[at]), d(sw))
        close(lse[at], *f["lse"], "lse")
        close(loss[at], *f["loss"], "loss")
    again = torch.full_like(loss, float("nan"))
    op(qx, qw, target, again, lse, bias=b, x_scale=sx, w_scale=sw)
    assert torch.equal(again, loss)
    return loss, lse


@pytest.mark.parametrize("rows,c,v", [(64, 1024, 12), (65, 1024, 12), (65, 1008, 12), (128, 4096, 1000), (129, 2560, 300), (129, 2544, 300), (197, 2992, 232),
                                      (90, 2001, 333), (2000, 4000, 64), (70, 1100, 4097)])
def test_either_way_of_e4m3(handle, rows, c, v):
    check_e4m3(handle, *e4m3_case(rows, c, v))


@pytest.mark.parametrize("rows,c,v", [(70, 1024, 333), (197, 2993, 232), (33, 257, 5000)])
@pytest.mark.parametrize("layout,by", [("odd", 1), ("pitch", 7)])
def test_e4m3_operands_at_any_address(handle, rows, c, v, layout, by):
    qx, qw, sx, sw, b, target = e4m3_case(rows, c, v)
    check_e4m3(handle, laid_out(qx, layout), shifted(qw, by), sx, sw, b, target)


def test_e4m3_of_few_rows_and_millions_of_classes(handle):
    """Logits in memory, in two pieces."""
    check_e4m3(handle, *e4m3_case(32, 16, 4300000))


def test_e4m3_of_many_rows_in_pieces(handle):
    """The rows' sums join those of the pieces before."""
    check_e4m3(handle, *e4m3_case(60000, 32, 20011), rows_at_once=10000)


@pytest.mark.parametrize("rows,c,v", [(3, 64, 1000), (40, 64, 5000), (300, 64, 3000), (100, 1024, 1000), (197, 2992, 232)])
def test_e4m3_of_masked_classes(handle, rows, c, v):
    qx, qw, sx, sw, b, target = e4m3_case(rows, c, v)
    b[::3] = float("-inf")
    b[1::3] = torch.finfo(F32).min
    target = torch.where(target < 3, -1, target // 3 * 3 - 1)
    loss, lse = check_e4m3(handle, qx, qw, sx, sw, b, target)
    target[0] = 3
    op = api.CrossEntropyForward(handle, qx, qw, target)
    op(qx, qw, target, loss, lse, bias=b, x_scale=sx, w_scale=sw)
    assert loss[0] == float("inf") and torch.isfinite(lse).all()
    b[:] = float("-inf")
    op(qx, qw, target, loss, lse, bias=b, x_scale=sx, w_scale=sw)
    assert (lse == float("-inf")).all() and torch.isnan(loss[target >= 0]).all() and (loss[target < 0] == 0).all()
    # rows of zeros: all classes that are left alike
    zero = torch.zeros_like(qx.float()).to(F8)
    b = torch.where(torch.arange(v, device="cuda") % 4 == 0, 0.0, float("-inf"))
    op(zero, qw, target, loss, lse, bias=b, x_scale=sx, w_scale=sw)
    close(lse, torch.full_like(lse, math.log((v + 3) // 4)).double(), torch.tensor(1e-5, device="cuda"), "lse")


@pytest.mark.parametrize("rows", [17, 33, 1000, 2 ** 17, 2 ** 20, 2 ** 25])
@pytest.mark.parametrize("v", [10, 1000, 131072])
def test_workspace_is_what_the_pieces_take(handle, rows, v):
    """Pieces of 512 MB of dz or logits, 256 MB of parts, and never less than 256 and 1024 classes."""
    c, mb = 64, 1 << 20
    x, w = B.dlcCreateTensorDescriptor(), B.dlcCreateFilterDescriptor()
    try:
        B.dlcSetTensor4dDescriptorEx(x, B.DLC_DATA_BFLOAT16, rows, c, 1, 1, c, 1, 0, 0)
        B.dlcSetFilter4dDescriptor(w, B.DLC_DATA_BFLOAT16, B.DLC_TENSOR_NCHW, v, c, 1, 1)
        forward, backward = (f(handle.h, x, 0, w, 0) for f in (B.dlcGetCrossEntropyForwardWorkspaceSize, B.dlcGetCrossEntropyBackwardWorkspaceSize))
    finally:
        B.dlcDestroyTensorDescriptor(x)
        B.dlcDestroyFilterDescriptor(w)
    # split products' partial sums: a tile of 256 x 256 for each pair of SMs; 64 rows at most keep logits
    products = 76 * 256 * 256 * 4 + mb
    parts = max(256 * mb, 33 * 8 * rows)
    logits = min(512 * mb, 4 * rows * (v + 3)) if rows <= 64 else 0
    assert forward <= parts + logits + 4 * rows + products
    dz = min(max(512 * mb, 512 * rows), (4 if rows <= 128 or rows * v * c <= 2 ** 30 else 2) * rows * (v + 7))
    assert backward <= dz + dz // 16 + 128 * (v + 7) + 1024 * v + (8 if rows <= 128 else 4) * rows * c + products
