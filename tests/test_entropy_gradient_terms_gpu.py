"""Gradients of the cross entropy where dz enters the products in two BF16 terms: up to 128 rows, and up
to 2^30 products of a row, class and channel.  FP32 outputs show what the products were given."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from tests import channel_ref as cref
from tests import train_ref as ref
from tests.test_channel_ops_gpu import BF, F32, laid_out, out_like
from tests.test_train_ops_gpu import close, d, entropy_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


def gradients(handle, x, w, b, target, dloss, dx_dtype=F32, dw_dtype=F32, layout="dense"):
    rows, (v, c) = x.shape[0], w.shape
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse, bias=b)
    dx, dw, db = out_like(rows, c, dx_dtype, layout), out_like(v, c, dw_dtype), torch.full((v,), float("nan"), device="cuda")
    api.CrossEntropyBackward(handle, x, w, target, dx, dw)(x, w, target, lse, dloss, dx, dw, bias=b, dbias=db)
    return lse, dx, dw, db


def wanted(x, w, b, target, dloss, lse):
    """dx and dw of dz from the lse that the call was given, in FP64, and bounds of a step whose dz keeps 16 bits: its rounding
    2^-16, the exponential's 4e-6, and the logits' error, which the tensor core's additions leave."""
    z = d(x) @ d(w).t() + (0 if b is None else d(b))
    there = target >= 0
    p = torch.exp(z - d(lse)[:, None])
    one = torch.zeros_like(p).scatter_(1, target.clamp(min=0)[:, None], 1.0)
    weight = torch.where(there, d(dloss), 0.0)[:, None]
    dz = weight * (p - one)
    return dz @ d(w), dz.t() @ d(x), weight.abs() * p, dz


# one row, fragments of eight and sixteen, both sides of 16 and of 128 rows, single k-blocks and several, odd
# channels (no vectors), and sizes up to 2^30
SIZES = [(1, 64, 50), (2, 512, 3000), (5, 272, 80), (8, 41, 700), (9, 1024, 5000), (16, 784, 1392), (17, 96, 300), (40, 50, 1001), (63, 256, 2000),
         (64, 128, 777), (65, 64, 4000), (89, 64, 45120), (100, 333, 500), (127, 72, 1000), (128, 2048, 1000), (129, 128, 600), (256, 2048, 1000),
         (1000, 96, 400), (5000, 33, 70)]


@pytest.mark.parametrize("rows,c,v", SIZES)
@pytest.mark.parametrize("bias", [False, True])
def test_gradients_keep_the_bits_that_a_rounded_dz_has_not(handle, rows, c, v, bias):
    x, w, b, target, dloss = entropy_case(rows, c, v, bias)
    target[0] = 0
    lse, dx, dw, _ = gradients(handle, x, w, b, target, dloss)
    wx, ww, size, dz = wanted(x, w, b, target, dloss, lse)
    # in norm: dz's terms 2^-16; a logit is off by some 2^-24 (c / 16 + 8) of the sum of its |x w| (the accumulator's
    # additions of 16 products truncate), which is at most |x| |w|; the products' own additions likewise; a form that rounds
    # dz once is off by about 2^-9.3 = 0.0016 or, where the targets' -1 are most of dz, half of that
    logit = 2.0 ** -24 * (c / 16 + 8) * d(x).norm(dim=1).max() * d(w).norm(dim=1).max() + 4e-6
    shaken = (size * logit).norm()
    noise = dz * (torch.rand_like(dz) * 2 - 1) * 2.0 ** -8
    for got, want, other, rounded, chain in ((dx, wx, d(w), noise @ d(w), v), (dw, ww, d(x), noise.t() @ d(x), rows)):
        own = 2.0 ** -24 * (chain / 16 + 8)
        spread = torch.linalg.matrix_norm(other, 2)
        bound = (shaken + (2.0 ** -16 + own) * dz.norm()) * spread
        err = (d(got) - want).norm()
        assert err <= bound, (err / want.norm(), bound / want.norm())
        # and the bound says something: a tenth of a rounding of dz, taken through the same product
        assert err <= 0.1 * rounded.norm(), (err / want.norm(), rounded.norm() / want.norm())


@pytest.mark.parametrize("rows,c,v", [(1, 7, 9), (16, 200, 333), (33, 130, 257), (100, 51, 700), (128, 64, 100), (200, 147, 1003),
                                      (9, 1025, 600), (33, 530, 1100), (128, 1023, 700)])
@pytest.mark.parametrize("dx_dtype,dw_dtype,layout", [(BF, BF, "odd"), (F32, BF, "columns"), (BF, F32, "pitch")])
def test_types_and_layouts(handle, rows, c, v, dx_dtype, dw_dtype, layout):
    x, w, b, target, dloss = entropy_case(rows, c, v, True)
    x = laid_out(x, layout)
    lse, dx, dw, db = gradients(handle, x, w, b, target, dloss, dx_dtype, dw_dtype, layout)
    f = ref.cross_entropy(d(x), d(w), target, d(b))
    (wx, ex), (ww, ew), (wb, eb) = ref.cross_entropy_backward(d(x), d(w), target, f, d(dloss), dx_dtype, dw_dtype)
    close(dx, wx, ex, "dx")
    close(dw, ww, ew, "dw")
    close(db, wb, eb, "dbias")
    # BF16 outputs are the FP32 ones rounded
    _, fx, fw, _ = gradients(handle, x, w, b, target, dloss, layout=layout)
    for got, full in ((dx, fx), (dw, fw)):
        if got.dtype == BF:
            step = full.abs() * 2.0 ** -8 + 1e-38
            assert ((got.float() - full).abs() <= step).all()


@pytest.mark.parametrize("rows,c,v", [(16, 8, 4300000), (100, 16, 1500000)])
def test_terms_in_pieces_of_the_classes(handle, rows, c, v):
    x, w, b, target, dloss = entropy_case(rows, c, v, True)
    lse, dx, dw, db = gradients(handle, x, w, b, target, dloss, BF, F32)
    wx, ww, size, dz = wanted(x, w, b, target, dloss, lse)
    own = 2.0 ** -24 * (v / 16 + 8)
    close(dx, wx, cref.stored(wx, BF) + (size * 1e-5 + (2.0 ** -16 + own) * dz.abs()) @ d(w).abs(), "dx")
    close(dw, ww, (size * 1e-5 + 2.0 ** -15 * dz.abs()).t() @ d(x).abs() + 1e-30, "dw")


@pytest.mark.parametrize("rows,c,v", [(7, 600, 1200), (64, 601, 1100), (100, 64, 200)])
def test_each_alone_and_beside_others(handle, rows, c, v):
    """Any of the gradients without the others, a dx in the middle of a wider buffer."""
    x, w, b, target, dloss = entropy_case(rows, c, v, True)
    lse, dx, dw, db = gradients(handle, x, w, b, target, dloss, BF, F32)
    for which in range(3):
        outs = [torch.full_like(t, float("nan")) if i == which else None for i, t in enumerate((dx, dw, db))]
        op = api.CrossEntropyBackward(handle, x, w, target, outs[0], outs[1])
        op(x, w, target, lse, dloss, outs[0], outs[1], bias=b, dbias=outs[2])
        assert torch.equal(outs[which], (dx, dw, db)[which])
    wide = torch.full((rows + 2, c + 24), 7.0, dtype=BF, device="cuda")
    part = wide[1:-1, 8:8 + c]
    api.CrossEntropyBackward(handle, x, w, target, part)(x, w, target, lse, dloss, part, bias=b)
    assert torch.equal(part, dx)
    part.fill_(7.0)
    assert (wide == 7).all()


@pytest.mark.parametrize("rows", [5, 40, 200])
def test_non_finite_gradients_stay_where_they_are(handle, rows):
    """An infinite weight of a row: its infinities and NaN reach its dx, and dw, and no other row's dx."""
    x, w, b, target, dloss = entropy_case(rows, 64, 300, False)
    target = target.clamp(min=0)
    want = gradients(handle, x, w, None, target, dloss)[1]
    dloss[rows // 2] = float("inf")
    _, dx, dw, _ = gradients(handle, x, w, None, target, dloss)
    rest = [i for i in range(rows) if i != rows // 2]
    assert not torch.isfinite(dx[rows // 2]).any() and torch.equal(dx[rest], want[rest])
    assert not torch.isfinite(dw[target[rows // 2]]).any()
