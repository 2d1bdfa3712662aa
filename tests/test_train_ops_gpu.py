"""Layer norm, dropout, embedding and cross entropy on the GPU against their FP64
definitions, under the bounds derived in train_ref."""
import math

import numpy as np
import pytest
import torch

from deep_learning_convolution_gb300 import api
from deep_learning_convolution_gb300 import binding as B
from tests import channel_ref as cref
from tests import train_ref as ref
from tests.test_channel_ops_gpu import BF, F8, F32, laid_out, out_like, rand

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


def d(t):
    return None if t is None else t.double()


def close(got, want, err, what):
    bad = ~((got.double() - want).abs() <= err)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; first {bad.nonzero()[0].tolist()} "
                           f"got {got[bad][0].item()} want {want[bad][0].item()} err {err.expand_as(want)[bad][0].item()}")


def close_e4m3(q, scale, y, ey, what):
    """E4M3 values times their scales, and the scales themselves."""
    s, top = scale.double()[:, None], y.abs().amax(1, keepdim=True).clamp(min=1e-30)
    close(s, top / 448, (ey.amax(1, keepdim=True) + 4 * cref.U32 * top) / 448 + 1e-38, what + " scale")
    close(q.double() * s, y, cref.E4M3 * y.abs() + 1.1 * ey + 4 * cref.U32 * top + 2.0 ** -10 * s, what)


# ---- layer norm ------------------------------------------------------------------

SIZES = [(1, 1), (1, 4096), (3, 8), (5, 7), (2, 64), (33, 130), (300, 333), (65, 512), (17, 1000), (9, 1024), (4, 2048),
         (3, 5000), (2, 8192), (2, 12288), (1, 40000), (5000, 72), (3000, 768), (50, 300), (700, 2404), (3000, 1280), (400, 3584)]


@pytest.mark.parametrize("rows,c", SIZES)
@pytest.mark.parametrize("xdt,rdt,ydt", [(BF, BF, F8), (BF, BF, BF), (BF, F32, BF), (F32, F32, F32), (F32, BF, F8)])
def test_layer_norm(handle, rows, c, xdt, rdt, ydt):
    x, r = rand(rows, c, seed=1, dtype=xdt) + 1.5, rand(rows, c, seed=2, std=3.0, dtype=rdt)
    gamma, beta = 1 + 0.3 * rand(c, seed=3), rand(c, seed=4)
    total, y = out_like(rows, c, rdt), out_like(rows, c, ydt)
    scale = out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
    op = api.LayerNormForward(handle, x, y, residual=r, total=total, eps=EPS)
    op(x, gamma, y, beta=beta, residual=r, total=total, scale=scale)
    t, want, err = ref.layer_norm(d(x), d(r), d(gamma), d(beta), EPS)
    close(total, t, cref.stored(t, rdt) + cref.U32 * t.abs(), "total")
    if ydt == F8:
        close_e4m3(y, scale, want, err, "y")
    else:
        close(y, want, err + cref.stored(want, ydt), "y")


@pytest.mark.parametrize("layout", ["pitch", "odd", "columns"])
@pytest.mark.parametrize("rows,c", [(70, 96), (33, 51), (4, 1023)])
@pytest.mark.parametrize("ydt", [BF, F8])
def test_layer_norm_layouts_without_residual_or_beta(handle, rows, c, layout, ydt):
    x = laid_out(rand(rows, c, seed=1, dtype=BF), layout)
    y, gamma = out_like(rows, c, ydt, layout), 1 + 0.3 * rand(c, seed=3)
    scale = out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
    api.LayerNormForward(handle, x, y, eps=EPS)(x, gamma, y, scale=scale)
    _, want, err = ref.layer_norm(d(x), None, d(gamma), None, EPS)
    if ydt == F8:
        close_e4m3(y, scale, want, err, layout)
    else:
        close(y, want, err + cref.stored(want, ydt), layout)


@pytest.mark.parametrize("axes,crop", [("NCHW", False), ("NHWC", True), ("NHWC", False)])
def test_layer_norm_of_images(handle, axes, crop):
    big = rand(3, 7, 9, 40, seed=1, dtype=BF)
    image = big[:, 1:6, 2:8] if crop else big
    x = image.permute(0, 3, 1, 2).contiguous() if axes == "NCHW" else image
    y = torch.empty(x.shape, dtype=F32, device="cuda")
    gamma, beta = rand(40, seed=2), rand(40, seed=3)
    api.LayerNormForward(handle, x, y, eps=EPS, axes=axes)(x, gamma, y, beta=beta)
    _, want, err = ref.layer_norm(d(image).reshape(-1, 40), None, d(gamma), d(beta), EPS)
    rows = (y.permute(0, 2, 3, 1) if axes == "NCHW" else y).reshape(-1, 40)
    close(rows, want, err + cref.stored(want, F32), axes)


def pitched(t, pitch):
    """The same rows at a pitch of so many elements, NaN between them."""
    out = torch.full((t.shape[0], pitch), float("nan"), device=t.device).to(t.dtype)[:, :t.shape[1]]
    out.copy_(t)
    return out


# one thread's channels and a row's, vectors that begin with the last channel in front of a row, 257
# vectors of eight where 256 would do, rows with blocks of their own, and rows too long for shared memory
@pytest.mark.parametrize("rows,c", [(1, 5), (9, 8), (300, 1), (70, 57), (1000, 130), (41, 250), (33, 1024), (4001, 256), (700, 1001), (64, 2048),
                                    (19, 4033), (7, 4096), (11, 8185), (3, 16381)])
@pytest.mark.parametrize("pad,y_pad", [(0, 0), (5, 0), (5, 5), (3, 1), (8, 7), (1, 16)])
@pytest.mark.parametrize("dtype,ydt", [(BF, BF), (BF, F8), (BF, F32), (F32, F32), (F32, BF), (F32, F8)])
def test_layer_norm_of_rows_that_begin_anywhere(handle, rows, c, pad, y_pad, dtype, ydt):
    x, r = (pitched(rand(rows, c, seed=s, std=2.0, dtype=dtype), c + pad) for s in (1, 2))
    gamma, beta = 1 + 0.3 * rand(c, seed=3), rand(c, seed=4)
    whole = torch.full((rows, c + y_pad), 7.0, device="cuda").to(ydt)
    y, scale = whole[:, :c], out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
    t, want, err = ref.layer_norm(d(x), d(r), d(gamma), d(beta), EPS)
    dy, dt = (pitched(rand(rows, c, seed=s, dtype=dtype), c + pad) for s in (5, 6))
    api.LayerNormForward(handle, x, y, residual=r, total=x, eps=EPS)(x, gamma, y, beta=beta, residual=r, total=x, scale=scale)
    close(x, t, cref.stored(t, dtype) + cref.U32 * t.abs(), "total")
    if ydt == F8:
        close_e4m3(y, scale, want, err, "y")
    else:
        close(y, want, err + cref.stored(want, ydt), "y")
    assert (whole[:, c:].float() == 7).all()
    between = x.as_strided((rows - 1, pad), (c + pad, 1), c)  # (behind the last row is nothing that a view has)
    assert torch.isnan(between.float()).all()
    dx, dg, db = pitched(torch.zeros(rows, c, device="cuda").to(dtype), c + pad), out_like(c, 1, F32)[:, 0], out_like(c, 1, F32)[:, 0]
    (want, ex), (wg, eg), (wb, eb) = ref.layer_norm_backward(d(dy), d(x), d(gamma), d(dt), EPS)
    api.LayerNormBackward(handle, dy, x, dx, dtotal=dt, eps=EPS)(dy, x, gamma, dx, dgamma=dg, dbeta=db, dtotal=dt)
    close(dx, want, ex + cref.stored(want, dtype), "dx")
    close(dg, wg, eg + 1e-30, "dgamma")
    close(db, wb, eb + 1e-30, "dbeta")
    assert torch.isnan(dx.as_strided((rows - 1, pad), (c + pad, 1), c).float()).all()


@pytest.mark.parametrize("c", [256, 100, 5000])
@pytest.mark.parametrize("layout", ["dense", "columns"])
def test_layer_norm_in_place_equal_and_non_finite_rows(handle, c, layout):
    r, x = laid_out(rand(6, c, seed=1), layout), laid_out(rand(6, c, seed=2, dtype=BF), layout)
    x[1], r[1] = 0, 0.5
    r[2, c // 2], r[4, 0] = float("nan"), float("inf")
    gamma, beta = 1 + 0.3 * rand(c, seed=3), rand(c, seed=4)
    y, scale = out_like(6, c, F8, layout), out_like(6, 1, F32)[:, 0]
    t, want, err = ref.layer_norm(d(x), d(r), d(gamma), d(beta), EPS)
    api.LayerNormForward(handle, x, y, residual=r, total=r, eps=EPS)(x, gamma, y, beta=beta, residual=r, total=r, scale=scale)
    good = [0, 1, 3, 5]
    close(r[good], t[good], cref.stored(t[good], F32) + cref.U32 * t[good].abs(), "total in place")
    close_e4m3(y[good], scale[good], want[good], err[good], "y")
    assert torch.isnan(y[2].float()).all() and torch.isnan(y[4].float()).all()


@pytest.mark.parametrize("rows,c,dtype", [(40, 768, BF), (700, 2048, BF), (33, 300, F32), (9, 100, BF)])
def test_layer_norm_of_one_type_in_place(handle, rows, c, dtype):
    """The sum in the place of either operand, the gradient in that of dtotal."""
    gamma, beta, y = 1 + 0.3 * rand(c, seed=3), rand(c, seed=4), torch.empty(rows, c, dtype=dtype, device="cuda")
    for place in range(2):
        ops = [laid_out(rand(rows, c, seed=s, dtype=dtype), "pitch") for s in (1, 2)]
        t, want, err = ref.layer_norm(d(ops[0]), d(ops[1]), d(gamma), d(beta), EPS)
        api.LayerNormForward(handle, ops[0], y, residual=ops[1], total=ops[place], eps=EPS)(
            ops[0], gamma, y, beta=beta, residual=ops[1], total=ops[place])
        close(ops[place], t, cref.stored(t, dtype) + cref.U32 * t.abs(), "total")
        close(y, want, err + cref.stored(want, dtype), "y")
    dt = ops[0]
    (want, ex), _, _ = ref.layer_norm_backward(d(y), d(ops[1]), d(gamma), d(dt), EPS)
    api.LayerNormBackward(handle, y, ops[1], dt, dtotal=dt, eps=EPS)(y, ops[1], gamma, dt, dtotal=dt)
    close(dt, want, ex + cref.stored(want, dtype), "dx")


@pytest.mark.parametrize("rows,c,pad", [(70, 256, 0), (70, 1001, 7), (70, 1001, 0)])
def test_broadcast_residuals_are_read_by_their_strides(handle, rows, c, pad):
    """A residual of one row for all."""
    x, one = pitched(rand(rows, c, seed=1, dtype=BF), c + pad), rand(1, c, seed=2, dtype=BF)
    y = pitched(torch.zeros(rows, c, device="cuda").to(BF), c + pad)
    many, g = one.expand(rows, c), torch.ones(c, device="cuda")
    try:
        op = api.LayerNormForward(handle, x, y, residual=many, eps=EPS)
    except B.DlcError as e:  # strides of zero are none that a descriptor takes
        assert e.status == B.DLC_STATUS_BAD_PARAM
        return
    op(x, g, y, residual=many)
    _, want, err = ref.layer_norm(d(x), d(many), d(g), None, EPS)
    close(y, want, err + cref.stored(want, BF), "layer norm")
    api.DropoutForward(handle, x, y, p=0.5, residual=many)(x, words(1, 2), y, residual=many)
    want, _ = ref.dropout(d(x), d(many), 0.5, 1, 2)
    close(y, want, cref.stored(want, BF) + 4 * cref.U32 * (want.abs() + d(many).abs()), "dropout")


@pytest.mark.parametrize("c", [64, 768, 5000])
def test_layer_norm_of_rows_far_from_zero(handle, c):
    """The variance is about the mean: a mean of 300 deviations costs what the rounding of the
    mean costs, and one large channel nothing."""
    x = rand(40, c, seed=1) + 300.0
    x[20:] -= 300.0
    x[20:, 0] += 1000.0
    y, gamma = torch.empty_like(x), torch.ones(c, device="cuda")
    api.LayerNormForward(handle, x, y, eps=EPS)(x, gamma, y)
    _, want, err = ref.layer_norm(d(x), None, d(gamma), None, EPS)
    close(y, want, err + cref.stored(want, F32), "y")
    # the bound says something: 300 U32 (c / 8 + 64) (1 + |n| mean |n|), 0.062 for 5000 channels and
    # |n| = 5; a mean square less the squared mean is off by 300^2 U32 (c / 8 + 64), 0.39 for 64
    assert err[:20].max() < 0.1


@pytest.mark.parametrize("rows,c", [(1, 1), (1, 4096), (3, 7), (100, 96), (257, 333), (1000, 512), (40, 1024), (9, 4097),
                                    (5, 8192), (3, 12288), (2, 20000), (7000, 64), (50, 300), (700, 2404), (900, 2560), (500, 3600), (3000, 768)])
@pytest.mark.parametrize("dt,with_dt,sums", [(BF, True, "both"), (F32, False, "both"), (BF, False, None), (F32, True, "gamma"),
                                             (BF, True, "beta")])
def test_layer_norm_backward(handle, rows, c, dt, with_dt, sums):
    dy, t = rand(rows, c, seed=1, dtype=dt), rand(rows, c, seed=2, std=2.0, dtype=dt) + 1
    dtot = rand(rows, c, seed=3, dtype=dt) if with_dt else None
    gamma, dx = 1 + 0.3 * rand(c, seed=4), out_like(rows, c, dt)
    dgamma = out_like(c, 1, F32)[:, 0] if sums in ("both", "gamma") else None
    dbeta = out_like(c, 1, F32)[:, 0] if sums in ("both", "beta") else None
    api.LayerNormBackward(handle, dy, t, dx, dtotal=dtot, eps=EPS)(dy, t, gamma, dx, dgamma=dgamma, dbeta=dbeta, dtotal=dtot)
    (want, ex), (wg, eg), (wb, eb) = ref.layer_norm_backward(d(dy), d(t), d(gamma), d(dtot), EPS)
    close(dx, want, ex + cref.stored(want, dt), "dx")
    if dgamma is not None:
        close(dgamma, wg, eg + 1e-30, "dgamma")
    if dbeta is not None:
        close(dbeta, wb, eb + 1e-30, "dbeta")


@pytest.mark.parametrize("layout", ["pitch", "odd", "columns"])
@pytest.mark.parametrize("ydt", [BF, F32])
def test_layer_norm_backward_layouts_in_place(handle, layout, ydt):
    rows, c = 77, 90
    dy, t = laid_out(rand(rows, c, seed=1, dtype=ydt), layout), laid_out(rand(rows, c, seed=2, dtype=BF), layout)
    dx = laid_out(rand(rows, c, seed=3, dtype=BF), layout)  # dtotal, overwritten
    gamma, dgamma, dbeta = 1 + 0.3 * rand(c, seed=4), out_like(c, 1, F32)[:, 0], out_like(c, 1, F32)[:, 0]
    (want, ex), (wg, eg), (wb, eb) = ref.layer_norm_backward(d(dy), d(t), d(gamma), d(dx), EPS)
    api.LayerNormBackward(handle, dy, t, dx, dtotal=dx, eps=EPS)(dy, t, gamma, dx, dgamma=dgamma, dbeta=dbeta, dtotal=dx)
    close(dx, want, ex + cref.stored(want, BF), "dx")
    close(dgamma, wg, eg + 1e-30, "dgamma")
    close(dbeta, wb, eb + 1e-30, "dbeta")


def test_layer_norm_gradient_is_that_of_the_forward_call(handle):
    """dx, dgamma and dbeta against central differences of the FP32 forward call."""
    rows, c, h = 6, 48, 2.0 ** -6
    t, dy, gamma, beta = rand(rows, c, seed=1), rand(rows, c, seed=2), 1 + 0.3 * rand(c, seed=3), rand(c, seed=4)
    dx, dgamma, dbeta, y = torch.empty_like(t), torch.empty_like(gamma), torch.empty_like(beta), torch.empty_like(t)
    api.LayerNormBackward(handle, dy, t, dx, eps=EPS)(dy, t, gamma, dx, dgamma=dgamma, dbeta=dbeta)
    op = api.LayerNormForward(handle, t, y, eps=EPS)

    def along(which, step):
        args = [t.clone(), gamma.clone(), beta.clone()]
        args[which] += step
        op(args[0], args[1], y, beta=args[2])
        return (d(dy) * d(y)).sum().item()

    # FP32 outputs of size 4 at most, 288 of them: 2^-24 * 4 * 288 / h rounding at most;
    # the cubic term of a step h in a row of size one: h^2 times derivatives of order one
    for which, grad in ((0, dx), (1, dgamma), (2, dbeta)):
        v = rand(*grad.shape, seed=9)
        v /= v.norm()
        got = (along(which, h * v) - along(which, -h * v)) / (2 * h)
        want = (d(grad) * d(v)).sum().item()
        assert abs(got - want) <= 2.0 ** -24 * 4 * 288 / h + 4 * h * h * d(dy).norm().item(), which


# ---- dropout ---------------------------------------------------------------------

def words(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("rows,c", [(1, 1), (3, 5), (1, 4096), (70, 96), (33, 51), (777, 1001), (4001, 256), (2, 40000)])
@pytest.mark.parametrize("xdt,rdt,ydt", [(BF, None, BF), (BF, BF, BF), (F32, F32, F32), (F32, BF, BF), (BF, F32, F32), (F32, None, F32)])
@pytest.mark.parametrize("p", [0.1, 0.75])
def test_dropout(handle, rows, c, xdt, rdt, ydt, p):
    x, r = rand(rows, c, seed=1, dtype=xdt), None if rdt is None else rand(rows, c, seed=2, dtype=rdt)
    y, seed, step = out_like(rows, c, ydt), -5 - rows, 2 ** 40 + c
    api.DropoutForward(handle, x, y, p=p, residual=r)(x, words(seed, step), y, residual=r)
    want, keep = ref.dropout(d(x), d(r), p, seed, step)
    # the scale's rounding, the product's and the sum's
    scaled = want if r is None else want - d(r)
    close(y, want, cref.stored(want, ydt) + cref.U32 * (2 * scaled.abs() + want.abs()), "y")
    if r is None:
        assert torch.equal(y != 0, keep & (x != 0))
    dy, dx = rand(rows, c, seed=3, dtype=ydt), out_like(rows, c, xdt)
    api.DropoutBackward(handle, dy, dx, p=p)(dy, words(seed, step), dx)
    want, _ = ref.dropout(d(dy), None, p, seed, step)
    close(dx, want, cref.stored(want, xdt) + 3 * cref.U32 * want.abs(), "dx")


@pytest.mark.parametrize("layout", ["pitch", "odd", "columns"])
@pytest.mark.parametrize("rows,c", [(70, 96), (33, 51), (300, 3)])
def test_dropout_layouts_have_one_mask(handle, rows, c, layout):
    dense = rand(rows, c, seed=1, dtype=BF)
    x, r, y = laid_out(dense, layout), laid_out(rand(rows, c, seed=2, dtype=BF), layout), out_like(rows, c, BF, layout)
    api.DropoutForward(handle, x, y, p=0.3, residual=r)(x, words(1, 2), y, residual=r)
    want, keep = ref.dropout(d(dense), d(r), 0.3, 1, 2)
    close(y, want, cref.stored(want, BF) + 4 * cref.U32 * (want.abs() + d(r).abs()), layout)
    mixed = torch.empty(rows, c, device="cuda")  # one side dense, the other in this layout
    api.DropoutForward(handle, x, mixed, p=0.3)(x, words(1, 2), mixed)
    assert torch.equal(mixed != 0, keep & (dense != 0))
    image = laid_out(rand(rows, c, seed=4, dtype=F32), layout)
    api.DropoutBackward(handle, dense, image, p=0.3)(dense, words(1, 2), image)
    assert torch.equal(image != 0, keep & (dense != 0))


@pytest.mark.parametrize("rows,c", [(1, 192), (2, 1001), (7, 250), (9, 333), (1000, 257), (4001, 198), (31, 4093)])
@pytest.mark.parametrize("pad", [0, 1, 2, 3, 4, 5, 6, 7])
def test_dropout_of_rows_that_begin_anywhere(handle, rows, c, pad):
    x, r = (pitched(rand(rows, c, seed=s, dtype=BF), c + pad) for s in (1, 2))
    for res in (r, None):
        y = pitched(torch.zeros(rows, c, device="cuda").to(BF), c + pad)
        api.DropoutForward(handle, x, y, p=0.4, residual=res)(x, words(7, rows), y, residual=res)
        want, _ = ref.dropout(d(x), d(res), 0.4, 7, rows)
        close(y, want, cref.stored(want, BF) + cref.U32 * (3 * want.abs() + (0 if res is None else 3 * d(res).abs())), "y")
        assert torch.isnan(y.as_strided((rows - 1, pad), (c + pad, 1), c).float()).all()
    # in place, and the neighbours of the first and the last row
    whole = torch.full((rows * (c + pad) + 16,), 3.0, device="cuda").to(BF)
    y = whole[8:8 + rows * (c + pad)].view(rows, c + pad)[:, :c]
    y.copy_(x)
    want, _ = ref.dropout(d(x), None, 0.4, 7, rows)
    api.DropoutBackward(handle, y, y, p=0.4)(y, words(7, rows), y)
    close(y, want, cref.stored(want, BF) + 3 * cref.U32 * want.abs(), "in place")
    y.fill_(3.0)
    assert (whole == 3).all()


def test_dropout_of_images_counts_pixels_in_order(handle):
    x = rand(2, 20, 5, 6, seed=1)  # NCHW
    y = torch.empty_like(x)
    api.DropoutForward(handle, x, y, p=0.4, axes="NCHW")(x, words(3, 4), y)
    _, keep = ref.dropout(d(x.permute(0, 2, 3, 1).reshape(-1, 20)), None, 0.4, 3, 4)
    assert torch.equal((y != 0).permute(0, 2, 3, 1).reshape(-1, 20), keep)
    crop = rand(2, 7, 9, 32, seed=1, dtype=BF)[:, 1:6, 2:8]
    z = torch.empty(2, 5, 6, 32, dtype=BF, device="cuda")
    api.DropoutForward(handle, crop, z, p=0.4)(crop, words(3, 4), z)
    _, keep = ref.dropout(d(crop).reshape(-1, 32), None, 0.4, 3, 4)
    assert torch.equal((z != 0).reshape(-1, 32), keep & (crop != 0).reshape(-1, 32))


def test_dropout_in_place_of_everything_nothing_and_not_finite(handle):
    x, r = rand(50, 64, seed=1, dtype=BF), rand(50, 64, seed=2, dtype=BF)
    want, keep = ref.dropout(d(x), d(r), 0.5, 9, 9)
    y = r.clone()
    api.DropoutForward(handle, x, y, p=0.5, residual=y)(x, words(9, 9), y, residual=y)
    close(y, want, cref.stored(want, BF) + 4 * cref.U32 * (want.abs() + d(r).abs()), "residual in place")
    z = x.clone()
    api.DropoutForward(handle, z, z, p=0.5)(z, words(9, 9), z)
    assert torch.equal(z, torch.where(keep, 2 * x, 0.0))  # exact: a scale of two
    api.DropoutForward(handle, x, z, p=0.0)(x, words(9, 9), z)
    assert torch.equal(z, x)
    bad = torch.where(keep, x, float("nan"))
    bad[0] = torch.where(keep[0], bad[0], float("inf"))
    api.DropoutForward(handle, bad, z, p=0.5)(bad, words(9, 9), z)
    assert torch.equal(z, torch.where(keep, 2 * x, 0.0))
    most = 1 - 2.0 ** -31  # two words of 2^32 keep
    api.DropoutForward(handle, x, z, p=most)(x, words(9, 9), z)
    assert (z == 0).all()


def test_dropout_of_a_replayed_graph_follows_its_words(handle):
    x, y, state = rand(100, 96, seed=1), torch.empty(100, 96, device="cuda"), words(5, 0)
    op = api.DropoutForward(handle, x, y, p=0.5)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        handle.set_stream(stream)
        try:
            op(x, state, y)
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                handle.set_stream(torch.cuda.current_stream())
                op(x, state, y)
                state[1:] += 1
        finally:
            handle.set_stream(stream)
        for step in range(3):
            graph.replay()
            stream.synchronize()
            assert torch.equal(y != 0, ref.dropout(d(x), None, 0.5, 5, step)[1])
    handle.set_stream(torch.cuda.current_stream())


# ---- embedding -------------------------------------------------------------------

def tokens_of(n, v, seed, dtype=torch.int64):
    """Tokens of very different frequencies, some of none."""
    g = torch.Generator().manual_seed(seed)
    t = (torch.rand(n, generator=g).double() * math.log(v + 1)).exp().long().clamp(max=v) - 1
    t = torch.where(torch.rand(n, generator=g) < 0.1, -1, t * 7919 % v)
    return t.to(dtype).cuda()


@pytest.mark.parametrize("rows,c,v", [(1, 1, 1), (1, 4096, 50), (64, 512, 1000), (33, 51, 7), (4001, 96, 70000), (3, 8, 300)])
@pytest.mark.parametrize("tdt,ydt,idt", [(BF, BF, torch.int64), (F32, F32, torch.int32), (BF, F32, torch.int32), (F32, BF, torch.int64)])
@pytest.mark.parametrize("layout", ["dense", "pitch", "odd", "columns"])
def test_embedding(handle, rows, c, v, tdt, ydt, idt, layout):
    table, tokens = rand(v, c, seed=1, dtype=tdt), tokens_of(rows, v, 2, idt)
    y = out_like(rows, c, ydt, layout)
    api.EmbeddingForward(handle, tokens, table, y, scale=3.7)(tokens, table, y)
    want = ref.embedding(tokens, d(table), float(np.float32(3.7)))
    close(y, want, cref.stored(want, ydt) + cref.U32 * want.abs(), "y")


@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 64, 100, 2047, 2048, 2049, 5000, 70000])
@pytest.mark.parametrize("c,v", [(64, 1000), (51, 3), (16, 70000)])
@pytest.mark.parametrize("ddt,tdt", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_backward(handle, rows, c, v, ddt, tdt, accumulate):
    dy, tokens = rand(rows, c, seed=1, dtype=ddt), tokens_of(rows, v, rows, torch.int32 if rows % 2 else torch.int64)
    before = rand(v, c, seed=3, dtype=tdt)
    dt = before.clone() if accumulate else out_like(v, c, tdt)
    op = api.EmbeddingBackward(handle, tokens, dy, dt, scale=0.5, accumulate=accumulate)
    op(tokens, dy, dt)
    want, err = ref.embedding_backward(tokens, d(dy), v, 0.5, d(before) if accumulate else None)
    close(dt, want, err + cref.stored(want, tdt), "dtable")
    if accumulate:  # rows of no token: not touched
        rest = torch.ones(v, dtype=torch.bool, device="cuda")
        rest[tokens[tokens >= 0].long()] = False
        assert torch.equal(dt[rest], before[rest])
    again = before.clone() if accumulate else out_like(v, c, tdt)
    op(tokens, dy, again)
    assert torch.equal(dt, again)


@pytest.mark.parametrize("rows,c,v", [(9000, 264, 5), (300, 2056, 1), (130000, 8, 40), (300001, 8, 3), (300001, 8, 200000)])
def test_embedding_backward_of_few_tokens(handle, rows, c, v):
    """Every token's rows reach over many blocks."""
    dy, dt = rand(rows, c, seed=1, dtype=BF), out_like(v, c, F32)
    tokens = torch.randint(-1, v, (rows,), generator=torch.Generator().manual_seed(2)).cuda()
    api.EmbeddingBackward(handle, tokens, dy, dt)(tokens, dy, dt)
    want, err = ref.embedding_backward(tokens, d(dy), v, 1.0)
    close(dt, want, err + cref.stored(want, F32), "dtable")


@pytest.mark.parametrize("layout", ["pitch", "odd", "columns"])
def test_embedding_backward_layouts(handle, layout):
    rows, c, v = 333, 90, 64
    dy, tokens, dt = laid_out(rand(rows, c, seed=1, dtype=BF), layout), tokens_of(rows, v, 5), out_like(v, c, BF)
    api.EmbeddingBackward(handle, tokens, dy, dt)(tokens, dy, dt)
    want, err = ref.embedding_backward(tokens, d(dy), v, 1.0)
    close(dt, want, err + cref.stored(want, BF), layout)


def test_embedding_of_pixels_and_no_tokens_at_all(handle):
    tokens = tokens_of(2 * 5 * 6, 30, 1).view(2, 5, 6)
    table, y = rand(30, 24, seed=2, dtype=BF), torch.empty(2, 24, 5, 6, device="cuda")
    api.EmbeddingForward(handle, tokens, table, y, axes="NCHW")(tokens, table, y)
    want = ref.embedding(tokens.view(-1), d(table), 1.0)
    assert torch.equal(d(y).permute(0, 2, 3, 1).reshape(-1, 24), want)
    dt, grad = out_like(30, 24, F32), rand(2, 24, 5, 6, seed=3)
    api.EmbeddingBackward(handle, tokens, grad, dt, axes="NCHW")(tokens, grad, dt)
    want, err = ref.embedding_backward(tokens.view(-1), d(grad.permute(0, 2, 3, 1).reshape(-1, 24)), 30, 1.0)
    close(dt, want, err + 1e-30, "dtable")
    none = torch.full((60,), -7, device="cuda").view(2, 5, 6)
    api.EmbeddingForward(handle, none, table, y, axes="NCHW", scale=2.0)(none, table, y)
    assert (y == 0).all()
    api.EmbeddingBackward(handle, none, grad, dt, axes="NCHW")(none, grad, dt)
    assert (dt == 0).all()


@pytest.mark.parametrize("rows", [40, 5000])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_tokens_beyond_the_table_are_reported(rows, idt):
    with api.Handle() as h:
        table, y, dt = rand(30, 24, seed=2), out_like(rows, 24, F32), out_like(30, 24, F32)
        tokens = torch.randint(0, 30, (rows,), generator=torch.Generator().manual_seed(2)).to(idt)
        far = [30, 2 ** 31 - 1] if idt == torch.int32 else [30, 2 ** 32, 2 ** 62]
        for i, t in enumerate(far):
            tokens[17 + i] = t
        tokens = tokens.cuda()
        good = torch.where(tokens < 30, tokens, -1)
        fwd, bwd = api.EmbeddingForward(h, tokens, table, y), api.EmbeddingBackward(h, tokens, y, dt)
        for call in (lambda: fwd(tokens, table, y), lambda: bwd(tokens, y, dt)):
            call()
            torch.cuda.synchronize()
            with pytest.raises(B.DlcError):
                fwd(tokens, table, y)  # the handle's next call
            code, detail = B.dlcGetLastDeviceError(h.h)
            assert code == B.DLC_DEVERR_INDEX and 17 <= detail < 17 + len(far)
        assert torch.equal(d(y), ref.embedding(good, d(table), 1.0))
        want, err = ref.embedding_backward(good, d(y), 30, 1.0)
        close(dt, want, err + 1e-30, "dtable")
        fwd(good, table, y)
        h.synchronize()


# ---- cross entropy ----------------------------------------------------------------

def classes_of(rows, v, seed):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, v, (rows,), generator=g)
    return torch.where(torch.rand(rows, generator=g) < 0.15, -100, t).cuda()


def entropy_case(rows, c, v, bias, seed=0):
    x, w = rand(rows, c, seed=seed + 1, dtype=BF), rand(v, c, seed=seed + 2, std=3 * c ** -0.5, dtype=BF)
    b = rand(v, seed=seed + 3) if bias else None
    return x, w, b, classes_of(rows, v, seed + 4), rand(rows, seed=seed + 5).abs() / rows


def check_entropy(handle, x, w, b, target, dloss, dx_dtype=BF, dw_dtype=BF, layout="dense"):
    rows, (v, c) = x.shape[0], w.shape
    loss, lse = out_like(rows, 1, F32)[:, 0], out_like(rows, 1, F32)[:, 0]
    fwd = api.CrossEntropyForward(handle, x, w, target)
    fwd(x, w, target, loss, lse, bias=b)
    f = ref.cross_entropy(d(x), d(w), target, d(b))
    close(lse, *f["lse"], "lse")
    close(loss, *f["loss"], "loss")
    dx, dw = out_like(rows, c, dx_dtype, layout), out_like(v, c, dw_dtype)
    db = out_like(v, 1, F32)[:, 0]
    bwd = api.CrossEntropyBackward(handle, x, w, target, dx, dw)
    bwd(x, w, target, lse, dloss, dx, dw, bias=b, dbias=db)
    (wx, ex), (ww, ew), (wb, eb) = ref.cross_entropy_backward(d(x), d(w), target, f, d(dloss), dx_dtype, dw_dtype)
    close(dx, wx, ex, "dx")
    close(dw, ww, ew, "dw")
    close(db, wb, eb, "dbias")
    again = [torch.full_like(t, float("nan")) for t in (loss, lse, dx, dw, db)]
    fwd(x, w, target, again[0], again[1], bias=b)
    if layout == "dense":  # (an example's strides are its own)
        bwd(x, w, target, lse, dloss, again[2], again[3], bias=b, dbias=again[4])
        for one, two in zip((loss, lse, dx, dw, db), again):
            assert torch.equal(one, two)
    return loss, lse, dx, dw, db


ENTROPY_SIZES = [(1, 1, 1), (100, 64, 1), (90, 8, 7), (1, 64, 1000), (3, 8, 2), (5, 7, 11), (4, 512, 5001), (33, 130, 257), (64, 256, 1000), (200, 147, 1003),
                 (300, 64, 256), (256, 512, 4096), (513, 72, 777), (1000, 128, 9000), (2, 64, 70000), (17, 1032, 12345)]


@pytest.mark.parametrize("rows,c,v", ENTROPY_SIZES)
@pytest.mark.parametrize("bias", [False, True])
def test_cross_entropy(handle, rows, c, v, bias):
    check_entropy(handle, *entropy_case(rows, c, v, bias))


@pytest.mark.parametrize("rows,c,v", [(77, 96, 500), (300, 51, 333), (600, 128, 6000)])
@pytest.mark.parametrize("dx_dtype,dw_dtype,layout", [(F32, F32, "dense"), (BF, F32, "odd"), (F32, BF, "columns"), (BF, BF, "pitch")])
def test_cross_entropy_types_and_layouts(handle, rows, c, v, dx_dtype, dw_dtype, layout):
    x, w, b, target, dloss = entropy_case(rows, c, v, True)
    check_entropy(handle, laid_out(x, layout), w, b, target.to(torch.int32), dloss, dx_dtype, dw_dtype, layout)


@pytest.mark.parametrize("rows", [1, 2, 3])
@pytest.mark.parametrize("c,v,layout", [(5, 64, "dense"), (41, 5003, "odd"), (38, 700, "pitch"), (64, 900, "odd"), (64, 901, "columns"), (1, 88, "dense"),
                                        (366, 1, "columns")])
def test_cross_entropy_of_single_rows_of_any_layout(handle, rows, c, v, layout):
    """Operands that vectors do not reach, as they are and as copies with padded rows."""
    x, w, b, target, dloss = entropy_case(rows, c, v, True)
    x, target = laid_out(x, layout), torch.arange(rows, device="cuda") % v
    check_entropy(handle, x, w, b, target, dloss, layout=layout)
    shifted = torch.empty(v * c + 1, dtype=BF, device="cuda")[1:].view(v, c)  # not at a vector's address
    shifted.copy_(w)
    check_entropy(handle, x, shifted, b, target, dloss, layout=layout)


@pytest.mark.parametrize("rows,c,v", [(16, 200, 333), (32, 4096, 70), (31, 24, 15), (17, 8, 1), (8, 72, 40000), (15, 64, 16), (33, 128, 100), (1, 1024, 5)])
@pytest.mark.parametrize("dw_dtype,layout", [(BF, "dense"), (F32, "columns"), (BF, "odd")])
def test_cross_entropy_filters_of_few_rows(handle, rows, c, v, dw_dtype, layout):
    x, w, b, target, dloss = entropy_case(rows, c, v, True)
    loss, lse, dx, dw, db = check_entropy(handle, laid_out(x, layout), w, b, target, dloss, dw_dtype=dw_dtype, layout=layout)
    # the rows of its own and no others
    whole = torch.full((v + 2, c), 5.0, dtype=dw_dtype, device="cuda")
    api.CrossEntropyBackward(handle, x, w, target, None, whole[1:-1])(x, w, target, lse, dloss, dw=whole[1:-1], bias=b)
    assert torch.equal(whole[1:-1], dw) and (whole[0] == 5).all() and (whole[-1] == 5).all()


@pytest.mark.parametrize("rows,c,v", [(1, 40, 600), (2, 24, 513), (3, 41, 700), (1, 41, 5000), (1, 7, 1)])
def test_cross_entropy_of_single_e4m3_rows(handle, rows, c, v):
    x, w = rand(rows, c, seed=1).to(F8), rand(v, c, seed=2, std=0.5).to(F8)
    sx, sw, target = rand(rows, seed=3).abs() + 0.1, rand(v, seed=4).abs() + 0.1, torch.arange(rows, device="cuda") % v
    loss, lse = out_like(rows, 1, F32)[:, 0], out_like(rows, 1, F32)[:, 0]
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse, x_scale=sx, w_scale=sw)
    f = ref.cross_entropy(d(x), d(w), target, None, d(sx), d(sw))
    close(lse, *f["lse"], "lse")
    close(loss, *f["loss"], "loss")


@pytest.mark.parametrize("rows,c,v", [(8192, 64, 40000), (5000, 40, 70001), (9000, 41, 33001)])
@pytest.mark.parametrize("dx_dtype", [F32, BF])
def test_cross_entropy_in_pieces_of_the_classes(handle, rows, c, v, dx_dtype):
    check_entropy(handle, *entropy_case(rows, c, v, True), dx_dtype=dx_dtype)


def test_cross_entropy_of_few_rows_and_millions_of_classes(handle):
    """Logits in memory, in two pieces."""
    check_entropy(handle, *entropy_case(32, 8, 4300000, True))


def test_cross_entropy_of_many_rows_in_pieces(handle):
    """The rows' sums join those of the pieces before."""
    rows, c, v = 60000, 16, 20011
    x, w, b, target, _ = entropy_case(rows, c, v, True)
    loss, lse = out_like(rows, 1, F32)[:, 0], out_like(rows, 1, F32)[:, 0]
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse, bias=b)
    for r in range(0, rows, 10000):
        at = slice(r, r + 10000)
        f = ref.cross_entropy(d(x[at]), d(w), target[at], d(b))
        close(lse[at], *f["lse"], "lse")
        close(loss[at], *f["loss"], "loss")


@pytest.mark.parametrize("rows,v", [(70000, 19), (140001, 300)])
def test_bias_gradient_of_many_rows(handle, rows, v):
    x, w, b, target, dloss = entropy_case(rows, 16, v, True)
    loss, lse, db = (torch.empty(n, device="cuda") for n in (rows, rows, v))
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse, bias=b)
    api.CrossEntropyBackward(handle, x, w, target)(x, w, target, lse, dloss, bias=b, dbias=db)
    f = ref.cross_entropy(d(x), d(w), target, d(b))
    close(db, *ref.cross_entropy_backward(d(x), d(w), target, f, d(dloss), BF, BF)[2], "dbias")


def test_cross_entropy_of_images(handle):
    """A class for every pixel, planar and channels last."""
    x, w = rand(3, 24, 9, 11, seed=1, dtype=BF), rand(19, 24, seed=2, std=0.5, dtype=BF)
    target, dloss = classes_of(3 * 9 * 11, 19, 3).view(3, 9, 11), rand(3, 9, 11, seed=4).abs()
    last = x.permute(0, 2, 3, 1).contiguous()
    want = check_entropy(handle, last.view(-1, 24), w, None, target.view(-1), dloss.view(-1))
    for image, axes in ((x, "NCHW"), (last, "NHWC")):
        loss, lse, dx, dw = torch.empty_like(dloss), torch.empty_like(dloss), torch.empty_like(image), torch.empty_like(w)
        api.CrossEntropyForward(handle, image, w, target, axes=axes)(image, w, target, loss, lse)
        api.CrossEntropyBackward(handle, image, w, target, dx, dw, axes=axes)(image, w, target, lse, dloss, dx, dw)
        for got, ref_, rel in ((loss, want[0], 1e-5), (dw, want[3], 2.0 ** -7)):
            assert (got.reshape(ref_.shape).float() - ref_.float()).abs().max() <= rel * ref_.float().abs().max()
        rows = (dx.permute(0, 2, 3, 1) if axes == "NCHW" else dx).reshape(-1, 24)
        assert (rows.float() - want[2].float()).abs().max() <= 2.0 ** -7 * want[2].float().abs().max()


@pytest.mark.parametrize("rows,c,v", [(3, 64, 1000), (70, 160, 3001), (700, 256, 5000), (50, 33, 70)])
def test_cross_entropy_of_e4m3(handle, rows, c, v):
    x, w, b, target, _ = entropy_case(rows, c, v, True)
    sx, sw = (t.float().abs().amax(1) / 448 for t in (x, w))
    qx, qw = (x.float() / sx[:, None]).to(F8), (w.float() / sw[:, None]).to(F8)
    loss, lse = out_like(rows, 1, F32)[:, 0], out_like(rows, 1, F32)[:, 0]
    api.CrossEntropyForward(handle, qx, qw, target)(qx, qw, target, loss, lse, bias=b, x_scale=sx, w_scale=sw)
    f = ref.cross_entropy(d(qx), d(qw), target, d(b), d(sx), d(sw))
    close(lse, *f["lse"], "lse")
    close(loss, *f["loss"], "loss")


@pytest.mark.parametrize("rows,v", [(40, 500), (300, 3000)])
def test_cross_entropy_of_masked_classes(handle, rows, v):
    """Classes with a bias of -inf, or of FP32's lowest value, have probability 0; rows that leave
    only such classes have no loss."""
    x, w, b, target, dloss = entropy_case(rows, 64, v, True)
    b[::3] = float("-inf")
    b[1::3] = torch.finfo(F32).min
    target = target // 3 * 3 + 2
    target = torch.where(target < 2, -1, target.clamp(max=v // 3 * 3 - 1))
    loss, lse, dx, dw, db = check_entropy(handle, x, w, b, target, dloss)
    assert (db[::3] == 0).all() and (db[1::3] == 0).all() and (dw[::3] == 0).all()
    # a target that is masked: an infinite loss
    target[0] = 3
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse, bias=b)
    assert loss[0] == float("inf") and torch.isfinite(lse).all()
    b[:] = float("-inf")
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse, bias=b)
    assert (lse == float("-inf")).all() and torch.isnan(loss[target >= 0]).all() and (loss[target < 0] == 0).all()
    # nothing but FP32's lowest value: all classes alike (a logit is below its rounding)
    b[:] = torch.finfo(F32).min
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse, bias=b)
    assert (lse == torch.finfo(F32).min).all() and (loss[target < 0] == 0).all()
    close(loss[target >= 0], torch.full_like(loss[target >= 0], math.log(v)).double(), torch.tensor(1e-5, device="cuda"), "loss")


@pytest.mark.parametrize("rows", [20, 200])
@pytest.mark.parametrize("level", [1e3, 1e6])
def test_cross_entropy_far_from_zero(handle, rows, level):
    """Logits that a bias lifts: the loss keeps the digits that log-sum-exp has not.  Logits are rounded
    at their own size (2^-24 level), their products summed within the bound of the linear layer."""
    x, w, b, target, _ = entropy_case(rows, 64, 700, True)
    b += level
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse, bias=b)
    f = ref.cross_entropy(d(x), d(w), target, d(b))
    at = 2 * cref.U32 * level * 1.01  # the chosen logit's and the others' rounding
    close(loss, f["loss"][0], 2 * (f["ez"].amax(1) + at) + 8 * cref.U32 * 20, "loss")
    close(lse, f["lse"][0], f["ez"].amax(1) + 2 * at + 8 * cref.U32 * 20, "lse")


def test_cross_entropy_of_large_logits_and_sure_rows(handle):
    """Logits of some hundreds, and rows whose target has nearly all of the probability: the
    gradient at the target keeps its digits."""
    rows, c, v = 130, 64, 900
    w = rand(v, c, seed=1, std=2.0, dtype=BF)
    target = classes_of(rows, v, 2).clamp(min=0)
    x = (w[target].float() * torch.linspace(0.02, 1.5, rows, device="cuda")[:, None]).to(BF)
    check_entropy(handle, x, w, None, target, torch.full((rows,), 1.0 / rows, device="cuda"))


def test_cross_entropy_of_non_finite_rows(handle):
    x, w, b, target, dloss = entropy_case(300, 64, 700, False)
    target = target.clamp(min=0)
    want = check_entropy(handle, x, w, b, target, dloss)
    x = x.clone()
    x[7, 3], x[250, 0] = float("nan"), float("inf")
    loss, lse = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse)
    rest = [i for i in range(300) if i not in (7, 250)]
    assert torch.isnan(loss[7]) and not torch.isfinite(loss[250])
    assert torch.equal(loss[rest], want[0][rest]) and torch.equal(lse[rest], want[1][rest])


def test_cross_entropy_of_rows_that_count_for_nothing(handle):
    """Padding rows give no gradient, whatever their loss's gradient or log-sum-exp is."""
    x, w, b, target, dloss = entropy_case(90, 64, 300, True)
    target[:] = -1
    target[10] = 4
    dloss[:10] = float("nan")
    dloss[20] = float("inf")
    loss, lse = torch.empty(90, device="cuda"), torch.empty(90, device="cuda")
    api.CrossEntropyForward(handle, x, w, target)(x, w, target, loss, lse, bias=b)
    assert (loss[target < 0] == 0).all() and loss[10] > 0
    lse[30] = float("nan")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    api.CrossEntropyBackward(handle, x, w, target, dx, dw)(x, w, target, lse, dloss, dx, dw, bias=b, dbias=db)
    assert (dx[target < 0] == 0).all() and (dx[10] != 0).any()
    assert torch.isfinite(dw.float()).all() and torch.isfinite(db).all()
    handle.synchronize()


def test_targets_beyond_the_classes_are_reported():
    with api.Handle() as h:
        x, w, b, target, dloss = entropy_case(90, 64, 300, True)
        target[40] = 300
        target[41] = 2 ** 32 + 5
        loss, lse, dx, dw = torch.empty(90, device="cuda"), torch.empty(90, device="cuda"), torch.empty_like(x), torch.empty_like(w)
        fwd, bwd = api.CrossEntropyForward(h, x, w, target), api.CrossEntropyBackward(h, x, w, target, dx, dw)
        fwd(x, w, target, loss, lse, bias=b)
        with pytest.raises(B.DlcError):
            h.synchronize()
        assert torch.isnan(loss[40]) and torch.isnan(loss[41]) and torch.isfinite(loss[:40]).all() and torch.isfinite(loss[42:]).all()
        bwd(x, w, target, lse, dloss, dx, dw, bias=b)
        torch.cuda.synchronize()
        code, detail = B.dlcGetLastDeviceError(h.h)
        assert code == B.DLC_DEVERR_INDEX and detail in (40, 41)
        assert (dx[40] == 0).all() and (dx[41] == 0).all()
        h.synchronize()


def test_any_of_the_gradients_alone(handle):
    x, w, b, target, dloss = entropy_case(200, 96, 1000, True)
    loss, lse, dx, dw, db = check_entropy(handle, x, w, b, target, dloss)
    for which in range(3):
        outs = [torch.empty_like(t) if i == which else None for i, t in enumerate((dx, dw, db))]
        op = api.CrossEntropyBackward(handle, x, w, target, outs[0], outs[1])
        op(x, w, target, lse, dloss, outs[0], outs[1], bias=b, dbias=outs[2])
        assert torch.equal(outs[which], (dx, dw, db)[which])


def test_cross_entropy_gradient_is_that_of_the_forward_call(handle):
    """dbias (FP32) against central differences of the loss."""
    x, w, b, target, dloss = entropy_case(60, 64, 90, True)
    loss, lse, _, _, db = check_entropy(handle, x, w, b, target, dloss)
    op = api.CrossEntropyForward(handle, x, w, target)
    v, h = rand(90, seed=8), 2.0 ** -5

    def at(step):
        op(x, w, target, loss, lse, bias=b + step * v)
        return (d(loss) * d(dloss)).sum().item()

    # losses of 10 at most, their rounding 2^-24 * 16 each (TC of the logits cancels: the same
    # products on both sides); the third derivative of log-sum-exp along v is below |v|_inf^3
    total = d(dloss).sum().item()
    got, want = (at(h) - at(-h)) / (2 * h), (d(db) * d(v)).sum().item()
    assert abs(got - want) <= total * (2.0 ** -20 / h + h * h / 6 * 2 * v.abs().max().item() ** 3) + 1e-5 * d(db).abs().sum().item()
