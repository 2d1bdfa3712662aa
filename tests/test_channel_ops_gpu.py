"""The channel operators on the GPU against their FP64 definitions, under the
error bounds derived in channel_ref."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from deep_learning_convolution_gb300 import binding as B
from tests import channel_ref as ref

pytestmark = pytest.mark.gpu

F32, BF, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-5


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


def rand(*shape, seed=0, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def laid_out(t, layout):
    """The values of a [rows, channels] tensor in another storage."""
    rows, c = t.shape
    if layout == "dense":
        return t
    if layout == "pitch":      # rows of a wider, 16-byte aligned matrix
        big = torch.zeros(rows, c + 64 - c % 8, dtype=t.dtype, device="cuda")[:, :c]
    elif layout == "odd":      # rows at an odd pitch, from an odd address
        big = torch.zeros(rows * (c + 3) + 1, dtype=t.dtype, device="cuda")[1:].view(rows, c + 3)[:, :c]
    elif layout == "columns":  # channels apart, rows adjacent
        big = torch.zeros(c, rows + 1, dtype=t.dtype, device="cuda").t()[:rows]
    else:
        raise ValueError(layout)
    big.copy_(t)
    return big


def out_like(rows, c, dtype, layout="dense"):
    t = laid_out(torch.zeros(rows, c, dtype=dtype, device="cuda"), layout)
    t.copy_(torch.full_like(t, float("nan"), dtype=F32))  # every element has to be written
    return t


def f64(t):
    return None if t is None else t.double().cpu()


def close(got, want, err, what):
    got = f64(got)
    bad = ~((got - want).abs() <= err)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; first "
                           f"{bad.nonzero()[0].tolist()} got {got[bad][0]} want {want[bad][0]} "
                           f"err {err[bad][0]}")


def close_e4m3(q, scale, want, rel, what):
    """E4M3 values times their scales against FP64, and the scales themselves."""
    s = f64(scale)[:, None]
    amax = want.abs().amax(1, keepdim=True).clamp(min=1e-30)
    close(s, amax / 448, 2 * rel * amax / 448 + 1e-38, what + " scale")
    close(f64(q) * s, want, (ref.E4M3 + 4 * rel) * want.abs() + 2.0 ** -10 * s, what)


# ---- RMS norm --------------------------------------------------------------------

NORM_SIZES = [(1, 1), (1, 4096), (3, 8), (5, 7), (2, 64), (33, 130), (300, 333), (65, 512),
              (17, 1000), (9, 1024), (4, 2048), (3, 5000), (2, 8192), (1, 40000), (5000, 72)]


@pytest.mark.parametrize("rows,c", NORM_SIZES)
@pytest.mark.parametrize("xdt,rdt,ydt", [(BF, BF, F8), (BF, F32, BF), (F32, F32, F32), (F32, BF, F8)])
def test_norm_forward(handle, rows, c, xdt, rdt, ydt):
    x, r = rand(rows, c, seed=1, dtype=xdt), rand(rows, c, seed=2, std=3.0, dtype=rdt)
    gamma = 1 + 0.3 * rand(c, seed=3)
    total, y = out_like(rows, c, rdt), out_like(rows, c, ydt)
    scale = out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
    op = api.RmsNormForward(handle, x, y, residual=r, total=total, eps=EPS)
    op(x, gamma, y, residual=r, total=total, scale=scale)
    t, want = ref.norm(f64(x), f64(r), f64(gamma), EPS)
    close(total, t, ref.stored(t, rdt) + ref.U32 * t.abs(), "total")
    rel = ref.norm_rel(c)
    if ydt == F8:
        close_e4m3(y, scale, want, rel, "y")
    else:
        close(y, want, rel * want.abs() + ref.stored(want, ydt), "y")


@pytest.mark.parametrize("layout", ["pitch", "odd", "columns"])
@pytest.mark.parametrize("rows,c", [(70, 96), (33, 51), (4, 1023)])
@pytest.mark.parametrize("ydt", [BF, F8])
def test_norm_layouts_without_residual(handle, rows, c, layout, ydt):
    x = laid_out(rand(rows, c, seed=1, dtype=BF), layout)
    y = out_like(rows, c, ydt, layout)
    gamma = 1 + 0.3 * rand(c, seed=3)
    scale = out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
    api.RmsNormForward(handle, x, y, eps=EPS)(x, gamma, y, scale=scale)
    _, want = ref.norm(f64(x), None, f64(gamma), EPS)
    if ydt == F8:
        close_e4m3(y, scale, want, ref.norm_rel(c), layout)
    else:
        close(y, want, ref.norm_rel(c) * want.abs() + ref.stored(want, ydt), layout)


def test_norm_of_an_image_in_both_formats(handle):
    n, c, h, w = 3, 40, 5, 6
    x = rand(n, c, h, w, seed=1, dtype=BF)  # NCHW
    gamma = 1 + 0.3 * rand(c, seed=3)
    y = torch.empty_like(x)
    api.RmsNormForward(handle, x, y, eps=EPS, axes="NCHW")(x, gamma, y)
    xl = x.permute(0, 2, 3, 1).contiguous()
    yl = torch.empty_like(xl)
    api.RmsNormForward(handle, xl, yl, eps=EPS)(xl, gamma, yl)
    _, want = ref.norm(f64(xl).view(-1, c), None, f64(gamma), EPS)
    err = ref.norm_rel(c) * want.abs() + ref.stored(want, BF)
    close(yl.view(-1, c), want, err, "NHWC")
    close(y.permute(0, 2, 3, 1).reshape(-1, c), want, err, "NCHW")


def test_norm_rows_of_a_cropped_image(handle):
    """Rows that no single pitch describes."""
    big = rand(2, 7, 9, 32, seed=1, dtype=BF)
    x = big[:, 1:6, 2:8]
    y = torch.empty(2, 5, 6, 32, dtype=F32, device="cuda")
    gamma = rand(32, seed=2)
    api.RmsNormForward(handle, x, y, eps=EPS)(x, gamma, y)
    _, want = ref.norm(f64(x).reshape(-1, 32), None, f64(gamma), EPS)
    close(y.view(-1, 32), want, ref.norm_rel(32) * want.abs() + ref.stored(want, F32), "crop")


@pytest.mark.parametrize("c", [256, 100, 5000])
def test_norm_in_place_zero_rows_and_non_finite_rows(handle, c):
    r = rand(6, c, seed=1, dtype=F32)
    x = rand(6, c, seed=2, dtype=BF)
    x[1] = 0
    r[1] = 0
    r[2, c // 2] = float("nan")
    r[4, 0] = float("inf")
    gamma = 1 + 0.3 * rand(c, seed=3)
    y, scale = out_like(6, c, F8), out_like(6, 1, F32)[:, 0]
    t, want = ref.norm(f64(x), f64(r), f64(gamma), EPS)
    api.RmsNormForward(handle, x, y, residual=r, total=r, eps=EPS)(
        x, gamma, y, residual=r, total=r, scale=scale)
    good = [0, 1, 3, 5]
    close(r[good], t[good], ref.stored(t[good], F32) + ref.U32 * t[good].abs(), "total in place")
    close_e4m3(y[good], scale[good], want[good], ref.norm_rel(c), "y")
    assert (y[1].float() == 0).all() and torch.isfinite(scale[1])
    assert torch.isnan(y[2].float()).all() and torch.isnan(y[4, 0].float())


@pytest.mark.parametrize("rows,c", [(1, 1), (1, 4096), (3, 7), (100, 96), (257, 333), (1000, 512),
                                    (40, 1024), (9, 4097), (2, 20000), (7000, 64)])
@pytest.mark.parametrize("dt,with_dt,with_dgamma", [(BF, True, True), (F32, False, True), (BF, False, False)])
def test_norm_backward(handle, rows, c, dt, with_dt, with_dgamma):
    dy, t = rand(rows, c, seed=1, dtype=dt), rand(rows, c, seed=2, std=2.0, dtype=dt)
    dtot = rand(rows, c, seed=3, dtype=dt) if with_dt else None
    gamma = 1 + 0.3 * rand(c, seed=4)
    dx = out_like(rows, c, dt)
    dgamma = out_like(c, 1, F32)[:, 0] if with_dgamma else None
    op = api.RmsNormBackward(handle, dy, t, dx, dtotal=dtot, eps=EPS)
    op(dy, t, gamma, dx, dgamma=dgamma, dtotal=dtot)
    want, wg, bx, bg = ref.norm_backward(f64(dy), f64(t), f64(gamma), f64(dtot), EPS)
    close(dx, want, 4 * ref.norm_rel(c) * bx + ref.stored(want, dt), "dx")
    if with_dgamma:
        close(dgamma, wg, (ref.norm_rel(c) + ref.U32 * (rows + 64)) * bg, "dgamma")


@pytest.mark.parametrize("layout", ["pitch", "odd", "columns"])
def test_norm_backward_layouts_in_place(handle, layout):
    rows, c = 77, 90
    dy, t = (laid_out(rand(rows, c, seed=s, dtype=BF), layout) for s in (1, 2))
    dx = laid_out(rand(rows, c, seed=3, dtype=BF), layout)  # dtotal, overwritten
    gamma, dgamma = 1 + 0.3 * rand(c, seed=4), out_like(c, 1, F32)[:, 0]
    want, wg, bx, bg = ref.norm_backward(f64(dy), f64(t), f64(gamma), f64(dx), EPS)
    api.RmsNormBackward(handle, dy, t, dx, dtotal=dx, eps=EPS)(dy, t, gamma, dx, dgamma=dgamma, dtotal=dx)
    close(dx, want, 4 * ref.norm_rel(c) * bx + ref.stored(want, BF), "dx")
    close(dgamma, wg, (ref.norm_rel(c) + ref.U32 * (rows + 64)) * bg, "dgamma")


def test_norm_gradient_is_that_of_the_forward_call(handle):
    """dgamma and dx against central differences of the FP32 forward call."""
    rows, c, h = 6, 48, 2.0 ** -6
    t, dy, gamma = rand(rows, c, seed=1), rand(rows, c, seed=2), 1 + 0.3 * rand(c, seed=3)
    dx, dgamma, y = torch.empty_like(t), torch.empty_like(gamma), torch.empty_like(t)
    api.RmsNormBackward(handle, dy, t, dx, eps=EPS)(dy, t, gamma, dx, dgamma=dgamma)
    op = api.RmsNormForward(handle, t, y, eps=EPS)

    def loss(tt, gg):
        op(tt, gg, y)
        return (f64(dy) * f64(y)).sum().item()

    # y is linear in gamma; in t the cubic term of a step h is h^2 / 6 of
    # derivatives of order one for rows of size one (2^-12 / 6 = 4e-5 of the
    # absolute terms); FP32 outputs are off by 1e-6 of theirs, over 2h = 1/32
    d = rand(c, seed=5)
    got = (loss(t, gamma + h * d) - loss(t, gamma - h * d)) / (2 * h)
    noise = 3e-6 * (f64(dy) * f64(y)).abs().sum().item() * 32
    assert abs(got - (f64(dgamma) * f64(d)).sum().item()) < noise
    d = rand(rows, c, seed=6)
    got = (loss(t + h * d, gamma) - loss(t - h * d, gamma)) / (2 * h)
    assert abs(got - (f64(dx) * f64(d)).sum().item()) < noise + 1e-3 * (f64(dx) * f64(d)).abs().sum().item()


# ---- linear and gated layers --------------------------------------------------------

def quantized(t):
    s = t.abs().amax(1, keepdim=True).clamp(min=1e-20) / 448
    return (t / s).to(F8), s[:, 0].contiguous()


SIZES = [  # rows, channels, filters (gated: of each half)
    (1, 1, 1), (1, 64, 64), (1, 1000, 200), (2, 333, 77), (3, 128, 256), (4, 2048, 130), (7, 96, 1001),
    (8, 512, 512), (9, 520, 264), (17, 147, 65), (32, 1024, 128), (64, 72, 1000), (100, 100, 100),
    (128, 256, 256), (129, 257, 255), (200, 64, 520), (256, 640, 384), (300, 1024, 96), (513, 40, 48),
    (777, 136, 1032), (2049, 192, 320), (5000, 24, 40)]


def run_forward(handle, rows, c, k, *, gated, dtype=BF, ydt=BF, kind="identity", bias=False, residual=None,
                z=None, layout="dense", zr_layout="dense"):
    n = 2 * k if gated else k
    x, w = rand(rows, c, seed=1), rand(n, c, seed=2, std=c ** -0.5)
    sx = sw = None
    if dtype == F8:
        (x, sx), (w, sw) = quantized(x), quantized(w)
    else:
        x, w = x.to(BF), w.to(BF)
    x = laid_out(x, layout)
    b = rand(n, seed=3, std=0.5) if bias else None
    r = laid_out(rand(rows, k, seed=4, std=2.0, dtype=residual), zr_layout) if residual else None
    zt = out_like(rows, n, z, zr_layout) if z else None
    y = out_like(rows, k, ydt, layout)
    cls = api.GatedForward if gated else api.LinearForward
    kw = {} if gated else {"residual": r}
    op = cls(handle, x, w, y, act=kind, z=zt, **kw)
    op(x, w, y, bias=b, z=zt, x_scale=sx, w_scale=sw, **kw)
    zw, ez = ref.product(f64(x), f64(w), f64(b), f64(sx), f64(sw))
    if gated:
        want, err = ref.gated(zw, ez, kind, ydt)
    else:
        want, err = ref.linear(zw, ez, kind, f64(r), ydt)
    what = f"{rows}x{c}x{k} {op.kernel(x, w, y)}"
    close(y, want, err, what)
    if z:
        close(zt, zw, ez + ref.stored(zw, z), what + " z")


@pytest.mark.parametrize("rows,c,k", SIZES)
@pytest.mark.parametrize("dtype,ydt,kind,bias,residual,z", [
    (BF, F32, "identity", False, None, None), (BF, BF, "gelu", True, BF, BF), (F8, BF, "silu", True, F32, None),
    (BF, F32, "relu", True, BF, F32)])
def test_linear_forward(handle, rows, c, k, dtype, ydt, kind, bias, residual, z):
    run_forward(handle, rows, c, k, gated=False, dtype=dtype, ydt=ydt, kind=kind, bias=bias,
                residual=residual, z=z)


@pytest.mark.parametrize("rows,c,k", SIZES)
@pytest.mark.parametrize("dtype,ydt,kind,bias,z", [
    (BF, BF, "silu", False, None), (BF, F32, "gelu", True, BF), (F8, BF, "silu", True, None),
    (BF, BF, "identity", False, F32)])
def test_gated_forward(handle, rows, c, k, dtype, ydt, kind, bias, z):
    run_forward(handle, rows, c, k, gated=True, dtype=dtype, ydt=ydt, kind=kind, bias=bias, z=z)


@pytest.mark.parametrize("kind", ["sigmoid", "tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows", [1, 200])
def test_other_activations(handle, kind, gated, rows):
    run_forward(handle, rows, 128, 192, gated=gated, kind=kind, ydt=F32, z=F32)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("layout", ["pitch", "odd", "columns"])
@pytest.mark.parametrize("rows,c,k", [(1, 100, 60), (3, 96, 64), (150, 130, 90), (300, 256, 512)])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_product_layouts(handle, gated, layout, rows, c, k, dtype):
    run_forward(handle, rows, c, k, gated=gated, dtype=dtype, kind="silu", bias=True,
                residual=None if gated else BF, z=BF, layout=layout, zr_layout=layout)


@pytest.mark.parametrize("rows", [2, 500])
def test_linear_residual_in_place(handle, rows):
    x, w, y = rand(rows, 128, seed=1, dtype=BF), rand(96, 128, seed=2, dtype=BF), rand(rows, 96, seed=3, dtype=F32)
    z, ez = ref.product(f64(x), f64(w))
    want, err = ref.linear(z, ez, "identity", f64(y), F32)
    api.LinearForward(handle, x, w, y, residual=y)(x, w, y, residual=y)
    close(y, want, err, "in place")


def test_linear_on_images(handle):
    """NHWC and NCHW activations, [K, C, 1, 1] filters: a 1x1 convolution."""
    n, c, h, w_, k = 2, 48, 9, 7, 80
    x, w = rand(n, c, h, w_, seed=1, dtype=BF), rand(k, c, 1, 1, seed=2, std=0.1, dtype=BF)
    y = torch.empty(n, k, h, w_, dtype=F32, device="cuda")
    api.LinearForward(handle, x, w, y, axes="NCHW", act="relu")(x, w, y)
    yl = torch.empty(n, h, w_, k, dtype=F32, device="cuda")
    xl = x.permute(0, 2, 3, 1).contiguous()
    api.LinearForward(handle, xl, w, yl, act="relu")(xl, w, yl)
    z, ez = ref.product(f64(xl).view(-1, c), f64(w).view(k, c))
    want, err = ref.linear(z, ez, "relu", None, F32)
    close(yl.view(-1, k), want, err, "NHWC")
    close(y.permute(0, 2, 3, 1).reshape(-1, k), want, err, "NCHW")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,c,k", [(1, 64, 96), (5, 256, 100), (40, 520, 300), (333, 130, 77), (1000, 200, 256),
                                      (4096, 64, 128)])
def test_non_finite_rows_stay_in_their_rows(handle, gated, rows, c, k):
    x, w = rand(rows, c, seed=1, dtype=BF), rand(2 * k if gated else k, c, seed=2, std=c ** -0.5, dtype=BF)
    bad = rows // 2
    x[bad, c - 1] = float("nan")
    y = out_like(rows, k, BF)
    (api.GatedForward if gated else api.LinearForward)(handle, x, w, y, act="silu")(x, w, y)
    nan = torch.isnan(y.float())
    assert nan[bad].all() and int(nan.sum()) == k


# ---- backward ----------------------------------------------------------------------

def run_backward(handle, rows, c, k, *, gated, kind="silu", zdt=BF, dydt=BF, dxdt=BF, dwdt=BF, bias=True,
                 layout="dense", want=("dx", "dw")):
    n = 2 * k if gated else k
    x = laid_out(rand(rows, c, seed=1, dtype=BF), layout)
    w = rand(n, c, seed=2, std=c ** -0.5, dtype=BF)
    dy = laid_out(rand(rows, k, seed=3, dtype=dydt), layout)
    z = laid_out(rand(rows, n, seed=4, dtype=zdt), layout) if gated or kind != "identity" else None
    dx = out_like(rows, c, dxdt, layout) if "dx" in want else None
    dw = out_like(n, c, dwdt) if "dw" in want else None
    db = out_like(n, 1, F32)[:, 0] if bias else None
    cls = api.GatedBackward if gated else api.LinearBackward
    cls(handle, x, w, dy, dx, dw, z=z, act=kind)(x, w, dy, dx, dw, dbias=db, z=z)
    dz, e = ref.act_grad(f64(dy), f64(z), kind, gated)
    (dxw, ex), (dww, ew), (dbw, eb) = ref.backward(f64(x), f64(w), dz, e, dxdt, dwdt)
    what = f"{rows}x{c}x{k}"
    if dx is not None:
        close(dx, dxw, ex, what + " dx")
    if dw is not None:
        close(dw, dww, ew, what + " dw")
    if bias:
        close(db, dbw, eb, what + " dbias")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,c,k", SIZES)
def test_backward(handle, gated, rows, c, k):
    run_backward(handle, rows, c, k, gated=gated, kind="silu", zdt=BF)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ["identity", "relu", "sigmoid", "tanh", "gelu"])
@pytest.mark.parametrize("rows,c,k", [(3, 40, 24), (260, 264, 136)])
def test_backward_activations(handle, gated, kind, rows, c, k):
    run_backward(handle, rows, c, k, gated=gated, kind=kind, zdt=F32, dydt=F32, dxdt=F32, dwdt=F32)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("layout", ["pitch", "odd", "columns"])
@pytest.mark.parametrize("kind", ["identity", "gelu"])
def test_backward_layouts(handle, gated, layout, kind):
    run_backward(handle, 150, 130, 90, gated=gated, kind=kind, layout=layout)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("want,bias", [(("dx",), False), (("dw",), False), ((), True)])
def test_backward_of_some(handle, gated, want, bias):
    run_backward(handle, 100, 64, 48, gated=gated, want=want, bias=bias)
    run_backward(handle, 100, 64, 48, gated=gated, kind="identity", want=want, bias=bias)


@pytest.mark.parametrize("gated", [False, True])
def test_gradient_is_that_of_the_forward_call(handle, gated):
    """dx, dw and dbias against central differences of the FP32-output call,
    on values and steps that BF16 holds exactly."""
    rows, c, k, h = 8, 32, 16, 2.0 ** -6
    n = 2 * k if gated else k

    def grid(*shape, seed, step=2.0 ** -4, top=1.0):
        g = torch.Generator().manual_seed(seed)
        m = int(top / step)
        return torch.randint(-m, m + 1, shape, generator=g).float().cuda() * step

    # |x| <= 1, steps of 2^-6: 65 values a side, within BF16's 8 bits
    x, w, b = grid(rows, c, seed=1), grid(n, c, seed=2, top=0.25), grid(n, seed=3)
    dx_, dw_, db_ = (grid(*s, seed=i, step=1.0) for s, i in (((rows, c), 4), ((n, c), 5), ((n,), 6)))
    dy = grid(rows, k, seed=7, step=0.25)
    y, z = torch.empty(rows, k, device="cuda"), torch.empty(rows, n, device="cuda")
    f = (api.GatedForward if gated else api.LinearForward)(handle, x.to(BF), w.to(BF), y, act="silu", z=z)

    def loss(x, w, b):
        f(x.to(BF), w.to(BF), y, bias=b, z=z)
        return (f64(dy) * f64(y)).sum().item()

    got = [(loss(x + h * dx_, w, b) - loss(x - h * dx_, w, b)) / (2 * h),
           (loss(x, w + h * dw_, b) - loss(x, w - h * dw_, b)) / (2 * h),
           (loss(x, w, b + h * db_) - loss(x, w, b - h * db_)) / (2 * h)]
    size = (f64(dy) * f64(y)).abs().sum().item()
    loss(x, w, b)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    bwd = (api.GatedBackward if gated else api.LinearBackward)(
        handle, x.to(BF), w.to(BF), dy.to(BF), dx, dw, z=z, act="silu")
    bwd(x.to(BF), w.to(BF), dy.to(BF), dx, dw, dbias=db, z=z)
    for name, g, grad, d in (("x", got[0], dx, dx_), ("w", got[1], dw, dw_), ("b", got[2], db, db_)):
        s = (f64(grad) * f64(d)).abs().sum().item()
        # dz in BF16 (2^-8); steps of up to h * sum|d w| = 2 in z for x and w
        # would leave a cubic term, so they are compared to 5 % of the absolute
        # terms; FP32 outputs over 2h = 1/32 add 1e-5 * 32 of the loss's terms
        tol = 0.05 * s + 3.2e-4 * size
        assert abs(g - (f64(grad) * f64(d)).sum().item()) < tol, (name, g)


# ---- as a program uses them ------------------------------------------------------------

def test_reproducible_and_on_another_stream(handle):
    x, w = rand(300, 1000, seed=1, dtype=BF), rand(512, 1000, seed=2, dtype=BF)
    dy, z = rand(300, 256, seed=3, dtype=BF), rand(300, 512, seed=4, dtype=BF)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(512, device="cuda")
    op = api.GatedBackward(handle, x, w, dy, dx, dw, z=z)
    op(x, w, dy, dx, dw, dbias=db, z=z)
    first = [t.clone() for t in (dx, dw, db)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    handle.set_stream(s)
    try:
        for _ in range(3):
            for t in (dx, dw, db):
                with torch.cuda.stream(s):
                    t.fill_(float("nan"))
            op(x, w, dy, dx, dw, dbias=db, z=z)
            s.synchronize()
            for a, b in zip(first, (dx, dw, db)):
                assert torch.equal(a, b)
    finally:
        handle.set_stream(torch.cuda.current_stream())


def test_graph_replay(handle):
    rows, c, f = 40, 256, 512
    x, r, gamma = rand(rows, c, seed=1, dtype=BF), rand(rows, c, seed=2, dtype=BF), 1 + 0.1 * rand(c, seed=3)
    w1, w2 = rand(2 * f, c, seed=4, std=c ** -0.5, dtype=BF), rand(c, f, seed=5, std=f ** -0.5, dtype=BF)
    t, y, h, out = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, f, dtype=BF, device="cuda"), torch.empty_like(x)
    s = torch.cuda.Stream()
    handle.set_stream(s)
    try:
        norm = api.RmsNormForward(handle, x, y, residual=r, total=t)
        up = api.GatedForward(handle, y, w1, h)
        down = api.LinearForward(handle, h, w2, out, residual=t)

        def step():
            norm(x, gamma, y, residual=r, total=t)
            up(y, w1, h)
            down(h, w2, out, residual=t)

        with torch.cuda.stream(s):
            step()
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step()
            x.copy_(rand(rows, c, seed=9, dtype=BF))
            out.fill_(float("nan"))
            g.replay()
            s.synchronize()
            replayed = out.clone()
            step()
            s.synchronize()
        assert torch.equal(replayed, out) and torch.isfinite(out.float()).all()
    finally:
        handle.set_stream(torch.cuda.current_stream())


def test_refusals(handle):
    x, w, y = rand(8, 64, dtype=BF), rand(32, 64, dtype=BF), torch.empty(8, 32, dtype=BF, device="cuda")
    gamma = torch.ones(64, device="cuda")

    def refused(status, fn):
        with pytest.raises(B.DlcError) as e:
            fn()
        assert e.value.status == status

    bad, unsupported = B.DLC_STATUS_BAD_PARAM, B.DLC_STATUS_NOT_SUPPORTED
    lin = api.LinearForward(handle, x, w, y)
    refused(bad, lambda: api.LinearForward(handle, x, rand(32, 65, dtype=BF), y))
    refused(bad, lambda: api.LinearForward(handle, x, w, torch.empty(7, 32, dtype=BF, device="cuda")))
    refused(bad, lambda: api.GatedForward(handle, x, rand(31, 64, dtype=BF), y))
    refused(bad, lambda: api.LinearForward(handle, x, w.to(F8), y))
    refused(unsupported, lambda: api.LinearForward(handle, x.float(), w.float(), y))
    refused(bad, lambda: lin(x, w, y, x_scale=torch.ones(8, device="cuda"), w_scale=torch.ones(32, device="cuda")))
    x8, w8 = x.to(F8), w.to(F8)
    refused(bad, lambda: api.LinearForward(handle, x8, w8, y)(x8, w8, y))  # no scales
    sq = torch.empty(8, 64, dtype=BF, device="cuda")
    refused(bad, lambda: api.LinearForward(handle, sq, rand(64, 64, dtype=BF), sq)(sq, rand(64, 64, dtype=BF), sq))
    refused(unsupported, lambda: B.dlcLinearForward(
        handle.h, lin.x_desc, x.data_ptr(), 0, lin.w_desc, w.data_ptr(), 0, 0, B.DLC_ACTIVATION_CLIPPED_RELU,
        None, 0, None, 0, lin.y_desc, y.data_ptr(), 0, 0))
    refused(bad, lambda: B.dlcLinearForward(handle.h, lin.x_desc, x.data_ptr(), 0, lin.w_desc, w.data_ptr(), 0, 0, 9,
                                            None, 0, None, 0, lin.y_desc, y.data_ptr(), 0, 0))
    with pytest.raises(ValueError):
        lin(x, w, y, bias=torch.ones(31, device="cuda"))
    with pytest.raises(ValueError):
        lin(x, w, y, residual=y)  # not among the example tensors
    # backward: nothing wanted, no z, too small a workspace
    dy, z = rand(8, 32, dtype=BF), rand(8, 32, dtype=BF)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    back = api.LinearBackward(handle, x, w, dy, dx, dw, z=z, act="silu")
    refused(bad, lambda: back(x, w, dy, z=z))
    refused(bad, lambda: back(x, w, dy, dx, dw))
    back._ws_bytes -= 1
    refused(bad, lambda: back(x, w, dy, dx, dw, z=z, dbias=torch.empty(32, device="cuda")))
    refused(unsupported, lambda: api.LinearBackward(handle, x8, w8, dy, dx, dw))
    # norm
    y8 = torch.empty(8, 64, dtype=F8, device="cuda")
    yn = torch.empty_like(x)
    refused(bad, lambda: api.RmsNormForward(handle, x, y8)(x, gamma, y8))  # E4M3 without scales
    refused(bad, lambda: api.RmsNormForward(handle, x, yn)(x, gamma, yn, scale=torch.ones(8, device="cuda")))
    refused(bad, lambda: api.RmsNormForward(handle, x, x)(x, gamma, x))
    refused(bad, lambda: api.RmsNormForward(handle, x, yn, eps=-1.0)(x, gamma, yn))
    refused(unsupported, lambda: api.RmsNormForward(handle, y8, yn)(y8, gamma, yn))
    refused(bad, lambda: api.RmsNormForward(handle, x, torch.empty(8, 63, dtype=BF, device="cuda"))(
        x, gamma, torch.empty(8, 63, dtype=BF, device="cuda")))
    # an E4M3 tensor is for the channel operators alone
    refused(unsupported, lambda: api.activation_forward(
        handle, y8.view(8, 64, 1, 1), yn.view(8, 64, 1, 1), mode="relu"))
    # nothing of this reached the device as an error
    assert handle.last_device_error() == (0, 0)


def test_long_offsets(handle):
    """Rows whose element offsets pass 32 bits, forward and backward."""
    pitch, rows, c, k = 1 << 22, 1200, 64, 40
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB free")
    big = torch.empty(rows * pitch, dtype=BF, device="cuda").view(rows, pitch)
    x = big[:, :c]
    x.copy_(rand(rows, c, seed=1, dtype=BF))
    w = rand(k, c, seed=2, std=c ** -0.5, dtype=BF)
    y = big[:, 1024:1024 + k]
    yd = torch.empty(rows, k, dtype=F32, device="cuda")
    api.LinearForward(handle, x, w, yd)(x, w, yd)
    z, ez = ref.product(f64(x), f64(w))
    close(yd, z, ez + ref.stored(z, F32), "x strided")
    gamma = 1 + 0.3 * rand(c, seed=3)
    n = torch.empty(rows, c, dtype=F32, device="cuda")
    api.RmsNormForward(handle, x, n, eps=EPS)(x, gamma, n)
    _, want = ref.norm(f64(x), None, f64(gamma), EPS)
    close(n, want, ref.norm_rel(c) * want.abs() + ref.stored(want, F32), "norm")
    xd = x.contiguous()
    api.LinearForward(handle, xd, w, y)(xd, w, y)
    close(y, z, ez + ref.stored(z, BF), "y strided")
    dx, dw = torch.empty_like(xd), torch.empty_like(w)
    api.LinearBackward(handle, x, w, y, dx, dw)(x, w, y, dx, dw)
    (dxw, ex), (dww, ew), _ = ref.backward(f64(x), f64(w), f64(y), 0 * f64(y), BF, BF)
    close(dx, dxw, ex, "dx")
    close(dw, dww, ew, "dw")
