"""The channel operators where one kernel hands over to another, on seeded
random problems, and on values and orders of calls that have gone wrong in
kernels of their kind; against FP64 under channel_ref's bounds."""
import random

import pytest
import torch

from deep_learning_convolution_gb300 import api
from deep_learning_convolution_gb300 import binding as B
from tests import channel_ref as ref
from tests.test_channel_ops_gpu import (BF, EPS, F8, F32, close, close_e4m3, f64, laid_out, out_like, quantized,
                                        rand, run_backward, run_forward)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = api.Handle()
    yield h
    h.synchronize()
    h.close()


def kernel_of(handle, rows, c, k, gated=False, dtype=BF):
    x = torch.empty(rows, c, dtype=dtype, device="cuda")
    w = torch.empty(2 * k if gated else k, c, dtype=dtype, device="cuda")
    y = torch.empty(rows, k, dtype=BF, device="cuda")
    return (api.GatedForward if gated else api.LinearForward)(handle, x, w, y).kernel(x, w, y)


def test_kernel_choice(handle):
    assert kernel_of(handle, 1, 2048, 8192, gated=True) == "gemv"
    assert kernel_of(handle, 4, 4096, 1000) == "gemv"
    assert kernel_of(handle, 4, 4096, 8192, gated=True) == "few_rows"   # 134 MB of filters
    assert kernel_of(handle, 64, 4096, 8192, gated=True, dtype=F8) == "few_rows"
    assert kernel_of(handle, 1, 333, 1001) == "gemv"                    # element by element
    assert kernel_of(handle, 3, 333, 1001) == "few_rows"                # packed first
    assert kernel_of(handle, 8192, 2048, 2048) == "gemm_pair"


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF, F8])
def test_row_counts(handle, rows, gated, dtype):
    run_forward(handle, rows, 272, 144, gated=gated, dtype=dtype, kind="silu", bias=True, z=BF)


@pytest.mark.parametrize("c", [1, 2, 7, 8, 15, 16, 63, 64, 65, 127, 128, 129, 4096, 20000])
@pytest.mark.parametrize("rows", [1, 2, 40, 300])
def test_reduction_lengths(handle, c, rows):
    run_forward(handle, rows, c, 72, gated=False, ydt=F32)
    run_forward(handle, rows, c, 40, gated=True, dtype=F8, kind="gelu")


@pytest.mark.parametrize("k", [1, 3, 8, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 256, 257, 1000])
@pytest.mark.parametrize("rows", [3, 300])
def test_filter_counts(handle, k, rows):
    run_forward(handle, rows, 96, k, gated=False, kind="gelu", bias=True, residual=BF, z=F32)
    run_forward(handle, rows, 96, k, gated=True, kind="silu", z=BF)


@pytest.mark.parametrize("rows,c,k", [(20480, 512, 256), (19500, 320, 520), (300, 6000, 256), (1500, 3000, 256)])
def test_split_tails(handle, rows, c, k):
    """Last waves whose tiles are split along the reduction, whole and ragged."""
    run_forward(handle, rows, c, k, gated=False, kind="relu", bias=True, residual=BF, z=BF)
    run_forward(handle, rows, c, k // 2, gated=True, kind="silu", z=BF)


def test_backward_with_long_reductions(handle):
    run_backward(handle, 30000, 64, 40, gated=True)
    run_backward(handle, 300, 48, 5000, gated=False, kind="gelu", dwdt=F32)


@pytest.mark.parametrize("seed", range(24))
def test_random_forward(handle, seed):
    r = random.Random(1000 + seed)

    def size(lo, hi):
        return int(round(lo * (hi / lo) ** r.random()))

    rows, c, k = size(1, 3000), size(1, 1500), size(1, 1200)
    gated, dtype = r.random() < 0.5, r.choice([BF, F8])
    run_forward(handle, rows, c, k, gated=gated, dtype=dtype, ydt=r.choice([BF, F32]),
                kind=r.choice(["identity", "relu", "sigmoid", "tanh", "silu", "gelu"]), bias=r.random() < 0.5,
                residual=None if gated else r.choice([None, BF, F32]), z=r.choice([None, BF, F32]),
                layout=r.choice(["dense", "pitch", "odd", "columns"]),
                zr_layout=r.choice(["dense", "pitch", "odd", "columns"]))


@pytest.mark.parametrize("seed", range(12))
def test_random_backward(handle, seed):
    r = random.Random(2000 + seed)

    def size(lo, hi):
        return int(round(lo * (hi / lo) ** r.random()))

    gated = r.random() < 0.5
    kind = r.choice(["relu", "sigmoid", "tanh", "silu", "gelu", "identity"])
    run_backward(handle, size(1, 2000), size(1, 600), size(1, 600), gated=gated, kind=kind, zdt=r.choice([BF, F32]),
                 dydt=r.choice([BF, F32]), dxdt=r.choice([BF, F32]), dwdt=r.choice([BF, F32]), bias=r.random() < 0.5,
                 layout=r.choice(["dense", "pitch", "odd", "columns"]))


@pytest.mark.parametrize("seed", range(16))
def test_random_norm(handle, seed):
    r = random.Random(3000 + seed)
    rows, c = int(round(3000 ** r.random())), int(round(9000 ** r.random()))
    layout = r.choice(["dense", "pitch", "odd", "columns"])
    xdt, tdt, ydt = r.choice([BF, F32]), r.choice([BF, F32]), r.choice([BF, F32, F8])
    x, res = laid_out(rand(rows, c, seed=1, dtype=xdt), layout), laid_out(rand(rows, c, seed=2, dtype=tdt), layout)
    gamma = 1 + 0.3 * rand(c, seed=3)
    total, y = out_like(rows, c, tdt, layout), out_like(rows, c, ydt, r.choice(["dense", layout]))
    scale = out_like(rows, 1, F32)[:, 0] if ydt == F8 else None
    api.RmsNormForward(handle, x, y, residual=res, total=total, eps=EPS)(x, gamma, y, residual=res, total=total, scale=scale)
    t, want = ref.norm(f64(x), f64(res), f64(gamma), EPS)
    close(total, t, ref.stored(t, tdt) + ref.U32 * t.abs(), "total")
    if ydt == F8:
        close_e4m3(y, scale, want, ref.norm_rel(c), layout)
    else:
        close(y, want, ref.norm_rel(c) * want.abs() + ref.stored(want, ydt), layout)
    dy, dx, dgamma = laid_out(rand(rows, c, seed=4, dtype=xdt), layout), out_like(rows, c, xdt, layout), torch.empty(c, device="cuda")
    api.RmsNormBackward(handle, dy, total, dx, dtotal=res, eps=EPS)(dy, total, gamma, dx, dgamma=dgamma, dtotal=res)
    want, wg, bx, bg = ref.norm_backward(f64(dy), f64(total), f64(gamma), f64(res), EPS)
    close(dx, want, 4 * ref.norm_rel(c) * bx + ref.stored(want, xdt), "dx")
    close(dgamma, wg, (ref.norm_rel(c) + ref.U32 * (rows + 64)) * bg, "dgamma")


@pytest.mark.parametrize("rows", [1, 2, 40, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_e4m3_nan_and_zero_rows(handle, rows, gated):
    """A NaN of E4M3 spoils its own row and no other; zero operands give the bias."""
    c, k = 160, 96
    n = 2 * k if gated else k
    (x, sx), (w, sw) = quantized(rand(rows, c, seed=1)), quantized(rand(n, c, seed=2))
    x[rows - 1, c // 2] = float("nan")
    x[0] = 0 if rows > 1 else x[0]
    bias = rand(n, seed=3)
    y = out_like(rows, k, F32)
    (api.GatedForward if gated else api.LinearForward)(handle, x, w, y, act="relu")(x, w, y, bias=bias, x_scale=sx, w_scale=sw)
    assert torch.isnan(y[rows - 1]).all() and int(torch.isnan(y).sum()) == k
    if rows > 1:
        b = f64(bias)
        want = b[:k].clamp(min=0) * (b[k:] if gated else 1)
        close(y[0], want, 1e-6 * want.abs() + 1e-30, "bias only")


@pytest.mark.parametrize("kind", ["silu", "gelu", "tanh", "sigmoid", "relu"])
def test_activations_far_out(handle, kind):
    """Arguments from -200 to 200 and infinities, forward and backward."""
    v = torch.tensor([-float("inf"), -200.0, -90.0, -30.0, -8.0, -3.0, -1e-3, 0.0, 1e-3, 3.0, 8.0, 30.0, 90.0, 200.0, float("inf"),
                      1.0]).to(BF).cuda()
    x, w = torch.ones(1, 1, dtype=BF, device="cuda"), v.view(-1, 1).contiguous()
    y, z = torch.empty(1, 16, device="cuda"), torch.empty(1, 16, device="cuda")
    api.LinearForward(handle, x, w, y, act=kind, z=z)(x, w, y, z=z)
    assert torch.equal(z[0].to(BF), v)
    f, df = ref.act(f64(v), kind)
    finite = torch.isfinite(f64(v))
    close(y[0][finite.cuda()], f[finite], ref.ACT_REL * f[finite].abs() + 2e-6, kind)
    if kind in ("tanh", "sigmoid", "relu"):
        assert torch.equal(f64(y[0])[~finite], f[~finite])
    dy, db = torch.ones(1, 16, dtype=F32, device="cuda"), torch.empty(16, device="cuda")
    api.LinearBackward(handle, x, w, dy, z=z, act=kind)(x, w, dy, dbias=db, z=z)
    close(db[finite.cuda()], df[finite], ref.ACT_REL * (1 + f64(v)[finite].abs()), kind + " slope")


def test_norm_of_tiny_and_large_rows(handle):
    """Rows of size 1e-12 (epsilon rules) and 1e12."""
    gamma = 1 + 0.3 * rand(300, seed=3)
    x = rand(4, 300, seed=1)
    x[1] *= 1e-12
    x[2] *= 1e12
    x[3] = 0
    y = torch.empty_like(x)
    api.RmsNormForward(handle, x, y, eps=EPS)(x, gamma, y)
    _, want = ref.norm(f64(x), None, f64(gamma), EPS)
    close(y, want, ref.norm_rel(300) * want.abs() + 1e-30, "y")


def test_arguments_written_just_before_the_call(handle):
    """Each launch may overlap the one before it; what that one wrote is read
    all the same: gamma, bias, filters and rows changed right before each call."""
    rows, c, k = 64, 512, 256
    x, w, y = rand(rows, c, seed=1, dtype=BF), rand(k, c, seed=2, std=c ** -0.5, dtype=BF), torch.empty(rows, k, device="cuda")
    n, gamma, bias = torch.empty(rows, c, device="cuda"), torch.ones(c, device="cuda"), torch.zeros(k, device="cuda")
    norm, lin = api.RmsNormForward(handle, x, n, eps=EPS), api.LinearForward(handle, x, w, y)
    got = []
    for i in range(20):
        gamma.fill_(float(i))
        norm(x, gamma, n)
        bias.fill_(float(i))
        lin(x, w, y, bias=bias)
        w.mul_(-1.0)
        got.append((n.clone(), y.clone()))
    _, unit = ref.norm(f64(x), None, torch.ones(c, dtype=torch.float64), EPS)
    z, ez = ref.product(f64(x), f64(w))
    for i, (a, b) in enumerate(got):
        close(a, i * unit, ref.norm_rel(c) * (i * unit).abs() + 1e-30, f"gamma {i}")
        close(b, z * (-1) ** i + i, ez + 1e-6 * (i + 1), f"filters {i}")


def test_e4m3_belongs_to_the_channel_operators(handle):
    x = torch.zeros(1, 16, 4, 4, device="cuda").to(F8)
    w, y = torch.zeros(16, 16, 1, 1, device="cuda").to(F8), torch.empty(1, 16, 4, 4, device="cuda")
    for call in (lambda: api.Conv2dForward(handle, x, w, y, math="bf16")(x, w, y),
                 lambda: api.Pool2dForward(handle, x, y, window=(1, 1), stride=(1, 1))(x, y),
                 lambda: api.Conv2dBackwardData(handle, w, x, x.clone(), math="bf16")(w, x, x.clone())):
        with pytest.raises(B.DlcError) as e:
            call()
        assert e.value.status == B.DLC_STATUS_NOT_SUPPORTED
