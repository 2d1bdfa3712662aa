"""The feed-forward example: its gradients against autograd in FP64, its
training and its E4M3 serving."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from examples import feed_forward_block as ex

pytestmark = pytest.mark.gpu


def test_gradients_of_the_block():
    rows, c, f = 96, 64, 80
    handle = api.Handle()
    block = ex.FeedForwardBlock(handle, rows, c, f, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    stream, residual, dout = (torch.randn(rows, c, generator=g, device="cuda").to(ex.BF16) for _ in range(3))
    out = block.forward(stream, residual)
    dstream = block.backward(dout)
    torch.cuda.synchronize()
    x = stream.double().requires_grad_()
    gamma, up, down, bias = (v.double().detach().requires_grad_() for v in
                             (block.master["gamma"], block.up, block.down, block.master["bias"]))
    t = x + residual.double()
    n = gamma * t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    z = n @ up.t()
    h = torch.nn.functional.silu(z[:, :f]) * z[:, f:]
    want = h @ down.t() + bias + t
    want.backward(dout.double())

    def off(a, b):
        return ((a.double() - b).norm() / b.norm()).item()

    # every tensor between the operators is BF16 (2^-9 relative, uniformly
    # spread: 1.7e-3 a rounding); at most eight roundings meet in a gradient
    assert off(out, want.detach()) < 5e-3
    for name, a, b in (("stream", dstream, x.grad), ("gamma", block.grad["gamma"], gamma.grad),
                       ("up", block.grad["up"], up.grad), ("down", block.grad["down"], down.grad),
                       ("bias", block.grad["bias"], bias.grad)):
        assert off(a, b) < 8 * 1.7e-3, name
    handle.close()


def test_example_trains_and_serves():
    losses, off = ex.main(steps=40, verbose=False)
    assert losses[-1] < 0.7 * losses[0]
    # E4M3 operands: 2^-5 relative rms a rounding at most in each of gate and up,
    # two operands each, on a part of the output that the stream dominates
    assert off < 0.06
