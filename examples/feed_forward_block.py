"""A convolution followed by a feed-forward block, trained and then served.

    s = conv3x3(image)                         the residual stream, NHWC pixels
    t = s + r;  n = gamma * t / rms(t)         RmsNormForward
    h = silu(n Wg^T) * (n Wu^T)                GatedForward
    out = h Wd^T + bd + t                      LinearForward

A training step runs the block forward and backward in BF16 with FP32 master
weights and plain gradient descent; serving takes the trained weights to E4M3
with one scale a filter and runs single pixels, the norm writing E4M3 rows with
their scales for the gated projections to read.

    python -m examples.feed_forward_block
"""
from __future__ import annotations

import torch

from deep_learning_convolution_gb300 import api

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


class FeedForwardBlock:
    """The block on `rows` pixels of `channels`, with its gradients."""

    def __init__(self, handle, rows, channels, hidden, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std

        def bf16(*shape):
            return torch.empty(*shape, dtype=BF16, device=device)

        # FP32 master weights; the gate's filters come first, then the up filters
        self.master = {"gamma": torch.ones(channels, device=device),
                       "up": randn(2 * hidden, channels, std=channels ** -0.5),
                       "down": randn(channels, hidden, std=0.5 * hidden ** -0.5),
                       "bias": torch.zeros(channels, device=device)}
        self.up, self.down = self.master["up"].to(BF16), self.master["down"].to(BF16)
        self.total, self.normed, self.out = bf16(rows, channels), bf16(rows, channels), bf16(rows, channels)
        self.z, self.hidden = bf16(rows, 2 * hidden), bf16(rows, hidden)
        self.dhidden, self.dnormed, self.dstream = bf16(rows, hidden), bf16(rows, channels), bf16(rows, channels)
        self.grad = {k: torch.empty_like(v) for k, v in self.master.items()}
        self.norm = api.RmsNormForward(handle, self.out, self.normed, residual=self.out, total=self.total)
        self.gated = api.GatedForward(handle, self.normed, self.up, self.hidden, z=self.z)
        self.linear = api.LinearForward(handle, self.hidden, self.down, self.out, residual=self.total)
        self.linear_back = api.LinearBackward(handle, self.hidden, self.down, self.out, self.dhidden, self.grad["down"])
        self.gated_back = api.GatedBackward(handle, self.normed, self.up, self.dhidden, self.dnormed, self.grad["up"],
                                            z=self.z)
        self.norm_back = api.RmsNormBackward(handle, self.dnormed, self.total, self.dstream, dtotal=self.out)

    def forward(self, stream, residual):
        self.norm(stream, self.master["gamma"], self.normed, residual=residual, total=self.total)
        self.gated(self.normed, self.up, self.hidden, z=self.z)
        return self.linear(self.hidden, self.down, self.out, bias=self.master["bias"], residual=self.total)

    def backward(self, dout):
        """Gradients of every weight, and of the stream (which is the residual's too)."""
        self.linear_back(self.hidden, self.down, dout, self.dhidden, self.grad["down"], dbias=self.grad["bias"])
        self.gated_back(self.normed, self.up, self.dhidden, self.dnormed, self.grad["up"], z=self.z)
        return self.norm_back(self.dnormed, self.total, self.master["gamma"], self.dstream, dgamma=self.grad["gamma"],
                              dtotal=dout)

    def step(self, rate):
        for k, v in self.master.items():
            v.sub_(self.grad[k], alpha=rate)
        self.up.copy_(self.master["up"])
        self.down.copy_(self.master["down"])


class ServedBlock:
    """The block's forward pass for a few rows, up projections in E4M3."""

    def __init__(self, handle, block: FeedForwardBlock, rows):
        channels, hidden = block.down.shape
        dev = block.down.device
        self.gamma, self.bias, self.down = block.master["gamma"], block.master["bias"], block.down
        scale = block.master["up"].abs().amax(1, keepdim=True).clamp_min(1e-30) / 448.0
        self.up, self.up_scale = (block.master["up"] / scale).to(E4M3), scale[:, 0].contiguous()
        self.total, self.out = (torch.empty(rows, channels, dtype=BF16, device=dev) for _ in range(2))
        self.normed = torch.empty(rows, channels, dtype=E4M3, device=dev)
        self.scale = torch.empty(rows, device=dev)
        self.hidden = torch.empty(rows, hidden, dtype=BF16, device=dev)
        self.norm = api.RmsNormForward(handle, self.total, self.normed, residual=self.total, total=self.total)
        self.gated = api.GatedForward(handle, self.normed, self.up, self.hidden)
        self.linear = api.LinearForward(handle, self.hidden, self.down, self.out, residual=self.total)

    def __call__(self, stream, residual):
        self.norm(stream, self.gamma, self.normed, residual=residual, total=self.total, scale=self.scale)
        self.gated(self.normed, self.up, self.hidden, x_scale=self.scale, w_scale=self.up_scale)
        return self.linear(self.hidden, self.down, self.out, bias=self.bias, residual=self.total)


def main(steps=60, images=4, size=14, channels=128, hidden=344, rate=40.0, verbose=True):
    """Trains the block to a teacher's outputs; returns the losses and how far
    the served block's outputs are from the trained one's."""
    handle = api.Handle()
    g = torch.Generator(device="cuda").manual_seed(1)
    image = torch.randn(images, size, size, channels, generator=g, device="cuda").to(BF16)
    filters = (torch.randn(channels, 3, 3, channels, generator=g, device="cuda") / (3 * channels ** 0.5)).to(BF16)
    features = torch.empty_like(image)
    conv = api.Conv2dForward(handle, image, filters, features, x_axes="NHWC", w_axes="KRSC", y_axes="NHWC",
                             pads=(1, 1, 1, 1), math="bf16")
    conv(image, filters, features, relu=True)
    rows = images * size * size
    stream, residual = features.view(rows, channels), image.view(rows, channels)
    teacher = FeedForwardBlock(handle, rows, channels, hidden, seed=2)
    target = teacher.forward(stream, residual).float()
    block = FeedForwardBlock(handle, rows, channels, hidden, seed=3)
    losses = []
    for i in range(steps):
        error = block.forward(stream, residual).float() - target
        losses.append(error.square().mean().item())
        block.backward((error * (2.0 / error.numel())).to(BF16))
        block.step(rate)
        if verbose and i % 10 == 0:
            print(f"step {i:3d}  loss {losses[-1]:.4f}")
    want = block.forward(stream, residual).float()
    served = ServedBlock(handle, block, 1)
    far, size_ = 0.0, 0.0
    for row in range(0, rows, max(1, rows // 16)):
        got = served(stream[row:row + 1], residual[row:row + 1]).float()
        far += (got - want[row]).square().sum().item()
        size_ += want[row].square().sum().item()
    off = (far / size_) ** 0.5
    if verbose:
        print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; served in E4M3, one pixel at a time: {off:.4f} off")
    handle.synchronize()
    handle.close()
    return losses, off


if __name__ == "__main__":
    main()
