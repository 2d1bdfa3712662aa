"""A small token model trained from token ids to its loss, every step one replayed graph.

    s = dropout(scale * E[tokens])                       EmbeddingForward, DropoutForward
    n = layer_norm(s);  h = silu(n Wg^T) * (n Wu^T)      LayerNormForward, GatedForward
    t = s + dropout(h Wd^T)                              LinearForward, DropoutForward
    m = layer_norm(t);  loss = cross_entropy(m E^T, next token)    CrossEntropyForward

The table E is the classifier's weight too: the loss's gradient is written to it and
the embedding's added.  Padded rows (tokens and targets of -1) take no part.  A step
of plain gradient descent, the dropout's step counter and the refreshed BF16 weights are
captured in one CUDA graph with the forward and backward pass.

    python -m examples.token_model
"""
from __future__ import annotations

import torch

from deep_learning_convolution_gb300 import api

BF16 = torch.bfloat16


class TokenModel:
    """The model on `rows` tokens at a time, with its gradients (FP32 master weights)."""

    def __init__(self, handle, rows, vocabulary, channels, hidden, p=0.1, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std

        def bf16(*shape):
            return torch.empty(*shape, dtype=BF16, device=device)

        def fp32(*shape):
            return torch.empty(*shape, device=device)

        self.master = {"table": randn(vocabulary, channels, std=channels ** -0.5),
                       "up": randn(2 * hidden, channels, std=channels ** -0.5),
                       "down": randn(channels, hidden, std=hidden ** -0.5),
                       "gamma": torch.ones(channels, device=device), "beta": torch.zeros(channels, device=device),
                       "gamma2": torch.ones(channels, device=device), "beta2": torch.zeros(channels, device=device)}
        self.weights = {k: self.master[k].to(BF16) for k in ("table", "up", "down")}
        self.grad = {k: torch.empty_like(v) for k, v in self.master.items()}
        self.scale, self.p = channels ** 0.5, p
        # seed and step of the two dropouts; a step counter for each call
        self.random = [torch.tensor([seed, i], dtype=torch.int64, device=device) for i in range(2)]
        self.tokens = torch.zeros(rows, dtype=torch.int64, device=device)
        self.target = torch.zeros(rows, dtype=torch.int64, device=device)
        self.embedded, self.stream, self.normed, self.down = (bf16(rows, channels) for _ in range(4))
        self.total, self.final = bf16(rows, channels), bf16(rows, channels)
        self.z, self.hidden = bf16(rows, 2 * hidden), bf16(rows, hidden)
        self.loss, self.lse, self.weight = fp32(rows), fp32(rows), fp32(rows)
        self.dfinal, self.dtotal, self.ddown, self.dnormed, self.dstream, self.dembedded = (bf16(rows, channels) for _ in range(6))
        self.dhidden = bf16(rows, hidden)
        w, h = self.weights, handle
        self.embed = api.EmbeddingForward(h, self.tokens, w["table"], self.embedded, scale=self.scale)
        self.drop = api.DropoutForward(h, self.embedded, self.stream, p=p)
        self.norm = api.LayerNormForward(h, self.stream, self.normed)
        self.gated = api.GatedForward(h, self.normed, w["up"], self.hidden, z=self.z)
        self.linear = api.LinearForward(h, self.hidden, w["down"], self.down)
        self.drop2 = api.DropoutForward(h, self.down, self.total, p=p, residual=self.stream)
        self.norm2 = api.LayerNormForward(h, self.total, self.final)
        self.entropy = api.CrossEntropyForward(h, self.final, w["table"], self.target)
        self.entropy_back = api.CrossEntropyBackward(h, self.final, w["table"], self.target, self.dfinal, self.grad["table"])
        self.norm2_back = api.LayerNormBackward(h, self.dfinal, self.total, self.dtotal)
        self.drop2_back = api.DropoutBackward(h, self.dtotal, self.ddown, p=p)
        self.linear_back = api.LinearBackward(h, self.hidden, w["down"], self.ddown, self.dhidden, self.grad["down"])
        self.gated_back = api.GatedBackward(h, self.normed, w["up"], self.dhidden, self.dnormed, self.grad["up"], z=self.z)
        self.norm_back = api.LayerNormBackward(h, self.dnormed, self.stream, self.dstream, dtotal=self.dtotal)
        self.drop_back = api.DropoutBackward(h, self.dstream, self.dembedded, p=p)
        self.embed_back = api.EmbeddingBackward(h, self.tokens, self.dembedded, self.grad["table"], scale=self.scale,
                                                accumulate=True)

    def forward(self):
        """The rows' losses, of the tokens and targets in self.tokens and self.target."""
        w, m = self.weights, self.master
        self.embed(self.tokens, w["table"], self.embedded)
        self.drop(self.embedded, self.random[0], self.stream)
        self.norm(self.stream, m["gamma"], self.normed, beta=m["beta"])
        self.gated(self.normed, w["up"], self.hidden, z=self.z)
        self.linear(self.hidden, w["down"], self.down)
        self.drop2(self.down, self.random[1], self.total, residual=self.stream)
        self.norm2(self.total, m["gamma2"], self.final, beta=m["beta2"])
        return self.entropy(self.final, w["table"], self.target, self.loss, self.lse)

    def backward(self):
        """Gradients of the mean loss over the rows that have a target."""
        w, m, g = self.weights, self.master, self.grad
        counted = (self.target >= 0).float()
        torch.div(counted, counted.sum().clamp(min=1), out=self.weight)
        self.entropy_back(self.final, w["table"], self.target, self.lse, self.weight, self.dfinal, g["table"])
        self.norm2_back(self.dfinal, self.total, m["gamma2"], self.dtotal, dgamma=g["gamma2"], dbeta=g["beta2"])
        self.drop2_back(self.dtotal, self.random[1], self.ddown)
        self.linear_back(self.hidden, w["down"], self.ddown, self.dhidden, g["down"])
        self.gated_back(self.normed, w["up"], self.dhidden, self.dnormed, g["up"], z=self.z)
        self.norm_back(self.dnormed, self.stream, m["gamma"], self.dstream, dgamma=g["gamma"], dbeta=g["beta"],
                       dtotal=self.dtotal)
        self.drop_back(self.dstream, self.random[0], self.dembedded)
        self.embed_back(self.tokens, self.dembedded, g["table"])

    def step(self, rate):
        for k, v in self.master.items():
            v.sub_(self.grad[k], alpha=rate)
        for k, v in self.weights.items():
            v.copy_(self.master[k])
        for r in self.random:
            r[1] += 2  # other elements are dropped in the next step


def main(steps=200, rows=512, vocabulary=2003, channels=128, hidden=344, rate=2.0, verbose=True):
    """Trains the model to continue sequences t -> a t + b (mod vocabulary); returns the losses."""
    stream = torch.cuda.Stream()
    with api.Handle(stream) as handle, torch.cuda.stream(stream):
        model = TokenModel(handle, rows, vocabulary, channels, hidden, seed=1)
        g = torch.Generator().manual_seed(2)

        def batch():
            tokens = torch.randint(0, vocabulary, (rows,), generator=g)
            tokens[torch.rand(rows, generator=g) < 0.05] = -1  # padding
            model.tokens.copy_(tokens)
            model.target.copy_(torch.where(tokens < 0, -1, (17 * tokens + 5) % vocabulary))

        def train():
            model.forward()
            model.backward()
            model.step(rate)

        batch()
        train()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            train()
        losses = []
        for i in range(steps):
            batch()
            graph.replay()
            losses.append((model.loss * model.weight).sum().item())
            if verbose and i % 20 == 0:
                print(f"step {i:3d}  loss {losses[-1]:.4f}")
        handle.synchronize()
    return losses


if __name__ == "__main__":
    main()
