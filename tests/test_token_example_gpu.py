"""The token model: its gradients against autograd in FP64 (the same masks), and that its
captured steps run."""
import math

import pytest
import torch

from deep_learning_convolution_gb300 import api
from examples import token_model as ex
from tests import train_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocabulary,channels,hidden", [(96, 50, 64, 80), (300, 1003, 128, 200)])
def test_gradients_of_the_model(rows, vocabulary, channels, hidden):
    with api.Handle() as handle:
        model = ex.TokenModel(handle, rows, vocabulary, channels, hidden, p=0.2, seed=3)
        g = torch.Generator().manual_seed(4)
        model.tokens.copy_(torch.randint(-1, vocabulary, (rows,), generator=g))
        model.target.copy_(torch.randint(-1, vocabulary, (rows,), generator=g))
        for k in ("gamma", "beta", "gamma2", "beta2"):
            model.master[k].add_(0.2 * torch.randn(channels, generator=g).cuda())
        loss = model.forward()
        model.backward()
        handle.synchronize()
        # BF16 weights are the leaves; the table is two of them, whose gradients add up
        leaf = {k: (model.weights.get(k, v)).double().detach().requires_grad_() for k, v in model.master.items()}
        there = (model.tokens >= 0)[:, None]
        x = torch.where(there, leaf["table"][model.tokens.clamp(min=0)] * model.scale, 0.0)
        keep = [ref.dropout(torch.ones(rows, channels, dtype=torch.float64, device="cuda"), None, 0.2, *r.tolist())[0]
                for r in model.random]
        s = x * keep[0]

        def norm(t, gamma, beta):
            return torch.nn.functional.layer_norm(t, (channels,), gamma, beta, 1e-5)

        z = norm(s, leaf["gamma"], leaf["beta"]) @ leaf["up"].t()
        h = torch.nn.functional.silu(z[:, :hidden]) * z[:, hidden:]
        t = s + (h @ leaf["down"].t()) * keep[1]
        logits = norm(t, leaf["gamma2"], leaf["beta2"]) @ leaf["table"].t()
        want = torch.nn.functional.cross_entropy(logits, model.target, reduction="none", ignore_index=-1)
        (want.sum() / (model.target >= 0).sum()).backward()

        def off(a, b):
            return ((a.double() - b).norm() / b.norm()).item()

        # every tensor between the operators is BF16: 2^-9 relative at most, uniformly spread 1.7e-3 a
        # rounding; sixteen tensors lie on the longest way from a weight to its gradient and
        # their errors are independent
        assert off(loss, want.detach()) < 4 * 1.7e-3
        for k, v in leaf.items():
            assert off(model.grad[k], v.grad) < math.sqrt(16) * 2 * 1.7e-3, k
        # padded rows leave nothing behind
        assert (loss[model.target < 0] == 0).all()


def test_example_runs():
    losses = ex.main(steps=12, verbose=False)
    assert len(losses) == 12 and all(math.isfinite(v) and v > 0 for v in losses)
