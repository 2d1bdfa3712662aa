"""The FP64 definitions that the tests of layer norm, dropout, embedding and cross
entropy compare with, against independent forms of them."""
import numpy as np
import pytest
import torch

from tests import train_ref as ref


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_philox_known_answers():
    """The known answers of the generator's reference: a zero counter and key, and all ones."""
    assert [hex(v) for v in ref.philox(0, 0, [0], 4)[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    ones = 2 ** 64 - 1
    # counter (c / 4, row, step): all ones needs group 2^32 - 1, so the rounds by hand
    x, k = [2 ** 32 - 1] * 4, [2 ** 32 - 1] * 2
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(b >> 32) ^ x[1] ^ k[0], b % 2 ** 32, (a >> 32) ^ x[3] ^ k[1], a % 2 ** 32]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    assert [hex(v) for v in x] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]
    assert ref.philox(-1, -1, [5], 9).tolist() == ref.philox(ones, ones, [5], 9).tolist()


def test_layer_norm_is_torchs():
    x, g, b = randn(7, 33, seed=1), randn(33, seed=2), randn(33, seed=3)
    _, y, _ = ref.layer_norm(x, None, g, b, 1e-5)
    assert torch.allclose(y, torch.nn.functional.layer_norm(x, (33,), g, b, 1e-5))


def test_layer_norm_gradient_is_autograds():
    x, g, b, dy, dt = (randn(*s, seed=i).requires_grad_(i < 3) for i, s in enumerate([(7, 33), (33,), (33,), (7, 33), (7, 33)]))
    torch.nn.functional.layer_norm(x, (33,), g, b, 1e-5).backward(dy)
    (dx, _), (dg, _), (db, _) = ref.layer_norm_backward(dy, x.detach(), g.detach(), dt, 1e-5)
    assert torch.allclose(dx, x.grad + dt) and torch.allclose(dg, g.grad) and torch.allclose(db, b.grad)


def test_embedding_gradient_is_autograds():
    table, dy = randn(11, 5, seed=1).requires_grad_(), randn(40, 5, seed=2)
    tokens = torch.randint(0, 11, (40,), generator=torch.Generator().manual_seed(3))
    y = 3.0 * table[tokens]
    y.backward(dy)
    assert torch.equal(ref.embedding(tokens, table.detach(), 3.0), y.detach())
    assert torch.allclose(ref.embedding_backward(tokens, dy, 11, 3.0)[0], table.grad)
    tokens[::3] = -1
    assert torch.allclose(ref.embedding_backward(tokens, dy, 11, 1.0)[0],
                          torch.zeros(11, 5, dtype=torch.float64).index_add_(0, tokens[tokens >= 0], dy[tokens >= 0]))


def test_cross_entropy_and_its_gradient_are_torchs():
    x, w, b = (randn(*s, seed=i).requires_grad_() for i, s in enumerate([(20, 6), (9, 6), (9,)]))
    target = torch.randint(0, 9, (20,), generator=torch.Generator().manual_seed(4))
    target[3] = target[11] = -100
    weight = randn(20, seed=5).abs()
    loss = torch.nn.functional.cross_entropy(x @ w.t() + b, target, reduction="none")
    (loss * weight).sum().backward()
    f = ref.cross_entropy(x.detach(), w.detach(), target, b.detach())
    assert torch.allclose(f["loss"][0], loss.detach())
    got = ref.cross_entropy_backward(x.detach(), w.detach(), target, f, weight, torch.float32, torch.float32)
    for (g, _), leaf in zip(got, (x, w, b)):
        assert torch.allclose(g, leaf.grad)


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9])
def test_dropout_keeps_the_share_it_says(p):
    x = torch.ones(400, 250, dtype=torch.float64)
    y, keep = ref.dropout(x, None, p, 7, 3)
    n = keep.numel()
    assert abs(keep.double().mean().item() - (1 - p)) <= 5 * (p * (1 - p) / n) ** 0.5
    assert torch.equal(y > 0, keep) and np.isclose(y.max().item(), 1 / (1 - p))
