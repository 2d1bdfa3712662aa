"""The token model's training steps: each takes the gradients off the weights and advances the masks, and a
replayed step does what an eager one does."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from examples import token_model as ex
from tests import channel_ref as cref

pytestmark = pytest.mark.gpu
ROWS, VOCABULARY, CHANNELS, HIDDEN, RATE = 200, 503, 64, 136, 1.5


def model(handle):
    return ex.TokenModel(handle, ROWS, VOCABULARY, CHANNELS, HIDDEN, p=0.1, seed=5)


def batch(m, i):
    g = torch.Generator().manual_seed(100 + i)
    for t in (m.tokens, m.target):
        t.copy_(torch.randint(-1, VOCABULARY, (ROWS,), generator=g))


def train(m):
    m.forward()
    m.backward()
    m.step(RATE)


def state(m):
    tensors = {**{"master " + k: v for k, v in m.master.items()}, **{"weight " + k: v for k, v in m.weights.items()},
               **{"gradient " + k: v for k, v in m.grad.items()}, "loss": m.loss, "masks 1": m.random[0], "masks 2": m.random[1]}
    return {k: v.clone() for k, v in tensors.items()}


def test_steps_take_the_gradients_off_the_weights():
    stream = torch.cuda.Stream()
    with api.Handle(stream) as handle, torch.cuda.stream(stream):
        m = model(handle)
        for i in range(3):
            batch(m, i)
            before = state(m)
            train(m)
            stream.synchronize()
            after = state(m)
            for k in m.master:
                old, new, grad = (s[n + k].double() for s, n in ((before, "master "), (after, "master "), (after, "gradient ")))
                # the product's and the difference's rounding
                assert ((new - (old - RATE * grad)).abs() <= 2 * cref.U32 * (old.abs() + RATE * grad.abs())).all(), k
                assert (new != old).any(), k
            for k in m.weights:
                assert torch.equal(after["weight " + k], after["master " + k].to(torch.bfloat16)), k
                assert not torch.equal(after["weight " + k], before["weight " + k]), k
            for k in ("masks 1", "masks 2"):
                assert (after[k] - before[k]).tolist() == [0, 2]
        handle.synchronize()


def test_replayed_steps_are_eager_ones():
    stream = torch.cuda.Stream()
    with api.Handle(stream) as handle, torch.cuda.stream(stream):
        eager, replayed = model(handle), model(handle)
        for m in (eager, replayed):
            batch(m, 0)
            train(m)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            train(replayed)
        for i in range(1, 5):
            batch(eager, i)
            batch(replayed, i)
            train(eager)
            graph.replay()
            stream.synchronize()
            a, b = state(eager), state(replayed)
            for k in a:
                assert torch.equal(a[k], b[k]), (i, k)
        assert eager.random[0].tolist() == [5, 10]
        handle.synchronize()
