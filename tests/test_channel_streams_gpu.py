"""The channel operators' workspaces between streams."""
import pytest
import torch

from deep_learning_convolution_gb300 import api
from tests.test_channel_ops_gpu import BF, rand

pytestmark = pytest.mark.gpu


def calls(op, n, stream, x, w, dy, want, got):
    """n calls on `stream`; whether any of them differs from `want` (a flag on the GPU)."""
    with torch.cuda.stream(stream):
        bad = torch.zeros((), dtype=torch.bool, device="cuda")
        for _ in range(n):
            op(x, w, dy, dw=got)
            bad |= (got != want).any()
    return bad


def problem():
    """A backward pass that reads copies of its operands in the workspace (rows at no
    multiple of 16 bytes) for most of its time."""
    x, w = rand(4000, 999, seed=1, dtype=BF), rand(1024, 999, seed=2, dtype=BF)
    dy = rand(4000, 1024, seed=3, dtype=BF)
    want, got = (torch.empty(1024, 999, dtype=BF, device="cuda") for _ in range(2))
    with api.Handle() as h:
        op = api.LinearBackward(h, x, w, dy, dw=want)
        size = op.workspace.numel()
        op(x, w, dy, dw=want)
        # (every kernel the tests queue up is loaded here: loading one waits for the GPU)
        assert not calls(op, 1, torch.cuda.current_stream(), x, w, dy, want, got).item()
        torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda._sleep(1)
        torch.cuda.synchronize()
        op.close()
    return x, w, dy, want, got, size


def test_workspace_is_not_another_streams_freed_memory():
    """Memory that was just released on torch's current stream, where kernels
    still write it, is no workspace for a handle on another stream."""
    x, w, dy, want, got, size = problem()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    with api.Handle(s) as h:
        old = torch.empty(size, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # some 10 ms: what follows queues up behind it
        for _ in range(1000):
            old.fill_(255)  # NaN, as BF16 and as FP32
        del old
        op = api.LinearBackward(h, x, w, dy, dw=got)
        bad = calls(op, 300, s, x, w, dy, want, got)
        torch.cuda.synchronize()
        op.close()
    assert not bad.item()


def test_workspace_outlives_work_on_every_stream_it_was_used_on():
    x, w, dy, want, got, size = problem()
    torch.cuda.empty_cache()
    busy, idle = torch.cuda.Stream(), torch.cuda.Stream()
    with api.Handle() as h:
        op = api.LinearBackward(h, x, w, dy, dw=got)
        torch.cuda.synchronize()
        with torch.cuda.stream(busy):
            torch.cuda._sleep(20_000_000)
        h.set_stream(busy)
        bad = calls(op, 100, busy, x, w, dy, want, got)
        h.set_stream(idle)
        op.close()
        idle.synchronize()
        other = torch.empty(size, dtype=torch.uint8, device="cuda")
        for _ in range(3000):  # before, beside and after the calls
            other.fill_(255)
        torch.cuda.synchronize()
    assert not bad.item()
