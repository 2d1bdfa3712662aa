"""Layer norm, dropout, embedding and cross entropy without a GPU: what their C entries
refuse before they look at a handle's device, and what their sources must not do."""
import os
import re

import pytest

from deep_learning_convolution_gb300 import binding as B
from deep_learning_convolution_gb300 import build as dlc_build

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deep_learning_convolution_gb300", "csrc")
NAMES = ("layernorm", "dropout", "embedding", "cross_entropy", "norm_rows", "channel_train")


@pytest.fixture(scope="module", autouse=True)
def lib():
    dlc_build.build()
    return B.load_library()


@pytest.mark.parametrize("call", [
    lambda: B.dlcLayerNormForward(None, 1e-5, None, 0, None, 0, 0, 0, None, 0, None, 0, 0),
    lambda: B.dlcGetLayerNormBackwardWorkspaceSize(None, None),
    lambda: B.dlcLayerNormBackward(None, 1e-5, None, 0, None, 0, 0, None, 0, None, 0, 0, 0, 0, 0),
    lambda: B.dlcDropoutForward(None, 0.1, 0, None, 0, None, 0, None, 0),
    lambda: B.dlcDropoutBackward(None, 0.1, 0, None, 0, None, 0),
    lambda: B.dlcEmbeddingForward(None, 1.0, B.DLC_INDEX_INT32, 0, None, 0, None, 0),
    lambda: B.dlcGetEmbeddingBackwardWorkspaceSize(None, None, None),
    lambda: B.dlcEmbeddingBackward(None, 1.0, B.DLC_INDEX_INT64, 0, None, 0, 0, None, 0, 0, 0),
    lambda: B.dlcCrossEntropyForward(None, None, 0, 0, None, 0, 0, 0, B.DLC_INDEX_INT32, 0, 0, 0, 0, 0),
    lambda: B.dlcGetCrossEntropyForwardWorkspaceSize(None, None, 0, None, 0),
    lambda: B.dlcCrossEntropyBackward(None, None, 0, None, 0, 0, B.DLC_INDEX_INT32, 0, 0, 0, None, 0, None, 0, 0, 0, 0),
    lambda: B.dlcGetCrossEntropyBackwardWorkspaceSize(None, None, 0, None, 0),
])
def test_calls_without_a_handle_are_refused(call):
    with pytest.raises(B.DlcError) as e:
        call()
    assert e.value.status == B.DLC_STATUS_NOT_INITIALIZED


def sources():
    for name in sorted(os.listdir(CSRC)):
        if name.startswith(NAMES):
            yield name, re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_nothing_is_read_by_the_read_only_path():
    """The grid ahead may still be writing what a kernel is about to read."""
    found = 0
    for name, text in sources():
        found += 1
        assert "__ldg(" not in text and "global.nc" not in text and "__restrict__" not in text, name
    assert found >= 7


def test_every_kernel_waits_for_the_grid_ahead():
    """Every kernel lets the next grid start early and waits itself before it touches memory."""
    for name, text in sources():
        kernels = re.split(r"__global__", text)[1:]
        for k in kernels:
            body = k[:k.index("\n}\n")]
            assert body.count("griddep_launch_dependents()") == 1 and "griddep_wait()" in body, name


def test_no_sum_depends_on_the_order_of_atomics():
    """Atomic additions only of whole numbers (histograms): gradients are the same every time."""
    for name, text in sources():
        for m in re.finditer(r"atomicAdd\(([^;]*);", text):
            assert name == "embedding.cu" and ("count" in m.group(1) or "hist" in m.group(1)), (name, m.group(0))
        assert "red.global" not in text, name
