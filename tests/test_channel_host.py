"""What the channel operators' host code must not keep between handles."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deep_learning_convolution_gb300", "csrc")


def test_counts_of_a_device_belong_to_its_handle():
    """How many clusters a device holds at once goes into a plan, and the plan into the
    workspace's size: one number for all devices of a process, or one that changes
    between the query and the call, would make them disagree."""
    asked = []
    for name in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        if name.startswith(("gemm", "gemv", "channel", "rmsnorm", "act_grad")):
            for line in text.splitlines():
                assert not re.search(r"\bstatic\s+(std::atomic<\s*int|int)\b[^()]*\bknown\b", line), f"{name}: {line.strip()}"
            asked += [name] * text.count("cudaOccupancyMaxActiveClusters(")
    assert asked == ["channel_api.cu"]  # one place, keeping its answers in the handle


def test_nothing_is_read_by_the_read_only_path():
    """The kernels start while the grid ahead of them runs, which may write anything they
    read: data of the read-only path must not change during a kernel."""
    for name in sorted(os.listdir(CSRC)):
        if name.startswith(("gemm", "gemv", "channel", "rmsnorm", "act_grad", "row_ring")):
            text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
            assert "__ldg(" not in text and "global.nc" not in text and "__restrict__" not in text, name
