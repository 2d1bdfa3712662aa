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
