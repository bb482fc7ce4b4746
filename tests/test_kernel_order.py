"""Orders that the kernels' sources have to keep, read from the sources (no
GPU): what breaks one of them is a race, which a run may not show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "long_context_hga_b200", "csrc")


def _function(file, name):
    """The text of a function, without its comments."""
    with open(os.path.join(CSRC, file)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = re.search(r"\b%s\s*\(" % re.escape(name), text).start()
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(name)


def test_a_kernel_that_writes_q_lets_no_dependent_start():
    """params.q_ready lets a kernel read q before it waits for the kernel ahead
    of it, so one that writes q must not let its dependents start early."""
    assert "griddep_launch" not in _function("rope.cuh", "rope_kernel")
