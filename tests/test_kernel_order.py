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


def test_the_abort_flag_is_cleared_before_any_warp_reads_it():
    """Thread 0 clears the block's abort flag; a warp that polled it before the
    store is ordered would take what an earlier block left for an abort and
    drop its tokens."""
    body = _function("q4_attend.cuh", "q4_attend_kernel")
    cleared = body.index("s_abort = 0")
    barrier = body.index("__syncthreads()", cleared)
    assert barrier < body.index("return", cleared)
    assert barrier < body.index("&s_abort", cleared)


def test_a_load_is_announced_after_every_lanes_entries():
    """The lanes of a fetching warp write the load's entries, lane 0 arrives for
    all of them: shuffles and ballots between do not order memory, so a
    __syncwarp has to stand before the arrive."""
    fetch = _function("q4_attend.cuh", "q4_fetch8")
    assert "__syncwarp()" in fetch[:fetch.index("mbar_arrive_expect_tx")]
    # and the entries are written before that call
    for file, kernel in (("q4_attend_tc.cuh", "q4_attend_tc_kernel"),
                         ("q4_attend.cuh", "q4_attend_kernel")):
        body = _function(file, kernel)
        assert 0 <= re.search(r"ents\[[^;]*\] = at", body).start() < body.index("q4_fetch8(")
