"""Limits of the serving calls that the host checks (no GPU)."""
import ctypes

import pytest

from test_serving_abi import FAKE, _pool


@pytest.fixture(scope="module")
def hga():
    from long_context_hga_b200 import build
    build.build()
    from long_context_hga_b200 import hga as mod
    return mod


def test_append_takes_as_many_sequences_as_the_attention(hga):
    """The search for rows that two sequences name grows with their square."""
    p, n0 = hga.Params(8, 2, 128).c(), hga.launch_count()

    def append(n_seq):
        b = hga.CQ4Batch(FAKE, FAKE, n_seq, 4)
        return hga.LIB.hga_q4_append(ctypes.byref(p), ctypes.byref(_pool(hga)), 0, ctypes.byref(b), 8,
                                     FAKE, 256, 128, FAKE, 256, 128, None)

    assert append(65536) == 2
    assert append(0) == 0
    assert hga.launch_count() == n0
