"""hga_q4_append: rows that several sequences of a call name (needs a B200)."""
import numpy as np
import pytest
import torch

import q4_ref
from test_gpu_q4 import _f64, _i32, _lib

pytestmark = pytest.mark.gpu


def _append(rows, counts, n_rows, length, off=True):
    """One call on a fresh pool: status, the tokens read back, the tokens."""
    hga = _lib()
    p = hga.Params(2, 1, 64)
    pool = hga.PagePool.allocate(1, 2 * n_rows, hga.q4_page_bytes(p, 8), 8, n_rows, 2)
    hga.pages_reserve(pool, _i32(np.arange(n_rows)), _i32([length] * n_rows))
    n = int(np.sum(counts))
    k, v = (torch.randn(n, 1, 64, device="cuda").bfloat16() for _ in range(2))
    b = hga.Q4Batch(_i32(rows), _i32(np.concatenate([[0], np.cumsum(counts)])) if off else None,
                    max(counts))
    hga.q4_append(p, pool, 0, b, k, v)
    status = hga.check()
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    hga.q4_read(p, pool, 0, b, ko, vo)
    assert hga.check() == 0
    same = np.array_equal(_f64(ko), q4_ref.stored(_f64(k))) and np.array_equal(_f64(vo), q4_ref.stored(_f64(v)))
    return status, same


@pytest.mark.parametrize("rows,counts", [([0, 0, 1], [9, 0, 9]), ([0, 0], [0, 9]),
                                         ([1, 1, 1, 0, 1], [0, 0, 9, 9, 0])])
def test_a_sequence_without_tokens_writes_nothing(rows, counts):
    assert _append(rows, counts, 2, 9) == (0, True)


@pytest.mark.parametrize("n,off", [(40, True), (1000, True), (1000, False), (3000, False)])
def test_many_sequences(n, off):
    hga = _lib()
    rows = np.random.default_rng(n).permutation(n)
    assert _append(rows, [1] * n, n, 3, off) == (0, True)
    rows[-1] = rows[7]
    assert _append(rows, [1] * n, n, 3, off)[0] == hga.HGA_ERR_DEVICE_CHECK
    rows[-1] = rows[n - 2]
    assert _append(rows, [1] * n, n, 3, off)[0] == hga.HGA_ERR_DEVICE_CHECK


def test_inactive_sequences_share_their_mark():
    hga = _lib()
    p = hga.Params(2, 1, 64)
    pool = hga.PagePool.allocate(1, 4, hga.q4_page_bytes(p, 8), 8, 2, 2)
    hga.pages_reserve(pool, _i32([0, 1]), _i32([1, 1]))
    k = torch.randn(600, 1, 64, device="cuda").bfloat16()
    rows = np.full(600, -1)
    rows[[3, 590]] = [0, 1]
    hga.q4_append(p, pool, 0, hga.Q4Batch(_i32(rows)), k, k)
    assert hga.check() == 0
