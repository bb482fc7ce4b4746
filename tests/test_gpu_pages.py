"""Pages of a cache (hga_pages_*) against plain bookkeeping (needs a B200)."""
import numpy as np
import pytest
import torch

import q4_ref

pytestmark = pytest.mark.gpu


def _lib():
    from long_context_hga_b200 import hga
    return hga


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _pair(planes, pages, page_bytes, pt, rows, row_pages, seed=0):
    hga = _lib()
    ref = q4_ref.Pool(planes, pages, page_bytes, pt, rows, row_pages, np.random.default_rng(seed))
    dev = hga.PagePool(torch.from_numpy(ref.data.copy()).cuda(), _i32(ref.table), _i32(ref.len),
                       _i32(ref.ref), pt)
    return hga, ref, dev


def _same(hga, ref, dev, what):
    want = hga.HGA_ERR_DEVICE_CHECK if ref.bad else 0
    assert hga.check() == want, what
    ref.bad = 0
    for name, x in (("table", ref.table), ("length", ref.len), ("ref", ref.ref), ("data", ref.data)):
        got = getattr(dev, name).cpu().numpy()
        assert np.array_equal(got, x), (what, name, np.argwhere(got != x)[:5])


@pytest.mark.parametrize("planes,pages,page_bytes,pt,rows,row_pages", [
    (1, 40, 16, 8, 12, 5),
    (3, 300, 1152 * 2, 16, 50, 9),
    (2, 5000, 576, 64, 70, 40),
])
def test_random_histories(planes, pages, page_bytes, pt, rows, row_pages):
    """200 calls in a row, refused entries among them: rows outside the table,
    rows named twice, children in use, parents that are children, pools that
    run out, padding."""
    hga, ref, dev = _pair(planes, pages, page_bytes, pt, rows, row_pages)
    rng = np.random.default_rng(pages)
    for step in range(200):
        op = rng.choice(["reserve", "reserve", "fork", "fork", "free", "compact", "copy"])
        n = int(rng.integers(1, min(rows, 8) + 1))
        rs = rng.integers(-1, rows + (rng.random() < 0.1), n)
        if op == "reserve":
            grow = np.array([ref.len[r] if 0 <= r < rows else 0 for r in rs])
            new = grow + rng.integers(-1 if rng.random() < 0.2 else 0, 3 * pt, n)
            ref.reserve(rs, new)
            hga.pages_reserve(dev, _i32(rs), _i32(new))
        elif op == "fork":
            kids = rng.integers(-1, rows, n)
            if rng.random() < 0.7:                       # mostly empty, distinct children
                empty = rng.permutation(np.flatnonzero(ref.len == 0))
                kids[:len(empty[:n])] = empty[:n]
            ref.fork(rs, kids)
            hga.pages_fork(dev, _i32(rs), _i32(kids))
        elif op == "free":
            ref.free(rs)
            hga.pages_free(dev, _i32(rs))
        elif op == "compact":
            ref.compact()
            hga.pages_compact(dev)
        else:
            # into free pages, now and then into a source or twice
            src, dst = rng.integers(-1, pages, n), rng.integers(-1, pages, n)
            free = np.flatnonzero(ref.ref == 0)
            if len(free):
                dst = np.where(dst < 0, -1, rng.choice(free, n))
            else:
                src[:], dst[:] = -1, -1
            ref.copy(src, dst)
            hga.pages_copy(dev, _i32(src), _i32(dst))
        _same(hga, ref, dev, (step, op))
    # nothing leaks: with every row freed the pool is empty
    everything = np.arange(rows)
    ref.free(everything)
    hga.pages_free(dev, _i32(everything))
    _same(hga, ref, dev, "end")
    assert not ref.ref.any()


def test_pool_that_runs_out_serves_in_order():
    hga, ref, dev = _pair(1, 6, 32, 8, 5, 4)
    for rows, new in (([0, 1], [20, 8]), ([2, 3, 4], [9, 8, 0]), ([3], [8])):
        ref.reserve(rows, new)
        hga.pages_reserve(dev, _i32(rows), _i32(new))
        _same(hga, ref, dev, rows)
    assert ref.len.tolist() == [20, 8, 9, 0, 0]


def test_tables_without_data():
    """A pool may keep tables only (the bytes live elsewhere)."""
    hga, ref, dev = _pair(1, 16, 16, 8, 4, 4)
    dev._c.data = None
    ref.reserve([0], [13])
    hga.pages_reserve(dev, _i32([0]), _i32([13]))
    ref.fork([0], [1])
    ref.data = dev.data.cpu().numpy()                   # nothing was copied
    hga.pages_fork(dev, _i32([0]), _i32([1]))
    _same(hga, ref, dev, "tables")


def test_broken_tables_are_reported_and_left():
    hga, ref, dev = _pair(1, 8, 32, 8, 4, 4)
    ref.reserve([0], [16])
    hga.pages_reserve(dev, _i32([0]), _i32([16]))
    _same(hga, ref, dev, "start")
    dev.table[0, 1] = 99                                # no such page
    hga.pages_fork(dev, _i32([0]), _i32([1]))
    assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
    assert dev.table[1].tolist() == [0, -1, -1, -1] and dev.ref.tolist() == [2, 1] + [0] * 6
    hga.pages_compact(dev)
    assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
    hga.pages_free(dev, _i32([0, 1]))
    assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
    assert dev.ref.tolist() == [0, 1] + [0] * 6         # the page that lost its entry


def test_captured_step_replays():
    """free + fork captured once: each replay gives what the calls give."""
    hga, ref, dev = _pair(2, 64, 1152, 16, 8, 6)
    ref.reserve([0, 1], [40, 33])
    hga.pages_reserve(dev, _i32([0, 1]), _i32([40, 33]))
    parents, kids = _i32([0, 0, 1, 1]), _i32([2, 3, 4, 5])
    hga.pages_fork(dev, parents, kids)
    ref.fork([0, 0, 1, 1], [2, 3, 4, 5])
    _same(hga, ref, dev, "eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hga.pages_free(dev, kids)
        hga.pages_fork(dev, parents, kids)
    for turn in range(3):
        dev.data[:, 0].random_(0, 256)
        ref.data = dev.data.cpu().numpy()
        parents.copy_(_i32([turn % 2, 1, 0, 1]))
        graph.replay()
        ref.free([2, 3, 4, 5])
        ref.fork([turn % 2, 1, 0, 1], [2, 3, 4, 5])
        _same(hga, ref, dev, turn)
