"""Page calls with lists longer than a block has threads (needs a B200)."""
import numpy as np
import pytest

from test_gpu_pages import _i32, _pair, _same

pytestmark = pytest.mark.gpu


def test_lists_of_thousands():
    """Reserve, fork, copy, free and compact with 1500 to 3000 entries, refused
    and padded ones among them: the counts carried from turn to turn."""
    rows, pages, pt = 3000, 9000, 8
    hga, ref, dev = _pair(1, pages, 16, pt, rows, 6)
    rng = np.random.default_rng(0)

    def reserve(rs, new):
        ref.reserve(rs, new)
        hga.pages_reserve(dev, _i32(rs), _i32(new))

    rs = rng.permutation(rows)
    rs[rng.integers(0, rows, 40)] = -1
    rs[rng.integers(0, rows, 20)] = rows
    rs[2900:2910] = rs[:10]                                 # named before
    rs = np.where(rs >= 1500, np.where(rs == rows, rows, -1), rs)
    reserve(rs, rng.integers(0, 30, rows))
    _same(hga, ref, dev, "reserve")
    parents, kids = rng.integers(-1, 1500, 1400), rng.permutation(np.arange(1500, 2900))
    kids[rng.integers(0, 1400, 50)] = -1
    kids[1300] = kids[3]
    ref.fork(parents, kids)
    hga.pages_fork(dev, _i32(parents), _i32(kids))
    _same(hga, ref, dev, "fork")
    free = np.flatnonzero(ref.ref == 0)
    src, dst = rng.integers(0, pages, 2500), np.full(2500, -1)
    dst[:len(free[:2000])] = rng.permutation(free)[:2000]
    dst[2100:] = dst[:400]
    src[2000:2100] = -1
    ref.copy(src, dst)
    hga.pages_copy(dev, _i32(src), _i32(dst))
    _same(hga, ref, dev, "copy")
    gone = rng.permutation(rows)[:2000]
    ref.free(gone)
    hga.pages_free(dev, _i32(gone))
    _same(hga, ref, dev, "free")
    ref.compact()
    hga.pages_compact(dev)
    _same(hga, ref, dev, "compact")
    # every row at once, until the pages run out somewhere past entry 1024
    everything = np.arange(rows)
    reserve(everything, ref.len + 25)
    _same(hga, ref, dev, "run out")
    assert 0 < (ref.ref == 0).sum() < 4 or (ref.ref == 0).sum() == 0


def test_a_row_of_thousands_of_pages():
    hga, ref, dev = _pair(1, 5000, 16, 8, 3, 4096)
    for rows, new in (([1, 0], [3 * 8, 1000 * 8 + 1]), ([0, 1], [4000 * 8, 90 * 8]), ([2], [2000 * 8])):
        ref.reserve(rows, new)
        hga.pages_reserve(dev, _i32(rows), _i32(new))
        _same(hga, ref, dev, rows)
    ref.free([1])
    hga.pages_free(dev, _i32([1]))
    ref.fork([0], [1])
    hga.pages_fork(dev, _i32([0]), _i32([1]))
    _same(hga, ref, dev, "fork")
    assert ref.len.tolist() == [32000, 32000, 0]
