"""The 4-bit cache (hga_q4_append, hga_q4_read, hga_q4_attend,
hga_q4_attend_routed) against float64 (needs a B200)."""
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


def _f64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A pool whose rows hold the given tokens, and the values it keeps of them."""

    def __init__(self, hga, p, lens, page, planes=1, plane=0, seed=0, spare=3, filled=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.p, self.plane, self.lens = p, plane, list(lens)
        n_rows = len(lens) + 2
        need = sum(-(-x // page) for x in lens)
        row_pages = max(1, max(-(-x // page) for x in lens)) + 1
        self.pool = hga.PagePool.allocate(planes, need + spare, hga.q4_page_bytes(p, page), page,
                                          n_rows, row_pages)
        self.pool.data.fill_(0xff)                  # what no token was stored into is NaN scales
        # pages in a mixed order: every row grows by turns
        for part in (2, 1):
            hga.pages_reserve(self.pool, _i32(np.arange(len(lens))[::part]),
                              _i32([x // part for x in lens][::part]))
        hga.pages_reserve(self.pool, _i32(np.arange(len(lens))), _i32(lens))
        n = sum(lens)
        shape = (n, p.n_kv_heads, p.head_dim)
        self.k = torch.randn(shape, generator=g, device="cuda").to(p.torch_dtype)
        self.v = torch.randn(shape, generator=g, device="cuda").to(p.torch_dtype)
        self.off = np.concatenate([[0], np.cumsum(lens)])
        if filled and n:
            b = hga.Q4Batch(_i32(np.arange(len(lens))), _i32(self.off), max(lens))
            hga.q4_append(p, self.pool, plane, b, self.k, self.v)
            assert hga.check() == 0
        self.k64, self.v64 = q4_ref.stored(_f64(self.k)), q4_ref.stored(_f64(self.v))

    def kv(self, row, h):
        a, b = self.off[row], self.off[row + 1]
        return self.k64[a:b, h], self.v64[a:b, h]


def _check_row(p, got_o, got_lse, q, k, v, allowed, what, max_q=1):
    o, lse, *size = q4_ref.attention(q, k, v, allowed)
    tc = p.dtype == "bf16" and max_q * p.n_q_heads // p.n_kv_heads >= 64
    to, tl = q4_ref.tolerance(p.dtype, o, *size, tc=tc)
    err = np.abs(got_o - o)
    assert np.all(err <= to), (what, float((err / to).max()))
    if got_lse is not None:
        empty = np.isneginf(lse)
        assert np.array_equal(empty, np.isneginf(got_lse)), what
        assert np.all(np.abs(got_lse - lse)[~empty] <= (tl + 2.0 ** -22 * np.abs(lse))[~empty]), what


# ---------------------------------------------------------------- append and read

@pytest.mark.parametrize("d,hkv,page,dtype,lens", [
    (128, 4, 64, "bf16", [1]),
    (128, 2, 8, "bf16", [7, 64, 1, 33]),
    (64, 3, 16, "bf16", [100, 17]),
    (64, 1, 128, "fp32", [129, 5]),
    (128, 5, 32, "fp32", [31, 32, 33, 1000]),
])
def test_stored_values_are_the_formats(d, hkv, page, dtype, lens):
    hga = _lib()
    p = hga.Params(hkv, hkv, d, dtype=dtype)
    c = Cache(hga, p, lens, page, planes=2, plane=1, filled=False)
    # magnitudes over the whole range, zeros, ties and the largest values among them
    g = torch.Generator(device="cuda").manual_seed(5)
    for x in (c.k, c.v):
        x.mul_(10 ** (torch.rand(x.shape[:2], generator=g, device="cuda") * 8 - 4)[..., None])
        x.clamp_(-61440, 61440)
        x[0, 0, :16] = 0
        x[-1, -1, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5] * 2, device="cuda") * 1.625
        x[0, -1, 16:32] = torch.tensor([61440.0, -61440.0] * 8, device="cuda")
        x[-1, 0, 32:48] = 2.0 ** -18
    other = c.pool.data[0].clone()
    b = hga.Q4Batch(_i32(np.arange(len(lens))), _i32(c.off), max(lens))
    hga.q4_append(p, c.pool, 1, b, c.k, c.v)
    ko, vo = torch.empty_like(c.k), torch.empty_like(c.v)
    hga.q4_read(p, c.pool, 1, b, ko, vo)
    assert hga.check() == 0
    assert np.array_equal(_f64(ko), q4_ref.stored(_f64(c.k)))
    assert np.array_equal(_f64(vo), q4_ref.stored(_f64(c.v)))
    assert torch.equal(c.pool.data[0], other)


def test_bytes_are_the_documented_layout():
    """One record read by hand: codes, nibbles and scales where the header says."""
    hga = _lib()
    p = hga.Params(2, 2, 64)
    c = Cache(hga, p, [11], 16)
    rec = c.pool.data[0, int(c.pool.table[0, 0])].cpu().numpy().reshape(2, 2, 576)
    mag = np.concatenate([q4_ref.MAG, -q4_ref.MAG])
    for h in range(2):
        for tok in (0, 7, 8, 10):
            r, t = rec[h, tok // 8], tok % 8
            for at, sc, x in ((0, 512, c.k64), (256, 544, c.v64)):
                code = r[at + 32 * t:at + 32 * t + 32]
                val = mag[np.stack([code & 15, code >> 4], -1).reshape(-1)]
                s = (r[sc + 4 * t:sc + 4 * t + 4].astype(np.uint16) << 7).view(np.float16)
                assert np.array_equal(val * np.repeat(s.astype(np.float64), 16), x[tok, h])
    assert np.all(rec[:, 1, 3 * 32:256] == 0xff)            # tokens that were not stored


def test_append_touches_only_its_tokens():
    """Single tokens into part-filled records, inactive rows, packed rows
    behind the last sequence, strided and unlike k and v."""
    hga = _lib()
    p = hga.Params(4, 2, 128)
    c = Cache(hga, p, [21, 40, 8], 16, seed=3)
    before = c.pool.data.clone()
    new = _i32([22, 41, 9])
    hga.pages_reserve(c.pool, _i32([0, 1, 2]), new)
    fused = torch.randn(5, 12 * 128, device="cuda").bfloat16()
    k = fused[:, 256:512].unflatten(1, (2, 128))
    v = torch.randn(2, 7, 128, device="cuda").bfloat16()[:, 1:6].transpose(0, 1)
    b = hga.Q4Batch(_i32([2, -1, 0]))                       # one token each; row 1 waits
    hga.q4_append(p, c.pool, 0, b, k, v)
    ko, vo = (torch.full((5, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    hga.q4_read(p, c.pool, 0, b, ko, vo)
    assert hga.check() == 0
    for i in (0, 2):
        assert np.array_equal(_f64(ko)[i], q4_ref.stored(_f64(k))[i])
        assert np.array_equal(_f64(vo)[i], q4_ref.stored(_f64(v))[i])
    assert torch.all(ko[[1, 3, 4]] == 9) and torch.all(vo[[1, 3, 4]] == 9)
    changed = (c.pool.data != before).sum().item()
    assert changed <= 2 * 2 * 2 * (64 + 8)                  # two tokens, heads, K and V
    everything = hga.Q4Batch(_i32([0, 1, 2]), _i32([0, 21, 61, 69]), 40)
    hga.pages_reserve(c.pool, _i32([0, 1, 2]), new)         # already there: nothing changes
    ko = torch.zeros(69, 2, 128, dtype=torch.bfloat16, device="cuda")
    vo = torch.zeros_like(ko)
    c.pool.length[:3].copy_(_i32([21, 40, 8]))
    hga.q4_read(p, c.pool, 0, everything, ko, vo)
    assert hga.check() == 0
    assert np.array_equal(_f64(ko), c.k64) and np.array_equal(_f64(vo), c.v64)


def test_values_out_of_range_and_broken_rows_are_reported():
    hga = _lib()
    p = hga.Params(1, 1, 64)
    for bad, kept in ((float("nan"), 0.0), (float("inf"), 61440.0), (-70000.0, -61440.0)):
        c = Cache(hga, p, [9], 8, filled=False)
        c.k[3, 0, 5] = bad
        b = hga.Q4Batch(_i32([0]), _i32([0, 9]), 9)
        hga.q4_append(p, c.pool, 0, b, c.k, c.v)
        assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
        ko, vo = torch.zeros_like(c.k), torch.zeros_like(c.v)
        hga.q4_read(p, c.pool, 0, b, ko, vo)
        assert hga.check() == 0
        want = q4_ref.stored(_f64(c.k))
        assert want[3, 0, 5] == kept
        assert np.array_equal(_f64(ko), want) and np.array_equal(_f64(vo), q4_ref.stored(_f64(c.v)))
    c = Cache(hga, p, [9, 9], 8, filled=False)
    for rows, off in (([0, 0], [0, 9, 18]), ([5, 1], [0, 9, 18]), ([0, 1], [0, 9, 19])):
        # a row named twice, a row outside the table, more tokens than the row has
        k = torch.zeros(19, 1, 64, dtype=torch.bfloat16, device="cuda")
        hga.q4_append(p, c.pool, 0, hga.Q4Batch(_i32(rows), _i32(off), 10), k, k)
        assert hga.check() == hga.HGA_ERR_DEVICE_CHECK, rows
    before = c.pool.data.clone()
    c.pool.table[0, 0] = 1000
    c.pool.table[1, 0] = -1
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    c.pool.length.fill_(1)
    hga.q4_append(p, c.pool, 0, hga.Q4Batch(_i32([0, 1])), k, k)
    assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
    assert torch.equal(before, c.pool.data)


# ---------------------------------------------------------------- dense attention

DENSE = [
    # hq, hkv, d, page, dtype, (context, queries) of each sequence
    (1, 1, 64, 8, "bf16", [(1, 1)]),
    (8, 1, 128, 64, "bf16", [(64, 1), (65, 1), (1, 1), (63, 1)]),
    (32, 4, 128, 64, "bf16", [(1000, 1), (2500, 1)]),
    (2, 1, 64, 16, "fp32", [(700, 1), (9, 1), (513, 1)]),
    (8, 2, 128, 8, "fp32", [(130, 5), (77, 77)]),
    (5, 1, 128, 32, "bf16", [(300, 7), (33, 2)]),
    (16, 1, 64, 64, "bf16", [(129, 1), (600, 3)]),
    (40, 8, 128, 128, "bf16", [(257, 1)]),
    (4, 4, 128, 64, "bf16", [(200, 200), (130, 64), (65, 65), (8, 8)]),
    (8, 2, 64, 64, "bf16", [(333, 190), (1, 1), (700, 33)]),
    (32, 4, 128, 64, "bf16", [(1100, 150)]),
    (6, 2, 128, 24, "bf16", [(515, 100), (300, 299)]),
    (4, 2, 64, 64, "fp32", [(300, 140)]),
    (8, 1, 128, 64, "bf16", [(9000, 1), (20, 1)]),
    (8, 1, 128, 64, "bf16", [(5000, 129)]),
]


@pytest.mark.parametrize("hq,hkv,d,page,dtype,seqs", DENSE)
def test_dense_attention(hq, hkv, d, page, dtype, seqs):
    hga = _lib()
    p = hga.Params(hq, hkv, d, dtype=dtype)
    c = Cache(hga, p, [s[0] for s in seqs], page, seed=hq + d)
    nq = [s[1] for s in seqs]
    off = np.concatenate([[0], np.cumsum(nq)])
    g = torch.Generator(device="cuda").manual_seed(7)
    n = int(off[-1])
    # rows behind the last sequence stay as they are
    q = torch.randn(n + 3, hq, d, generator=g, device="cuda").to(p.torch_dtype)
    b = hga.Q4Batch(_i32(np.arange(len(seqs))), _i32(off), max(nq))
    q64 = _f64(q)
    # a tight bound of the lengths and a loose one: the work is cut, and its
    # kernel chosen, by the bound
    for bound in (max(s[0] for s in seqs), 1 << 21):
        o = torch.full_like(q, 5.0)
        lse = torch.full((n + 3, hq), 5.0, device="cuda")
        hga.q4_attend(p, c.pool, 0, b, q, o, lse, max_ctx=bound)
        assert hga.check() == 0
        assert torch.all(o[n:] == 5) and torch.all(lse[n:] == 5)
        o64, l64 = _f64(o), _f64(lse)
        _check_dense(p, c, seqs, off, q64, o64, l64, max(nq))
        # a repeat is equal bit for bit
        o2, lse2 = torch.full_like(o, 5.0), torch.full_like(lse, 5.0)
        hga.q4_attend(p, c.pool, 0, b, q, o2, lse2, max_ctx=bound)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def _check_dense(p, c, seqs, off, q64, o64, l64, max_q):
    hkv, d, G = p.n_kv_heads, p.head_dim, p.n_q_heads // p.n_kv_heads
    for i, (ctx, m) in enumerate(seqs):
        pos = ctx - m + np.arange(m)
        for h in range(hkv):
            k, v = c.kv(i, h)
            rows = slice(off[i], off[i + 1]), slice(h * G, (h + 1) * G)
            allowed = np.repeat(np.arange(ctx)[None] <= pos[:, None], G, 0)
            _check_row(p, o64[rows].reshape(-1, d), l64[rows].reshape(-1), q64[rows].reshape(-1, d),
                       k, v, allowed, (i, h), max_q)


def test_inactive_rows_one_token_form_and_no_lse():
    hga = _lib()
    p = hga.Params(8, 2, 128)
    c = Cache(hga, p, [100, 300], 64)
    q = torch.randn(4, 8, 128, device="cuda").bfloat16()
    o, lse = torch.full_like(q, 3.0), torch.full((4, 8), 3.0, device="cuda")
    b = hga.Q4Batch(_i32([1, -1, 0, -7]))
    hga.q4_attend(p, c.pool, 0, b, q, o, lse)
    assert hga.check() == 0
    assert torch.all(o[[1, 3]] == 0) and torch.all(lse[[1, 3]] == -float("inf"))
    one = hga.Q4Batch(_i32([1, 0]), _i32([0, 1, 2]), 1)
    o2 = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    hga.q4_attend(p, c.pool, 0, one, q[[0, 2]].contiguous(), o2)
    assert hga.check() == 0
    assert torch.equal(o2, o[[0, 2]])


@pytest.mark.parametrize("nq,bound", [(1, 200), (40, 200), (40, 1 << 21)])
def test_missing_pages_and_short_rows_are_left_out(nq, bound):
    hga = _lib()
    p = hga.Params(4, 1, 64)
    c = Cache(hga, p, [200, 50], 16)
    c.pool.table[0, 2] = -1                          # tokens 32 .. 47
    c.pool.table[0, 5] = 1 << 20                     # tokens 80 .. 95
    q = torch.randn(2 * nq, 4, 64, device="cuda").bfloat16()
    o, lse = torch.zeros_like(q), torch.zeros(2 * nq, 4, device="cuda")
    c.pool.length[1] = nq - 1                        # fewer tokens than queries
    b = hga.Q4Batch(_i32([0, 1]), _i32([0, nq, 2 * nq]), nq)
    hga.q4_attend(p, c.pool, 0, b, q, o, lse, max_ctx=bound)
    assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
    k, v = c.kv(0, 0)
    pos = 200 - nq + np.arange(nq)
    t = np.arange(200)
    allowed = (t <= pos[:, None]) & ~((t >= 32) & (t < 48)) & ~((t >= 80) & (t < 96))
    _check_row(p, _f64(o[:nq]).reshape(-1, 64), _f64(lse[:nq]).reshape(-1),
               _f64(q[:nq]).reshape(-1, 64), k, v, np.repeat(allowed, 4, 0), "holes", nq)
    assert torch.all(o[nq:] == 0) and torch.all(lse[nq:] == -float("inf"))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 300.0, 1e30])
def test_queries_of_any_magnitude(dtype, scale):
    """q is held relative to a power of two of its row: neither tiny nor huge
    queries lose it (huge ones give a one-hot softmax)."""
    hga = _lib()
    p = hga.Params(8, 1, 128, dtype=dtype)
    c = Cache(hga, p, [150], 64)
    for nq, bound in ((1, 150), (100, 150), (100, 1 << 21)):
        q = (torch.randn(nq, 8, 128, device="cuda") * scale).to(p.torch_dtype)
        q[:, 3] = 0                                  # a zero row
        o, lse = torch.zeros_like(q), torch.zeros(nq, 8, device="cuda")
        hga.q4_attend(p, c.pool, 0, hga.Q4Batch(_i32([0]), _i32([0, nq]), nq), q, o, lse,
                      max_ctx=bound)
        assert hga.check() == 0
        k, v = c.kv(0, 0)
        allowed = np.repeat(np.arange(150)[None] <= (150 - nq + np.arange(nq))[:, None], 8, 0)
        q64, o64 = _f64(q).reshape(-1, 128), _f64(o).reshape(-1, 128)
        if scale < 1000:
            _check_row(p, o64, _f64(lse).reshape(-1), q64, k, v, allowed, scale, nq)
            continue
        ref, *_ = q4_ref.attention(q64, k, v, allowed)
        assert np.all(np.abs(o64 - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * 10)


# ---------------------------------------------------------------- routed attention

def _lists(hga, p, q0, n, t_cap, rng, fill):
    """Random ascending lists of legal groups, [-1]-padded, as routing writes them."""
    nb = -(-n // 64)
    cap = hga.index_capacity(p, t_cap, 1)
    idx = np.full((p.n_kv_heads, nb, max(cap, 1)), -1, np.int32)
    cnt = np.zeros((p.n_kv_heads, nb), np.int32)
    for h in range(p.n_kv_heads):
        for b in range(nb):
            lo, hi = p.sink // 8, max(p.sink, q0 + 64 * b - p.local) // 8
            m = min(hi - lo, cap) if fill == "all" else int(rng.integers(0, min(hi - lo, cap) + 1))
            idx[h, b, :m] = np.sort(rng.permutation(np.arange(lo, hi))[:m])
            cnt[h, b] = m
    return idx, cnt


@pytest.mark.parametrize("hq,hkv,d,page,dtype,q0,n,sink,local,top,pos_lo", [
    (8, 2, 128, 64, "bf16", 0, 1, 64, 128, 8, None),
    (8, 2, 128, 64, "bf16", 0, 200, 64, 128, 8, None),
    (32, 4, 128, 64, "bf16", 2048, 130, 64, 512, 64, None),
    (32, 4, 128, 64, "bf16", 2048, 41, 64, 512, 64, 2088),      # a decode step's row
    (8, 1, 64, 16, "bf16", 640, 64, 0, 0, 16, None),
    (5, 1, 128, 8, "bf16", 640, 70, 128, 64, 12, 700),
    (4, 2, 64, 32, "fp32", 320, 100, 64, 64, 8, None),
    (4, 4, 128, 64, "fp32", 320, 3, 64, 64, 8, 322),
    (2, 1, 128, 128, "bf16", 1024, 64, 64, 0, 0, None),         # every group
    (32, 4, 128, 64, "bf16", 4096, 500, 64, 512, 64, None),
    (32, 4, 64, 8, "bf16", 4096, 450, 64, 512, 64, 4170),
    (40, 4, 128, 16, "bf16", 2048, 390, 0, 512, 64, None),      # 10 heads a KV head
])
def test_routed_attention(hq, hkv, d, page, dtype, q0, n, sink, local, top, pos_lo):
    hga = _lib()
    p = hga.Params(hq, hkv, d, sink=sink, local=local, top_chunks=0, top_groups=top, dtype=dtype)
    T = q0 + n
    t_cap = -(-T // 64) * 64
    c = Cache(hga, p, [13, T], page)
    idx, cnt = _lists(hga, p, q0, n, t_cap, np.random.default_rng(q0 + n), "all" if top == 0 else "")
    q = torch.randn(n, hq, d, device="cuda").to(p.torch_dtype)
    o, lse = torch.full_like(q, 5.0), torch.full((n, hq), 5.0, device="cuda")
    hga.q4_attend_routed(p, c.pool, 0, 1, q, q0, t_cap, _i32(idx), _i32(cnt), o, lse, pos_lo=pos_lo)
    assert hga.check() == 0
    first = 0 if pos_lo is None else pos_lo - q0
    assert torch.all(o[:first] == 5) and torch.all(lse[:first] == 5)
    G = hq // hkv
    q64, o64, l64 = _f64(q), _f64(o), _f64(lse)
    t = np.arange(T)
    for b in range(-(-n // 64)):
        b0 = q0 + 64 * b
        rows = np.arange(max(64 * b, first), min(64 * b + 64, n))
        if not len(rows):
            continue
        for h in range(hkv):
            keep = (t < min(sink, b0)) | ((t >= b0 - local) & (t >= 0) & (t < b0 + 64))
            for j in idx[h, b, :cnt[h, b]]:
                keep[8 * j:8 * j + 8] = True
            k, v = c.kv(1, h)
            allowed = np.repeat(keep[None] & (t <= (q0 + rows)[:, None]), G, 0)
            s = (rows, slice(h * G, (h + 1) * G))
            _check_row(p, o64[s].reshape(-1, d), l64[s].reshape(-1), q64[s].reshape(-1, d), k, v,
                       allowed, (b, h), min(n - first, 64))


def test_routed_reports_bad_lists_and_skips_them():
    hga = _lib()
    p = hga.Params(4, 1, 64, sink=64, local=64, top_chunks=0, top_groups=8)
    c = Cache(hga, p, [704], 64)
    q = torch.randn(64, 4, 64, device="cuda").bfloat16()
    good = np.array([[[10, 20, 30, -1, -1, -1, -1, -1]]], np.int32)
    o, o2 = torch.zeros_like(q), torch.zeros_like(q)
    hga.q4_attend_routed(p, c.pool, 0, 0, q, 640, 704, _i32(good), _i32([[3]]), o)
    assert hga.check() == 0
    t = np.arange(704)
    keep = (t < 64) | (t >= 576)
    for j in (10, 20, 30):
        keep[8 * j:8 * j + 8] = True
    allowed = np.repeat(keep[None] & (t <= (640 + np.arange(64))[:, None]), 4, 0)

    def same(x, what):
        # the entry that is skipped keeps its slot, so the groups behind it are
        # summed in another order: equal to the tolerance, not bit for bit
        _check_row(p, _f64(x).reshape(-1, 64), None, _f64(q).reshape(-1, 64), *c.kv(0, 0), allowed, what, 64)

    same(o, "good")
    # outside the candidates (a sink group, the local window, beyond the context, negative)
    for wrong in (3, 75, 1 << 28, -5):
        bad = np.array([[[10, 20, 30, wrong, -1, -1, -1, -1]]], np.int32)
        hga.q4_attend_routed(p, c.pool, 0, 0, q, 640, 704, _i32(bad), _i32([[4]]), o2)
        assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
        same(o2, wrong)
    for count in (-1, 9):
        hga.q4_attend_routed(p, c.pool, 0, 0, q, 640, 704, _i32(good), _i32([[count]]), o2)
        assert hga.check() == hga.HGA_ERR_DEVICE_CHECK


def test_two_streams_and_a_graph():
    """Two calls at once on two streams with their own workspaces, and a
    captured append + attend that replays on new data and longer rows."""
    hga = _lib()
    p = hga.Params(8, 2, 128)
    c = Cache(hga, p, [3000, 2999], 64, spare=8)
    q = torch.randn(2, 2, 8, 128, device="cuda").bfloat16()
    b = [hga.Q4Batch(_i32([i])) for i in (0, 1)]
    want = []
    for i in (0, 1):
        o = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device="cuda")
        hga.q4_attend(p, c.pool, 0, b[i], q[i, :1].contiguous(), o, max_ctx=3000)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(10):
        got = [torch.zeros_like(o) for o in want]
        qs = [q[i, :1].contiguous() for i in (0, 1)]
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            hga.q4_attend(p, c.pool, 0, b[i], qs[i], got[i], max_ctx=3000, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a decode step as a graph: reserve, append, attend
    both = hga.Q4Batch(_i32([0, 1]))
    work = hga.q4_workspace(p, both, 2, 3100)
    new_len, rows = _i32([3001, 3000]), _i32([0, 1])
    k, v = (torch.zeros(2, 2, 128, device="cuda").bfloat16() for _ in range(2))
    x, y = q[:, 0].contiguous(), torch.zeros(2, 8, 128, device="cuda").bfloat16()
    lse = torch.zeros(2, 8, device="cuda")

    def step():
        hga.pages_reserve(c.pool, rows, new_len)
        hga.q4_append(p, c.pool, 0, both, k, v)
        hga.q4_attend(p, c.pool, 0, both, x, y, lse, max_ctx=3100, work=work)
        new_len.add_(1)

    graph = torch.cuda.CUDAGraph()
    two_more = [torch.randn(4, 2, 2, 128, device="cuda").bfloat16() for _ in range(2)]
    k.copy_(two_more[0][0])
    v.copy_(two_more[1][0])
    step()                                                  # eager first
    with torch.cuda.graph(graph):
        step()
    for turn in range(1, 4):
        k.copy_(two_more[0][turn])
        v.copy_(two_more[1][turn])
        x.normal_()
        graph.replay()
        assert hga.check() == 0
        assert c.pool.length[:2].tolist() == [3001 + turn, 3000 + turn]
        for i in (0, 1):
            n = [3000, 2999][i]
            for h in (0, 1):
                kk, vv = c.kv(i, h)
                kk = np.concatenate([kk, q4_ref.stored(_f64(two_more[0][:turn + 1, i, h]))])
                vv = np.concatenate([vv, q4_ref.stored(_f64(two_more[1][:turn + 1, i, h]))])
                _check_row(p, _f64(y[i, 4 * h:4 * h + 4]), _f64(lse[i, 4 * h:4 * h + 4]),
                           _f64(x[i, 4 * h:4 * h + 4]), kk, vv, np.ones((4, n + turn + 1), bool),
                           (turn, i, h))


def test_pages_far_into_a_large_pool():
    """Byte offsets past 2^32: the last pages of a 5 GB pool."""
    hga = _lib()
    p = hga.Params(8, 8, 128)
    page_bytes = hga.q4_page_bytes(p, 64)                   # 73,728
    n_pages = 5 * 2 ** 30 // page_bytes
    pool = hga.PagePool(torch.empty(1, n_pages, page_bytes, dtype=torch.uint8, device="cuda"),
                        _i32([[n_pages - 1, n_pages - 2, n_pages - 3]]), _i32([150]),
                        torch.zeros(n_pages, dtype=torch.int32, device="cuda"), 64)
    b = hga.Q4Batch(_i32([0]), _i32([0, 150]), 150)
    k, v, q = (torch.randn(150, 8, 128, device="cuda").bfloat16() for _ in range(3))
    hga.q4_append(p, pool, 0, b, k, v)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    hga.q4_read(p, pool, 0, b, ko, vo)
    o, lse = torch.zeros_like(q), torch.zeros(150, 8, device="cuda")
    hga.q4_attend(p, pool, 0, b, q, o, lse, max_ctx=1 << 21)
    assert hga.check() == 0
    k64, v64 = q4_ref.stored(_f64(k)), q4_ref.stored(_f64(v))
    assert np.array_equal(_f64(ko), k64) and np.array_equal(_f64(vo), v64)
    allowed = np.tril(np.ones((150, 150), bool))
    for h in (0, 7):
        _check_row(p, _f64(o[:, h]), _f64(lse[:, h]), _f64(q[:, h]), k64[:, h], v64[:, h], allowed, h, 150)
