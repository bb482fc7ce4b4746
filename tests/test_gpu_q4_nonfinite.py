"""Queries that are not finite in the 4-bit attentions: NaN in their own output
rows, a report, and nothing in any other row (needs a B200)."""
import numpy as np
import pytest
import torch

import q4_ref
from test_gpu_q4 import Cache, _f64, _i32, _lib

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

CASES = [
    # hq, hkv, d, dtype, context, queries, bound, on tcgen05
    (8, 2, 128, "bf16", 100, 1, 100, False),                # one CTA a sequence
    (8, 2, 128, "bf16", 3000, 1, 3000, False),              # split and joined
    (16, 4, 64, "bf16", 700, 5, 700, False),                # tiles of 16 rows
    (4, 2, 128, "fp32", 100, 1, 100, False),
    (4, 2, 64, "fp32", 2000, 9, 2000, False),
    (64, 8, 128, "bf16", 400, 320, 500, True),              # 80 CTAs: not split
    (64, 8, 64, "bf16", 400, 320, 500, True),
    (8, 1, 128, "bf16", 300, 100, 1 << 21, True),           # split and joined
]


def _cache(hga, p, ctx, seed):
    """A row of ctx tokens whose K is negative in dim 3 of every head."""
    c = Cache(hga, p, [ctx], 64, seed=seed, filled=False)
    c.k[..., 3] = -(c.k[..., 3].abs() + 1)
    hga.q4_append(p, c.pool, 0, hga.Q4Batch(_i32([0]), _i32([0, ctx]), ctx), c.k, c.v)
    assert hga.check() == 0
    c.k64, c.v64 = q4_ref.stored(_f64(c.k)), q4_ref.stored(_f64(c.v))
    assert np.all(c.k64[..., 3] < 0)
    return c


@pytest.mark.parametrize("hq,hkv,d,dtype,ctx,nq,bound,tc", CASES)
def test_queries_that_are_not_finite(hq, hkv, d, dtype, ctx, nq, bound, tc):
    hga = _lib()
    p = hga.Params(hq, hkv, d, dtype=dtype)
    G = hq // hkv
    c = _cache(hga, p, ctx, hq + d)
    b = hga.Q4Batch(_i32([0]), _i32([0, nq]), nq)
    g = torch.Generator(device="cuda").manual_seed(3)
    for j, value in ((5, NAN), (5, INF), (5, -INF), (3, INF), (3, -INF)):   # dim 3: all scores one sign
        q = torch.randn(nq, hq, d, generator=g, device="cuda").to(p.torch_dtype)
        bad = np.zeros((nq, hq), bool)
        bad[nq // 2, 1] = bad[nq - 1, hq - 1] = True
        q[torch.from_numpy(bad).cuda()] = q[torch.from_numpy(bad).cuda()].index_fill(
            1, torch.tensor([j], device="cuda"), value)
        o, lse = torch.zeros_like(q), torch.zeros(nq, hq, device="cuda")
        hga.q4_attend(p, c.pool, 0, b, q, o, lse, max_ctx=bound)
        assert hga.check() == hga.HGA_ERR_DEVICE_CHECK, (j, value)
        o64, l64, q64 = _f64(o), _f64(lse), _f64(q)
        assert np.isnan(o64[bad]).all() and np.isnan(l64[bad]).all(), (j, value)
        pos = ctx - nq + np.arange(nq)
        for h in range(hkv):
            hs = slice(h * G, (h + 1) * G)
            good = ~bad[:, hs].reshape(-1)
            allowed = np.repeat(np.arange(ctx)[None] <= pos[:, None], G, 0)[good]
            ref, rl, *size = q4_ref.attention(q64[:, hs].reshape(-1, d)[good], *c.kv(0, h), allowed)
            to, tl = q4_ref.tolerance(dtype, ref, *size, tc=tc)
            assert np.all(np.abs(o64[:, hs].reshape(-1, d)[good] - ref) <= to), (j, value, h)
            assert np.all(np.abs(l64[:, hs].reshape(-1)[good] - rl) <= tl + 2.0 ** -22 * np.abs(rl))


@pytest.mark.parametrize("hq,hkv,d,dtype,ctx,nq,bound,tc", CASES)
def test_a_query_that_attends_nothing_stays_zero(hq, hkv, d, dtype, ctx, nq, bound, tc):
    """Inactive sequences, and rows whose tokens' pages are all missing, give 0
    and -inf whatever their queries hold; the inactive ones without a report."""
    hga = _lib()
    p = hga.Params(hq, hkv, d, dtype=dtype)
    c = _cache(hga, p, ctx, 1)
    q = torch.full((nq, hq, d), NAN, device="cuda").to(p.torch_dtype)
    for row, status in ((-1, 0), (0, hga.HGA_ERR_DEVICE_CHECK)):
        if row == 0:
            c.pool.table.fill_(-1)
        o, lse = torch.ones_like(q), torch.ones(nq, hq, device="cuda")
        hga.q4_attend(p, c.pool, 0, hga.Q4Batch(_i32([row]), _i32([0, nq]), nq), q, o, lse,
                      max_ctx=bound)
        assert hga.check() == status
        assert torch.all(o == 0) and torch.all(lse == -INF)


@pytest.mark.parametrize("nq", [3, 130])
def test_rows_that_attend_one_or_a_few_tokens(nq):
    """The first rows attend one to eight tokens of a single record (the one
    before has no page): NaN all the same."""
    hga = _lib()
    p = hga.Params(8, 1, 128)
    c = Cache(hga, p, [16 + nq], 8, seed=2)
    c.pool.table[0, 0] = -1                                  # tokens 0 .. 7
    q = torch.full((nq, 8, 128), NAN, device="cuda").bfloat16()
    o, lse = torch.zeros_like(q), torch.zeros(nq, 8, device="cuda")
    c.pool.length[0] = 8 + nq                                # queries stand at 8 ..
    hga.q4_attend(p, c.pool, 0, hga.Q4Batch(_i32([0]), _i32([0, nq]), nq), q, o, lse, max_ctx=1 << 21)
    assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
    assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("n,pos_lo", [(1, None), (200, None), (200, 1024 + 199)])
def test_routed_queries_that_are_not_finite(n, pos_lo):
    hga = _lib()
    p = hga.Params(32, 4, 128, sink=64, local=128, top_chunks=0, top_groups=16)
    q0, t_cap = 1024, 1024 + -(-n // 64) * 64
    c = _cache(hga, p, q0 + n, 4)
    nb, cap = -(-n // 64), hga.index_capacity(p, t_cap, 1)
    idx = np.full((4, nb, cap), -1, np.int32)
    idx[..., :4] = [9, 30, 31, 70]
    cnt = np.full((4, nb), 4, np.int32)
    for value in (NAN, INF):
        q = torch.randn(n, 32, 128, device="cuda").bfloat16()
        q[n - 1, 7, 3] = value
        o, lse = torch.zeros_like(q), torch.zeros(n, 32, device="cuda")
        hga.q4_attend_routed(p, c.pool, 0, 0, q, q0, t_cap, _i32(idx), _i32(cnt), o, lse, pos_lo=pos_lo)
        assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
        assert torch.isnan(o[n - 1, 7]).all() and torch.isnan(lse[n - 1, 7])
        o[n - 1, 7], lse[n - 1, 7] = 0, 0
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype,nq,bound", [("bf16", 1, 200), ("fp32", 1, 200), ("bf16", 100, 200),
                                            ("bf16", 100, 1 << 21)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_beyond_the_range_of_fp32_are_reported(dtype, nq, bound, sign):
    hga = _lib()
    p = hga.Params(8, 1, 128, dtype=dtype)
    c = _cache(hga, p, 200, 6)
    q = torch.zeros(nq, 8, 128, device="cuda").to(p.torch_dtype)
    q[..., 3] = sign * 3.3e38
    c.k.fill_(600.0)
    hga.q4_append(p, c.pool, 0, hga.Q4Batch(_i32([0]), _i32([0, 200]), 200), c.k, c.v)
    o = torch.zeros_like(q)
    hga.q4_attend(p, c.pool, 0, hga.Q4Batch(_i32([0]), _i32([0, nq]), nq), q, o, max_ctx=bound)
    assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
