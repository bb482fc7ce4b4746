"""The 4-bit attentions over batches and sizes that take other turns of the
code than a few sequences do (needs a B200)."""
import numpy as np
import pytest
import torch

import q4_ref
from test_gpu_q4 import Cache, _f64, _i32, _lib, _lists

pytestmark = pytest.mark.gpu


def _on_tcgen05(p, units, rows, max_tok):
    """The rule by which a call takes the kernel of many query rows."""
    return p.dtype == "bf16" and rows >= 64 and units * (-(-rows // 16)) * max_tok > 1 << 19


def _check(p, o, lse, q, k, v, allowed, tc, what):
    ref, rl, *size = q4_ref.attention(q, k, v, allowed)
    to, tl = q4_ref.tolerance(p.dtype, ref, *size, tc=tc)
    err = np.abs(o - ref)
    assert np.all(err <= to), (what, float((err / to).max()))
    assert np.all(np.abs(lse - rl) <= tl + 2.0 ** -22 * np.abs(rl)), what


def _dense(p, c, rows, nq, bound, tc, sample=None, seed=9):
    """One dense call over table rows (negative: inactive); every row, or a
    sample of the sequences, against float64."""
    hga = _lib()
    hq, hkv, d = p.n_q_heads, p.n_kv_heads, p.head_dim
    G = hq // hkv
    off = np.concatenate([[0], np.cumsum(nq)])
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(int(off[-1]), hq, d, generator=g, device="cuda").to(p.torch_dtype)
    o, lse = torch.full_like(q, 5.0), torch.full((len(q), hq), 5.0, device="cuda")
    hga.q4_attend(p, c.pool, 0, hga.Q4Batch(_i32(rows), _i32(off), max(nq)), q, o, lse, max_ctx=bound)
    assert hga.check() == 0
    q64, o64, l64 = _f64(q), _f64(o), _f64(lse)
    for i, r in enumerate(rows):
        s = slice(off[i], off[i + 1])
        if r < 0:
            assert np.all(o64[s] == 0) and np.all(np.isneginf(l64[s])), i
            continue
        if sample is not None and i not in sample:
            assert np.isfinite(o64[s]).all() and np.isfinite(l64[s]).all(), i
            continue
        ctx = c.lens[r]
        pos = ctx - nq[i] + np.arange(nq[i])
        allowed = np.repeat(np.arange(ctx)[None] <= pos[:, None], G, 0)
        for h in range(hkv):
            hs = slice(h * G, (h + 1) * G)
            _check(p, o64[s, hs].reshape(-1, d), l64[s, hs].reshape(-1), q64[s, hs].reshape(-1, d),
                   *c.kv(r, h), allowed, tc, (i, r, h))


@pytest.mark.parametrize("n,hq,hkv,d,dtype", [
    (33, 8, 1, 128, "bf16"),       # slots to spare: the search goes past 32 sequences
    (100, 8, 1, 64, "bf16"),
    (200, 4, 2, 64, "bf16"),
    (40, 32, 8, 128, "bf16"),      # a few more slots than sequences
    (54, 16, 8, 64, "bf16"),       # one more slot than sequences
    (55, 16, 8, 64, "bf16"),       # as many: every sequence has a CTA of its own
    (100, 16, 8, 64, "bf16"),
    (70, 4, 2, 64, "fp32"),
])
def test_generated_tokens_of_many_sequences(n, hq, hkv, d, dtype):
    """Ragged lengths, one of them long, some sequences inactive, rows in a
    mixed order; a tight bound and a loose one."""
    hga = _lib()
    p = hga.Params(hq, hkv, d, dtype=dtype)
    rng = np.random.default_rng(n)
    lens = rng.integers(1, 700, n)
    lens[n // 3], lens[n - 1], lens[0] = 5000, 1, 64
    c = Cache(hga, p, lens.tolist(), 64, seed=n)
    rows = rng.permutation(n)
    rows[[2, n // 2]] = -1
    for bound in (5000, 1 << 20):
        _dense(p, c, rows.tolist(), [1] * n, bound, False)


def test_generated_tokens_beside_short_prompts():
    """Sequences of one to nine tokens, and of none, in one call of 60."""
    hga = _lib()
    p = hga.Params(16, 2, 64)
    rng = np.random.default_rng(60)
    lens = rng.integers(9, 400, 60)
    lens[50] = 3000
    c = Cache(hga, p, lens.tolist(), 16, seed=60)
    nq = rng.integers(0, 10, 60)
    nq[:3] = 9
    _dense(p, c, rng.permutation(60).tolist(), nq.tolist(), 3000, False)


@pytest.mark.parametrize("hq,hkv,d,dtype,lens,nq,low,tc", [
    (8, 2, 128, "bf16", [3000, 77, 1500], [1, 1, 1], 64, False),
    (8, 2, 128, "bf16", [3000, 77, 1500], [1, 1, 1], 0, False),
    (16, 1, 64, "bf16", [2000, 130], [3, 2], 100, False),
    (4, 2, 64, "fp32", [1800, 300], [5, 1], 10, False),
    # tcgen05: split for 1024 tokens, where the sequences have three times that
    (16, 2, 128, "bf16", [3100, 2900, 3000], [300, 129, 260], 1024, True),
])
def test_sequences_longer_than_the_bound(hq, hkv, d, dtype, lens, nq, low, tc):
    """max_ctx decides how the work is cut; results stay right beyond it."""
    hga = _lib()
    p = hga.Params(hq, hkv, d, dtype=dtype)
    assert _on_tcgen05(p, len(lens) * hkv, max(nq) * hq // hkv, low) == tc
    c = Cache(hga, p, lens, 64, seed=low)
    _dense(p, c, list(range(len(lens))), nq, low, tc)


@pytest.mark.parametrize("hq,hkv,d", [(64, 8, 128), (64, 8, 64), (40, 8, 128), (12, 4, 64)])
def test_prompts_that_fill_the_gpu_without_a_split(hq, hkv, d):
    """At least 75 (unit, tile) CTAs: outputs and lse straight from TMEM.  Whole
    and part-filled tiles, one with a single row of 128 left over."""
    hga = _lib()
    p = hga.Params(hq, hkv, d)
    G = hq // hkv
    lens = [900, 700, 650, 40]
    nq = [640, 333, 260 // G * 2 + 1, 40]
    tiles = -(-max(nq) * G // 256)
    assert len(lens) * hkv * tiles >= 75
    assert _on_tcgen05(p, len(lens) * hkv, max(nq) * G, 900)
    c = Cache(hga, p, lens, 64, seed=d)
    _dense(p, c, [2, 0, 3, 1], [nq[2], nq[0], nq[3], nq[1]], 900, True)


@pytest.mark.parametrize("hq,hkv,d", [(64, 8, 64), (64, 8, 128)])
def test_routed_blocks_without_a_split(hq, hkv, d):
    hga = _lib()
    p = hga.Params(hq, hkv, d, sink=64, local=512, top_chunks=0, top_groups=64)
    q0, n = 2048, 330
    T, t_cap, G = q0 + n, 2432, hq // hkv
    assert 6 * hkv * 2 >= 75 and _on_tcgen05(p, 6 * hkv, 64 * G, 64 + 512 + 64 * 8 + 64)
    c = Cache(hga, p, [T], 64, seed=d)
    idx, cnt = _lists(hga, p, q0, n, t_cap, np.random.default_rng(d), "")
    q = torch.randn(n, hq, d, device="cuda").bfloat16()
    o, lse = torch.full_like(q, 5.0), torch.full((n, hq), 5.0, device="cuda")
    hga.q4_attend_routed(p, c.pool, 0, 0, q, q0, t_cap, _i32(idx), _i32(cnt), o, lse)
    assert hga.check() == 0
    q64, o64, l64, t = _f64(q), _f64(o), _f64(lse), np.arange(T)
    for b in range(6):
        b0 = q0 + 64 * b
        rows = np.arange(64 * b, min(64 * b + 64, n))
        for h in (0, 3, 7):
            keep = (t < 64) | ((t >= b0 - 512) & (t < b0 + 64))
            for j in idx[h, b, :cnt[h, b]]:
                keep[8 * j:8 * j + 8] = True
            allowed = np.repeat(keep[None] & (t <= (q0 + rows)[:, None]), G, 0)
            s = (rows, slice(h * G, (h + 1) * G))
            _check(p, o64[s].reshape(-1, d), l64[s].reshape(-1), q64[s].reshape(-1, d), *c.kv(0, h),
                   allowed, True, (b, h))


def test_what_the_two_kernels_say_of_one_call():
    """64 rows a unit or more do not always go to tcgen05: the other kernel's
    result is within its own, narrower bound."""
    hga = _lib()
    p = hga.Params(32, 4, 128)
    c = Cache(hga, p, [1024] * 3, 64, seed=5)
    assert not _on_tcgen05(p, 12, 128, 1024) and _on_tcgen05(p, 12, 128, 1 << 16)
    for bound in (1024, 1 << 16):
        _dense(p, c, [0, 1, 2], [16, 15, 16], bound, bound > 1024)
