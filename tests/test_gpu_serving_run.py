"""The rotary, page and 4-bit cache calls together, as a program uses them:
prompts, forks, generated tokens, requests that leave, the routed form with
lists that routing made, and a training segment (needs a B200)."""
import numpy as np
import pytest
import torch

import q4_ref
from test_gpu_q4 import _check_row, _f64, _i32, _lib

pytestmark = pytest.mark.gpu


def test_prompts_forks_and_generated_tokens():
    """Two layers, two prompts in one ragged call, three forks, 20 generated
    tokens, requests that leave and a compacted pool; every attention output
    against float64 over what the history should hold."""
    hga = _lib()
    hq, hkv, d, page, planes = 8, 2, 128, 16, 2
    p = hga.Params(hq, hkv, d)
    G = hq // hkv
    pool = hga.PagePool.allocate(planes, 80, hga.q4_page_bytes(p, page), page, 6, 40)
    plan = hga.Rope.make(d, 1e6, sections=(16, 24, 24))
    gen = torch.Generator(device="cuda").manual_seed(11)
    past = {}                                        # row -> per plane [(k, v)] float64, stored

    def step(rows, counts, max_ctx):
        """counts[i] new tokens of rows[i] in every plane: qkv, rope, append, attend."""
        n = sum(counts)
        off = np.concatenate([[0], np.cumsum(counts)])
        b = hga.Q4Batch(_i32(rows), _i32(off), max(counts))
        new = [past[r][0][0].shape[0] + c for r, c in zip(rows, counts)]
        hga.pages_reserve(pool, _i32(rows), _i32(new))
        work = hga.q4_workspace(p, b, n, max_ctx)
        pos = torch.cat([torch.arange(m - c, m) for m, c in zip(new, counts)]).int().cuda()
        pos = torch.stack([pos, pos // 3, pos % 5])
        for plane in range(planes):
            qkv = torch.randn(n, hq + 2 * hkv, d, generator=gen, device="cuda").bfloat16()
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            qr = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
            hga.rope(plan, pos, q, qr, k, k)          # k in place
            hga.q4_append(p, pool, plane, b, k, v)
            o, lse = torch.empty_like(qr), torch.empty(n, hq, device="cuda")
            hga.q4_attend(p, pool, plane, b, qr, o, lse, max_ctx=max_ctx, work=work)
            assert hga.check() == 0
            k64, v64 = q4_ref.stored(_f64(k)), q4_ref.stored(_f64(v))
            q64, o64, l64 = _f64(qr), _f64(o), _f64(lse)
            for i, r in enumerate(rows):
                s = slice(off[i], off[i + 1])
                past[r][plane] = [np.concatenate([x, y[s]]) for x, y in zip(past[r][plane], (k64, v64))]
                kk, vv = past[r][plane]
                at = new[i] - counts[i] + np.arange(counts[i])
                allowed = np.repeat(np.arange(new[i])[None] <= at[:, None], G, 0)
                for h in range(hkv):
                    hs = slice(h * G, (h + 1) * G)
                    _check_row(p, o64[s, hs].reshape(-1, d), l64[s, hs].reshape(-1),
                               q64[s, hs].reshape(-1, d), kk[:, h], vv[:, h], allowed,
                               (plane, r, h), max(counts))

    empty = lambda: [[np.zeros((0, hkv, d))] * 2 for _ in range(planes)]
    past[0], past[1] = empty(), empty()
    step([0, 1], [150, 67], 1 << 16)
    hga.pages_fork(pool, _i32([0, 0, 1]), _i32([2, 3, 4]))
    for child, parent in ((2, 0), (3, 0), (4, 1)):
        past[child] = [list(x) for x in past[parent]]
    for t in range(10):
        step([4, 0, 3, 1, 2], [1] * 5, 200)
    hga.pages_free(pool, _i32([0, 4, -1]))            # the parent of two of them leaves
    del past[0], past[4]
    hga.pages_compact(pool)
    assert hga.check() == 0
    used = int((pool.ref > 0).sum())
    assert torch.all(pool.ref[:used] > 0) and torch.all(pool.ref[used:] == 0)
    for t in range(10):
        step([3, 1, 2], [1, 2, 1], 200)
    hga.pages_free(pool, _i32([1, 2, 3]))
    assert hga.check() == 0 and not pool.ref.any() and torch.all(pool.table == -1)


def test_routed_attention_on_lists_that_routing_made():
    """A context in 4 bits, read back into the buffers that routing and the
    16-bit attention use: both attentions of the same lists agree with float64,
    for a segment and for its last row alone."""
    hga = _lib()
    p = hga.Params(32, 4, 128, sink=64, local=512, top_chunks=16, top_groups=64)
    T, n = 4096 + 37, 485                             # the segment starts at 3648
    q0, t_cap = T - n, 4160
    assert q0 % 64 == 0
    pool = hga.PagePool.allocate(1, 70, hga.q4_page_bytes(p, 64), 64, 1, 66)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(T, 4, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    b = hga.Q4Batch(_i32([0]), _i32([0, T]), T)
    hga.pages_reserve(pool, _i32([0]), _i32([T]))
    hga.q4_append(p, pool, 0, b, k, v)
    kb, vb = (torch.zeros(4, t_cap, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    hga.q4_read(p, pool, 0, b, kb[:, :T].transpose(0, 1), vb[:, :T].transpose(0, 1))
    q = torch.randn(n, 32, 128, generator=g, device="cuda").bfloat16()
    bufs = hga.allocate(p, t_cap, n)
    hga.forward(p, q, q0, kb, vb, bufs)
    o, lse = torch.full_like(bufs.o, 7.0), torch.full_like(bufs.lse, 7.0)
    hga.q4_attend_routed(p, pool, 0, 0, q, q0, t_cap, bufs.group_idx, bufs.group_cnt, o, lse)
    last, ll = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    hga.q4_attend_routed(p, pool, 0, 0, q, q0, t_cap, bufs.group_idx, bufs.group_cnt, last, ll,
                         pos_lo=T - 1)
    assert hga.check() == 0
    assert torch.all(last[:-1] == 7) and torch.all(ll[:-1] == 7)
    k64, v64 = q4_ref.stored(_f64(k)), q4_ref.stored(_f64(v))
    assert np.array_equal(_f64(kb[:, :T].transpose(0, 1)), k64)
    idx, cnt = bufs.group_idx.cpu().numpy(), bufs.group_cnt.cpu().numpy()
    q64, o64, l64 = _f64(q), _f64(o), _f64(lse)
    d64, e64, a64 = _f64(last), _f64(ll), _f64(bufs.o)
    t = np.arange(T)
    for blk in (0, 3, 7):
        b0 = q0 + 64 * blk
        rows = np.arange(64 * blk, min(64 * blk + 64, n))
        for h in (0, 3):
            keep = (t < 64) | ((t >= b0 - 512) & (t < b0 + 64))
            assert cnt[h, blk] > 0
            for j in idx[h, blk, :cnt[h, blk]]:
                keep[8 * j:8 * j + 8] = True
            allowed = np.repeat(keep[None] & (t <= (q0 + rows)[:, None]), 8, 0)
            s = (rows, slice(8 * h, 8 * h + 8))
            x = q64[s].reshape(-1, 128)
            _check_row(p, o64[s].reshape(-1, 128), l64[s].reshape(-1), x, k64[:, h], v64[:, h],
                       allowed, (blk, h), 64)
            ref = q4_ref.attention(x, k64[:, h], v64[:, h], allowed)[0]
            # the 16-bit attention's own bound
            assert np.all(np.abs(a64[s].reshape(-1, 128) - ref) <= 2e-3 + 1e-2 * np.abs(ref))
            if blk == 7:
                y = slice(8 * h, 8 * h + 8)
                _check_row(p, d64[-1, y], e64[-1, y], q64[-1, y], k64[:, h], v64[:, h], allowed[-8:],
                           ("last", h))


def test_training_segment_through_the_rotation():
    """rope -> attend -> attend_backward -> rope_backward: the projections'
    gradients are the rotated ones turned back, straight from the attention's
    fp32 buffers and layouts, and the loss's differences follow them."""
    hga = _lib()
    p = hga.Params(4, 2, 64, sink=64, local=64, top_chunks=0, top_groups=0, dtype="fp32")
    n, t_cap = 192, 192
    g = torch.Generator(device="cuda").manual_seed(4)
    plan = hga.Rope.make(64, 1e4)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q, w = (torch.randn(n, 4, 64, generator=g, device="cuda") for _ in range(2))
    k, v = (torch.randn(n, 2, 64, generator=g, device="cuda") for _ in range(2))
    vb = v.transpose(0, 1).contiguous()

    def forward(q, k):
        qr, kb = torch.empty_like(q), torch.zeros(2, t_cap, 64, device="cuda")
        hga.rope(plan, pos, q, qr, k, kb.transpose(0, 1))
        bufs = hga.allocate(p, t_cap, n)
        hga.forward(p, qr, 0, kb, vb, bufs)
        return qr, kb, bufs

    qr, kb, bufs = forward(q, k)
    d_q, d_k, d_v = torch.empty_like(q), torch.empty_like(kb), torch.empty_like(kb)
    hga.attend_backward(p, qr, 0, kb, vb, bufs.group_idx, bufs.group_cnt, bufs.o, bufs.lse, w, d_q,
                        d_k, d_v)
    g_q, g_k = torch.empty_like(q), torch.empty_like(k)
    hga.rope_backward(plan, pos, d_q, g_q, d_k.transpose(0, 1), g_k)
    assert hga.check() == 0
    freq, axis = plan.freq.cpu().numpy(), plan.axis.cpu().numpy()
    for got, x in ((g_q, d_q), (g_k, d_k.transpose(0, 1))):
        want = q4_ref.rotate(_f64(x), pos.cpu().numpy()[None], freq, axis, False, -1)
        assert np.all(np.abs(_f64(got) - want) <= 6.5e-7 * 2 * np.abs(_f64(x)).max() + 1e-12)
    # differences: float64 attention over all earlier tokens (everything is kept)
    def loss(q, k):
        total = 0.0
        mask = np.tril(np.ones((n, n), bool))
        qr = q4_ref.rotate(q, pos.cpu().numpy()[None], freq, axis, False)
        kr = q4_ref.rotate(k, pos.cpu().numpy()[None], freq, axis, False)
        for h in range(4):
            o = q4_ref.attention(qr[:, h], kr[:, h // 2], _f64(v)[:, h // 2], mask)[0]
            total += (o * _f64(w)[:, h]).sum()
        return total

    rng = np.random.default_rng(5)
    for grad, which in ((g_q, 0), (g_k, 1)):
        u = rng.standard_normal(grad.shape)
        e = 1e-4
        args = [_f64(q), _f64(k)]
        hi, lo = list(args), list(args)
        hi[which], lo[which] = args[which] + e * u, args[which] - e * u
        diff = (loss(*hi) - loss(*lo)) / (2 * e)
        mine = float((_f64(grad) * u).sum())
        # each gradient value is good to about 1e-5 of the largest; the sum of
        # as many products with random signs to their root; e^2 of the third derivative
        tol = 1e-5 * np.abs(_f64(grad)).max() * np.sqrt(u.size) * 4 + 1e-5 * abs(diff)
        assert abs(diff - mine) <= tol, (which, diff, mine, tol)


def test_captured_prompt_replays():
    """A captured append + attend of many query rows (its own workspace) on new
    data, while another stream runs the same call with its own workspace."""
    hga = _lib()
    p = hga.Params(8, 1, 64)
    pool = hga.PagePool.allocate(1, 64, hga.q4_page_bytes(p, 64), 64, 2, 32)
    hga.pages_reserve(pool, _i32([0, 1]), _i32([700, 700]))
    b = [hga.Q4Batch(_i32([i]), _i32([0, 300]), 300) for i in (0, 1)]
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v = (torch.randn(700, 1, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    for i in (0, 1):
        hga.q4_append(p, pool, 0, hga.Q4Batch(_i32([i]), _i32([0, 700]), 700), k, v)
    x = [torch.randn(300, n, 64, generator=g, device="cuda").bfloat16() for n in (8, 1, 1)]
    o = [torch.zeros(300, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bound = 1 << 21                                   # the kernel of long histories
    work = [hga.q4_workspace(p, b[i], 300, bound) for i in (0, 1)]

    def run(i):
        hga.q4_append(p, pool, 0, b[i], x[1], x[2])
        hga.q4_attend(p, pool, 0, b[i], x[0], o[i], max_ctx=bound, work=work[i])

    run(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(0)
    side = torch.cuda.Stream()
    for turn in range(5):
        for t in x:
            t.normal_(generator=g)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            run(1)
        torch.cuda.synchronize()
        assert hga.check() == 0
        assert torch.equal(o[0], o[1])
    k64 = np.concatenate([q4_ref.stored(_f64(k))[:400], q4_ref.stored(_f64(x[1]))])
    v64 = np.concatenate([q4_ref.stored(_f64(v))[:400], q4_ref.stored(_f64(x[2]))])
    allowed = np.repeat(np.arange(700)[None] <= 400 + np.arange(300)[:, None], 8, 0)
    _check_row(p, _f64(o[0]).reshape(-1, 64), None, _f64(x[0]).reshape(-1, 64), k64[:, 0], v64[:, 0],
               allowed, "replay", 300)
