"""hga_rope right before a call with q_ready (needs a B200)."""
import dataclasses

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,n", [(32, 4, 128, 2048), (4, 4, 64, 511), (8, 1, 128, 64)])
def test_a_rotation_before_a_q_ready_call(hq, hkv, d, n):
    """rope -> route_chunks and rope -> attend on queries that change every
    turn: with q_ready they give what they give without, bit for bit."""
    from long_context_hga_b200 import hga
    T = 4096 + n
    t_cap, q0 = -(-T // 64) * 64, 4096
    p = hga.Params(hq, hkv, d, sink=64, local=128, top_chunks=8, top_groups=32)
    ready = dataclasses.replace(p, q_ready=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn(hkv, t_cap, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    plan = hga.Rope.make(d, 1e6)
    pos = torch.arange(q0, T, dtype=torch.int32, device="cuda")
    q = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    lists = hga.allocate(p, t_cap, n)
    hga.commit(p, k, v, 0, T, lists.chunk_sum, lists.group_sum)
    for turn in range(8):
        x = torch.randn(n, hq, d, generator=g, device="cuda").bfloat16()
        got = []
        for pp in (p, ready):
            b = hga.allocate(p, t_cap, n)
            q.fill_(turn)                               # what a read that comes too early sees
            hga.rope(plan, pos, x, q)
            hga.route_chunks(pp, q, q0, lists.chunk_sum, t_cap, b.chunk_idx, b.chunk_cnt)
            hga.route_groups(p, q, q0, lists.group_sum, t_cap, b.chunk_idx, b.chunk_cnt,
                             b.group_idx, b.group_cnt)
            q.fill_(-turn)
            hga.rope(plan, pos, x, q)
            hga.attend(pp, q, q0, k, v, b.group_idx, b.group_cnt, b.o, b.lse)
            got.append(b)
        assert hga.check() == 0
        for name in ("chunk_cnt", "chunk_idx", "group_cnt", "group_idx", "o", "lse"):
            assert torch.equal(getattr(got[0], name), getattr(got[1], name)), (turn, name)
