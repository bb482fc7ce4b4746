"""hga_rope with one position for all axes (needs a B200)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 2, 37, 2500])
@pytest.mark.parametrize("fn", ["rope", "rope_backward"])
def test_a_position_that_all_axes_share(n, fn):
    """A text token stands at one position on every axis: pos.expand(axes, n),
    without a copy, gives what the copy gives."""
    from long_context_hga_b200 import hga
    g = torch.Generator(device="cuda").manual_seed(n)
    plan = hga.Rope.make(128, 1e6, sections=(16, 24, 24))
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(n, 4, 128, generator=g, device="cuda").bfloat16()
    k = torch.randn(n, 2, 128, generator=g, device="cuda").bfloat16()
    got = []
    for p in (pos.expand(3, n), pos.expand(3, n).contiguous()):
        qo, ko = torch.zeros_like(q), torch.zeros_like(k)
        getattr(hga, fn)(plan, p, q, qo, k, ko)
        assert hga.check() == 0
        got.append((qo, ko))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert not torch.equal(got[0][0], q)
