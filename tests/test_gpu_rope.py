"""Rotary positions (hga_rope, hga_rope_backward) against float64 (needs a B200)."""
import numpy as np
import pytest
import torch

import q4_ref

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def _lib():
    from long_context_hga_b200 import hga
    return hga


def _check(got, ref, mag, what=""):
    """fp32 arithmetic: the angle's fraction of a turn is rounded to fp32
    (pi 2^-24), sine and cosine are good to 2 ulp (2^-23), two products and a
    sum (3 * 2^-24): together under 6.5e-7 of |x| + |y|; one rounding to the
    output's type."""
    eps = torch.finfo(got.dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = 6.5e-7 * mag * (1 + eps) + eps * np.abs(ref) + 1e-30
    assert np.all(err <= tol), (what, float((err / tol).max()))


def _mag(x, half, adjacent):
    m = np.abs(x)
    out = np.zeros_like(m)
    a = slice(0, 2 * half, 2) if adjacent else slice(0, half)
    b = slice(1, 2 * half, 2) if adjacent else slice(half, 2 * half)
    out[..., a] = out[..., b] = m[..., a] + m[..., b]
    return out


@pytest.mark.parametrize("n,hq,hkv,d,rot,axes,adjacent,tin,tout,fn", [
    (1, 1, 1, 128, 128, 1, False, BF16, BF16, "rope"),
    (7, 32, 4, 128, 128, 3, False, BF16, BF16, "rope"),
    (130, 5, 3, 64, 64, 2, True, BF16, FP32, "rope"),
    (1300, 8, 2, 128, 128, 3, False, FP32, FP32, "rope_backward"),
    (33, 4, 1, 128, 64, 1, False, FP32, BF16, "rope_backward"),
    (33, 4, 1, 80, 80, 3, False, BF16, BF16, "rope"),          # 40 pairs
    (9, 3, 2, 72, 36, 2, True, FP32, FP32, "rope"),            # 18 pairs: no vectors
    (5, 2, 1, 33, 32, 1, False, BF16, BF16, "rope_backward"),  # an odd head
    (4, 2, 1, 128, 0, 1, False, BF16, BF16, "rope"),           # nothing turns
    (6, 2, 2, 256, 256, 4, False, BF16, BF16, "rope"),
])
def test_against_float64(n, hq, hkv, d, rot, axes, adjacent, tin, tout, fn):
    hga = _lib()
    g = torch.Generator().manual_seed(n * 1000 + d)
    half = rot // 2
    freq = 1e6 ** (-torch.arange(half, dtype=torch.float64) * 2 / max(rot, 1))
    axis = torch.randint(0, axes, (half,), generator=g, dtype=torch.uint8)
    pos = torch.randint(-1000, 1 << 20, (axes, n), generator=g, dtype=torch.int32)
    pos[:, 0] = torch.tensor([0, 2 ** 31 - 1, -2 ** 31, 1])[:axes]
    q = torch.randn(n, hq, d, generator=g).to(tin)
    k = torch.randn(n, hkv, d, generator=g).to(tin)
    plan = hga.Rope(freq.cuda(), axis.cuda(), d, n_axes=axes, adjacent=adjacent)
    qo = torch.full((n, hq, d), float("nan"), dtype=tout, device="cuda")
    ko = torch.full((n, hkv, d), float("nan"), dtype=tout, device="cuda")
    getattr(hga, fn)(plan, pos.cuda(), q.cuda(), qo, k.cuda(), ko)
    assert hga.check() == 0
    sign = 1 if fn == "rope" else -1
    for x, got in ((q, qo), (k, ko)):
        x64 = x.double().numpy()
        ref = q4_ref.rotate(x64, pos.numpy(), freq.numpy(), axis.numpy(), adjacent, sign)
        _check(got, ref, _mag(x64, half, adjacent), fn)


@pytest.mark.parametrize("unaligned", [False, True])
def test_strides_in_place_and_cache_layout(unaligned):
    """q and k from the rows of a fused projection, k into a cache's tokens
    [Hkv, t_cap, d], q in place; everything around stays as it was."""
    hga = _lib()
    n, hq, hkv, d, t_cap, t0 = 21, 6, 2, 64, 50, 13
    g = torch.Generator(device="cuda").manual_seed(1)
    pad = 1 if unaligned else 8
    rows = torch.randn(n, (hq + 2 * hkv) * d + pad, generator=g, device="cuda").to(BF16)
    q = rows[:, :hq * d].unflatten(1, (hq, d))
    k = rows[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    before = rows.clone()
    cache = torch.full((hkv, t_cap, d), 7.0, dtype=BF16, device="cuda")
    plan = hga.Rope.make(d, 1e4)
    pos = torch.arange(t0, t0 + n, dtype=torch.int32, device="cuda")
    hga.rope(plan, pos, q, q, k, cache[:, t0:t0 + n].transpose(0, 1))
    assert hga.check() == 0
    b = before.double().cpu().numpy()
    freq, axis = plan.freq.cpu().numpy(), plan.axis.cpu().numpy()
    p = pos.cpu().numpy()[None]
    x = b[:, :hq * d].reshape(n, hq, d)
    _check(q, q4_ref.rotate(x, p, freq, axis, False), _mag(x, d // 2, False), "q")
    x = b[:, hq * d:(hq + hkv) * d].reshape(n, hkv, d)
    _check(cache[:, t0:t0 + n].transpose(0, 1), q4_ref.rotate(x, p, freq, axis, False),
           _mag(x, d // 2, False), "k")
    assert torch.equal(rows[:, hq * d:], before[:, hq * d:])
    assert torch.all(cache[:, :t0] == 7) and torch.all(cache[:, t0 + n:] == 7)


def test_backward_is_the_adjoint_and_the_difference_quotient():
    """<rope(x), g> = <x, rope_backward(g)>, and the loss's difference along a
    direction equals the gradient's product with it (the rotation is linear, so
    a difference of any length is the derivative)."""
    hga = _lib()
    n, h, d = 50, 3, 128
    gen = torch.Generator(device="cuda").manual_seed(2)
    plan = hga.Rope.make(d, 1e6, sections=(16, 24, 24))
    pos = torch.randint(0, 100000, (3, n), generator=gen, device="cuda", dtype=torch.int32)
    x, g, u = (torch.randn(n, h, d, generator=gen, device="cuda") for _ in range(3))
    y, y2, gx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    hga.rope(plan, pos, x, y)
    hga.rope(plan, pos, x + u, y2)
    hga.rope_backward(plan, pos, g, gx)
    assert hga.check() == 0
    # each value is good to 6.5e-7 of its pair's magnitude (see _check), the
    # sum of n h d products with random signs keeps at most that of sum |.||.|
    size = float((x.abs().double() * g.abs().double()).sum()) * 2
    assert abs(float((y.double() * g).sum() - (x.double() * gx).sum())) <= 2 * 6.5e-7 * 2 * size
    diff = float(((y2.double() - y.double()) * g).sum())
    size = float(((x.abs() + u.abs()).double() * 2 * g.abs().double()).sum()) * 2
    assert abs(diff - float((u.double() * gx).sum())) <= 4 * 6.5e-7 * 2 * size
    back = torch.empty_like(x)
    hga.rope_backward(plan, pos, y, back)
    assert float((back - x).abs().max()) <= 2 * 6.5e-7 * 2 * float(x.abs().max()) * 2


def test_axis_out_of_range_is_reported():
    hga = _lib()
    plan = hga.Rope.make(64, 1e4, sections=(16, 16))
    plan._c.n_axes = 1
    q = torch.randn(3, 1, 64, device="cuda")
    hga.rope(plan, torch.zeros(2, 3, dtype=torch.int32, device="cuda"), q, torch.empty_like(q))
    assert hga.check() == hga.HGA_ERR_DEVICE_CHECK
    assert hga.check() == 0
