"""Refusals of the rotary, page and 4-bit cache calls (no GPU): every bad
argument is found on the host, before anything is launched, and the structs'
mirrors match the header."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x100000                      # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def hga():
    from long_context_hga_b200 import build
    build.build()
    from long_context_hga_b200 import hga as mod
    return mod


STRUCTS = {"hga_rope_plan": "CRopePlan", "hga_rope_io": "CRopeIo", "hga_page_pool": "CPagePool",
           "hga_q4_batch": "CQ4Batch"}


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_struct_mirrors_match_the_header(hga, tmp_path):
    lines = ['#include "hga.h"', "#include <stdio.h>", "int main(void) {"]
    for cname, pyname in STRUCTS.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        for field, _ in getattr(hga, pyname)._fields_:
            lines.append(f'  printf("{cname} {field} %zu\\n", offsetof({cname}, {field.rstrip("_")}));')
    lines += ["  return 0;", "}"]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines) + "\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout
    for line in out.splitlines():
        cname, key, value = line.split()
        cls = getattr(hga, STRUCTS[cname])
        assert int(value) == (ctypes.sizeof(cls) if key == "size" else getattr(cls, key).offset), line


def _plan(hga, **kw):
    f = dict(freq=FAKE, axis=FAKE, n_axes=1, head_dim=128, rot_dim=128, adjacent=0)
    f.update(kw)
    return hga.CRopePlan(*f.values())


def _io(hga, **kw):
    f = dict(in_=FAKE, out=FAKE, its=128, ihs=128, ots=128, ohs=128, heads=1, idt=0, odt=0)
    f.update(kw)
    return hga.CRopeIo(*f.values())


def test_rope_refuses(hga):
    L, B, n0 = hga.LIB, ctypes.byref, hga.launch_count()

    def call(plan=None, q=None, k=None, pos=FAKE, stride=8, n=8, fn=L.hga_rope):
        return fn(B(plan or _plan(hga)), pos, stride, n, B(q or _io(hga)), None if k is None else B(k), None)

    for fn in (L.hga_rope, L.hga_rope_backward):
        assert fn(None, FAKE, 8, 8, B(_io(hga)), None, None) == 1
        assert fn(B(_plan(hga)), FAKE, 8, 8, None, None, None) == 1
        assert call(fn=fn, n=0, pos=None) == 0
        for bad in (dict(n_axes=0), dict(head_dim=0), dict(rot_dim=127), dict(rot_dim=130),
                    dict(rot_dim=-2), dict(adjacent=2), dict(freq=None), dict(axis=None)):
            assert call(plan=_plan(hga, **bad), fn=fn) == 1, bad
        assert call(plan=_plan(hga, head_dim=258), fn=fn) == 2
        for bad in (dict(in_=None), dict(out=None), dict(in_=FAKE + 1), dict(out=FAKE + 1),
                    dict(heads=0), dict(idt=2), dict(odt=-1)):
            assert call(q=_io(hga, **bad), fn=fn) == 1, bad
            assert call(k=_io(hga, **bad), fn=fn) == 1, bad
        assert call(k=_io(hga, idt=1), fn=fn) == 1          # q and k of two types
        assert call(k=_io(hga, odt=1), fn=fn) == 1
        assert call(n=-1, fn=fn) == 1
        assert call(stride=7, fn=fn) == 1
        assert call(pos=None, fn=fn) == 1
    assert hga.launch_count() == n0


def _pool(hga, **kw):
    f = dict(data=FAKE, page_bytes=2 * 8 * 1152, plane_stride=16 * 2 * 8 * 1152, n_pages=16,
             n_planes=2, page_tokens=64, n_rows=4, row_pages=8, table=FAKE, len=FAKE, ref=FAKE,
             work=FAKE)
    f.update(kw)
    return hga.CPagePool(*f.values())


BAD_POOLS = (dict(page_bytes=8), dict(page_bytes=2 * 8 * 1152 + 8), dict(plane_stride=16),
             dict(plane_stride=16 * 2 * 8 * 1152 + 8), dict(n_pages=0), dict(n_planes=0),
             dict(page_tokens=0), dict(page_tokens=12), dict(n_rows=0), dict(row_pages=0),
             dict(table=None), dict(len=None), dict(ref=None), dict(data=FAKE + 8))


def test_pages_refuse(hga):
    L, B, n0 = hga.LIB, ctypes.byref, hga.launch_count()
    calls = {
        "reserve": lambda p, n, x=FAKE: L.hga_pages_reserve(p, x, FAKE, n, None),
        "fork": lambda p, n, x=FAKE: L.hga_pages_fork(p, x, FAKE, n, None),
        "free": lambda p, n, x=FAKE: L.hga_pages_free(p, x, n, None),
        "copy": lambda p, n, x=FAKE: L.hga_pages_copy(p, x, FAKE, n, None),
    }
    for name, call in calls.items():
        assert call(None, 1) == 1
        for bad in BAD_POOLS + (dict(work=None),):
            assert call(B(_pool(hga, **bad)), 1) == 1, (name, bad)
        ok = B(_pool(hga))
        assert call(ok, 0) == 0 and call(ok, 0, None) == 0
        assert call(ok, -1) == 1
        assert call(ok, 1, None) == 1
        assert call(ok, 17 if name == "copy" else 5) == 1   # longer than the pool allows
        for big in (dict(row_pages=1 << 30, page_tokens=64), dict(row_pages=1, page_tokens=(1 << 31) - 4088),
                    dict(n_rows=1 << 20, row_pages=1 << 11, page_tokens=8),
                    dict(n_pages=(1 << 30) + 1, plane_stride=1 << 62)):
            assert call(B(_pool(hga, **big)), 1) == 2, (name, big)
    assert L.hga_pages_copy(B(_pool(hga, data=None)), FAKE, FAKE, 1, None) == 1
    assert L.hga_pages_compact(None, None) == 1
    for bad in BAD_POOLS + (dict(work=None),):
        assert L.hga_pages_compact(B(_pool(hga, **bad)), None) == 1, bad
    assert L.hga_pages_work_ints(None) == -1
    assert L.hga_pages_work_ints(B(_pool(hga, n_pages=0))) == -1
    assert L.hga_pages_work_ints(B(_pool(hga))) >= 3 * 16 + 3 * 4
    assert hga.launch_count() == n0


def test_q4_refuses(hga):
    L, B, n0 = hga.LIB, ctypes.byref, hga.launch_count()
    P = hga.Params
    ok = P(8, 2, 128).c()
    batch = lambda **kw: hga.CQ4Batch(*{**dict(rows=FAKE, off=FAKE, n_seq=2, max_q=4), **kw}.values())

    def io(fn, p=ok, pool=None, plane=0, b=None, n=8, k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128):
        return fn(B(p) if p else None, B(pool or _pool(hga)), plane, B(b or batch()), n, k, kt, kh, v,
                  vt, vh, None)

    def att(p=ok, pool=None, plane=0, b=None, n=8, q=FAKE, ctx=512, o=FAKE, work=FAKE,
            size=1 << 40):
        return L.hga_q4_attend(B(p) if p else None, B(pool or _pool(hga)), plane, B(b or batch()), n,
                               q, ctx, o, None, work, size, None)

    def routed(p=ok, pool=None, plane=0, row=0, q=FAKE, q0=64, n=64, lo=64, cap=512, gi=FAKE, o=FAKE,
               work=FAKE, size=1 << 40):
        return L.hga_q4_attend_routed(B(p) if p else None, B(pool or _pool(hga)), plane, row, q, q0, n,
                                      lo, cap, gi, FAKE, o, None, work, size, None)

    every = [lambda **kw: io(L.hga_q4_append, **kw), lambda **kw: io(L.hga_q4_read, **kw), att, routed]
    for call in every:
        assert call(p=None) == 1
        assert call(p=P(8, 3, 128).c()) == 1
        assert call(p=P(8, 2, 96).c()) == 2
        assert call(p=P(8, 4, 128).c()) == 1                 # the pages are of 2 KV heads
        assert call(p=P(8, 2, 64).c()) == 1
        assert call(plane=2) == 1 and call(plane=-1) == 1
        for bad in BAD_POOLS + (dict(data=None),):
            assert call(pool=_pool(hga, **bad)) == 1, bad
    for call in every[:3]:
        assert call(n=0) == 0
        assert call(n=-1) == 1
        assert call(b=batch(n_seq=0)) == 0
        assert call(b=batch(n_seq=-1)) == 1
        assert call(b=batch(max_q=-1)) == 1
        assert call(b=batch(rows=None)) == 1
        assert call(b=batch(off=None)) == 1                  # several tokens need off
        assert call(b=batch(off=None, max_q=1), n=1) == 1    # fewer rows than sequences
    for call in every[:2]:
        for bad in (dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 8), dict(kt=257),
                    dict(kh=4), dict(vt=260), dict(vh=7)):
            assert call(**bad) == 1, bad
    for bad in (dict(q=None), dict(o=None), dict(q=FAKE + 8), dict(o=FAKE + 8), dict(ctx=-1)):
        assert att(**bad) == 1, bad
    # a long context is split: the workspace has to be there
    assert att(ctx=1 << 20, work=None) == 1
    assert att(ctx=1 << 20, work=FAKE + 8) == 1
    assert att(ctx=1 << 20, size=16) == 1
    assert att(b=batch(n_seq=65536)) == 2
    for bad in (dict(row=-1), dict(row=4), dict(q0=32), dict(n=512), dict(lo=63), dict(q=None),
                dict(o=None), dict(gi=None), dict(q=FAKE + 8),
                dict(n=-1), dict(cap=64 * 8 * 9, q0=64 * 8, n=64, lo=64 * 8)):
        assert routed(**bad) == 1, bad
    wide = P(8, 2, 128, top_chunks=0, top_groups=200).c()                  # enough tokens to be split
    for bad in (dict(work=None), dict(work=FAKE + 8), dict(size=16)):
        assert routed(p=wide, q0=2048, lo=2048, cap=4096, pool=_pool(hga, row_pages=64), **bad) == 1
    assert routed(lo=128) == 0                               # no row is asked for
    assert L.hga_q4_page_bytes(B(ok), 64) == 2 * 8 * 1152
    assert L.hga_q4_page_bytes(B(P(8, 2, 64).c()), 8) == 2 * 576
    assert L.hga_q4_page_bytes(B(ok), 60) == -1 and L.hga_q4_page_bytes(None, 64) == -1
    assert L.hga_q4_attend_work(B(ok), 2, 1, 2, 1 << 20) > 0
    assert L.hga_q4_attend_work(B(ok), 2, 1, 2, 64) == 0
    assert L.hga_q4_attend_work(B(ok), -1, 1, 2, 64) == -1
    assert L.hga_q4_attend_work(None, 1, 1, 2, 64) == -1
    assert L.hga_q4_attend_routed_work(None, 1) == -1
    assert hga.launch_count() == n0


def test_binding_refuses_what_it_cannot_pass_on(hga):
    import torch
    i32 = torch.int32
    with pytest.raises(hga.HgaError):
        hga.Rope(torch.zeros(64), torch.zeros(64, dtype=torch.uint8), 128)       # not float64
    with pytest.raises(hga.HgaError):
        hga.Rope.make(128, 1e6, sections=(16, 24, 23), device="cpu")
    plan = hga.Rope.make(128, 1e6, sections=(16, 24, 24), device="cpu")
    assert plan.axis.tolist() == [0] * 16 + [1] * 24 + [2] * 24 and plan.n_axes == 3
    turn = hga.Rope.make(16, 1e4, sections=(2, 3, 3), interleaved=True, device="cpu")
    assert turn.axis.tolist() == [0, 1, 2, 0, 1, 2, 1, 2]
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    pos = torch.zeros(3, 4, dtype=i32)
    with pytest.raises(hga.HgaError):                                             # not on a GPU
        hga.rope(plan, pos, q, q)
    for bad in (pos[:2], pos[:, :3], pos.long()):
        with pytest.raises(hga.HgaError):
            hga.rope(plan, bad, q, q)
    data = torch.zeros(1, 4, 1152 * 8, dtype=torch.uint8)
    table, length, ref = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(4, dtype=i32)
    pool = hga.PagePool(data, table, length, ref, 64)
    for args in ((data.float(), table, length, ref), (data, table.long(), length, ref),
                 (data, table, length[:1], ref), (data, table, length, ref[:3]), (data[0], table, length, ref)):
        with pytest.raises(hga.HgaError):
            hga.PagePool(*args, 64)
    with pytest.raises(hga.HgaError):
        hga.pages_free(pool, torch.zeros(2))                                      # not int32
    with pytest.raises(hga.HgaError):
        hga.pages_fork(pool, torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32))
    with pytest.raises(hga.HgaError):
        hga.pages_free(pool, torch.zeros(2, dtype=i32))                           # not on a GPU
    with pytest.raises(hga.HgaError):
        hga.Q4Batch(torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32))
    p = hga.Params(2, 1, 128)
    batch = hga.Q4Batch(torch.zeros(4, dtype=i32))
    k = torch.zeros(4, 1, 128, dtype=torch.bfloat16)
    for kk, vv in ((k.float(), k), (k, k.half()), (k[:, :, :64], k), (k, k[:3])):
        with pytest.raises(hga.HgaError):
            hga.q4_append(p, pool, 0, batch, kk, vv)
    with pytest.raises(hga.HgaError):
        hga.q4_append(p, pool, 0, batch, k, k)                                    # not on a GPU
    for qq in (q.float(), q[:, :1], q.transpose(0, 1)):
        with pytest.raises(hga.HgaError):
            hga.q4_attend(p, pool, 0, batch, qq, torch.zeros_like(qq))


def test_reference_format_is_its_definition():
    """The reference's own checks: representable values stay, ties go to the
    even code, and no value of a block moves by more than half its code step."""
    import q4_ref
    assert len(q4_ref.SCALES) == 227 and q4_ref.SCALES[-1] == 10240.0
    halves = (np.arange(227, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(halves, q4_ref.SCALES)
    x = np.zeros((1, 16))
    x[0, :8] = q4_ref.MAG * 1.25
    assert np.array_equal(q4_ref.stored(x), x)
    x[0, 8:15] = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5]) * -1.25
    got = q4_ref.stored(x)
    assert np.array_equal(got[0, 8:15], np.array([0, 1, 1, 2, 2, 4, 4]) * -1.25)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((1000, 16)) * 10.0 ** rng.uniform(-4, 4, (1000, 1))
    got = q4_ref.stored(x)
    top = np.abs(x).max(-1, keepdims=True)
    # the scale is the next one above top / 6: 3 mantissa bits (9/8 apart), or
    # 2^-17 apart below 2^-14; the widest code step is 2 scales
    assert np.all(np.abs(got - x) <= np.maximum(top / 6 * 9 / 8, top / 6 + 2.0 ** -17) * (1 + 1e-12))
