"""Cases of the serving and training operators around the routed attention,
with their plain forms.

Operators:
  rope      rotary positions with one to three axes on q and k, read from a
            fused projection and written where the attention reads them, and
            the backward pass from the attention's fp32 gradients;
  append    K/V tokens of several sequences into pages of 4-bit codes, and the
            same tokens read back as the values the codes stand for;
  attend    attention over such a cache: one token per sequence (decode), many
            (prefill), and the routed form with its kept groups of 8 tokens;
  pages     forking, freeing and compacting the pages of a cache.

The 4-bit format: 16 neighbouring values of a head share one scale.  A scale
is a byte b standing for the IEEE half with bits b << 7 (5 exponent bits, 3
mantissa bits, no sign); it is the smallest one with 6 * scale >= max|x|, at
most 10240.  A code is sign and magnitude index of {0, .5, 1, 1.5, 2, 3, 4, 6},
the one nearest to x / scale, ties to the even index.  A record holds 8 tokens
of one KV head: K codes [8][d/2], V codes [8][d/2] (dim 2i in the low nibble),
K scales [8][d/16], V scales [8][d/16].  A page is [KV head][tokens / 8] records.
"""
import math
import random

import torch

own = False

MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token of 8 requests: 32 query heads on 4 KV heads
        dict(name="rope_step_8", op="rope", n=8, hq=32, hkv=4, d=128, axes=1, adjacent=False,
             backward=False, dtype="bf16", far=65536),
        # a 16K prompt with image tokens (time, height, width), 32 heads on 8
        dict(name="rope_prompt_16k", op="rope", n=16384, hq=32, hkv=8, d=128, axes=3,
             adjacent=False, backward=False, dtype="bf16", far=131072),
        # a training segment: gradients of the rotated q and k come in fp32
        dict(name="rope_grad_4k", op="rope", n=4096, hq=32, hkv=8, d=128, axes=3, adjacent=False,
             backward=True, dtype="fp32", far=131072),
        # the prompts of some short requests enter the cache (ragged)
        dict(name="append_ragged_1k", op="append", n_seq=5, n=1009, hkv=4, d=128, page=64,
             dtype="bf16"),
        # a 32K context is stored in one go
        dict(name="append_32k", op="append", n_seq=1, n=32768, hkv=8, d=128, page=64,
             dtype="bf16"),
        # a small fp32 model: 2 query heads on one KV head, head_dim 64
        dict(name="decode_small_fp32", op="attend", n_seq=3, ctx=1024, nq=1, hq=2, hkv=1, d=64,
             page=16, dtype="fp32"),
        # 8 requests at up to 64K tokens, one new token each
        dict(name="decode_8x64k", op="attend", n_seq=8, ctx=65536, nq=1, hq=32, hkv=4, d=128,
             page=64, dtype="bf16"),
        # chunked prefill: up to 1K new tokens of 3 requests on up to 8K of history
        dict(name="prefill_3x1k_of_8k", op="attend", n_seq=3, ctx=8192, nq=1024, hq=32, hkv=8,
             d=128, page=64, dtype="bf16"),
        # the routed attention of the last 2K queries of a 64K context
        dict(name="routed_64k_last2k", op="routed", T=65536, nq=2048, hq=32, hkv=4, d=128,
             sink=64, local=512, groups=64, page=64, dtype="bf16"),
        # parallel sampling: 4 requests fork into 4 samples each, one layer
        dict(name="fork_4x4", op="fork", parents=4, each=4, len=700, planes=1, hkv=4, d=128,
             page=64),
        # beams over every layer's pages: 16 requests, 8 beams
        dict(name="fork_16x8_layers", op="fork", parents=16, each=8, len=500, planes=36, hkv=8,
             d=128, page=64),
        # half the requests have left a pool of 24 layers; the rest moves together
        dict(name="compact_24_layers", op="compact", rows=64, len=640, planes=24, hkv=4, d=128,
             page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "routed", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([x for x in (1, 2, 4, 5, 8) if x * hkv <= 32])
    page = rng.choice([8, 16, 32, 64, 64, 128])
    if op == "rope":
        return dict(op=op, n=_log(rng, 1, 16384), hq=hq, hkv=hkv, d=d, axes=rng.choice([1, 2, 3]),
                    adjacent=rng.random() < 0.3, backward=rng.random() < 0.4, dtype=dtype,
                    far=_log(rng, 100, 1000000))
    if op == "append":
        n = _log(rng, 1, 32768)
        return dict(op=op, n_seq=min(n, _log(rng, 1, 64)), n=n, hkv=hkv, d=d, page=page,
                    dtype=dtype)
    if op == "attend":
        form = rng.choice(["one", "few", "many"])
        if form == "one":
            n_seq = _log(rng, 1, 128)
            ctx = _log(rng, 16, 2 ** 21 // (n_seq * hkv))
            nq = 1
        elif form == "few":
            n_seq = _log(rng, 1, 16)
            ctx = _log(rng, 16, 2 ** 19 // (n_seq * hkv))
            nq = min(ctx, rng.randint(2, 16))
        else:
            n_seq = _log(rng, 1, 4)
            ctx = _log(rng, 256, 8192)
            nq = min(ctx, _log(rng, 17, 1024))
            n_seq = max(1, min(n_seq, 3 * 1024 * 8192 // (nq * ctx)))
        return dict(op=op, n_seq=n_seq, ctx=ctx, nq=nq, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype)
    if op == "routed":
        T = _log(rng, 256, 65536)
        nq = min(T, rng.choice([1, 17, 64, _log(rng, 2, 2048)]))
        return dict(op=op, T=T, nq=nq, hq=hq, hkv=hkv, d=d, sink=64 * rng.randint(0, 2),
                    local=64 * rng.randint(0, 8), groups=_log(rng, 1, 64), page=page, dtype=dtype)
    if op == "fork":
        planes = _log(rng, 1, 36)
        return dict(op=op, parents=_log(rng, 1, 16), each=_log(rng, 1, 8), len=_log(rng, 1, 800),
                    planes=planes, hkv=hkv, d=d, page=min(page, 64))
    return dict(op=op, rows=_log(rng, 2, 64), len=_log(rng, 8, 640), planes=_log(rng, 1, 24),
                hkv=min(hkv, 4), d=d, page=min(page, 64))


# ------------------------------------------------------------------ the 4-bit format (plain)

def _tables(dev):
    mag = torch.tensor(MAG, device=dev)
    both = torch.cat([mag, -mag])
    byte = torch.arange(256, device=dev)
    pair = torch.stack([both[byte & 15], both[byte >> 4]], -1)          # [256][2]
    scale = (torch.arange(256, device=dev, dtype=torch.int32) << 7).to(torch.int16)
    return pair, scale.view(torch.float16).float()


def _encode(x, tab):
    """x [..., d] -> codes [..., d/2] and scale bytes [..., d/16] (uint8)."""
    f = x.float().unflatten(-1, (-1, 16))
    a = f.abs()
    steps = 6 * tab[1][:227]
    b = torch.searchsorted(steps, a.amax(-1).contiguous()).clamp(max=226)
    s = tab[1][b].unsqueeze(-1)
    idx = ((a > .25 * s).byte() + (a >= .75 * s).byte() + (a > 1.25 * s).byte()
           + (a >= 1.75 * s).byte() + (a > 2.5 * s).byte() + (a >= 3.5 * s).byte()
           + (a > 5 * s).byte())
    code = torch.where(s > 0, idx, 0) + 8 * (f < 0).byte()
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), b.to(torch.uint8)


def _decode(codes, scales, tab):
    """codes [..., d/2], scales [..., d/16] -> fp32 [..., d]."""
    v = tab[0][codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    return (v * tab[1][scales.int()].unsqueeze(-1)).flatten(-2)


def _split(rec, d):
    """records [..., 72 d / 8] -> K codes, V codes [..., 8, d/2], K scales, V scales."""
    a, b = 4 * d, d // 2
    return (rec[..., :a].unflatten(-1, (8, -1)), rec[..., a:2 * a].unflatten(-1, (8, -1)),
            rec[..., 2 * a:2 * a + b].unflatten(-1, (8, -1)),
            rec[..., 2 * a + b:].unflatten(-1, (8, -1)))


def _rec_bytes(d):
    return 9 * d


def _records(st, k, v):
    """k, v [n][Hkv][d] with n % 8 == 0 -> records [n / 8][Hkv][bytes]."""
    parts = []
    kc, ks = _encode(k, st["tab"])
    vc, vs = _encode(v, st["tab"])
    for x in (kc, vc, ks, vs):
        parts.append(x.unflatten(0, (-1, 8)).transpose(1, 2).flatten(-2))
    return torch.cat(parts, -1)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ragged(lo, hi, n, salt):
    """n whole numbers in [lo, hi], the first one hi: a case's own, whatever the seed, so that
    its outputs keep their shapes."""
    r = random.Random("%d %d %d %d" % (lo, hi, n, salt))
    return [hi] + [r.randint(lo, hi) for _ in range(n - 1)]


def _cache(case, lens, g, planes=1, extra=0, fill=True):
    """A pool whose sequences (table rows) hold `lens` tokens, its pages in a random order."""
    page, d, hkv = case["page"], case["d"], case["hkv"]
    n = [-(-x // page) for x in lens]
    row_pages = max(n)
    total = sum(n)
    n_pages = total + extra
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), row_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(n):
        table[i, :c] = order[at:at + c]
        at += c
    page_bytes = hkv * (page // 8) * _rec_bytes(d)
    st = dict(tab=_tables("cuda"), table=table,
              length=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              ref=torch.zeros(n_pages, dtype=torch.int32, device="cuda"),
              data=torch.empty(planes, n_pages, page_bytes, dtype=torch.uint8, device="cuda"))
    st["ref"][order[:total].long()] = 1
    if fill:
        view = st["data"].view(planes, n_pages, hkv, page // 8, _rec_bytes(d))
        step = max(1, 2 ** 25 // (page * hkv * d))
        for a in range(0, n_pages, step):
            c = min(step, n_pages - a)
            k = torch.randn(c * page, hkv, d, generator=g, device="cuda").bfloat16()
            v = torch.randn(c * page, hkv, d, generator=g, device="cuda").bfloat16()
            r = _records(st, k, v).view(c, page // 8, hkv, -1).transpose(1, 2)
            view[0, a:a + c] = r
    return st


# ------------------------------------------------------------------ prepare

def _sections(case):
    """How many frequencies each axis takes."""
    r = case["d"] // 2
    return {1: [r], 2: [r // 2, r - r // 2], 3: [r // 4, r * 3 // 8, r - r // 4 - r * 3 // 8]}[case["axes"]]


def _prepare_rope(case, seed):
    g = _gen(seed)
    n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
    dt = _dt(case)
    st = dict(case=case)
    st["pos"] = torch.randint(0, case["far"], (case["axes"], n), generator=g, device="cuda",
                              dtype=torch.int32)
    st["freq"] = 1e6 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2 / d)
    st["axis"] = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"),
                                         torch.tensor(_sections(case), device="cuda")).to(torch.uint8)
    if case["backward"]:
        # the attention's gradients: q's in its rows, k's in the cache's layout
        st["q"] = torch.randn(n, hq, d, generator=g, device="cuda")
        st["k"] = torch.randn(hkv, n, d, generator=g, device="cuda").transpose(0, 1)
        rows = torch.zeros(n, hq + 2 * hkv, d, device="cuda", dtype=dt)
        st["q_out"], st["k_out"] = rows[:, :hq], rows[:, hq:hq + hkv]
    else:
        # the fused projection's rows in, q's rows and the cache's layout out
        rows = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda").to(dt)
        st["q"], st["k"] = rows[:, :hq], rows[:, hq:hq + hkv]
        st["q_out"] = torch.zeros(n, hq, d, device="cuda", dtype=dt)
        st["k_out"] = torch.zeros(hkv, n, d, device="cuda", dtype=dt).transpose(0, 1)
    return st


def _prepare_append(case, seed):
    g = _gen(seed)
    n, n_seq = case["n"], case["n_seq"]
    r = random.Random("%d %d" % (n, n_seq))
    cuts = [0] + sorted(r.randint(0, n - n_seq) for _ in range(n_seq - 1)) + [n - n_seq]
    add = [b - a + 1 for a, b in zip(cuts, cuts[1:])]   # n tokens in all, at least one each
    before = [r.randint(0, 200) for _ in add]
    st = _cache(case, [a + b for a, b in zip(add, before)], g, fill=False)
    st["case"] = case
    st["off"] = torch.tensor([0] + add, device="cuda").cumsum(0).int()
    st["rows"] = torch.randperm(n_seq, generator=g, device="cuda").int()
    # rows are taken in a random order: sequence i of the call is table row rows[i]
    st["table"][st["rows"].long()] = st["table"].clone()
    st["length"][st["rows"].long()] = st["length"].clone()
    st["max_q"] = max(add)
    st["k"], st["v"] = (torch.randn(n, case["hkv"], case["d"], generator=g, device="cuda").to(_dt(case))
                        for _ in range(2))
    st["k_out"], st["v_out"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
    return st


def _prepare_attend(case, seed):
    g = _gen(seed)
    n_seq, nq = case["n_seq"], case["nq"]
    ctx = _ragged(max(nq, case["ctx"] // 2), case["ctx"], n_seq, 0)
    add = _ragged(max(1, nq // 2), nq, n_seq, 1)
    st = _cache(case, ctx, g, extra=3)
    st["case"] = case
    st["rows"] = torch.arange(n_seq, device="cuda", dtype=torch.int32)
    st["off"] = torch.tensor([0] + add, device="cuda").cumsum(0).int()
    n = sum(add)
    dt = _dt(case)
    st["q"] = torch.randn(n, case["hq"], case["d"], generator=g, device="cuda").to(dt)
    st["k"], st["v"] = (torch.randn(n, case["hkv"], case["d"], generator=g, device="cuda").to(dt)
                        for _ in range(2))
    st["o"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros(n, case["hq"], device="cuda")
    return st


def _prepare_routed(case, seed):
    g = _gen(seed)
    T, nq, hkv = case["T"], case["nq"], case["hkv"]
    q0 = (T - nq) // 64 * 64
    T = q0 + nq
    st = _cache(case, [T], g, extra=3)
    st["case"], st["q0"] = case, q0
    n_blocks = -(-nq // 64)
    b0 = q0 + 64 * torch.arange(n_blocks, device="cuda")
    # candidates: groups between the sink and the local window of the block
    first = case["sink"] // 8
    n_cand = ((b0 - case["local"]).clamp(min=case["sink"]) // 8 - first)
    total = max(1, T // 8)
    score = torch.rand(hkv, n_blocks, total, generator=g, device="cuda")
    j = torch.arange(total, device="cuda")
    ok = (j >= first) & (j < first + n_cand[:, None])
    keep = min(case["groups"], total)
    top = torch.where(ok, score, -1.0).topk(keep, -1)
    idx = torch.where(top.values >= 0, top.indices, total).sort(-1).values
    st["cnt"] = (idx < total).sum(-1).int()
    st["idx"] = torch.where(idx < total, idx, -1).int().contiguous()
    st["t_cap"] = -(-T // 64) * 64
    dt = _dt(case)
    st["q"] = torch.randn(nq, case["hq"], case["d"], generator=g, device="cuda").to(dt)
    st["o"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros(nq, case["hq"], device="cuda")
    return st


def _prepare_fork(case, seed):
    g = _gen(seed)
    P, n = case["parents"], case["parents"] * case["each"]
    lens = _ragged(max(1, case["len"] // 2), case["len"], P, 0)
    st = _cache(case, lens, g, planes=case["planes"], extra=n, fill=False)
    st["case"] = case
    st["data"].random_(0, 256, generator=g)
    st["table"] = torch.cat([st["table"], st["table"].new_full((n, st["table"].shape[1]), -1)])
    st["length"] = torch.cat([st["length"], st["length"].new_zeros(n)])
    st["from"] = torch.arange(P, device="cuda", dtype=torch.int32).repeat_interleave(case["each"])
    st["to"] = torch.arange(P, P + n, device="cuda", dtype=torch.int32)
    return st


def _prepare_compact(case, seed):
    g = _gen(seed)
    R = case["rows"]
    lens = _ragged(max(1, case["len"] // 2), case["len"], R, 0)
    st = _cache(case, lens, g, planes=case["planes"], fill=False)
    st["case"] = case
    st["data"].random_(0, 256, generator=g)
    # every second request has left
    gone = torch.randperm(R, generator=g, device="cuda")[:R // 2]
    left = st["table"][gone]
    st["ref"][left[left >= 0].long()] = 0
    st["table"][gone] = -1
    st["length"][gone] = 0
    st["table0"], st["ref0"] = st["table"].clone(), st["ref"].clone()
    return st


def prepare(case, seed):
    st = globals()["_prepare_" + case["op"]](case, seed)
    if own:
        _handles(case, st)
    return st


# ------------------------------------------------------------------ the framework's calls

def _handles(case, st):
    """The objects that a program keeps between calls."""
    from long_context_hga_b200 import hga
    st["hga"] = hga
    if case["op"] == "rope":
        st["plan"] = hga.Rope(st["freq"], st["axis"], case["d"], adjacent=case["adjacent"])
        return
    st["pool"] = hga.PagePool(st["data"], st["table"], st["length"], st["ref"], case["page"])
    if case["op"] in ("fork", "compact"):
        return
    hq = case.get("hq", case["hkv"])
    st["p"] = hga.Params(hq, case["hkv"], case["d"], sink=case.get("sink", 64),
                         local=case.get("local", 128), top_chunks=0,
                         top_groups=st["idx"].shape[-1] if "idx" in st else 8, dtype=case["dtype"])
    if case["op"] == "routed":
        st["work"] = hga.q4_routed_workspace(st["p"], st["q"].shape[0])
        return
    max_q = st.get("max_q", case.get("nq"))
    st["batch"] = hga.Q4Batch(st["rows"], None if max_q == 1 and case["op"] == "attend" else st["off"], max_q)
    if case["op"] == "attend":
        st["work"] = hga.q4_workspace(st["p"], st["batch"], st["q"].shape[0], case["ctx"])


def _own(st):
    case, hga = st["case"], st["hga"]
    op = case["op"]
    if op == "rope":
        call = hga.rope_backward if case["backward"] else hga.rope
        call(st["plan"], st["pos"], st["q"], st["q_out"], st["k"], st["k_out"])
        return [st["q_out"], st["k_out"]]
    pool = st["pool"]
    if op == "append":
        hga.q4_append(st["p"], pool, 0, st["batch"], st["k"], st["v"])
        hga.q4_read(st["p"], pool, 0, st["batch"], st["k_out"], st["v_out"])
        return [st["k_out"], st["v_out"]]
    if op == "attend":
        hga.q4_append(st["p"], pool, 0, st["batch"], st["k"], st["v"])
        hga.q4_attend(st["p"], pool, 0, st["batch"], st["q"], st["o"], st["lse"],
                      max_ctx=case["ctx"], work=st["work"])
        return [st["o"], st["lse"]]
    if op == "routed":
        hga.q4_attend_routed(st["p"], pool, 0, 0, st["q"], st["q0"], st["t_cap"], st["idx"], st["cnt"],
                             st["o"], st["lse"], work=st["work"])
        return [st["o"], st["lse"]]
    if op == "fork":
        hga.pages_free(pool, st["to"])
        hga.pages_fork(pool, st["from"], st["to"])
        return [st["data"], st["table"], st["length"], st["ref"]]
    st["table"].copy_(st["table0"])
    st["ref"].copy_(st["ref0"])
    hga.pages_compact(pool)
    return [st["data"], st["table"], st["ref"]]


# ------------------------------------------------------------------ the plain forms

def _rotate(st, x, sign):
    case = st["case"]
    ang = st["pos"].double()[st["axis"].long()].T * st["freq"]       # [n][d/2], in 64 bits
    c, s = ang.cos().float()[:, None], (sign * ang.sin()).float()[:, None]
    x = x.float()
    if case["adjacent"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_rope(st):
    sign = -1 if st["case"]["backward"] else 1
    st["q_out"].copy_(_rotate(st, st["q"], sign))
    st["k_out"].copy_(_rotate(st, st["k"], sign))
    return [st["q_out"], st["k_out"]]


def _where(st):
    """Page, record and row in it of every token of the call."""
    off = st["off"].long()
    n = st["k"].shape[0]
    tok = torch.arange(n, device="cuda")
    seq = torch.searchsorted(off[1:].contiguous(), tok, right=True)
    row = st["rows"].long()[seq]
    pos = st["length"].long()[row] - off[seq + 1] + tok
    page = st["case"]["page"]
    return st["table"][row, pos // page].long(), pos % page // 8, pos % 8


def _view(st):
    case = st["case"]
    return st["data"][0].view(st["data"].shape[1], case["hkv"], case["page"] // 8, _rec_bytes(case["d"]))


def _plain_store(st):
    at, rec, r = _where(st)
    view = _view(st)
    parts = _split(view, st["case"]["d"])
    for part, x in zip((0, 2), (st["k"], st["v"])):
        code, scale = _encode(x, st["tab"])
        for y, z in ((parts[part // 2], code), (parts[2 + part // 2], scale)):
            y[at, :, rec, r] = z


def _plain_append(st):
    _plain_store(st)
    at, rec, r = _where(st)
    parts = [x[at, :, rec, r] for x in _split(_view(st), st["case"]["d"])]
    st["k_out"].copy_(_decode(parts[0], parts[2], st["tab"]))
    st["v_out"].copy_(_decode(parts[1], parts[3], st["tab"]))
    return [st["k_out"], st["v_out"]]


def _softmax(s, v, ok):
    """s, ok [..., r, t], v [..., t, d] -> output and log of the sum; empty rows 0 and -inf."""
    s = torch.where(ok, s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    o = (e / torch.where(l > 0, l, 1.0)) @ v
    return o, (torch.log(l) + m).squeeze(-1)


def _plain_attend(st):
    _plain_store(st)
    case = st["case"]
    d, hkv, G, page = case["d"], case["hkv"], case["hq"] // case["hkv"], case["page"]
    rec = _view(st)[st["table"].clamp(min=0).long()]       # [seq][page][Hkv][page/8][bytes]
    kc, vc, ks, vs = (x.permute(0, 2, 1, 3, 4, 5).flatten(2, 4) for x in _split(rec, d))
    k, v = _decode(kc, ks, st["tab"]), _decode(vc, vs, st["tab"])           # [seq][Hkv][t][d]
    n_seq, t = k.shape[0], k.shape[2]
    off = st["off"].long()
    n = off[1:] - off[:-1]
    m = case["nq"]
    j = torch.arange(m, device="cuda")
    tok = (off[:-1, None] + j).clamp(max=st["q"].shape[0] - 1)            # [seq][m], padded
    q = st["q"].float()[tok].view(n_seq, m, hkv, G, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    pos = st["length"].long()[:, None] - n[:, None] + j
    ok = torch.arange(t, device="cuda") <= pos.repeat_interleave(G, 1)[..., None]
    o, lse = _softmax(q @ k.transpose(-1, -2) / d ** 0.5, v, ok[:, None])
    live = j < n[:, None]
    o = o.view(n_seq, hkv, m, G, d).permute(0, 2, 1, 3, 4).reshape(n_seq, m, hkv * G, d)
    lse = lse.view(n_seq, hkv, m, G).permute(0, 2, 1, 3).reshape(n_seq, m, hkv * G)
    st["o"].copy_(o[live])
    st["lse"].copy_(lse[live])
    return [st["o"], st["lse"]]


def _plain_routed(st):
    case = st["case"]
    d, hkv, G, page = case["d"], case["hkv"], case["hq"] // case["hkv"], case["page"]
    nq, q0 = st["q"].shape[0], st["q0"]
    nb = -(-nq // 64)
    b0 = q0 + 64 * torch.arange(nb, device="cuda")
    # every group a block may attend: sink, routed, local window and diagonal; -1 = none
    sink = torch.arange(case["sink"] // 8, device="cuda").expand(hkv, nb, -1)
    sink = torch.where(sink * 8 < b0[:, None], sink, -1)
    lo = torch.maximum((b0 - case["local"]).clamp(min=0), torch.minimum(b0, b0.new_tensor(case["sink"])))
    loc = (b0 // 8)[:, None] - case["local"] // 8 + torch.arange(case["local"] // 8 + 8, device="cuda")
    loc = torch.where(loc * 8 >= lo[:, None], loc, -1).expand(hkv, -1, -1)
    grp = torch.cat([sink, st["idx"].long(), loc], -1)                       # [Hkv][nb][L]
    grp = torch.where(grp * 8 < q0 + nq, grp, -1)
    at = grp.clamp(min=0)
    head = torch.arange(hkv, device="cuda")[:, None, None]
    rec = _view(st)[st["table"][0].long()[at * 8 // page], head, at % (page // 8)]
    kc, vc, ks, vs = (x.flatten(2, 3) for x in _split(rec, d))
    k, v = _decode(kc, ks, st["tab"]), _decode(vc, vs, st["tab"])
    t = (at[..., None] * 8 + torch.arange(8, device="cuda")).flatten(-2)
    there = (grp >= 0)[..., None].expand(-1, -1, -1, 8).flatten(-2)
    row = torch.arange(nb * 64, device="cuda")
    q = st["q"].float()[row.clamp(max=nq - 1)].view(nb, 64, hkv, G, d).permute(2, 0, 1, 3, 4).flatten(2, 3)
    pos = (q0 + row).view(nb, 64).repeat_interleave(G, 1)
    ok = there[:, :, None] & (t[:, :, None] <= pos[..., None])
    v = torch.where((there & (t < q0 + nq))[..., None], v, 0.0)
    o, lse = _softmax(q @ k.transpose(-1, -2) / d ** 0.5, v, ok)
    st["o"].copy_(o.view(hkv, nb, 64, G, d).permute(1, 2, 0, 3, 4).reshape(nb * 64, hkv * G, d)[:nq])
    st["lse"].copy_(lse.view(hkv, nb, 64, G).permute(1, 2, 0, 3).reshape(nb * 64, hkv * G)[:nq])
    return [st["o"], st["lse"]]


def _plain_fork(st):
    case = st["case"]
    table, length, ref, page = st["table"], st["length"], st["ref"], case["page"]
    frm, to = st["from"].long(), st["to"].long()
    # the children's pages go back
    old = table[to]
    ref.index_put_((old.clamp(min=0).long().flatten(),), -(old >= 0).int().flatten(), accumulate=True)
    table[to] = -1
    length[to] = 0
    # whole pages are shared; a page that ends inside is copied to the lowest free one
    full, part = length[frm] // page, length[frm] % page > 0
    rows = table[frm]
    col = torch.arange(rows.shape[1], device="cuda")
    shared = col < full[:, None]
    ref.index_put_((rows.clamp(min=0).long().flatten(),), shared.int().flatten(), accumulate=True)
    free = torch.sort((ref != 0).int(), stable=True).indices
    rank = torch.cumsum(part.int(), 0) - 1
    new = free[rank.clamp(min=0)].int()
    last = part[:, None] & (col == full[:, None])
    table[to] = torch.where(shared, rows, torch.where(last, new[:, None], -1))
    length[to] = length[frm]
    src = rows.gather(1, full.long().clamp(max=rows.shape[1] - 1)[:, None])[:, 0]
    src, dst = src[part].long(), new[part].long()
    ref[dst] = 1
    st["data"][:, dst] = st["data"][:, src]
    return [st["data"], table, length, ref]


def _plain_compact(st):
    table, ref = st["table"], st["ref"]
    table.copy_(st["table0"])
    ref.copy_(st["ref0"])
    used = ref > 0
    n = used.sum()
    i = torch.arange(ref.numel(), device="cuda")
    src = torch.nonzero(used & (i >= n))[:, 0]
    dst = torch.nonzero(~used & (i < n))[:, 0]
    to = i.clone()
    to[src] = dst
    st["data"][:, dst] = st["data"][:, src]
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), -1))
    ref[dst] = ref[src]
    ref[src] = 0
    return [st["data"], table, ref]


def run(state):
    return _own(state) if own else globals()["_plain_" + state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, d = case["op"], case["d"]
    if op == "rope":
        x = case["n"] * (case["hq"] + case["hkv"]) * d
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": x * ((4 if case["backward"] else e) + e), "flops": 3 * x}
    rec = _rec_bytes(d) / 8                                   # bytes of a token's K and V of a head
    if op == "append":
        x = case["n"] * case["hkv"]
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * x * (2 * d * e + rec), "flops": 2 * x * d * 4}
    if op == "attend":
        e = 2 if case["dtype"] == "bf16" else 4
        n_seq, m = case["n_seq"], case["nq"]
        each = list(zip(_ragged(max(m, case["ctx"] // 2), case["ctx"], n_seq, 0),
                        _ragged(max(1, m // 2), m, n_seq, 1)))
        ctx, new = sum(c for c, _ in each), sum(n for _, n in each)
        pairs = sum(n * c - n * (n - 1) // 2 for c, n in each)
        io = new * (2 * case["hq"] * d * e + 4 * case["hq"] + 2 * case["hkv"] * d * e)
        return {"bytes": ctx * case["hkv"] * rec + io, "flops": 4 * pairs * case["hq"] * d}
    if op == "routed":
        e = 2 if case["dtype"] == "bf16" else 4
        nq, nb = case["nq"], -(-case["nq"] // 64)
        per = min(case["T"], case["sink"] + case["local"] + 8 * case["groups"])
        once = min(case["T"], case["sink"] + case["local"] + nq + 8 * case["groups"] * nb)
        return {"bytes": once * case["hkv"] * rec + nq * case["hq"] * (2 * d * e + 4),
                "flops": 4 * nq * case["hq"] * d * (per + 32)}
    page_bytes = case["hkv"] * (case["page"] // 8) * _rec_bytes(d)
    if op == "fork":
        lens = _ragged(max(1, case["len"] // 2), case["len"], case["parents"], 0)
        inside = sum(x % case["page"] > 0 for x in lens) * case["each"]
        shared = sum(x // case["page"] for x in lens) * case["each"]
        return {"bytes": 2 * inside * case["planes"] * page_bytes + 8 * (shared + inside), "flops": 0}
    lens = _ragged(max(1, case["len"] // 2), case["len"], case["rows"], 0)
    total = sum(-(-x // case["page"]) for x in lens)
    # half the rows have left: about a quarter of the pages are used and above the used count
    return {"bytes": 2 * total / 4 * case["planes"] * page_bytes + 8 * total, "flops": 0}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _two_to(e):
    """2^e in 64 bits for whole e in [-32, 32) (pow is not exact on the GPU)."""
    return torch.tensor([2.0 ** i for i in range(-32, 32)], dtype=torch.float64, device=e.device)[e + 32]


def _value(code):
    """A 4-bit code's value: sign, two exponent bits, one mantissa bit."""
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * _two_to(e - 1))
    return torch.where(code >= 8, -mag, mag)


def _scale_value(b):
    e, m = b >> 3, (b & 7).double()
    return torch.where(e == 0, m * 2.0 ** -17, (1 + m / 8) * _two_to(e - 15))


def _stored(x):
    """The values that 4 bits hold of x [..., d], in 64 bits."""
    x = x.double().unflatten(-1, (-1, 16))
    every = _scale_value(torch.arange(227, device=x.device))
    top = x.abs().amax(-1)
    b = torch.zeros_like(top, dtype=torch.int64)
    for bit in (128, 64, 32, 16, 8, 4, 2, 1):           # the smallest byte that is large enough
        c = (b + bit).clamp(max=227)
        b = torch.where(6 * every[(c - 1).clamp(max=226)] < top, c, b)
    s = every[b.clamp(max=226)].unsqueeze(-1)
    r = (x / torch.where(s > 0, s, 1.0)).abs().clamp(max=6)
    grid = torch.tensor(MAG, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(grid, r.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - r, r - grid[lo]
    pick = torch.where(up < down, hi, torch.where(up > down, lo, torch.where(hi % 2 == 0, hi, lo)))
    return (grid[pick] * x.sign() * s).flatten(-2)


def _exact_tokens(st, row, plane=0):
    """K and V of a table row from its pages, [Hkv][pages * page][d] in 64 bits."""
    case = st["case"]
    d, hkv, page = case["d"], case["hkv"], case["page"]
    pages = st["table"][row]
    pages = pages[pages >= 0].long()
    r = st["data"][plane][pages].view(-1, hkv, page // 8, 9 * d).long()
    out = []
    for a, b in ((0, 8 * d), (4 * d, 8 * d + d // 2)):
        c = r[..., a:a + 4 * d].unflatten(-1, (8, d // 2))
        code = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        s = _scale_value(r[..., b:b + d // 2].unflatten(-1, (8, d // 16)))
        x = _value(code) * s.repeat_interleave(16, -1)
        out.append(x.permute(1, 0, 2, 3, 4).reshape(hkv, -1, d))
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None
    g = globals()
    st = g["_prepare_" + op](case, seed)
    if op == "rope":
        out = []
        for x in (st["q"], st["k"]):
            ang = torch.stack([st["pos"][a].double() * f for a, f in zip(st["axis"].tolist(), st["freq"].tolist())], -1)
            if case["backward"]:
                ang = -ang
            w = torch.polar(torch.ones_like(ang), ang)[:, None]
            d = case["d"]
            z = x.double().unflatten(-1, (d // 2, 2)) if case["adjacent"] else x.double().unflatten(-1, (2, d // 2)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(z.contiguous()) * w)
            out.append((y if case["adjacent"] else y.transpose(-1, -2)).flatten(-2))
        return out
    if op == "append":
        return [_stored(st["k"]), _stored(st["v"])]
    d, hkv, G = case["d"], case["hkv"], case["hq"] // case["hkv"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    if op == "attend":
        if work(case)["flops"] > 3e12:
            return None
        off, lens = st["off"].tolist(), st["length"].tolist()
        nk, nv = _stored(st["k"]), _stored(st["v"])
        for i in range(case["n_seq"]):
            a, b = off[i], off[i + 1]
            k, v = _exact_tokens(st, i)
            k[:, lens[i] - b + a:lens[i]] = nk[a:b].transpose(0, 1)
            v[:, lens[i] - b + a:lens[i]] = nv[a:b].transpose(0, 1)
            for h in range(hkv):
                x = st["q"][a:b, h * G:(h + 1) * G].double()
                for c in range(0, b - a, 128):
                    y = x[c:c + 128]
                    pos = lens[i] - b + a + c + torch.arange(y.shape[0], device="cuda")
                    s = torch.einsum("igd,td->igt", y, k[h, :lens[i]]) / math.sqrt(d)
                    s.masked_fill_((torch.arange(lens[i], device="cuda") > pos[:, None])[:, None], -math.inf)
                    z = torch.logsumexp(s, -1)
                    lse[a + c:a + c + 128, h * G:(h + 1) * G][:b - a - c] = z
                    o[a + c:a + c + 128, h * G:(h + 1) * G][:b - a - c] = torch.exp(s - z[..., None]) @ v[h, :lens[i]]
        return [o, lse]
    k, v = _exact_tokens(st, 0)
    q0, nq = st["q0"], st["q"].shape[0]
    idx, cnt = st["idx"].cpu(), st["cnt"].cpu()
    for b in range(-(-nq // 64)):
        p0 = q0 + 64 * b
        n = min(64, q0 + nq - p0)
        pos = p0 + torch.arange(n, device="cuda")
        for h in range(hkv):
            here = torch.zeros(k.shape[1], dtype=torch.bool)
            here[:min(case["sink"], p0)] = True
            here[max(0, p0 - case["local"]):p0 + n] = True
            for j in idx[h, b, :int(cnt[h, b])].tolist():
                here[8 * j:8 * j + 8] = True
            t = torch.nonzero(here)[:, 0].to("cuda")
            t = t[t < q0 + nq]
            x = st["q"][64 * b:64 * b + n, h * G:(h + 1) * G].double()
            s = torch.einsum("igd,td->igt", x, k[h, t]) / math.sqrt(d)
            s.masked_fill_((t > pos[:, None])[:, None], -math.inf)
            z = torch.logsumexp(s, -1)
            lse[64 * b:64 * b + n, h * G:(h + 1) * G] = z
            o[64 * b:64 * b + n, h * G:(h + 1) * G] = torch.exp(s - z[..., None]) @ v[h, t]
    return [o, lse]
