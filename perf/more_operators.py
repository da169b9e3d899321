"""The serving operators' cases over an 8-bit cache and over selected pages of a cache.

    append   new tokens into a cache of e4m3 values with a power-of-two scale for each 16 positions and head
    attend   attention over that cache
    bounds   per page and head, bounds of its keys in 8 bits
    select   the pages that a cheap score over those bounds selects for each token and kv head
    sparse   attention over the selected pages

A case says which operator it is and its sizes. `run` computes it with elementary torch operations
in binary32 (binary64 for angles), or, with `own` set, through the library's public calls. Ragged
lengths come from the case's own fields.
"""
import math
import random

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
EPS = 1e-5
BLOCK = 16  # positions that share a scale


def listed():
    return [
        # one decode token of the 1.1B model's heads (32 query, 4 kv, 64 wide): pure latency
        dict(name="append_one", op="append", heads=32, kv=4, dim=64, rope_dim=64, interleaved=True, norm=False,
             fused=False, in_dtype="f32", page=16, seqs=1, q_lo=1, q_hi=1, ctx_lo=99, ctx_hi=99, mix=1),
        # a prompt step: five ragged prompts, about 8000 new tokens in all, normed heads, fused qkv rows
        dict(name="append_prompts", op="append", heads=32, kv=8, dim=128, rope_dim=96, interleaved=False, norm=True,
             fused=True, in_dtype="f32", page=32, seqs=5, q_lo=700, q_hi=2500, ctx_lo=0, ctx_hi=4000, mix=3),
        # one decode token at position 519 with the 1.1B model's heads: the smallest call
        dict(name="attend_one", op="attend", heads=32, kv=4, dim=64, out="f16", page=16, seqs=1, q_lo=1, q_hi=1,
             ctx_lo=519, ctx_hi=519, window=0, lse=False, mix=1),
        # a decode step of 64 sequences of very different lengths
        dict(name="attend_batch", op="attend", heads=32, kv=8, dim=128, out="bf16", page=64, seqs=64, q_lo=1, q_hi=1,
             ctx_lo=30, ctx_hi=8191, window=0, lse=False, mix=2),
        # a mixed step: ragged prompt pieces over a filled cache
        dict(name="attend_chunks", op="attend", heads=32, kv=8, dim=128, out="f16", page=16, seqs=6, q_lo=1, q_hi=700,
             ctx_lo=0, ctx_hi=6000, window=0, lse=True, mix=4),
        # a whole prompt at once
        dict(name="attend_prompt", op="attend", heads=32, kv=8, dim=128, out="bf16", page=32, seqs=1, q_lo=8191,
             q_hi=8191, ctx_lo=0, ctx_hi=0, window=0, lse=False, mix=6),
        # the pages that a decode step of 61 sequences wrote to
        dict(name="bounds_batch", op="bounds", heads=32, kv=8, dim=128, dtype="e4m3", page=64, seqs=61, q_lo=1, q_hi=1,
             ctx_lo=0, ctx_hi=9000, mix=2),
        # the pages that a prompt step wrote to, in a 16-bit cache
        dict(name="bounds_prompts", op="bounds", heads=32, kv=8, dim=128, dtype="bf16", page=32, seqs=5, q_lo=700,
             q_hi=2500, ctx_lo=0, ctx_hi=4000, mix=3),
        # one token against a long document in small pages
        dict(name="select_long", op="select", heads=32, kv=8, dim=128, dtype="f16", page=16, seqs=1, q_lo=1, q_hi=1,
             ctx_lo=131000, ctx_hi=131000, select=128, first=1, last=2, mix=3),
        # a decode step of 64 sequences over long texts
        dict(name="select_batch", op="select", heads=32, kv=8, dim=128, dtype="e4m3", page=64, seqs=64, q_lo=1, q_hi=1,
             ctx_lo=1000, ctx_hi=40000, select=32, first=1, last=2, mix=4),
        # the attention of one token over 2048 of its positions, the 1.1B model's heads
        dict(name="sparse_one", op="sparse", heads=32, kv=4, dim=64, dtype="f16", out="f16", page=16, seqs=1, q_lo=1,
             q_hi=1, ctx_lo=20000, ctx_hi=20000, select=128, lse=False, mix=5),
        # the attention of a decode step of 64 sequences over up to 2048 positions each
        dict(name="sparse_batch", op="sparse", heads=32, kv=8, dim=128, dtype="e4m3", out="bf16", page=64, seqs=64,
             q_lo=1, q_hi=1, ctx_lo=1000, ctx_hi=16000, select=32, lse=True, mix=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "bounds", "select", "sparse"))
    mix = rng.randrange(1 << 20)
    kv = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 128))
    heads = kv * rng.choice((1, 2, 3, 4, 5, 7, 8))
    page = rng.choice((16, 32, 64, 128, 256))
    c = dict(op=op, heads=heads, kv=kv, dim=dim, page=page, mix=mix)
    if op in ("append", "bounds"):
        tokens = _log(rng, 1, 8192)
        seqs = _log(rng, 1, min(64, tokens))
        c.update(seqs=seqs, q_lo=max(1, tokens // seqs // 2), q_hi=max(1, tokens // seqs), ctx_lo=0,
                 ctx_hi=_log(rng, 1, 6000))
        if op == "append":
            c.update(rope_dim=rng.choice((dim, dim, dim // 2)), interleaved=rng.random() < 0.5,
                     norm=rng.random() < 0.5, fused=rng.random() < 0.5, in_dtype=rng.choice(("f32", "f32", "f16", "bf16")))
        else:
            c.update(dtype=rng.choice(("e4m3", "e4m3", "f16", "bf16")))
        return c
    if op == "attend":
        while True:  # a drawn case costs no more than the largest listed one, padded as the plain form pads
            q_hi = rng.choice((1, 1, 4, _log(rng, 1, 4096)))
            seqs, ctx = _log(rng, 1, 64), _log(rng, 1, 100000)
            if seqs * (q_hi + ctx) * kv * dim <= 600_000_000 and seqs * q_hi * heads * (q_hi + ctx) <= 2_000_000_000:
                c.update(seqs=seqs, q_lo=max(1, q_hi // 3), q_hi=q_hi, ctx_lo=ctx // 8, ctx_hi=ctx,
                         window=rng.choice((0, 0, _log(rng, 16, 4096))), lse=rng.random() < 0.5,
                         out=rng.choice(("f16", "bf16", "bf16", "f32")))
                return c
    c.update(dtype=rng.choice(("e4m3", "e4m3", "f16", "bf16")))
    while True:
        seqs, ctx, q_hi, select = _log(rng, 1, 64), _log(rng, 100, 130000), rng.choice((1, 1, 1, 3)), _log(rng, 4, 256)
        pages = ctx // page + 1
        if op == "select":
            if seqs * q_hi * pages * kv * dim <= 64 * 626 * 1024:
                c.update(seqs=seqs, q_lo=1, q_hi=q_hi, ctx_lo=ctx // 8, ctx_hi=ctx, select=select,
                         first=rng.choice((0, 1, 1)), last=rng.choice((1, 2, 2)))
                return c
        elif seqs * q_hi * min(select, pages) * page * kv * dim <= 64 * 2048 * 1024 and seqs * ctx * kv * dim <= 600_000_000:
            c.update(seqs=seqs, q_lo=1, q_hi=q_hi, ctx_lo=ctx // 8, ctx_hi=ctx, select=select, lse=rng.random() < 0.5,
                     out=rng.choice((c["dtype"] if c["dtype"] != "e4m3" else "bf16", "f32")))
            return c


def _lengths(c):
    """New tokens and earlier positions of each sequence."""
    r = random.Random(c["mix"] * 7919 + c["seqs"])
    return [(r.randint(c["q_lo"], c["q_hi"]), r.randint(c["ctx_lo"], c["ctx_hi"])) for _ in range(c["seqs"])]


def _batch(c, gen, dev):
    """The batch: a shuffled page table, lengths, and of each token its sequence, its number there and its position."""
    lens = _lengths(c)
    need = [-(-(n + x) // c["page"]) for n, x in lens]
    n_pages, max_pages = sum(need) + 3, max(need)
    q_start = torch.tensor([0] + [n for n, _ in lens]).cumsum(0).to(torch.int32)
    kv_len = torch.tensor([n + x for n, x in lens], dtype=torch.int32)
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(c["seqs"], max_pages, dtype=torch.int32, device=dev)
    at = torch.arange(max_pages, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    table[at] = order[: sum(need)]
    seq = torch.repeat_interleave(torch.arange(c["seqs"]), q_start.diff().long())
    local = torch.arange(int(q_start[-1])) - q_start[seq].long()
    return dict(case=c, q_start=q_start.to(dev), kv_len=kv_len.to(dev), table=table, seq=seq.to(dev),
                local=local.to(dev), pos=(kv_len[seq] - q_start.diff()[seq] + local).to(dev), n_pages=n_pages,
                max_q=max(n for n, _ in lens), max_kv=max(n + x for n, x in lens), tokens=int(q_start[-1]))


def _scales(e):
    """E8M0 values of the exponents e."""
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _pools(c, n_pages, gen, dev, dtype):
    """Keys and values of about unit size, and their scales (None in a 16-bit cache)."""
    page, kv, dim = c["page"], c["kv"], c["dim"]
    if dtype != "e4m3":  # positions first
        pools = torch.empty(2, 1, n_pages, page, kv, dim, dtype=TYPES[dtype], device=dev)
        for p in pools.view(2, -1).split(1 << 28, dim=1):
            p.copy_(torch.empty(p.shape, dtype=p.dtype, device=dev).normal_(generator=gen))
        return dict(k_pages=pools[0], v_pages=pools[1])
    pools = torch.empty(2, 1, n_pages, kv, page, dim, dtype=torch.uint8, device=dev)  # heads first
    for p in pools.view(2, -1).split(1 << 28, dim=1):
        x = torch.empty(p.shape, device=dev).normal_(0.0, 96.0, generator=gen).clamp_(-448, 448)
        p.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
    e = torch.randint(-8, -5, (2, 1, n_pages, kv, page // BLOCK), generator=gen, device=dev)
    pools, e = pools.view(torch.float8_e4m3fn), _scales(e)
    return dict(k_pages=pools[0], v_pages=pools[1], k_scales=e[0], v_scales=e[1])


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    c = dict(case)
    st = _batch(c, gen, dev)
    dtype = c.get("dtype", "e4m3")
    h, kv, dim, n = c["heads"], c["kv"], c["dim"], st["tokens"]
    t = TYPES["f16" if dtype == "e4m3" else dtype]  # of the queries
    st.update(_pools(c, st["n_pages"], gen, dev, dtype))
    if c["op"] == "append":
        x = (torch.randn(n, (h + 2 * kv) * dim, generator=gen, device=dev) * 2).to(TYPES[c["in_dtype"]])
        q, k, v = x.split([h * dim, kv * dim, kv * dim], dim=1)
        if not c["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        norms = [torch.rand(dim, generator=gen, device=dev) + 0.5 for _ in range(2)] if c["norm"] else [None, None]
        st.update(q=q, k=k, v=v, q_norm=norms[0], k_norm=norms[1], q_out=torch.empty(n, h * dim, dtype=t, device=dev))
        return st
    # scores of a standard deviation of about two, as trained heads have
    st["q"] = (torch.randn(n, h * dim, generator=gen, device=dev) * 2).to(t)
    if c["op"] in ("bounds", "select"):
        b = torch.randn(2, 1, st["n_pages"], kv, dim, generator=gen, device=dev) * 30
        b = torch.stack([b.amax(0).ceil(), b.amin(0).floor()], dim=3).clamp(-127, 127).to(torch.int8)
        e = torch.randint(-6, -3, (1, st["n_pages"], kv), generator=gen, device=dev)
        st.update(bounds=b, bound_scales=_scales(e))
    if c["op"] == "select":
        st["pages"] = torch.empty(n, kv, c["select"], dtype=torch.int32, device=dev)
    if c["op"] == "sparse":
        # a random choice of each token's pages, the newest among them, in order
        m = st["table"].shape[1]
        held = st["pos"].long() // c["page"]
        rank = torch.rand(n, kv, m, generator=gen, device=dev)
        at = torch.arange(m, device=dev)
        rank = torch.where(at == held[:, None, None], 2.0, rank).masked_fill_(at > held[:, None, None], -1.0)
        width = min(c["select"], m)
        best = rank.topk(width, dim=2)
        pages = torch.where(best.values >= 0, best.indices, m).sort(2).values
        st["pages"] = torch.full((n, kv, c["select"]), -1, dtype=torch.int32, device=dev)
        st["pages"][:, :, :width] = torch.where(pages < m, pages, -1)
    if c["op"] in ("attend", "sparse"):
        st.update(out=torch.empty(n, h * dim, dtype=TYPES[c["out"]], device=dev),
                  lse=torch.empty(n, h, device=dev) if c["lse"] else None)
        # rows of a sequence's last page that nothing was written to hold whatever was there
        for s, (a, x) in enumerate(_lengths(c)):
            if (a + x) % c["page"]:
                last, row = st["table"][s, (a + x) // c["page"]].long(), (a + x) % c["page"]
                if dtype == "e4m3":
                    st["v_pages"].view(torch.uint8)[0, last, :, row:] = 0x7F
                else:
                    st["v_pages"][0, last, row:] = float("nan")
    return st


# ---- the plain forms ---------------------------------------------------------------------
def _norm(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _angles(pos, c):
    r = c["rope_dim"]
    f = 10000.0 ** (-2.0 * torch.arange(r // 2, device=pos.device, dtype=torch.float64) / r)
    a = pos.double()[:, None] * f
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, cos, sin, c):
    r = c["rope_dim"]
    y = x.clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _exponent(amax, mantissa, bits, lo, hi):
    """The least e in lo..hi with amax <= mantissa * 2^(bits + e), mantissa in [0.5, 1)."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, (x - bits + (m > mantissa)).clamp(lo, hi), lo)


def _store(x, pages, scales, st, c):
    """Quantises the rows x [tokens, kv, dim] into their blocks; earlier rows of a block whose scale grows are rescaled."""
    page, kv, dim = c["page"], c["kv"], c["dim"]
    pos = st["pos"].long()
    begins = (st["local"] == 0) | (pos % BLOCK == 0)
    of = begins.cumsum(0) - 1  # each token's block, counted over the batch
    p0 = pos[begins]
    where = st["table"][st["seq"][begins], p0 // page].long()
    block = (p0 % page) // BLOCK
    amax = torch.zeros(len(p0), kv, device=x.device).index_reduce_(0, of, x.abs().amax(-1), "amax")
    e = _exponent(amax, 0.875, 9, -40, 40)
    byte = scales.view(torch.uint8)[0]
    before = byte[where, :, block].int() - 127
    e = torch.where((p0 % BLOCK > 0)[:, None], torch.maximum(e, before), e)
    code = pages.view(torch.uint8)[0].view(-1, kv, page // BLOCK, BLOCK, dim)
    rows = code[where, :, block].view(torch.float8_e4m3fn).float()
    rows = torch.ldexp(rows, (before - e)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    earlier = torch.arange(BLOCK, device=x.device)[None] < (p0 % BLOCK)[:, None]
    code[where, :, block] = torch.where(earlier[:, None, :, None], rows, code[where, :, block])
    byte[where, :, block] = (e + 127).to(torch.uint8)
    y = torch.ldexp(x, -e[of][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    code[where[of], :, block[of], pos % BLOCK] = y


def _append(st):
    c = st["case"]
    n, dim = st["tokens"], c["dim"]
    cos, sin = _angles(st["pos"], c)
    q = _rotate(_norm(st["q"].float().reshape(n, -1, dim), st["q_norm"]), cos, sin, c)
    k = _rotate(_norm(st["k"].float().reshape(n, -1, dim), st["k_norm"]), cos, sin, c)
    _store(k, st["k_pages"], st["k_scales"], st, c)
    _store(st["v"].float().reshape(n, -1, dim), st["v_pages"], st["v_scales"], st, c)
    st["q_out"].copy_(q.reshape(n, -1))
    return _appended(st)


def _appended(st):
    return dict(q=st["q_out"], k_pages=st["k_pages"], v_pages=st["v_pages"], k_scales=st["k_scales"],
                v_scales=st["v_scales"])


def _values(st, name, pages):
    """Keys or values of the pages numbered by `pages`, in 32 bits: [*pages.shape, kv, page, dim]."""
    c, x = st["case"], st[name + "_pages"]
    if x.dtype != torch.float8_e4m3fn:
        return x[0][pages].transpose(-3, -2).float()
    f = x.view(torch.uint8)[0][pages].view(torch.float8_e4m3fn).float()
    e = st[name + "_scales"].view(torch.uint8)[0][pages].int() - 127
    return torch.ldexp(f, e.repeat_interleave(BLOCK, -1)[..., None])


def _attend(st):
    c = st["case"]
    h, kv, dim, page, dev = c["heads"], c["kv"], c["dim"], c["page"], st["q"].device
    nq, b, g = st["max_q"], c["seqs"], c["heads"] // c["kv"]
    nk = st["table"].shape[1] * page
    held = torch.arange(nk, device=dev)[None] < st["kv_len"][:, None]
    k, v = (_values(st, x, st["table"].long()).permute(0, 2, 1, 3, 4).reshape(b, kv, nk, dim) for x in "kv")
    v = v.masked_fill_(~held[:, None, :, None], 0.0)
    i = torch.arange(nq, device=dev)
    n_new = st["q_start"].diff()
    take = (st["q_start"][:-1, None] + i.clamp(max=nq)).clamp(max=st["tokens"] - 1).long()
    q = st["q"].view(-1, kv, g, dim)[take].float()
    s = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(b, kv, g * nq, dim), k.transpose(2, 3))
    s = s.view(b, kv, g, nq, nk).mul_(1.0 / math.sqrt(dim))
    pos = (st["kv_len"] - n_new)[:, None] + i
    j = torch.arange(nk, device=dev)
    seen = held[:, None] & (j <= pos[..., None])
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(b, kv, g * nq, nk), v).view(b, kv, g, nq, dim)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    st["out"].copy_(o.permute(0, 3, 1, 2, 4)[st["seq"], st["local"]].reshape(st["tokens"], h * dim))
    if not c["lse"]:
        return st["out"]
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)[st["seq"], st["local"]]
    st["lse"].copy_(lse.reshape(st["tokens"], h))
    return dict(out=st["out"], lse=st["lse"])


def _bounds(st):
    c = st["case"]
    page = c["page"]
    pos = st["pos"].long()
    begins = (st["local"] == 0) | (pos % page == 0)
    logical = pos[begins] // page
    where = st["table"][st["seq"][begins], logical].long()
    k = _values(st, "k", where)
    row = torch.arange(page, device=k.device)[None] + logical[:, None] * page
    off = (row >= st["kv_len"][st["seq"][begins], None])[:, None, :, None]
    top, least = k.masked_fill(off, float("-inf")).amax(2), k.masked_fill(off, float("inf")).amin(2)
    e = _exponent(torch.maximum(top.abs(), least.abs()).amax(-1), 127 / 128, 7, -100, 121)
    b = torch.stack([torch.ldexp(top, -e[..., None]).ceil(), torch.ldexp(least, -e[..., None]).floor()], dim=2)
    st["bounds"][0, where] = b.clamp(-127, 127).to(torch.int8)
    st["bound_scales"].view(torch.uint8)[0, where] = (e + 127).to(torch.uint8)
    return dict(bounds=st["bounds"], scales=st["bound_scales"])


def _select(st):
    c = st["case"]
    n, kv, dim, m = st["tokens"], c["kv"], c["dim"], st["table"].shape[1]
    q = st["q"].float().view(n, kv, -1, dim)
    eq = _exponent(q.abs().amax(-1), 127 / 128, 7, -100, 121)
    q = torch.ldexp(q, -eq[..., None]).round()
    table = st["table"].long()
    # (the integers' products and sums stay below 2^24, so 32-bit floats hold them exactly)
    per_seq = st["bounds"][0][table].float()
    eb = (st["bound_scales"].view(torch.uint8)[0][table].int() - 127).transpose(1, 2)[st["seq"]]
    top, least = (per_seq[:, :, :, i].permute(0, 2, 3, 1)[st["seq"]] for i in (0, 1))
    s = torch.matmul(q.clamp(min=0), top) + torch.matmul(q.clamp(max=0), least)
    s = torch.ldexp(s, (eq[..., None] + eb[:, :, None]).clamp(-100, 100)).amax(2)
    at = torch.arange(m, device=q.device)
    held = (st["pos"].long() // c["page"])[:, None, None]
    s.masked_fill_((at < c["first"]) | (at > held - c["last"]), float("inf"))
    s.masked_fill_(at > held, float("-inf"))
    value, index = s.sort(dim=2, descending=True, stable=True)
    width = min(c["select"], m)
    pages = torch.where(value[..., :width] > float("-inf"), index[..., :width], m).sort(2).values
    st["pages"].fill_(-1)
    st["pages"][..., :width] = torch.where(pages < m, pages, -1)
    return st["pages"]


def _sparse(st):
    c = st["case"]
    n, h, kv, dim, page = st["tokens"], c["heads"], c["kv"], c["dim"], c["page"]
    pages = st["pages"].long()
    width = pages.shape[2]
    where = st["table"].long()[st["seq"][:, None, None], pages.clamp(min=0)]
    head = torch.arange(kv, device=pages.device)[None, :, None]

    def rows(name):
        x = st[name + "_pages"]
        if x.dtype != torch.float8_e4m3fn:
            return x[0].transpose(1, 2)[where, head].float()
        f = x.view(torch.uint8)[0][where, head].view(torch.float8_e4m3fn).float()
        e = st[name + "_scales"].view(torch.uint8)[0][where, head].int() - 127
        return torch.ldexp(f, e.repeat_interleave(BLOCK, -1)[..., None])

    j = pages[..., None] * page + torch.arange(page, device=pages.device)
    seen = ((pages >= 0)[..., None] & (j <= st["pos"].long()[:, None, None, None])).view(n, kv, 1, -1)
    k = rows("k").view(n, kv, width * page, dim)
    v = rows("v").view(n, kv, width * page, dim).masked_fill_(~seen.transpose(2, 3), 0.0)
    s = torch.matmul(st["q"].float().view(n, kv, -1, dim), k.transpose(2, 3)).mul_(1.0 / math.sqrt(dim))
    s.masked_fill_(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v) / torch.where(total > 0, total, torch.ones_like(total))
    st["out"].copy_(o.reshape(n, h * dim))
    if not c["lse"]:
        return st["out"]
    st["lse"].copy_((top + total.log()).view(n, h))
    return dict(out=st["out"], lse=st["lse"])


# ---- the library's calls -------------------------------------------------------------------
def _own(st):
    from quant_dequant_gemv_gb300 import qdq

    c = st["case"]
    if "cache" not in st:  # made once for the pools, as a server does
        st["cache"] = qdq.PagedCache(st["k_pages"], st["v_pages"], c["heads"], rope_dim=c.get("rope_dim", c["dim"]),
                                     interleaved=c.get("interleaved", True), k_scales=st.get("k_scales"),
                                     v_scales=st.get("v_scales"))
        st["batch"] = qdq.PagedBatch(st["q_start"], st["kv_len"], st["table"], st["tokens"])
    cache, batch = st["cache"], st["batch"]
    if c["op"] == "append":
        cache.append(0, batch, st["q"], st["k"], st["v"], st["q_out"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS)
        return _appended(st)
    if c["op"] == "bounds":
        cache.key_bounds(0, batch, st["bounds"], st["bound_scales"])
        return dict(bounds=st["bounds"], scales=st["bound_scales"])
    if c["op"] == "select":
        cache.select_pages(0, batch, st["q"], st["bounds"], st["bound_scales"], st["pages"], first=c["first"],
                           last=c["last"])
        return st["pages"]
    if c["op"] == "attend":
        cache.attention(0, batch, st["q"], st["out"], window=c["window"], lse=st["lse"])
    else:
        cache.attention_pages(0, batch, st["q"], st["pages"], st["out"], lse=st["lse"])
    return dict(out=st["out"], lse=st["lse"]) if c["lse"] else st["out"]


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "bounds": _bounds, "select": _select,
            "sparse": _sparse}[state["case"]["op"]](state)


# ---- what a pass has to move and compute ----------------------------------------------------
def _page_bytes(c):
    """Bytes of one position of one head, keys and values, with their share of the scales."""
    return 2 * c["dim"] + 2 / BLOCK if c.get("dtype", "e4m3") == "e4m3" else 4 * c["dim"]


def work(case):
    c = case
    lens, page, kv, dim, h = _lengths(c), c["page"], c["kv"], c["dim"], c["heads"]
    tokens = sum(n for n, _ in lens)
    if c["op"] == "append":
        size = 4 if c["in_dtype"] == "f32" else 2
        return dict(bytes=tokens * ((h + 2 * kv) * dim * size + h * dim * 2 + kv * _page_bytes(c)),
                    flops=tokens * (h + 2 * kv) * dim * 6)
    if c["op"] == "bounds":
        rows = sum(n + x - x // page * page for n, x in lens)
        pages = sum((n + x - 1) // page - x // page + 1 for n, x in lens)
        return dict(bytes=kv * (rows * _page_bytes(c) / 2 + pages * (2 * dim + 1)), flops=rows * kv * dim * 2)
    if c["op"] == "select":
        pages = sum(-(-(n + x) // page) for n, x in lens)
        pairs = sum(n * -(-(n + x) // page) for n, x in lens)
        return dict(bytes=pages * kv * (2 * dim + 1) + tokens * (h * dim * 2 + kv * c["select"] * 4),
                    flops=pairs * h * dim * 4)
    io = tokens * h * (dim * (2 + (4 if c["out"] == "f32" else 2)) + (4 if c["lse"] else 0))
    if c["op"] == "sparse":
        pairs = 0
        for n, x in lens:
            for p in range(x, x + n):  # the newest page among the selected ones, as far as it is filled
                pairs += min((c["select"] - 1) * page, p // page * page) + p % page + 1
        return dict(bytes=pairs * kv * _page_bytes(c) + io + tokens * kv * c["select"] * 4, flops=4 * dim * h * pairs)
    w, pairs, rows = c["window"], 0, 0
    for n, x in lens:
        rows += n + (min(x, w - 1) if w else x)
        if not w:
            pairs += n * x + n * (n + 1) // 2
        else:
            pairs += sum(min(w, x + i + 1) for i in range(n))
    return dict(bytes=rows * kv * _page_bytes(c) + io, flops=4 * dim * h * pairs)


# ---- the definitions in 64 bits, sequence by sequence ----------------------------------------
def _exact_append(st):
    c = st["case"]
    dim, r, page = c["dim"], c["rope_dim"], c["page"]
    i = torch.arange(r // 2, device="cuda", dtype=torch.float64)
    turn = torch.polar(torch.ones_like(i)[None], st["pos"].double()[:, None] * torch.exp(-2 * i / r * math.log(10000.0)))

    def turned(x, w):
        x = x.double().reshape(st["tokens"], -1, dim)
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / dim + EPS).sqrt() * w.double()
        head, rest = x[..., :r], x[..., r:]
        pairs = head.unflatten(-1, (r // 2, 2)) if c["interleaved"] else head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
        head = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([head, rest], -1)

    found = dict(q=turned(st["q"], st["q_norm"]).reshape(st["tokens"], -1))
    for name, x in (("k", turned(st["k"], st["k_norm"])), ("v", st["v"].double().reshape(st["tokens"], -1, dim))):
        code = st[name + "_pages"].double()
        scale = torch.exp2(st[name + "_scales"].view(torch.uint8).double() - 127)
        for s, (n, p) in enumerate(_lengths(c)):
            at, end = int(st["q_start"][s]), p + n
            while p < end:  # block by block
                stop = min(end, p // BLOCK * BLOCK + BLOCK)
                rows = x[at : at + stop - p].transpose(0, 1)
                where, b, row = st["table"][s, p // page], p % page // BLOCK, p % BLOCK
                new = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / 448)).clamp(-40, 40))
                old = scale[0, where, :, b]
                if row:
                    new = torch.maximum(new, old)
                blk = code[0, where, :, b * BLOCK : (b + 1) * BLOCK]
                blk[:, :row] *= (old / new)[:, None, None]
                blk[:, row : row + stop - p] = rows / new[:, None, None]
                scale[0, where, :, b] = new
                at, p = at + stop - p, stop
        found[name + "_pages"], found[name + "_scales"] = code, scale
    return found


def _exact_rows(st, name, seq, n):
    """Keys or values of a sequence's first n positions in 64 bits: [kv, n, dim]."""
    c, x = st["case"], st[name + "_pages"]
    pages = st["table"][seq, : -(-n // c["page"])].long()
    if x.dtype != torch.float8_e4m3fn:
        return x[0, pages].flatten(0, 1)[:n].double().transpose(0, 1)
    x = x.view(torch.uint8)[0, pages].view(torch.float8_e4m3fn).double()
    e = st[name + "_scales"].view(torch.uint8)[0, pages].double() - 127
    x = x.unflatten(2, (-1, BLOCK)) * torch.exp2(e)[..., None, None]
    return x.flatten(2, 3).transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_attention(st):
    c = st["case"]
    dim, page, g = c["dim"], c["page"], c["heads"] // c["kv"]
    out = torch.zeros(st["tokens"], c["heads"], dim, dtype=torch.float64, device="cuda")
    lse = torch.full((st["tokens"], c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    q = st["q"].view(st["tokens"], c["heads"], dim)
    for s in range(c["seqs"]):
        a, b, n = int(st["q_start"][s]), int(st["q_start"][s + 1]), int(st["kv_len"][s])
        k, v = _exact_rows(st, "k", s, n), _exact_rows(st, "v", s, n).nan_to_num()
        j = torch.arange(n, device="cuda")
        p = torch.arange(n - (b - a), n, device="cuda")[:, None]
        hidden = j > p
        if c.get("window"):
            hidden = hidden | (j <= p - c["window"])
        for h in range(c["heads"]):
            off = hidden
            if c["op"] == "sparse":
                mine = torch.zeros(b - a, st["table"].shape[1] + 1, dtype=torch.bool, device="cuda")
                mine.scatter_(1, st["pages"][a:b, h // g].long().where(st["pages"][a:b, h // g] >= 0, mine.shape[1] - 1), True)
                off = hidden | ~mine[:, j // page]
            x = q[a:b, h].double() @ k[h // g].T / math.sqrt(dim)
            x.masked_fill_(off, -math.inf)
            e = torch.logsumexp(x, 1)
            out[a:b, h] = (x - e[:, None]).exp() @ v[h // g]
            lse[a:b, h] = e
    out = out.reshape(st["tokens"], -1)
    return dict(out=out, lse=lse) if c["lse"] else out


def exact(case, seed):
    if case["op"] in ("bounds", "select"):  # whole numbers
        return None
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attention(st)
