"""The serving operators' cases: cache append, attention over a paged cache, sampling.

A case says which operator it is and its sizes. `run` computes it with elementary torch
operations in binary32 (binary64 for angles and for the sums that decide a token), or, with
`own` set, through the library's public calls. Ragged lengths come from the case's own fields.
"""
import math
import random

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # one decode token of the 1.1B model's heads (32 query, 4 kv, 64 wide): pure latency
        dict(name="append_one", op="append", heads=32, kv=4, dim=64, rope_dim=64, interleaved=True, norm=False,
             fused=False, dtype="f16", in_dtype="f32", page=16, seqs=1, q_lo=1, q_hi=1, ctx_lo=99, ctx_hi=99, mix=1),
        # one token each of a batch of 61 sequences, heads of an 8B model, normed heads, fused qkv rows
        dict(name="append_batch", op="append", heads=32, kv=8, dim=128, rope_dim=128, interleaved=False, norm=True,
             fused=True, dtype="bf16", in_dtype="f32", page=64, seqs=61, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=9000, mix=2),
        # a prompt step: five ragged prompts, about 8000 new tokens in all
        dict(name="append_prompts", op="append", heads=32, kv=8, dim=128, rope_dim=96, interleaved=False, norm=True,
             fused=True, dtype="bf16", in_dtype="f32", page=32, seqs=5, q_lo=700, q_hi=2500, ctx_lo=0, ctx_hi=4000, mix=3),
        # one decode token at position 519 with the 1.1B model's heads: the smallest call
        dict(name="attend_one", op="attend", heads=32, kv=4, dim=64, dtype="f16", page=16, seqs=1, q_lo=1, q_hi=1,
             ctx_lo=519, ctx_hi=519, window=0, lse=False, mix=1),
        # a decode step of 64 sequences of very different lengths
        dict(name="attend_batch", op="attend", heads=32, kv=8, dim=128, dtype="bf16", page=64, seqs=64, q_lo=1, q_hi=1,
             ctx_lo=30, ctx_hi=8191, window=0, lse=False, mix=2),
        # one token against a long document
        dict(name="attend_long", op="attend", heads=32, kv=8, dim=128, dtype="f16", page=128, seqs=1, q_lo=1, q_hi=1,
             ctx_lo=131000, ctx_hi=131000, window=0, lse=True, mix=3),
        # a mixed step: ragged prompt pieces over a filled cache
        dict(name="attend_chunks", op="attend", heads=32, kv=8, dim=128, dtype="f16", page=16, seqs=6, q_lo=1, q_hi=700,
             ctx_lo=0, ctx_hi=6000, window=0, lse=False, mix=4),
        # prompts of the 1.1B model's heads with a sliding window
        dict(name="attend_window", op="attend", heads=32, kv=4, dim=64, dtype="f16", page=16, seqs=3, q_lo=700,
             q_hi=2100, ctx_lo=0, ctx_hi=3000, window=1000, lse=True, mix=5),
        # a whole prompt at once
        dict(name="attend_prompt", op="attend", heads=32, kv=8, dim=128, dtype="bf16", page=32, seqs=1, q_lo=8191,
             q_hi=8191, ctx_lo=0, ctx_hi=0, window=0, lse=False, mix=6),
        # the next token of one sequence, 32000 words
        dict(name="sample_one", op="sample", rows=1, vocab=32000, dtype="f32", mix=1),
        # a decode step of 64 sequences, every filter in use
        dict(name="sample_batch", op="sample", rows=64, vocab=32000, dtype="f32", mix=2),
        # a large batch over a large, odd vocabulary
        dict(name="sample_wide", op="sample", rows=256, vocab=131071, dtype="f32", mix=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "sample"))
    mix = rng.randrange(1 << 20)
    if op == "sample":
        while True:
            rows, vocab = _log(rng, 1, 300), _log(rng, 1000, 140000)
            if rows * vocab <= 256 * 131071:
                return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(("f32", "f32", "bf16", "f16")), mix=mix)
    kv = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 128))
    heads = kv * rng.choice((1, 2, 3, 4, 5, 7, 8))
    page = rng.choice((16, 32, 64, 128, 256))
    dtype = rng.choice(("f16", "bf16"))
    if op == "append":
        tokens = _log(rng, 1, 8192)
        seqs = _log(rng, 1, min(64, tokens))
        return dict(op=op, heads=heads, kv=kv, dim=dim, rope_dim=rng.choice((dim, dim, dim // 2)),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.5, fused=rng.random() < 0.5, dtype=dtype,
                    in_dtype=rng.choice(("f32", "f32", dtype)), page=page, seqs=seqs, q_lo=max(1, tokens // seqs // 2),
                    q_hi=max(1, tokens // seqs), ctx_lo=0, ctx_hi=_log(rng, 1, 6000), mix=mix)
    while True:  # a drawn case costs no more than the largest listed one, padded as the plain form pads
        q_hi = rng.choice((1, 1, 4, _log(rng, 1, 4096)))
        seqs, ctx = _log(rng, 1, 64), _log(rng, 1, 100000)
        if seqs * (q_hi + ctx) * kv * dim <= 600_000_000 and seqs * q_hi * heads * (q_hi + ctx) <= 2_000_000_000:
            return dict(op=op, heads=heads, kv=kv, dim=dim, dtype=dtype, page=page, seqs=seqs, q_lo=max(1, q_hi // 3),
                        q_hi=q_hi, ctx_lo=ctx // 8, ctx_hi=ctx, window=rng.choice((0, 0, _log(rng, 16, 4096))),
                        lse=rng.random() < 0.5, mix=mix)


def _lengths(c):
    """New tokens and earlier positions of each sequence."""
    r = random.Random(c["mix"] * 7919 + c["seqs"])
    return [(r.randint(c["q_lo"], c["q_hi"]), r.randint(c["ctx_lo"], c["ctx_hi"])) for _ in range(c["seqs"])]


def _paged(c, gen, dev):
    """The cache and the batch: page pools, a shuffled page table, lengths."""
    lens = _lengths(c)
    page, kv, dim, t = c["page"], c["kv"], c["dim"], TYPES[c["dtype"]]
    need = [-(-(n + x) // page) for n, x in lens]
    n_pages, max_pages = sum(need) + 3, max(need)
    q_start = torch.tensor([0] + [n for n, _ in lens]).cumsum(0).to(torch.int32)
    kv_len = torch.tensor([n + x for n, x in lens], dtype=torch.int32)
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(c["seqs"], max_pages, dtype=torch.int32, device=dev)
    at = torch.arange(max_pages, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    table[at] = order[: sum(need)]
    pools = torch.empty(2, 1, n_pages, page, kv, dim, dtype=t, device=dev)
    for p in pools.view(2, -1).split(1 << 28, dim=1):
        p.copy_(torch.empty(p.shape, dtype=t, device=dev).normal_(generator=gen))
    seq = torch.repeat_interleave(torch.arange(c["seqs"]), q_start.diff().long())
    local = torch.arange(int(q_start[-1])) - q_start[seq].long()
    return dict(case=c, k_pages=pools[0], v_pages=pools[1], q_start=q_start.to(dev), kv_len=kv_len.to(dev), table=table,
                seq=seq.to(dev), local=local.to(dev), pos=(kv_len[seq] - q_start.diff()[seq] + local).to(dev),
                max_q=max(n for n, _ in lens), max_kv=max(n + x for n, x in lens), tokens=int(q_start[-1]))


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    c = dict(case)
    if c["op"] == "sample":
        b, v = c["rows"], c["vocab"]
        width = 1 + 2 * torch.rand(b, 1, generator=gen, device=dev)  # peaked and flat rows
        logits = (torch.randn(b, v, generator=gen, device=dev) * width).to(TYPES[c["dtype"]])
        pick = torch.rand(4, b, generator=gen, device=dev)
        # a batch mixes greedy rows and rows with any of the filters
        top_k = torch.where(pick[0] < 0.6, (pick[0] * 120).int() + 1, torch.zeros_like(pick[0], dtype=torch.int32)).to(torch.int32)
        top_p = torch.where(pick[1] < 0.7, 0.6 + 0.5 * pick[1], torch.ones_like(pick[1]))
        min_p = torch.where(pick[2] < 0.3, 0.2 * pick[2], torch.zeros_like(pick[2]))
        temperature = torch.where(pick[3] < 0.1, torch.zeros_like(pick[3]), 0.4 + pick[3])
        if b == 1:
            top_k.fill_(40), top_p.fill_(0.95), min_p.fill_(0.0), temperature.fill_(0.8)
        return dict(case=c, logits=logits, top_k=top_k, top_p=top_p, min_p=min_p, temperature=temperature,
                    u=torch.rand(b, generator=gen, device=dev), tokens=torch.empty(b, dtype=torch.int64, device=dev),
                    logprobs=torch.empty(b, device=dev))
    st = _paged(c, gen, dev)
    h, kv, dim, t, n = c["heads"], c["kv"], c["dim"], TYPES[c["dtype"]], st["tokens"]
    if c["op"] == "append":
        ti = TYPES[c["in_dtype"]]
        x = (torch.randn(n, (h + 2 * kv) * dim, generator=gen, device=dev) * 2).to(ti)
        q, k, v = x.split([h * dim, kv * dim, kv * dim], dim=1)
        if not c["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        norms = [torch.rand(dim, generator=gen, device=dev) + 0.5 for _ in range(2)] if c["norm"] else [None, None]
        st.update(q=q, k=k, v=v, q_norm=norms[0], k_norm=norms[1], q_out=torch.empty(n, h * dim, dtype=t, device=dev))
        return st
    # scores of a standard deviation of about two, as trained heads have
    q = (torch.randn(n, h * dim, generator=gen, device=dev) * 2).to(t)
    st.update(q=q, out=torch.empty_like(q), lse=torch.empty(n, h, device=dev) if c["lse"] else None)
    # rows of a sequence's last page that nothing was written to hold whatever was there
    for s, (a, x) in enumerate(_lengths(c)):
        if (a + x) % c["page"]:
            st["v_pages"][0, st["table"][s, (a + x) // c["page"]].long(), (a + x) % c["page"]:] = float("nan")
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


def _append(st):
    c = st["case"]
    n, dim, page = st["tokens"], c["dim"], c["page"]
    cos, sin = _angles(st["pos"], c)
    q = _rotate(_norm(st["q"].float().reshape(n, -1, dim), st["q_norm"]), cos, sin, c)
    k = _rotate(_norm(st["k"].float().reshape(n, -1, dim), st["k_norm"]), cos, sin, c)
    at = st["table"][st["seq"], (st["pos"] // page).long()].long() * page + st["pos"].long() % page
    st["k_pages"].view(-1, c["kv"], dim)[at] = k.to(st["k_pages"].dtype)
    st["v_pages"].view(-1, c["kv"], dim)[at] = st["v"].reshape(n, -1, dim).to(st["v_pages"].dtype)
    st["q_out"].copy_(q.reshape(n, -1))
    return dict(q=st["q_out"], k_pages=st["k_pages"], v_pages=st["v_pages"])


def _attend(st):
    c = st["case"]
    h, kv, dim, page, dev = c["heads"], c["kv"], c["dim"], c["page"], st["q"].device
    nq, nk, b, g = st["max_q"], st["max_kv"], c["seqs"], c["heads"] // c["kv"]
    j = torch.arange(nk, device=dev)
    held = j[None] < st["kv_len"][:, None]
    rows = st["table"][:, (j // page)].long() * page + j % page
    k = st["k_pages"].view(-1, kv, dim)[rows].float()
    v = st["v_pages"].view(-1, kv, dim)[rows].float().masked_fill_(~held[:, :, None, None], 0.0)
    i = torch.arange(nq, device=dev)
    n_new = st["q_start"].diff()
    take = (st["q_start"][:-1, None] + i.clamp(max=nq)).clamp(max=st["tokens"] - 1).long()
    q = st["q"].view(-1, kv, g, dim)[take].float()
    s = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(b, kv, g * nq, dim), k.permute(0, 2, 3, 1))
    s = s.view(b, kv, g, nq, nk).mul_(1.0 / math.sqrt(dim))
    pos = (st["kv_len"] - n_new)[:, None] + i
    seen = held[:, None] & (j <= pos[..., None])
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(b, kv, g * nq, nk), v.permute(0, 2, 1, 3)).view(b, kv, g, nq, dim)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    pick = o.permute(0, 3, 1, 2, 4)[st["seq"], st["local"]].reshape(st["tokens"], h * dim)
    st["out"].copy_(pick)
    if not c["lse"]:
        return st["out"]
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)[st["seq"], st["local"]]
    st["lse"].copy_(lse.reshape(st["tokens"], h))
    return dict(out=st["out"], lse=st["lse"])


def _sample(st):
    x = st["logits"].float()
    x = torch.where(x.isnan(), float("-inf"), x)
    greedy = st["temperature"] <= 0
    inverse = 1.0 / torch.where(greedy, torch.ones_like(st["temperature"]), st["temperature"])
    z, order = x.sort(dim=1, descending=True, stable=True)
    w = ((z - z[:, :1]) * inverse[:, None]).exp().double()  # weights in 32 bits, their sums in 64
    rank = torch.arange(x.shape[1], device=x.device)[None]
    k = torch.where(greedy, 1, torch.where(st["top_k"] > 0, st["top_k"], x.shape[1]))
    w.masked_fill_(rank >= k[:, None], 0.0)
    mass = w.cumsum(1)
    p = st["top_p"].double()[:, None]
    w.masked_fill_((mass - w >= p * mass[:, -1:]) & (p < 1) & (rank > 0), 0.0)
    w.masked_fill_(w < st["min_p"].clamp(max=1.0)[:, None], 0.0)
    kept = torch.zeros_like(w).scatter_(1, order, w)
    run_mass = kept.cumsum(1)
    total = run_mass[:, -1:]
    token = (run_mass <= st["u"].double()[:, None] * total).sum(1, keepdim=True)
    st["tokens"].copy_(token[:, 0])
    st["logprobs"].copy_((kept.gather(1, token) / total).log()[:, 0])
    return dict(token=st["tokens"], logprob=st["logprobs"])


# ---- the library's calls -------------------------------------------------------------------
def _own(st):
    from quant_dequant_gemv_gb300 import qdq

    c = st["case"]
    if c["op"] == "sample":
        qdq.sample(st["logits"], st["u"], st["tokens"], temperature=st["temperature"], top_k=st["top_k"],
                   top_p=st["top_p"], min_p=st["min_p"], logprobs=st["logprobs"])
        return dict(token=st["tokens"], logprob=st["logprobs"])
    if "cache" not in st:  # made once for the pools, as a server does
        st["cache"] = qdq.PagedCache(st["k_pages"], st["v_pages"], c["heads"], rope_dim=c.get("rope_dim", c["dim"]),
                                     interleaved=c.get("interleaved", True))
        st["batch"] = qdq.PagedBatch(st["q_start"], st["kv_len"], st["table"], st["tokens"])
    if c["op"] == "append":
        st["cache"].append(0, st["batch"], st["q"], st["k"], st["v"], st["q_out"], q_norm=st["q_norm"],
                           k_norm=st["k_norm"], eps=EPS)
        return dict(q=st["q_out"], k_pages=st["k_pages"], v_pages=st["v_pages"])
    st["cache"].attention(0, st["batch"], st["q"], st["out"], window=c["window"], lse=st["lse"])
    return dict(out=st["out"], lse=st["lse"]) if c["lse"] else st["out"]


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "sample": _sample}[state["case"]["op"]](state)


# ---- what a pass has to move and compute ----------------------------------------------------
def work(case):
    c = case
    if c["op"] == "sample":
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=c["rows"] * (c["vocab"] * size + 32), flops=c["rows"] * c["vocab"] * 4)
    lens = _lengths(c)
    tokens = sum(n for n, _ in lens)
    if c["op"] == "append":
        values = tokens * (c["heads"] + 2 * c["kv"]) * c["dim"]
        return dict(bytes=values * ((4 if c["in_dtype"] == "f32" else 2) + 2), flops=values * 6)
    w, pairs, rows = c["window"], 0, 0
    for n, x in lens:
        rows += n + (min(x, w - 1) if w else x)
        if not w:
            pairs += n * x + n * (n + 1) // 2
        else:
            pairs += sum(min(w, x + i + 1) for i in range(n))
    return dict(bytes=rows * c["kv"] * c["dim"] * 4 + tokens * c["heads"] * (c["dim"] * 4 + (4 if c["lse"] else 0)),
                flops=4 * c["dim"] * c["heads"] * pairs)


# ---- the definitions in 64 bits, sequence by sequence ----------------------------------------
def _exact_sample(st):
    tokens, logs = [], []
    for b in range(st["case"]["rows"]):
        x = st["logits"][b].double()
        t, u = float(st["temperature"][b]), float(st["u"][b])
        if t <= 0:
            tokens.append(int(torch.nonzero(x == x.max())[0, 0]))
            logs.append(0.0)
            continue
        w = ((x - x.max()) / t).exp()
        by = torch.argsort(x, descending=True, stable=True)
        n = int(st["top_k"][b])
        by = by[:n] if n > 0 else by
        p = float(st["top_p"][b])
        if p < 1:
            before = w[by].cumsum(0) - w[by]
            n = int((before < p * w[by].sum()).sum())
            by = by[: max(n, 1)]
        by = by[w[by] >= float(st["min_p"][b])].sort().values
        mass = w[by].cumsum(0)
        at = min(int((mass <= u * mass[-1]).sum()), len(by) - 1)
        tokens.append(int(by[at]))
        logs.append(float((w[by[at]] / mass[-1]).log()))
    return dict(token=torch.tensor(tokens, device="cuda"), logprob=torch.tensor(logs, dtype=torch.float64, device="cuda"))


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

    k, v = turned(st["k"], st["k_norm"]), st["v"].double().reshape(st["tokens"], -1, dim)
    k_pages, v_pages = st["k_pages"].double(), st["v_pages"].double()
    for s in range(c["seqs"]):
        a, b = int(st["q_start"][s]), int(st["q_start"][s + 1])
        where = st["pos"][a:b].long()
        pages = st["table"][s].long()[where // page]
        k_pages[0, pages, where % page] = k[a:b]
        v_pages[0, pages, where % page] = v[a:b]
    return dict(q=turned(st["q"], st["q_norm"]).reshape(st["tokens"], -1), k_pages=k_pages, v_pages=v_pages)


def _exact_attend(st):
    c = st["case"]
    dim, page, g = c["dim"], c["page"], c["heads"] // c["kv"]
    out = torch.zeros(st["tokens"], c["heads"], dim, dtype=torch.float64, device="cuda")
    lse = torch.full((st["tokens"], c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    q = st["q"].view(st["tokens"], c["heads"], dim)
    for s in range(c["seqs"]):
        a, b, n = int(st["q_start"][s]), int(st["q_start"][s + 1]), int(st["kv_len"][s])
        pages = st["table"][s, : -(-n // page)].long()
        k = st["k_pages"][0, pages].flatten(0, 1)[:n]
        v = st["v_pages"][0, pages].flatten(0, 1)[:n]
        j = torch.arange(n, device="cuda")
        p = torch.arange(n - (b - a), n, device="cuda")[:, None]
        hidden = (j > p) | ((j <= p - c["window"]) if c["window"] else torch.zeros_like(j > p))
        for h in range(c["heads"]):
            x = q[a:b, h].double() @ k[:, h // g].double().T / math.sqrt(dim)
            x.masked_fill_(hidden, -math.inf)
            e = torch.logsumexp(x, 1)
            out[a:b, h] = (x - e[:, None]).exp() @ v[:, h // g].double()
            lse[a:b, h] = e
    out = out.reshape(st["tokens"], -1)
    return dict(out=out, lse=lse) if c["lse"] else out


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](st)
