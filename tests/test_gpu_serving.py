"""The serving calls on the GPU against the float64 oracle (oracle/serving.py).

* Append. A stored value is the fp32 result rounded once: half a step of the pools' type
  (finfo.eps / 2 relative, and half a subnormal step for fp16), plus the fp32 arithmetic's own
  error: the norm (a 12-term sum, a reciprocal root, two products: 12 x 2^-24), the angle (its
  fraction of a turn kept to 32 bits and rounded to fp32: pi x 2^-25; sine and cosine within two
  ulps) and three rounded operations; 32 x 2^-24 of the pair's magnitudes covers them.
* Attention. Half a step of the output's type on the value; half a step of the pools' type on each
  weight, so that times sum a|v|; scores in fp32, off by at most 2 D 2^-24 max sum|q k| scale,
  which moves a weight by as much relatively, twice for the normalisation; 2^-20 for the
  exponentials and the rescalings; n 2^-24 for the sums over n positions; fp16 weights below
  2^-14 of the largest are subnormal, 2^-25 each, times sum|v|.
* Sampling. Tokens equal the oracle's, with the random number and top_p moved by 1e-5 either way
  allowed for: fp32 weights are off by a few 2^-24 times the exponent (below 40 here), 5e-6 of the
  mass at most. The log-probability follows within 2e-5.
"""
import numpy as np
import pytest

from oracle import serving as sv

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def qdq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quant_dequant_gemv_gb300 import build, qdq
    build.build()
    torch.cuda.set_device(0)
    return qdq


DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().cpu().double().numpy()


def make(qdq, lens, heads=4, kv=2, dim=64, page=16, dtype="f16", layers=1, seed=0, extra_tokens=0, spare=3,
         rope_dim=None, interleaved=True, fill=float("nan")):
    """A cache whose pools hold `fill` and a batch of (new, earlier) lengths with shuffled pages."""
    rng = np.random.default_rng(seed)
    need = [-(-max(n + x, 1) // page) for n, x in lens]
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages)
    table = np.full((len(lens), max(need)), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    pools = torch.full((2, layers, n_pages, page, kv, dim), fill, dtype=DT[dtype], device="cuda")
    q_start = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
    kv_len = np.array([n + x for n, x in lens], np.int32)
    tokens = int(q_start[-1]) + extra_tokens
    b = dict(rng=rng, q_start=q_start, kv_len=kv_len, table=table, tokens=tokens, pools=pools, dtype=dtype, dim=dim,
             heads=heads, kv=kv, page=page, n_pages=n_pages)
    b["cache"] = qdq.PagedCache(pools[0], pools[1], heads, rope_dim=rope_dim, interleaved=interleaved)
    b["batch"] = batch_of(qdq, b)
    return b


def batch_of(qdq, b):
    return qdq.PagedBatch(*(torch.from_numpy(b[k]).cuda() for k in ("q_start", "kv_len", "table")), b["tokens"])


def fill_held(b, layer=0, scale=1.0):
    """Random keys and values at every held position of the batch; the rest keeps its fill."""
    for s, n in enumerate(b["kv_len"]):
        for j in range(int(n)):
            at = sv.row_of(b["table"], b["n_pages"], b["page"], s, j)
            if at is not None:
                x = torch.from_numpy(b["rng"].standard_normal((2, b["kv"], b["dim"])) * scale).to(DT[b["dtype"]])
                b["pools"][:, layer, at[0], at[1]] = x.cuda()


# ---- append -------------------------------------------------------------------------------
def check_append(qdq, b, in_dtype, norm, rope_dim, interleaved, layer=0, fused=False, eps=1e-5):
    T, H, G, D = b["tokens"], b["heads"], b["kv"], b["dim"]
    x = torch.from_numpy(b["rng"].standard_normal((T, (H + 2 * G) * D)) * 2).to(DT[in_dtype]).cuda()
    q, k, v = x.split([H * D, G * D, G * D], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = [torch.from_numpy(b["rng"].uniform(0.5, 1.5, D).astype(np.float32)).cuda() if norm else None for _ in "qk"]
    q_out = torch.full((T, H * D), 7.0, dtype=DT[b["dtype"]], device="cuda")
    before = f64(b["pools"])
    b["cache"].append(layer, b["batch"], q, k, v, q_out, q_norm=w[0], k_norm=w[1], eps=eps)
    assert qdq.get_device_status() == 0
    wn = [None if a is None else f64(a) for a in w]
    want_q, want = sv.append(f64(q), f64(k), f64(v), b["q_start"], b["kv_len"], b["table"], b["n_pages"], b["page"], D,
                             rope_dim, interleaved, q_norm=wn[0], k_norm=wn[1], eps=eps)
    half = torch.finfo(DT[b["dtype"]]).eps / 2
    tiny = 2.0 ** -25 if b["dtype"] == "f16" else 0.0

    def close(got, ref, turned, what):
        size = np.abs(ref)
        if turned and rope_dim:
            r, n = rope_dim, ref.shape[-1]
            i = np.arange(n)
            mate = np.where(i < r, i ^ 1 if interleaved else (i + r // 2) % r, i)
            size = np.hypot(size, size[:, mate]) * 2
        err = np.abs(got - ref)
        d = 32 * 2.0 ** -24 * size
        assert (err <= half * (np.abs(ref) + d) + d + tiny).all(), f"{what}: {err.max()}"

    got_q = f64(q_out).reshape(T, H, D)
    for t in range(T):
        if t in want_q:
            close(got_q[t], want_q[t], True, f"q of token {t}")
        else:
            assert (got_q[t] == 7).all(), f"token {t} is of no sequence"
    got = f64(b["pools"])
    touched = np.zeros(got.shape, bool)
    for (page, row), (kr, vr) in want.items():
        close(got[0, layer, page, row], kr, True, f"k at {page}, {row}")
        close(got[1, layer, page, row], vr, False, f"v at {page}, {row}")
        touched[:, layer, page, row] = True
    assert np.array_equal(got[~touched], before[~touched], equal_nan=True), "rows of no new token were written"


@pytest.mark.parametrize("dtype,in_dtype", [("f16", "f32"), ("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("dim,heads,kv", [(64, 4, 2), (128, 3, 1), (64, 7, 7), (128, 32, 1)])
@pytest.mark.parametrize("interleaved,part,norm", [(True, 1, True), (False, 1, False), (True, 2, False), (False, 2, True),
                                                   (False, 0, True)])
def test_append(qdq, dtype, in_dtype, dim, heads, kv, interleaved, part, norm):
    rope_dim = dim // part if part else 0
    b = make(qdq, [(1, 0), (5, 30), (0, 12), (33, 0), (1, 77)], heads, kv, dim, 16, dtype, rope_dim=rope_dim,
             interleaved=interleaved, seed=dim + heads, extra_tokens=2)
    check_append(qdq, b, in_dtype, norm, rope_dim, interleaved, fused=norm)


def test_append_one_token_and_a_second_layer(qdq):
    b = make(qdq, [(1, 518)], 32, 4, 64, 128, "f16", layers=3)
    check_append(qdq, b, "f32", False, 64, True, layer=2)


def test_append_many_sequences(qdq):
    lens = [(int(n), int(x)) for n, x in np.random.default_rng(5).integers(0, 3, (700, 2))]
    b = make(qdq, lens, 2, 1, 64, 16, "bf16", seed=3, interleaved=False)
    check_append(qdq, b, "f32", True, 64, False, fused=True)


def test_append_far_positions(qdq):
    """At a position near 2^29 the angles are still those of the formula."""
    far = (1 << 29) - 5
    b = make(qdq, [(3, 0)], 4, 2, 64, 256, "f16")
    pages = 1 << 21
    b["kv_len"] = np.array([far], np.int32)
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    at = (far - 1) // 256
    table[0, at] = 1

    class Far:  # the oracle's table: two million entries, one of them held
        shape = (1, pages)

        def __getitem__(self, key):
            return 1 if key[1] == at else -1
    b["table"] = Far()
    b["batch"] = qdq.PagedBatch(torch.from_numpy(b["q_start"]).cuda(), torch.from_numpy(b["kv_len"]).cuda(), table, 3)
    check_append(qdq, b, "f32", False, 64, True)


def test_append_bad_pages_and_negative_positions(qdq):
    b = make(qdq, [(40, 0), (6, 20), (9, 0)], 4, 2, 64, 16, "f16", seed=9)
    b["table"][0, 1], b["table"][1, 1] = -5, b["n_pages"]     # absent pages
    b["kv_len"][2] = 4                                         # the first five of its nine tokens lie before 0
    b["batch"] = batch_of(qdq, b)
    check_append(qdq, b, "f32", True, 64, True)


# ---- attention ----------------------------------------------------------------------------
def check_attention(qdq, b, window=0, scale=None, layer=0, out_dtype=None, q_scale=1.5, sample=None, pad=0,
                    weight_half=None):
    T, H, D = b["tokens"], b["heads"], b["dim"]
    scale = D ** -0.5 if scale is None else scale
    wide = torch.from_numpy(b["rng"].standard_normal((T, H * D + pad)) * q_scale).to(DT[b["dtype"]]).cuda()
    q = wide[:, :H * D]
    out = torch.full((T, H * D + pad), 7.0, dtype=DT[out_dtype or b["dtype"]], device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    b["cache"].attention(layer, b["batch"], q, out[:, :H * D], scale=scale, window=window, lse=lse)
    assert qdq.get_device_status() == 0
    ref, ref_lse, spread, reach = sv.attention(f64(q).reshape(T, H, D), f64(b["pools"][0, layer]),
                                               f64(b["pools"][1, layer]), b["q_start"], b["kv_len"], b["table"], scale,
                                               window)
    got, got_lse = f64(out[:, :H * D]).reshape(T, H, D), f64(lse)
    none = np.isnan(ref_lse)
    assert (got[none] == 7).all() and (got_lse[none] == 7).all(), "rows of no sequence were written"
    assert (f64(out[:, H * D:]) == 7).all()
    half = torch.finfo(DT[b["dtype"]]).eps / 2 if weight_half is None else weight_half
    half_out = torch.finfo(out.dtype).eps / 2
    n = int(b["kv_len"].max())
    ds = 2 * D * 2.0 ** -24 * reach
    v_max = np.nanmax(np.abs(f64(b["pools"][1, layer])), initial=0.0, where=np.isfinite(f64(b["pools"][1, layer])))
    tol = half_out * np.abs(ref) + (half + 2 * ds[..., None] + 2.0 ** -20 + n * 2.0 ** -24) * spread
    tol = tol + (n * 2.0 ** -25 * v_max if b["dtype"] == "f16" else 0.0) + 1e-30
    live = ~none
    err = np.abs(got - ref)
    assert np.isfinite(got[live]).all(), "a masked position reached the result"
    bad = np.argwhere(live[..., None] & ~(err <= tol))
    assert not len(bad), f"{len(bad)} of {err.size} out of tolerance, first {bad[0]}: {got[tuple(bad[0])]} vs {ref[tuple(bad[0])]}"
    empty = live & (ref_lse == -np.inf)
    assert (got[empty] == 0).all() and (got_lse[empty] == -np.inf).all()
    some = live & ~empty
    tol_l = 2 * ds + 2.0 ** -20 + n * 2.0 ** -24 + np.abs(ref_lse) * 2.0 ** -22
    assert (np.abs(got_lse[some] - ref_lse[some]) <= tol_l[some]).all()
    return out


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv,page", [(64, 4, 4, 16), (64, 8, 2, 32), (128, 8, 1, 64), (128, 6, 2, 16),
                                               (64, 5, 1, 128), (128, 32, 1, 256)])
@pytest.mark.parametrize("lens", [[(1, 0)], [(1, 130), (1, 0), (1, 257), (0, 9), (1, 15)], [(37, 0), (1, 200), (70, 61)],
                                  [(150, 150)]])
def test_attention(qdq, dtype, dim, heads, kv, page, lens):
    b = make(qdq, lens, heads, kv, dim, page, dtype, seed=dim + page, extra_tokens=1)
    fill_held(b)
    check_attention(qdq, b)


@pytest.mark.parametrize("window", [1, 16, 100, 129, 5000])
@pytest.mark.parametrize("lens", [[(1, 300)], [(90, 200), (1, 128), (260, 0)]])
def test_attention_window(qdq, window, lens):
    b = make(qdq, lens, 4, 2, 64, 16, "f16", seed=window)
    fill_held(b)
    check_attention(qdq, b, window=window)


def test_attention_fp32_output_strides_scale_and_layer(qdq):
    b = make(qdq, [(20, 50), (1, 90)], 4, 2, 128, 32, "bf16", layers=2, seed=4)
    fill_held(b, layer=1)
    check_attention(qdq, b, layer=1, out_dtype="f32", scale=0.3, pad=64)


def test_attention_bad_pages_and_empty_rows(qdq):
    b = make(qdq, [(40, 100), (1, 150), (9, 0), (3, 40)], 4, 2, 64, 16, "f16", seed=9)
    b["table"][0, 2], b["table"][1, 0], b["table"][1, 5] = -5, b["n_pages"], 1 << 30
    b["table"][3, :] = -1                                      # nothing to attend to
    b["kv_len"][2] = 4                                         # five tokens before position 0
    b["batch"] = batch_of(qdq, b)
    fill_held(b)
    check_attention(qdq, b)
    check_attention(qdq, b, window=30)


def test_attention_kv_len_past_the_table(qdq):
    b = make(qdq, [(4, 60), (1, 30)], 4, 2, 64, 16, "bf16", seed=2)
    fill_held(b)
    b["kv_len"] = np.array([70, 31], np.int32)                 # positions 64..69 have no page
    b["batch"] = batch_of(qdq, b)
    check_attention(qdq, b)


def test_attention_large_scores_and_infinite_stale_values(qdq):
    """Scores in the hundreds (a nearly one-hot softmax), stale rows of infinities."""
    for fill in (float("inf"), float("-inf")):
        b = make(qdq, [(30, 200), (1, 333)], 8, 2, 64, 32, "bf16", seed=6, fill=fill)
        fill_held(b, scale=8.0)
        check_attention(qdq, b, q_scale=8.0)


def test_attention_rising_and_falling_scores(qdq):
    """Keys that grow along the sequence raise the running maximum in every tile."""
    for sign in (1, -1):
        b = make(qdq, [(1, 1500), (140, 500)], 8, 2, 128, 64, "f16", seed=8)
        fill_held(b)
        for s, n in enumerate(b["kv_len"]):
            for j in range(int(n)):
                pg, rw = sv.row_of(b["table"], b["n_pages"], b["page"], s, j)
                b["pools"][0, 0, pg, rw] *= 1 + 3 * (j if sign > 0 else int(n) - j) / int(n)
        check_attention(qdq, b)


@pytest.mark.parametrize("kv_len", [1000, 4097, 20000])
def test_attention_long_single_tokens(qdq, kv_len):
    """One token over a long cache (the positions are split over CTAs and joined)."""
    b = make(qdq, [(1, kv_len - 1), (2, 700)], 8, 2, 128, 128, "f16", seed=kv_len)
    at = torch.randn(2, 1, b["n_pages"], b["page"], 2, 128, device="cuda").half()
    b["pools"].copy_(at)
    check_attention(qdq, b)


def test_attention_is_repeatable_and_reads_its_batch_when_it_runs(qdq):
    """The same call twice gives the same bits; a captured graph follows the batch's arrays."""
    b = make(qdq, [(1, 2000), (60, 400), (1, 9)], 8, 2, 64, 16, "bf16", seed=1)
    b["pools"].copy_(torch.randn(b["pools"].shape, device="cuda"))
    H, D, T = 8, 64, b["tokens"]
    q = torch.randn(T, H * D, device="cuda").bfloat16()
    o = [torch.zeros(T, H * D, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    for x in o[:2]:
        b["cache"].attention(0, b["batch"], q, x)
    assert torch.equal(o[0], o[1])
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        b["cache"].attention(0, b["batch"], q, o[2])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o[0], o[2])
    kv = b["batch"]._keep[1]
    kv[0] = 1200
    g.replay()
    b["cache"].attention(0, b["batch"], q, o[1])
    torch.cuda.synchronize()
    assert torch.equal(o[1], o[2]) and not torch.equal(o[0], o[2])
    assert qdq.get_device_status() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,window", [([(23, 1200), (55, 900)], 1000), ([(19, 3000), (40, 700), (3, 400)], 0)])
def test_attention_partly_filled_tiles_are_repeatable(qdq, dim, lens, window):
    """Tiles of rows in which whole warps have none: many passes, each with the oracle's result."""
    b = make(qdq, lens, 32, 4, dim, 16, "f16", seed=17)
    b["pools"].copy_(torch.randn(b["pools"].shape, device="cuda"))
    first = check_attention(qdq, b, window=window)
    q = torch.from_numpy(b["rng"].standard_normal((b["tokens"], 32 * dim))).half().cuda()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    outs = [torch.zeros_like(first) for _ in range(2)]
    b["cache"].attention(0, b["batch"], q, outs[0], window=window)
    for _ in range(400):
        outs[1].zero_()
        b["cache"].attention(0, b["batch"], q, outs[1], window=window)
        wrong += (outs[0] != outs[1]).any()
    assert int(wrong) == 0 and qdq.get_device_status() == 0


@pytest.mark.parametrize("lens", [[(1, 700)], [(1, 130), (1, 0), (1, 2000), (16, 300), (3, 900)]])
def test_attention_of_few_rows_keeps_what_the_weights_rounding_leaves(qdq, lens):
    """At 128 dims an fp16 weight is held in two terms, the second rounded by half a step of half a step."""
    b = make(qdq, lens, 16, 2, 128, 16, "f16", seed=31)
    fill_held(b)
    check_attention(qdq, b, out_dtype="f32", weight_half=(torch.finfo(torch.float16).eps / 2) ** 2)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [8, 14])
def test_attention_of_a_sequence_keeps_its_bits_whatever_its_neighbours_ask(qdq, heads, dim):
    """The rows of a tile after a sequence's last one hold the next sequence's queries."""
    b = make(qdq, [(5, 1500), (7, 1400)] * 20, heads, 2, dim, 16, "f16", seed=23)
    b["pools"].copy_(torch.randn(b["pools"].shape, device="cuda"))
    q = torch.from_numpy(b["rng"].standard_normal((b["tokens"], heads * dim))).half().cuda()
    mine = torch.from_numpy(np.arange(b["tokens"]) % 12 < 5).cuda()
    got = []
    for loud in (0.0, 12.0):
        x = torch.where(mine[:, None], q, q * loud)
        out, lse = torch.zeros_like(x), torch.zeros(b["tokens"], heads, device="cuda")
        b["cache"].attention(0, b["batch"], x, out, lse=lse)
        got.append((out[mine], lse[mine]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert qdq.get_device_status() == 0


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_is_repeatable_where_heads_do_not_fill_a_tile(qdq, dim):
    """Seven heads to a key head: 126 of a tile's 128 rows are of the sequence."""
    b = make(qdq, [(202, 1), (335, 0), (570, 2), (607, 1)] * 3, 14, 2, dim, 128, "f16", seed=29)
    b["pools"].copy_(torch.randn(b["pools"].shape, device="cuda"))
    q = 2 * torch.from_numpy(b["rng"].standard_normal((b["tokens"], 14 * dim))).half().cuda()
    out, other, junk = (torch.zeros_like(q) for _ in range(3))
    b["cache"].attention(0, b["batch"], q, out, window=263)
    for k in range(20):
        b["cache"].attention(0, b["batch"], q * (1 + k), junk, window=263)
        b["cache"].attention(0, b["batch"], q, other, window=263)
        assert torch.equal(out, other), k


@pytest.mark.parametrize("lens", [[(1, 0)], [(1, 700), (3, 5)], [(300, 40)]])
def test_attention_keeps_a_query_that_is_no_number_to_itself(qdq, lens):
    b = make(qdq, lens, 8, 2, 128, 32, "bf16", seed=5)
    fill_held(b)
    T = b["tokens"]
    q = torch.from_numpy(b["rng"].standard_normal((T, 8 * 128))).bfloat16().cuda()
    out, clean = (torch.zeros(T, 8 * 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.zeros(T, 8, device="cuda")
    b["cache"].attention(0, b["batch"], q, clean)
    q[T - 1, 3 * 128 + 7] = float("nan")
    b["cache"].attention(0, b["batch"], q, out, lse=lse)
    got = out.view(T, 8, 128)
    assert got[T - 1, 3].isnan().all() and lse[T - 1, 3].isnan()
    got[T - 1, 3] = clean.view(T, 8, 128)[T - 1, 3]
    assert torch.equal(out, clean)


def test_attention_without_any_page(qdq):
    b = make(qdq, [(3, 0), (1, 9)], 4, 2, 64, 16, "f16")
    b["batch"] = qdq.PagedBatch(torch.from_numpy(b["q_start"]).cuda(), torch.from_numpy(b["kv_len"]).cuda(),
                                torch.zeros(2, 0, dtype=torch.int32, device="cuda"), 4)
    q = torch.ones(4, 256, dtype=torch.float16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((4, 4), 7.0, device="cuda")
    b["cache"].attention(0, b["batch"], q, out, lse=lse)
    assert (out == 0).all() and (lse == -float("inf")).all()
    k = torch.ones(4, 128, dtype=torch.float16, device="cuda")
    b["cache"].append(0, b["batch"], q, k, k, out)
    assert out.isfinite().all() and b["pools"].isnan().all()


def test_a_step_in_a_graph(qdq):
    """Append, attention and sampling captured together, replayed on other tokens and lengths."""
    b = make(qdq, [(9, 0), (1, 70)], 4, 2, 64, 16, "f16", seed=21, spare=9)
    fill_held(b)
    T, V = b["tokens"], 5000
    rng = np.random.default_rng(1)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()
    q, k, v, w = new(T, 256), new(T, 128), new(T, 128), new(256, V)
    q16, att = (torch.zeros(T, 256, dtype=t, device="cuda") for t in (torch.float16, torch.float32))
    logits, u = torch.zeros(T, V, device="cuda"), torch.full((T,), 0.6, device="cuda")
    top_p = torch.full((T,), 0.8, device="cuda")
    tokens = [torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(2)]
    torch.mm(att, w, out=logits)  # (the matrix product's own first call)

    def step(out):
        b["cache"].append(0, b["batch"], q, k, v, q16)
        b["cache"].attention(0, b["batch"], q16, att)
        torch.mm(att, w, out=logits)
        qdq.sample(logits, u, out, top_p=top_p)

    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        step(tokens[0])
    for n in range(3):
        q.normal_()
        k.normal_()
        b["batch"]._keep[1][1] = 71 - 9 * n
        g.replay()
        torch.cuda.synchronize()
        step(tokens[1])
        torch.cuda.synchronize()
        assert torch.equal(tokens[0], tokens[1]) and qdq.get_device_status() == 0


def test_append_then_attention_on_a_side_stream(qdq):
    b = make(qdq, [(12, 0), (1, 0)], 4, 2, 64, 16, "f16", seed=12)
    T, H, G, D = 13, 4, 2, 64
    rng = np.random.default_rng(0)
    q, k, v = (torch.from_numpy(rng.standard_normal((T, n * D)).astype(np.float32)).cuda() for n in (H, G, G))
    q_out, out = (torch.empty(T, H * D, dtype=torch.float16, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b["cache"].append(0, b["batch"], q, k, v, q_out, stream=s)
    b["cache"].attention(0, b["batch"], q_out, out, stream=s)
    s.synchronize()
    ref, _, spread, _ = sv.attention(f64(q_out).reshape(T, H, D), f64(b["pools"][0, 0]), f64(b["pools"][1, 0]), b["q_start"],
                                     b["kv_len"], b["table"], D ** -0.5)
    assert (np.abs(f64(out).reshape(T, H, D) - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -10 * spread + 1e-6).all()


def test_paged_refusals(qdq):
    b = make(qdq, [(3, 0)], 4, 2, 64, 16, "f16")
    c, batch = b["cache"], b["batch"]
    new = lambda n, w, t=torch.float16: torch.zeros(n, w, dtype=t, device="cuda")
    q, k, out = new(3, 256), new(3, 128), new(3, 256)

    def refused(code, f):
        with pytest.raises(qdq.QdqError) as e:
            f()
        assert e.value.rc == code

    refused(-2, lambda: c.attention(1, batch, q, out))
    refused(-2, lambda: c.attention(-1, batch, q, out))
    refused(-2, lambda: c.attention(0, batch, q, out, window=-1))
    refused(-2, lambda: c.attention(0, batch, q, out, scale=float("nan")))
    refused(-1, lambda: c.attention(0, batch, q, new(3, 256, torch.bfloat16)))
    refused(-1, lambda: c.append(0, batch, *(x.bfloat16() for x in (q, k, k)), out))
    refused(-2, lambda: c.append(0, batch, q, k, k, out, eps=-1.0))
    refused(-4, lambda: c.attention(0, batch, q.cpu(), out))
    refused(-4, lambda: c.append(0, batch, q, k.cpu(), k, out))
    refused(-3, lambda: c.attention(0, batch, new(4, 257)[:, 1:][:3], out))
    refused(-3, lambda: c.attention(0, batch, new(4, 257)[:, :256][:3], out))
    many = qdq.PagedBatch(torch.zeros(1026, dtype=torch.int32).cuda(), torch.zeros(1025, dtype=torch.int32).cuda(),
                          torch.zeros(1025, 1, dtype=torch.int32).cuda(), 3)
    refused(-8, lambda: c.attention(0, many, q, out))
    host = qdq.PagedBatch(*(torch.from_numpy(b[n]) for n in ("q_start", "kv_len", "table")), 3)
    refused(-4, lambda: c.attention(0, host, q, out))
    for bad in (lambda: c.attention(0, batch, q[:2], out), lambda: c.attention(0, batch, q.float(), out),
                lambda: c.append(0, batch, q, q, k, out), lambda: c.attention(0, batch, q, out, lse=new(3, 4))):
        with pytest.raises(ValueError):
            bad()
    none = qdq.PagedBatch(torch.zeros(1, dtype=torch.int32).cuda(), torch.zeros(0, dtype=torch.int32).cuda(),
                          torch.zeros(0, 1, dtype=torch.int32).cuda(), 0)
    c.attention(0, none, q, out)                               # nothing to do
    c.append(0, none, q, k, k, out)
    refused(-4, lambda: qdq.sample(torch.zeros(2, 8), torch.zeros(2, device="cuda"),
                                   torch.zeros(2, dtype=torch.int64, device="cuda")))


# ---- sampling -----------------------------------------------------------------------------
def check_sample(qdq, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, stride=None):
    B, V = logits.shape
    dev = lambda a, t: None if a is None else torch.from_numpy(np.broadcast_to(a, B).astype(t)).cuda()
    if stride:
        wide = torch.full((B, stride), float("inf"), dtype=logits.dtype, device="cuda")
        wide[:, :V] = logits
        logits = wide[:, :V]
    tokens = torch.full((B,), -9, dtype=torch.int64, device="cuda")
    logp = torch.full((B,), 7.0, device="cuda")
    qdq.sample(logits, dev(u, np.float32), tokens, temperature=dev(temperature, np.float32), top_k=dev(top_k, np.int32),
               top_p=dev(top_p, np.float32), min_p=dev(min_p, np.float32), logprobs=logp)
    x, tok, lp = f64(logits), tokens.cpu().numpy(), f64(logp)
    at = lambda a, r, d: d if a is None else float(np.float32(np.broadcast_to(a, B)[r]))
    for r in range(B):
        p, m = at(top_p, r, 1.0), at(min_p, r, 0.0)

        def fits(du, dp, dm):
            token, share = sv.sample(x[r], min(max(at(u, r, 0) + du, 0), 1), at(temperature, r, 1.0),
                                     int(at(top_k, r, 0)), p + dp, m + dm * m)
            return token == tok[r] and (share == lp[r] or abs(share - lp[r]) <= 2e-5)

        moves = (0, -1e-5, 1e-5)
        assert any(fits(du, dp, dm) for du in moves for dp in (moves if 0 < p < 1 else (0,))
                   for dm in (moves if 0 < m < 1 else (0,))), f"row {r}: token {tok[r]}, log-probability {lp[r]}"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 31, 1000, 4097, 32000, 131071, 262144])
def test_sample(qdq, dtype, vocab):
    rng = np.random.default_rng(vocab)
    B = 9
    x = torch.from_numpy(rng.standard_normal((B, vocab)) * rng.uniform(0.5, 4, (B, 1))).to(DT[dtype]).cuda()
    u = rng.uniform(0, 1, B).astype(np.float32)
    check_sample(qdq, x, u)
    check_sample(qdq, x, u, temperature=rng.uniform(0.3, 2, B), top_k=rng.integers(0, 60, B),
                 top_p=rng.uniform(0.1, 1.2, B), min_p=rng.uniform(0, 0.2, B), stride=vocab + 5)
    check_sample(qdq, x, u, top_p=rng.uniform(0.05, 0.999, B))
    check_sample(qdq, x, u, temperature=0.7, top_k=rng.integers(1, max(2, vocab), B))
    check_sample(qdq, x, u, temperature=[0.0, 1.0, -1.0] * 3, min_p=0.01)


def test_sample_ties_and_extremes(qdq):
    V = 3001
    rng = np.random.default_rng(3)
    x = torch.zeros(8, V)
    x[1] = torch.from_numpy(rng.integers(0, 4, V) * 1.0)       # four values, many ties
    x[2, 5:] = float("-inf")
    x[3] = float("-inf")
    x[3, 2999] = -1e30
    x[4] = float("nan")
    x[4, 17] = -3.0
    x[5] = torch.finfo(torch.float32).min                      # a mask's lowest value everywhere but one
    x[5, 100] = 0.0
    x[6] = -0.0
    x[6, ::2] = 0.0
    x[7] = torch.from_numpy(rng.standard_normal(V) * 1e4)
    x = x.cuda()
    u = np.array([0.5, 0.31, 0.7, 0.2, 0.9, 0.99, 0.25, 0.6], np.float32)
    check_sample(qdq, x, u)
    check_sample(qdq, x, u, top_k=7)
    check_sample(qdq, x, u, top_p=0.3)
    check_sample(qdq, x, u, top_k=900, top_p=0.33, min_p=0.001)
    check_sample(qdq, x, u, top_p=0.0)
    check_sample(qdq, x, np.zeros(8, np.float32), top_k=3)
    check_sample(qdq, x, np.ones(8, np.float32), top_k=3)
    check_sample(qdq, x, u, temperature=0.0)
    check_sample(qdq, x, u, min_p=2.0)
    check_sample(qdq, x, u, top_k=V + 10)


def test_sample_rows_with_nothing(qdq):
    x = torch.full((3, 50), float("-inf"), device="cuda")
    x[1] = float("nan")
    x[2, 3] = 1.0
    tokens = torch.zeros(3, dtype=torch.int64, device="cuda")
    logp = torch.zeros(3, device="cuda")
    u = torch.full((3,), 0.5, device="cuda")
    qdq.sample(x, u, tokens, logprobs=logp, top_p=torch.full((3,), 0.9, device="cuda"))
    assert tokens.tolist() == [-1, -1, 3] and logp.tolist() == [float("-inf"), float("-inf"), 0.0]


def test_sample_follows_the_distribution(qdq):
    """Evenly spaced random numbers give each token its share of the mass."""
    V, B = 40, 4000
    rng = np.random.default_rng(11)
    row = rng.standard_normal(V).astype(np.float32) * 2
    x = torch.from_numpy(row).cuda().expand(B, V).contiguous()
    u = torch.from_numpy(((np.arange(B) + 0.5) / B).astype(np.float32)).cuda()
    tokens = torch.empty(B, dtype=torch.int64, device="cuda")
    qdq.sample(x, u, tokens, top_k=torch.full((B,), 12, dtype=torch.int32, device="cuda"))
    keep = np.argsort(-row, kind="stable")[:12]
    w = np.zeros(V)
    w[keep] = np.exp(row[keep].astype(np.float64))
    share = np.bincount(tokens.cpu().numpy(), minlength=V) / B
    assert np.abs(share - w / w.sum()).max() <= 1.5 / B


@pytest.mark.parametrize("dtype,vocab", [("f32", 50000), ("bf16", 200003)])
def test_sample_wide_cuts(qdq, dtype, vocab):
    """Kept sets from a handful of entries to most of the row: both sides of the gathered list's
    length, cuts in the open bin, and 16-bit logits whose cuts fall among thousands of ties."""
    rng = np.random.default_rng(vocab)
    B = 10
    x = torch.from_numpy(rng.standard_normal((B, vocab)) * np.linspace(0.3, 6, B)[:, None]).to(DT[dtype]).cuda()
    for k in (1, 2, 1500, 2047, 2048, 2049, 2500, vocab // 2, vocab - 1):
        check_sample(qdq, x, rng.uniform(0, 1, B).astype(np.float32), top_k=k, temperature=rng.uniform(0.2, 2, B))
    for p in (0.01, 0.3, 0.6, 0.9, 0.96, 0.999, 0.999999):
        check_sample(qdq, x, rng.uniform(0, 1, B).astype(np.float32), top_p=p, temperature=rng.uniform(0.2, 2, B))
        check_sample(qdq, x, rng.uniform(0, 1, B).astype(np.float32), top_p=p, top_k=5000, min_p=0.02)


def test_sample_extreme_parameters(qdq):
    """Temperatures near the ends of fp32, random numbers outside [0, 1), a top-k far in the open bin."""
    rng = np.random.default_rng(8)
    B, V = 6, 20011
    x = torch.from_numpy(rng.standard_normal((B, V)) * 3).float()
    x[1, ::3] = float("-inf")
    x = x.cuda()
    u = rng.uniform(0, 1, B).astype(np.float32)
    check_sample(qdq, x, u, temperature=[1e-30, 1e30, 0.02, 0.05, 50.0, 1.0], top_k=[0, 9000, 15000, 500, 19000, 20010])
    check_sample(qdq, x, u, temperature=[1e30, 1e30, 1e6, 300.0, 50.0, 10.0], top_p=[0.5, 0.9, 0.99, 0.25, 0.999, 0.01])
    check_sample(qdq, x, np.float32([-3.0, 1.5, 0.0, 1.0, -1e-9, 2.0]), top_k=40)
