"""The calls over a cache of e4m3 values and over chosen pages, on the GPU against the float64 oracle
(oracle/serving.py).

* Append. A scale is the oracle's, but where the largest value lies within the fp32 arithmetic's
  error of a power of two's border (then one exponent either way). A stored value is off by half a
  step: 2^-4 of it, or half e4m3's smallest step, 2^-10 * 2^e; the fp32 arithmetic before that by
  what tests/test_gpu_serving.py derives. Earlier rows of a block are rescaled to the bit.
* Attention. As there, with the weights in two fp16 terms (one, where blocks of many rows have a
  16-bit result): each is off by 2^-22 (2^-11) of itself and 2^-32 of the row's largest (its
  value's scale in it), which meets at most 448 * 2^e; t = s * c + e
  is rounded with |e| in it, which is counted as 4 * 2^-24 * |e| beside the scores' own error.
* Bounds and selections are whole numbers: equal.
"""
import numpy as np
import pytest

from oracle import serving as sv
from tests import test_gpu_serving as base
from tests.test_gpu_serving import DT, batch_of, f64, qdq  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def make(qdq, lens, heads=4, kv=2, dim=64, page=16, dtype="e4m3", layers=1, seed=0, extra_tokens=0, spare=3, rope_dim=None,
         interleaved=True, fill=0x7F, exponents=(-9, -5)):
    """A cache of e4m3 values whose pools hold `fill` (a NaN), and a batch; or base.make's of 16 bits."""
    if dtype != "e4m3":
        b = base.make(qdq, lens, heads, kv, dim, page, dtype, layers, seed, extra_tokens, spare, rope_dim, interleaved)
        b["q_dtype"] = b["dtype"]
        return b
    rng = np.random.default_rng(seed)
    need = [-(-max(n + x, 1) // page) for n, x in lens]
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages)
    table = np.full((len(lens), max(need)), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    pools = torch.full((2, layers, n_pages, kv, page, dim), fill, dtype=torch.uint8, device="cuda")
    e = rng.integers(*exponents, (2, layers, n_pages, kv, page // 16)) + 127
    q_start = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
    b = dict(rng=rng, q_start=q_start, kv_len=np.array([n + x for n, x in lens], np.int32), table=table,
             tokens=int(q_start[-1]) + extra_tokens, pools=pools, scales=torch.from_numpy(e.astype(np.uint8)).cuda(),
             dtype=dtype, q_dtype="f16", dim=dim, heads=heads, kv=kv, page=page, n_pages=n_pages)
    b["cache"] = qdq.PagedCache(*pools.view(torch.float8_e4m3fn), heads, rope_dim=rope_dim, interleaved=interleaved,
                                k_scales=b["scales"][0], v_scales=b["scales"][1].view(torch.float8_e8m0fnu))
    b["batch"] = batch_of(qdq, b)
    return b


def fill_held(b, layer=0, scale=1.0):
    """Random codes at every held position (values of about unit size), or base.fill_held's."""
    if b["dtype"] != "e4m3":
        return base.fill_held(b, layer, scale)
    host = b["pools"].cpu().numpy()
    for s, n in enumerate(b["kv_len"]):
        for j in range(int(n)):
            at = sv.row_of(b["table"], b["n_pages"], b["page"], s, j)
            if at is not None:
                x = np.clip(b["rng"].standard_normal((2, b["kv"], b["dim"])) * 96 * scale, -448, 448)
                host[:, layer, at[0], :, at[1]] = sv.e4m3_byte(x)
    b["pools"].copy_(torch.from_numpy(host))


def values(b, layer=0):
    """Keys and values [n_pages, page, kv, dim] in float64."""
    if b["dtype"] != "e4m3":
        return f64(b["pools"][0, layer]), f64(b["pools"][1, layer])
    codes, scales = b["pools"].cpu().numpy(), b["scales"].cpu().numpy()
    return tuple(sv.values_e4m3(codes[i, layer], scales[i, layer]) for i in range(2))


# ---- append -------------------------------------------------------------------------------
def check_append(qdq, b, in_dtype="f32", norm=False, rope_dim=None, interleaved=True, layer=0, fused=False, x=None, eps=1e-5):
    T, H, G, D = b["tokens"], b["heads"], b["kv"], b["dim"]
    rope_dim = D if rope_dim is None else rope_dim
    if x is None:
        x = b["rng"].standard_normal((T, (H + 2 * G) * D)) * 2
    x = torch.from_numpy(x).to(DT[in_dtype]).cuda()
    q, k, v = x.split([H * D, G * D, G * D], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = [torch.from_numpy(b["rng"].uniform(0.5, 1.5, D).astype(np.float32)).cuda() if norm else None for _ in "qk"]
    q_out = torch.full((T, H * D), 7.0, dtype=torch.float16, device="cuda")
    before, scales_before = b["pools"].cpu().numpy(), b["scales"].cpu().numpy()
    b["cache"].append(layer, b["batch"], q, k, v, q_out, q_norm=w[0], k_norm=w[1], eps=eps)
    assert qdq.get_device_status() == 0
    wn = [None if a is None else f64(a) for a in w]
    # the rows in float64, and what the fp32 arithmetic may be off by (tests/test_gpu_serving.py)
    turned, slack = np.zeros((2, T, G, D)), np.zeros((2, T, G, D))
    got_q = f64(q_out).reshape(T, H, D)
    told = np.zeros(T, bool)
    i = np.arange(D)
    mate = np.where(i < rope_dim, i ^ 1 if interleaved else (i + rope_dim // 2) % max(rope_dim, 1), i)
    d = lambda ref: 32 * 2.0 ** -24 * np.hypot(np.abs(ref), np.abs(ref[..., mate])) * 2
    for t, s, p in sv.tokens_of(b["q_start"], b["kv_len"], T):
        told[t] = True
        qh = sv.head_norm(f64(q[t]).reshape(H, D), wn[0], eps)
        ref = sv.rotate(qh, p, rope_dim, interleaved, 10000.0) if p >= 0 else np.zeros_like(qh)
        ref = np.clip(ref, -65504, 65504)
        assert (np.abs(got_q[t] - ref) <= 2.0 ** -11 * (np.abs(ref) + d(ref)) + d(ref) + 2.0 ** -25)[np.isfinite(ref)].all(), f"q of token {t}"
        turned[0, t] = sv.rotate(sv.head_norm(f64(k[t]).reshape(G, D), wn[1], eps), p, rope_dim, interleaved, 10000.0)
        turned[1, t] = f64(v[t]).reshape(G, D)
        slack[0, t] = d(turned[0, t])
    assert (got_q[~told] == 7).all()
    codes, scales = b["pools"].cpu().numpy(), b["scales"].cpu().numpy()
    for i in range(2):
        want, want_s, exact = sv.append_e4m3(turned[i], before[i, layer], scales_before[i, layer], b["q_start"], b["kv_len"],
                                             b["table"], T)
        off = np.argwhere(scales[i, layer] != want_s)
        for pg, g, blk in off:  # the border's other side, if the largest value is as near to it as that
            near = [np.abs(np.log2(np.abs(y).max() / 448) - np.round(np.log2(np.abs(y).max() / 448))) for (p_, g_, r), y in exact.items()
                    if (p_, g_, r // 16) == (pg, g, blk)]
            assert i == 0 and min(near) < 2.0 ** -16 and abs(int(scales[i, layer, pg, g, blk]) - int(want_s[pg, g, blk])) == 1
        touched = np.zeros(want.shape, bool)
        pos_of = {}
        for t, s, p in sv.tokens_of(b["q_start"], b["kv_len"], T):
            at = sv.row_of(b["table"], b["n_pages"], b["page"], s, p)
            if at is not None:
                pos_of[at] = t
        for (pg, g, r), y in exact.items():
            e = float(want_s[pg, g, r // 16]) - float(scales[i, layer, pg, g, r // 16])
            y = y * 2.0 ** e
            got = sv.E4M3[codes[i, layer, pg, g, r]]
            unit = 2.0 ** (127.0 - float(scales[i, layer, pg, g, r // 16]))
            lim = np.clip(y, -448, 448)
            tol = 2.0 ** -4 * np.abs(lim) + 2.0 ** -10 + slack[i, pos_of[pg, r], g] * unit * 1.0625
            ok = np.where(np.isnan(y), np.isnan(got), np.abs(got - lim) <= tol)
            assert ok.all(), (i, pg, g, r, got[~ok][:3], y[~ok][:3])
            touched[pg, g, r] = True
        if not len(off):
            assert np.array_equal(codes[i, layer][~touched], want[~touched]), "earlier rows, or rows of no new token"
        rest = [x for x in range(codes.shape[1]) if x != layer]
        assert np.array_equal(codes[i, rest], before[i, rest]) and np.array_equal(scales[i, rest], scales_before[i, rest])


@pytest.mark.parametrize("in_dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv,page", [(64, 4, 2, 16), (128, 3, 1, 32), (64, 7, 7, 256), (128, 32, 1, 64)])
@pytest.mark.parametrize("interleaved,part,norm", [(True, 1, True), (False, 1, False), (True, 2, False), (False, 2, True),
                                                   (False, 0, True)])
def test_append(qdq, in_dtype, dim, heads, kv, page, interleaved, part, norm):
    rope_dim = dim // part if part else 0
    b = make(qdq, [(1, 0), (5, 30), (0, 12), (33, 0), (1, 77), (17, 15)], heads, kv, dim, page, rope_dim=rope_dim,
             interleaved=interleaved, seed=dim + heads, extra_tokens=2)
    fill_held(b)
    check_append(qdq, b, in_dtype, norm, rope_dim, interleaved, fused=norm)


def test_append_a_second_layer(qdq):
    b = make(qdq, [(1, 518)], 32, 4, 64, 128, layers=3)
    check_append(qdq, b, layer=2)


def test_append_many_sequences_and_a_long_prompt(qdq):
    """Over 2048 tokens, where a CTA takes a window of them: blocks that reach over windows' ends."""
    lens = [(int(n), int(x)) for n, x in np.random.default_rng(5).integers(0, 40, (120, 2))]
    b = make(qdq, lens + [(700, 5)], 2, 1, 64, 16, seed=3, interleaved=False, extra_tokens=3)
    assert b["tokens"] >= 2048
    fill_held(b)
    check_append(qdq, b, "bf16", True, 64, False, fused=True)


@pytest.mark.parametrize("dim,kv", [(64, 2), (128, 1)])
def test_append_token_by_token(qdq, dim, kv):
    """A sequence that grows by pieces, with sizes that make scales grow inside blocks."""
    b = make(qdq, [(0, 0), (0, 20)], 2 * kv, kv, dim, 32, seed=7)
    b["table"] = np.array([[0, 1, -1], [2, 4, 3]], np.int32)
    kv_len = np.array([0, 20])
    fill_held(b)
    for step, new in enumerate([(1, 0), (1, 1), (3, 1), (1, 5), (0, 1), (20, 1), (1, 1), (16, 16), (30, 1)]):
        kv_len = kv_len + new
        b["q_start"], b["kv_len"] = np.array([0, new[0], sum(new)], np.int32), kv_len.astype(np.int32)
        b["tokens"] = sum(new)
        b["batch"] = batch_of(qdq, b)
        x = b["rng"].standard_normal((sum(new), 4 * kv * dim)) * 2.0 ** b["rng"].integers(-12, 12, (sum(new), 1))
        check_append(qdq, b, x=x)


def test_append_extreme_values(qdq):
    """Zeros, values beyond the exponents' range, infinities and NaN, and beyond fp16's range in q."""
    for scale in (0.0, 1e-30, 1e-12, 1e12, 1e30):
        b = make(qdq, [(20, 3), (1, 0)], 2, 1, 64, 16, seed=1, rope_dim=0)
        fill_held(b)
        check_append(qdq, b, rope_dim=0, x=b["rng"].standard_normal((21, 4 * 64)) * scale)
    b = make(qdq, [(20, 0)], 2, 1, 64, 16, seed=1, rope_dim=0)
    x = b["rng"].standard_normal((20, 4 * 64))
    x[3, 128:140], x[4, 200], x[5, 130], x[6, 5] = np.inf, -np.inf, np.nan, 1e9
    check_append(qdq, b, rope_dim=0, x=x)


def test_append_bad_pages_and_negative_positions(qdq):
    b = make(qdq, [(40, 0), (6, 20), (9, 0), (20, 100)], 4, 2, 64, 16, seed=9)
    b["table"][0, 1], b["table"][1, 1] = -5, b["n_pages"]     # absent pages
    b["kv_len"][2] = 4                                         # the first five of its nine tokens lie before 0
    b["kv_len"][3] = b["table"].shape[1] * 16 + 4              # the last four lie past the table
    b["batch"] = batch_of(qdq, b)
    check_append(qdq, b, norm=True)


# ---- attention ----------------------------------------------------------------------------
def check_attention(qdq, b, window=0, scale=None, layer=0, out_dtype="f32", q_scale=1.5, pad=0, lists=None, q=None):
    T, H, D = b["tokens"], b["heads"], b["dim"]
    scale = D ** -0.5 if scale is None else scale
    if q is None:
        q = torch.from_numpy(b["rng"].standard_normal((T, H * D + pad)) * q_scale).to(DT[b["q_dtype"]]).cuda()[:, :H * D]
    out = torch.full((T, H * D + pad), 7.0, dtype=DT[out_dtype], device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    K, V = values(b, layer)
    args = (b["q_start"], b["kv_len"], b["table"], scale)
    if lists is None:
        b["cache"].attention(layer, b["batch"], q, out[:, :H * D], scale=scale, window=window, lse=lse)
        want = sv.attention(f64(q).reshape(T, H, D), K, V, *args, window)
    else:
        b["cache"].attention_pages(layer, b["batch"], q, torch.from_numpy(lists.astype(np.int32)).cuda(), out[:, :H * D],
                                   scale=scale, lse=lse)
        want = sv.attention_pages(f64(q).reshape(T, H, D), K, V, lists, *args)
    assert qdq.get_device_status() == 0
    ref, ref_lse, spread, reach = want
    got, got_lse = f64(out[:, :H * D]).reshape(T, H, D), f64(lse)
    none = np.isnan(ref_lse)
    assert (got[none] == 7).all() and (got_lse[none] == 7).all(), "rows of no sequence were written"
    assert (f64(out[:, H * D:]) == 7).all()
    half_out = torch.finfo(out.dtype).eps / 2
    n = int(b["kv_len"].max())
    e = 0
    if b["dtype"] == "e4m3":
        e = int(np.abs(b["scales"][:, layer].cpu().numpy().astype(int) - 127).clip(max=40).max())
        v_max = 448 * 2.0 ** int(b["scales"][1, layer].cpu().numpy().astype(int).max() - 127)
    else:
        v_max = np.nanmax(np.abs(V), initial=0.0, where=np.isfinite(V))
    # two terms: 16 bits of a weight in bf16, 22 in fp16, whose smallest step counts too
    weight, least = (2.0 ** -17, 0.0) if b["q_dtype"] == "bf16" else (2.0 ** -22, 2.0 ** -32)
    if lists is None and out_dtype != "f32" and -(-T // len(b["kv_len"])) * (H // b["kv"]) > 16:
        # blocks of many rows with a 16-bit result: one fp16 term, rounded to nearest, off by 2^-11 of itself
        # (fp16's smallest step, 2^-24, is 2^-31 of the row's largest weight, which is kept times 2^7: half of it, 2^-32)
        weight = 2.0 ** -11
    ds = 2 * D * 2.0 ** -24 * reach + 4 * 2.0 ** -24 * e
    tol = half_out * np.abs(ref) + (weight + 2 * ds[..., None] + 2.0 ** -20 + n * 2.0 ** -24) * spread + n * least * v_max + 1e-30
    if out_dtype == "f16":
        tol = tol + 2.0 ** -25
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


@pytest.mark.parametrize("out_dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dim,heads,kv,page", [(64, 4, 4, 16), (64, 8, 2, 32), (128, 8, 1, 64), (128, 6, 2, 16),
                                               (64, 12, 1, 128), (128, 32, 1, 256)])
@pytest.mark.parametrize("lens", [[(1, 0)], [(1, 130), (1, 0), (1, 257), (0, 9), (1, 15)], [(37, 0), (1, 200), (70, 61)],
                                  [(150, 150)]])
def test_attention(qdq, out_dtype, dim, heads, kv, page, lens):
    b = make(qdq, lens, heads, kv, dim, page, seed=dim + page, extra_tokens=1)
    fill_held(b)
    check_attention(qdq, b, out_dtype=out_dtype)


@pytest.mark.parametrize("window", [1, 16, 100, 129, 5000])
@pytest.mark.parametrize("lens", [[(1, 300)], [(90, 200), (1, 128), (260, 0)]])
def test_attention_window(qdq, window, lens):
    b = make(qdq, lens, 4, 2, 64, 16, seed=window)
    fill_held(b)
    check_attention(qdq, b, window=window)


@pytest.mark.parametrize("scale", [0.3, -0.2, 0.0])
def test_attention_strides_scale_and_layer(qdq, scale):
    b = make(qdq, [(20, 50), (1, 90)], 4, 2, 128, 32, layers=2, seed=4)
    fill_held(b, layer=1)
    check_attention(qdq, b, layer=1, out_dtype="bf16", scale=scale, pad=64)


def test_attention_bad_pages_and_empty_rows(qdq):
    b = make(qdq, [(40, 100), (1, 150), (9, 0), (3, 40)], 4, 2, 64, 16, seed=9)
    b["table"][0, 2], b["table"][1, 0], b["table"][1, 5] = -5, b["n_pages"], 1 << 30
    b["table"][3, :] = -1                                      # nothing to attend to
    b["kv_len"][2] = 4                                         # five tokens before position 0
    b["batch"] = batch_of(qdq, b)
    fill_held(b)
    check_attention(qdq, b)
    check_attention(qdq, b, window=30)


def test_attention_kv_len_past_the_table_and_no_table(qdq):
    b = make(qdq, [(4, 60), (1, 30)], 4, 2, 64, 16, seed=2)
    fill_held(b)
    b["kv_len"] = np.array([70, 31], np.int32)                 # positions 64..69 have no page
    b["batch"] = batch_of(qdq, b)
    check_attention(qdq, b)
    b["table"] = np.zeros((2, 0), np.int32)
    b["batch"] = batch_of(qdq, b)
    check_attention(qdq, b)


@pytest.mark.parametrize("lens", [[(1, 700)], [(1, 130), (40, 900)]])
def test_attention_scales_far_apart(qdq, lens):
    """Scales that differ by 2^30 from block to block: a value's scale moves the weights' unit."""
    b = make(qdq, lens, 4, 2, 128, 32, seed=3, exponents=(-16, 14))
    fill_held(b)
    check_attention(qdq, b, q_scale=2.0 ** -6)
    e = b["scales"].cpu().numpy()
    e[0] = 120                                                 # the values' alone
    b["scales"].copy_(torch.from_numpy(e))
    check_attention(qdq, b)
    e[1], e[1, ..., 0] = 0, 255                                # beyond the range: its ends
    b["scales"].copy_(torch.from_numpy(e))
    b["rng"] = np.random.default_rng(1)
    K, V = values(b)
    assert np.nanmax(np.abs(V)) <= 448 * 2.0 ** 40
    out = torch.zeros(b["tokens"], 4 * 128, device="cuda")
    q = torch.randn(b["tokens"], 4 * 128, device="cuda").half()
    b["cache"].attention(0, b["batch"], q, out)
    ref, _, spread, _ = sv.attention(f64(q).reshape(-1, 4, 128), K, V, b["q_start"], b["kv_len"], b["table"], 128 ** -0.5)
    # (blocks 2^80 below the others' count for nothing; the rest as ever, in units of 2^40)
    assert (np.abs(f64(out).reshape(ref.shape) - ref) <= 2.0 ** -14 * spread + 448 * 2.0 ** (40 - 20)).all()


def test_attention_large_scores(qdq):
    b = make(qdq, [(30, 200), (1, 333)], 8, 2, 64, 32, seed=6)
    fill_held(b)
    check_attention(qdq, b, q_scale=60.0)


def test_attention_many_small_weights_beside_a_large_one(qdq):
    """One position with a score 13 above 20000 others: the small weights' sum is not lost."""
    b = make(qdq, [(1, 19999)], 4, 1, 64, 256, seed=3, exponents=(-8, -7))
    K = torch.zeros_like(b["pools"][0])
    K[0, b["table"][0, 0], 0, 5] = int(sv.e4m3_byte(np.array([208.0]))[0])
    b["pools"][0].copy_(K)
    b["pools"][1].copy_(torch.from_numpy(sv.e4m3_byte(b["rng"].standard_normal(b["pools"][1].shape) * 96 + 96)))
    b["scales"].fill_(127 - 7)
    q = torch.ones(1, 256, device="cuda").half()
    check_attention(qdq, b, q=q)


@pytest.mark.parametrize("kv_len", [1000, 4097, 20000])
@pytest.mark.parametrize("heads", [2, 8, 32])
def test_attention_long_single_tokens(qdq, kv_len, heads):
    """One token over a long cache (the positions are split over CTAs and joined), and two sequences."""
    b = make(qdq, [(1, kv_len - 1), (1, 700)], heads, 2, 128, 128, seed=kv_len)
    x = np.clip(b["rng"].standard_normal(b["pools"].shape) * 96, -448, 448)
    b["pools"].copy_(torch.from_numpy(sv.e4m3_byte(x)))
    check_attention(qdq, b)


def test_attention_many_sequences(qdq):
    lens = [(int(n), int(x)) for n, x in np.random.default_rng(5).integers(0, 3, (1024, 2))]
    b = make(qdq, lens, 2, 1, 64, 16, seed=3)
    fill_held(b)
    check_attention(qdq, b)


# ---- bounds and selection ---------------------------------------------------------------------
def bounds_of(b, layers=1):
    g = torch.Generator(device="cuda").manual_seed(3)
    bounds = torch.randint(-127, 128, (layers, b["n_pages"], b["kv"], 2, b["dim"]), generator=g, device="cuda", dtype=torch.int8)
    return bounds, torch.randint(100, 140, (layers, b["n_pages"], b["kv"]), generator=g, device="cuda", dtype=torch.uint8)


def check_bounds(qdq, b, layer=0, layers=1):
    bounds, scales = bounds_of(b, layers)
    was, was_s = bounds.cpu().numpy(), scales.cpu().numpy()
    K, _ = values(b, layer)
    b["cache"].key_bounds(layer, b["batch"], bounds, scales)
    assert qdq.get_device_status() == 0
    want, want_s = sv.key_bounds(K, was[layer], was_s[layer], b["q_start"], b["kv_len"], b["table"], b["tokens"])
    was[layer], was_s[layer] = want, want_s
    assert np.array_equal(scales.cpu().numpy(), was_s) and np.array_equal(bounds.cpu().numpy(), was)


@pytest.mark.parametrize("dtype", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("dim,kv,page", [(64, 2, 16), (128, 1, 32), (128, 3, 256), (64, 1, 128)])
def test_bounds(qdq, dtype, dim, kv, page):
    b = make(qdq, [(1, 0), (5, 30), (0, 12), (133, 0), (1, 300), (17, 15)], 2 * kv, kv, dim, page, dtype, layers=2, seed=dim,
             extra_tokens=2)
    fill_held(b, layer=1)
    check_bounds(qdq, b, 1, 2)


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
def test_bounds_of_many_tokens(qdq, dtype):
    """A window of tokens a CTA; absent pages, negative positions, positions past the table."""
    b = make(qdq, [(1500, 70), (40, 0), (0, 3), (9, 0), (1, 64), (600, 20)], 8, 8, 64, 32, dtype, seed=4)
    b["table"][0, 3], b["table"][1, 1] = -1, b["n_pages"] + 7
    b["kv_len"][3] = 4
    b["kv_len"][0] = b["table"].shape[1] * 32 + 5
    b["batch"] = batch_of(qdq, b)
    fill_held(b)
    check_bounds(qdq, b)


@pytest.mark.parametrize("dtype", ["e4m3", "f16", "bf16"])
def test_bounds_of_extreme_keys(qdq, dtype):
    """Zeros, one sign only, values at a power's border, and (16-bit) infinities and the type's ends."""
    b = make(qdq, [(64, 0)], 2, 2, 64, 16, dtype, seed=4)
    fill_held(b)
    if dtype == "e4m3":
        p = b["pools"][0, 0]
        p[b["table"][0, 0]] = 0
        p[b["table"][0, 1]] &= 0x7F
        p[b["table"][0, 2]] |= 0x80
        p[b["table"][0, 3]] = torch.where(p[b["table"][0, 3]] == 0x7F, 0, p[b["table"][0, 3]])
        for x in (1, 2):  # (a sign bit on a NaN is one)
            p[b["table"][0, x]] = torch.where(p[b["table"][0, x]] & 0x7F == 0x7F, 0x38, p[b["table"][0, x]])
    else:
        p = b["pools"][0, 0]
        p[b["table"][0, 0]] = 0
        p[b["table"][0, 1]] = p[b["table"][0, 1]].abs()
        p[b["table"][0, 2], :, 0] = 127.0
        p[b["table"][0, 2], :, 1] = torch.finfo(p.dtype).max
        p[b["table"][0, 3], 3, 0, 5], p[b["table"][0, 3], 4, 1, 6] = float("inf"), float("nan")
    check_bounds(qdq, b)


def check_select(qdq, b, n_select, first=1, last=1, bounds=None, layer=0, layers=1, pad=0):
    T, H, D = b["tokens"], b["heads"], b["dim"]
    q = torch.from_numpy(b["rng"].standard_normal((T, H * D + pad))).to(DT[b["q_dtype"]]).cuda()[:, :H * D]
    bounds, scales = bounds_of(b, layers) if bounds is None else bounds
    lists = torch.full((T, b["kv"], n_select), -2, dtype=torch.int32, device="cuda")
    b["cache"].select_pages(layer, b["batch"], q, bounds, scales, lists, first=first, last=last)
    assert qdq.get_device_status() == 0
    want = sv.select_pages(f64(q).reshape(T, H, D), bounds[layer].cpu().numpy(), scales[layer].cpu().numpy(), b["q_start"],
                           b["kv_len"], b["table"], b["page"], n_select, first, last)
    got = lists.cpu().numpy()
    bad = np.argwhere((got != want).any(-1))
    assert not len(bad), (bad[0], got[tuple(bad[0])], want[tuple(bad[0])])
    return got


@pytest.mark.parametrize("dtype", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv", [(64, 4, 2), (128, 3, 1), (64, 32, 1), (128, 8, 8), (128, 10, 2)])
@pytest.mark.parametrize("n_select,first,last", [(1, 0, 0), (1, 0, 1), (4, 1, 2), (37, 2, 1), (2000, 1, 1)])
def test_select(qdq, dtype, dim, heads, kv, n_select, first, last):
    b = make(qdq, [(1, 0), (2, 30), (0, 12), (1, 1333), (3, 700), (1, 15)], heads, kv, dim, 16, dtype, seed=dim, extra_tokens=2,
             layers=2)
    check_select(qdq, b, n_select, first, last, layer=1, layers=2)


def test_select_one_token_over_many_pages(qdq):
    """A cluster of CTAs scores one token's pages."""
    b = make(qdq, [(1, 40000)], 8, 2, 64, 16, "f16", seed=1)
    check_select(qdq, b, 128, 1, 2)
    check_select(qdq, b, 1, 0, 0)


@pytest.mark.parametrize("dtype,dim,heads", [("e4m3", 128, 8), ("bf16", 64, 36), ("f16", 128, 4)])
def test_select_many_items(qdq, dtype, dim, heads):
    """More tokens and heads than SMs: several share one."""
    lens = [(1, int(x)) for x in np.random.default_rng(5).integers(0, 900, 60)]
    b = make(qdq, lens, heads, 4, dim, 16, dtype, seed=4)
    for n in (1, 20):
        check_select(qdq, b, n, 0, 1)


def test_select_as_many_pages_as_there_may_be(qdq):
    """32768 entries of a table over a few pages: thousands of equal scores."""
    b = make(qdq, [(1, 200), (1, 40)], 2, 1, 64, 16, seed=1)
    b["table"] = b["rng"].integers(-1, b["n_pages"], (2, 32768)).astype(np.int32)
    b["kv_len"] = np.array([32768 * 16, 20000 * 16 - 3], np.int32)
    b["batch"] = batch_of(qdq, b)
    for n in (7, 5000):
        check_select(qdq, b, n, 1, 2)


def test_select_ties_and_absent_pages(qdq):
    """Equal scores take the lowest pages; absent pages and negative positions none."""
    b = make(qdq, [(1, 4000), (1, 900), (9, 0), (2, 500), (1, 100)], 4, 2, 64, 16, seed=2)
    bounds, scales = bounds_of(b)
    bounds[:] = bounds[0, 0, 0]
    scales[:] = 120
    for n in (1, 5, 64, 250):
        check_select(qdq, b, n, 0, 0, (bounds, scales))
        check_select(qdq, b, n, 1, n - 1, (bounds, scales))
    bounds, scales = bounds_of(b)
    bounds[:, ::2], scales[:, ::2] = 0, 127                    # half of them equal, at zero
    b["table"][0, 3:90:4], b["table"][1, 0], b["table"][3, 31] = -1, b["n_pages"], -7
    b["table"][4, :] = -1
    b["kv_len"][2] = 4                                         # five tokens before position 0
    b["kv_len"][0] += 200                                      # past the table
    b["batch"] = batch_of(qdq, b)
    for n in (1, 5, 64, 250):
        check_select(qdq, b, n, 1, 0, (bounds, scales), pad=64)


def test_select_scores_of_both_signs_and_scales_far_apart(qdq):
    b = make(qdq, [(1, 3000), (1, 2000)], 4, 2, 128, 16, "bf16", seed=2)
    bounds, scales = bounds_of(b)
    bounds[:, ::3] = -bounds[:, ::3].abs()                     # (mx and mn need not be bounds of anything)
    scales.copy_(torch.randint(0, 256, scales.shape, device="cuda", dtype=torch.uint8))
    for n in (3, 50):
        check_select(qdq, b, n, 0, 0, (bounds, scales))


# ---- attention over lists -----------------------------------------------------------------------
def random_lists(b, n, rng):
    lists = np.full((b["tokens"], b["kv"], n), -1)
    most = b["table"].shape[1]
    for t in range(b["tokens"]):
        for g in range(b["kv"]):
            k = rng.integers(0, min(n, most) + 1)
            lists[t, g, :k] = np.sort(rng.permutation(most)[:k])
    return lists


@pytest.mark.parametrize("dtype", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv,page", [(64, 4, 4, 16), (64, 8, 2, 32), (128, 8, 1, 64), (128, 6, 2, 16),
                                               (64, 12, 1, 128), (128, 32, 1, 256), (64, 48, 2, 256)])
@pytest.mark.parametrize("n", [1, 5, 24])
def test_attention_pages(qdq, dtype, dim, heads, kv, page, n):
    b = make(qdq, [(1, 130), (2, 0), (1, 300), (0, 9), (3, 15), (1, 700)], heads, kv, dim, page, dtype, seed=dim + page,
             extra_tokens=1, layers=2)
    fill_held(b, layer=1)
    check_attention(qdq, b, layer=1, lists=random_lists(b, n, b["rng"]), out_dtype=(dtype if n == 5 and dtype != "e4m3" else "f32"),
                    pad=64 * (n == 5))


@pytest.mark.parametrize("dtype", ["e4m3", "f16"])
def test_attention_pages_odd_lists(qdq, dtype):
    """Entries that repeat, fall, or name no page of the table; absent pages; empty lists."""
    b = make(qdq, [(1, 200), (1, 200), (2, 140), (4, 0)], 4, 2, 64, 16, dtype, seed=5)
    b["table"][1, 3] = -1
    b["kv_len"][3] = 2                                         # two tokens before position 0
    b["batch"] = batch_of(qdq, b)
    fill_held(b)
    lists = np.full((b["tokens"], 2, 6), -1)
    lists[0, 0], lists[0, 1] = [2, 2, 5, 4, 5, 7], [0, 1, 2, 3, 4, 5]
    lists[1, 0], lists[1, 1] = [-1, 3, 5, -1, 12, 400], [3, 3, 3, 3, 3, 3]
    lists[2, 0], lists[2, 1] = [8, 9, 10, 1 << 30, -5, -(1 << 31)], [7, 6, 5, 4, 3, 2]
    lists[4:, :, 0] = 0
    check_attention(qdq, b, lists=lists)


def test_attention_pages_of_everything_is_attention(qdq):
    for dtype in ("e4m3", "f16", "bf16"):
        b = make(qdq, [(1, 3000), (1, 77)], 8, 2, 128, 64, dtype, seed=8)
        x = torch.randn(b["pools"].shape, device="cuda") * (96 if dtype == "e4m3" else 1)
        b["pools"].copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if dtype == "e4m3" else x)
        every = np.tile(np.arange(b["table"].shape[1]), (2, 2, 1))
        check_attention(qdq, b, lists=every)


# ---- together -------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
def test_a_decode_step_over_chosen_pages(qdq, dtype):
    """Append, bounds, selection, attention over the selection, as a captured graph that replays step after
    step with the batch's arrays moved on; every step's results are the oracle's."""
    H, G, D, page = 8, 2, 64, 16
    lens = [(1, 0), (1, 250), (1, 31), (1, 500)]
    b = make(qdq, [(1, x + 8) for _, x in lens], H, G, D, page, dtype, seed=3)
    b["kv_len"] = np.array([x for _, x in lens], np.int32)
    fill_held(b)
    b["batch"] = batch_of(qdq, b)
    bounds, scales = torch.zeros(1, b["n_pages"], G, 2, D, dtype=torch.int8, device="cuda"), torch.zeros(1, b["n_pages"], G, dtype=torch.uint8, device="cuda")
    # the bounds of what is held already: a batch in which all of it is new
    old = qdq.PagedBatch(torch.tensor([0, *np.cumsum(b["kv_len"])], dtype=torch.int32, device="cuda"), *b["batch"]._keep[1:],
                         int(b["kv_len"].sum()))
    b["cache"].key_bounds(0, old, bounds, scales)
    T = 4
    x = torch.zeros(T, (H + 2 * G) * D, device="cuda")
    q, k, v = x.split([H * D, G * D, G * D], dim=1)
    q16 = torch.zeros(T, H * D, dtype=DT[b["q_dtype"]], device="cuda")
    lists = torch.zeros(T, G, 6, dtype=torch.int32, device="cuda")
    out = torch.zeros(T, H * D, device="cuda")

    def step():
        b["cache"].append(0, b["batch"], q, k, v, q16)
        b["cache"].key_bounds(0, b["batch"], bounds, scales)
        b["cache"].select_pages(0, b["batch"], q16, bounds, scales, lists, first=1, last=2)
        b["cache"].attention_pages(0, b["batch"], q16, lists, out)

    kv = b["batch"]._keep[1]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(6):
        kv += 1
        b["kv_len"] = kv.cpu().numpy()
        x.copy_(torch.from_numpy(b["rng"].standard_normal(tuple(x.shape))))
        graph.replay()
        torch.cuda.synchronize()
        assert qdq.get_device_status() == 0
        K, V = values(b)
        want = sv.select_pages(f64(q16).reshape(T, H, D), bounds[0].cpu().numpy(), scales[0].cpu().numpy(), b["q_start"],
                               b["kv_len"], b["table"], page, 6, 1, 2)
        assert np.array_equal(lists.cpu().numpy(), want)
        fresh, fresh_s = sv.key_bounds(K, bounds[0].cpu().numpy(), scales[0].cpu().numpy(), [0, *np.cumsum(b["kv_len"])], b["kv_len"],
                                       b["table"], int(b["kv_len"].sum()))
        assert np.array_equal(fresh, bounds[0].cpu().numpy()) and np.array_equal(fresh_s, scales[0].cpu().numpy())
        ref = sv.attention_pages(f64(q16).reshape(T, H, D), K, V, want, b["q_start"], b["kv_len"], b["table"], D ** -0.5)[0]
        assert np.abs(f64(out).reshape(T, H, D) - ref).max() < 1e-4


def test_results_repeat_and_graphs_follow_the_batch(qdq):
    """The same calls give the same bits, on other streams and in a replayed graph too."""
    b = make(qdq, [(1, 2000), (60, 400), (1, 9)], 8, 2, 64, 16, seed=1)
    x = torch.randn(b["pools"].shape, device="cuda") * 96
    b["pools"].copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    H, D, T = 8, 64, b["tokens"]
    q = torch.randn(T, H * D, device="cuda").half()
    lists = torch.from_numpy(random_lists(b, 40, b["rng"]).astype(np.int32)).cuda()
    o = [[torch.zeros(T, H * D, device="cuda") for _ in range(2)] for _ in range(3)]

    def both(to):
        b["cache"].attention(0, b["batch"], q, to[0])
        b["cache"].attention_pages(0, b["batch"], q, lists, to[1])

    both(o[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(50):
            both(o[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(o[0], o[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both(o[2])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(o[0], o[2]))
    b["batch"]._keep[1][0] = 1200
    graph.replay()
    both(o[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(o[1], o[2])) and not torch.equal(o[0][0], o[2][0])
    assert qdq.get_device_status() == 0


# ---- refusals --------------------------------------------------------------------------------------
def test_refusals_on_the_device(qdq):
    b = make(qdq, [(1, 100), (1, 40)], 4, 2, 64, 16)
    c, batch = b["cache"], b["batch"]
    q = torch.zeros(2, 256, device="cuda").half()
    out = torch.zeros(2, 256, device="cuda")
    lists = torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda")
    bounds, scales = bounds_of(b)
    for f, text in ((lambda: c.attention(0, batch, q.bfloat16(), out), "queries' type"),
                    (lambda: c.attention_pages(0, batch, q.bfloat16(), lists, out), "queries' type"),
                    (lambda: c.select_pages(0, batch, q.float(), bounds, scales, lists), "queries' type"),
                    (lambda: c.attention_pages(0, batch, q, lists[0], out), "n_select"),
                    (lambda: c.attention_pages(0, batch, q, lists[:1], out), "n_select"),
                    (lambda: c.attention_pages(0, batch, q, lists.long(), out), "int32"),
                    (lambda: c.key_bounds(0, batch, bounds.float(), scales), "int8"),
                    (lambda: c.key_bounds(0, batch, bounds[:, 1:].contiguous(), scales), "int8"),
                    (lambda: c.key_bounds(0, batch, bounds, scales.short()), "bytes")):
        with pytest.raises(ValueError, match=text):
            f()
    L, ref = qdq.lib(), batch._ref
    good = dict(n_select=4, first=1, last=1, layer=0, stride=256, pages=lists.data_ptr(), bounds=bounds.data_ptr(), scales=scales.data_ptr())

    def select(**k):
        a = {**good, **k}
        return L.qdq_paged_select_pages(c._h, a["layer"], ref, q.data_ptr(), a["stride"], a["bounds"], a["scales"], a["n_select"], a["first"],
                                        a["last"], a["pages"], 0)

    assert select() == 0
    assert [select(**k) for k in (dict(n_select=0), dict(first=-1), dict(last=-1), dict(first=3, last=2), dict(layer=1), dict(stride=255))] == [-2] * 6
    assert [select(**k) for k in (dict(pages=0), dict(bounds=0), dict(scales=0))] == [-4] * 3
    assert select(stride=260) == -3 and select(bounds=bounds.data_ptr() + 8) == -3 and select(pages=lists.data_ptr() + 2) == -3
    attend = lambda lists=lists.data_ptr(), n=4, out_type=1, scale=0.1: L.qdq_paged_attention_pages(
        c._h, 0, ref, q.data_ptr(), 256, lists, n, out_type, out.data_ptr(), 256, scale, 0, 0)
    assert attend() == 0 and attend(n=0) == -2 and attend(lists=0) == -4 and attend(out_type=4) == -1 and attend(scale=float("inf")) == -2
    wide = qdq.PagedBatch(*batch._keep[:2], torch.zeros(2, 32769, dtype=torch.int32, device="cuda"), 2)
    with pytest.raises(qdq.QdqError):
        c.select_pages(0, wide, q, bounds, scales, lists)
    torch.cuda.synchronize()
    assert qdq.get_device_status() == 0


@pytest.mark.parametrize("dtype", ["e4m3", "bf16"])
def test_pages_past_four_gigabytes(qdq, dtype):
    """The same batch in a small cache and in the last pages of a pool of over 4 GB: the same bits."""
    H, G, D, page = 8, 8, 128, 64
    lens = [(1, 700), (40, 100), (1, 0)]
    b = make(qdq, lens, H, G, D, page, dtype, seed=2)
    fill_held(b)
    far = 33000 if dtype == "bf16" else 66000
    assert far * page * G * D * b["pools"].element_size() > 1 << 32
    pools = torch.zeros(2, 2, far, *b["pools"].shape[3:], dtype=b["pools"].dtype, device="cuda")
    pools[:, 1, far - b["n_pages"]:] = b["pools"][:, 0]
    more = {}
    if dtype == "e4m3":
        scales = torch.zeros(2, 2, far, G, page // 16, dtype=torch.uint8, device="cuda")
        scales[:, 1, far - b["n_pages"]:] = b["scales"][:, 0]
        more = dict(k_scales=scales[0], v_scales=scales[1])
    big = qdq.PagedCache(*(pools.view(torch.float8_e4m3fn) if more else pools), H, **more)
    table = b["batch"]._keep[2]
    there = qdq.PagedBatch(*b["batch"]._keep[:2], torch.where(table >= 0, table + (far - b["n_pages"]), table), b["tokens"])
    T = b["tokens"]
    x = torch.from_numpy(b["rng"].standard_normal((T, (H + 2 * G) * D))).float().cuda()
    q, k, v = x.split([H * D, G * D, G * D], dim=1)
    got = []
    for cache, batch, layer, n in ((b["cache"], b["batch"], 0, b["n_pages"]), (big, there, 1, far)):
        q16 = torch.zeros(T, H * D, dtype=DT[b["q_dtype"]], device="cuda")
        bounds = torch.zeros(layer + 1, n, G, 2, D, dtype=torch.int8, device="cuda")
        bound_scales = torch.zeros(layer + 1, n, G, dtype=torch.uint8, device="cuda")
        lists = torch.zeros(T, G, 4, dtype=torch.int32, device="cuda")
        outs = [torch.zeros(T, H * D, device="cuda") for _ in range(2)]
        cache.append(layer, batch, q, k, v, q16)
        cache.key_bounds(layer, batch, bounds, bound_scales)
        cache.select_pages(layer, batch, q16, bounds, bound_scales, lists)
        cache.attention(layer, batch, q16, outs[0])
        cache.attention_pages(layer, batch, q16, lists, outs[1])
        got.append((q16, bounds[layer, -b["n_pages"]:], lists, *outs))
    assert qdq.get_device_status() == 0
    assert all(torch.equal(a, c) for a, c in zip(*got))
    assert torch.equal(pools[:, 1, far - b["n_pages"]:].view(torch.uint8), b["pools"][:, 0].view(torch.uint8))


def test_attention_pages_of_a_prompt_piece(qdq):
    """Hundreds of tokens, each with a list of its own."""
    for dtype in ("e4m3", "f16"):
        b = make(qdq, [(150, 60), (1, 300), (0, 5), (33, 0)], 8, 2, 64, 16, dtype, seed=5, extra_tokens=3)
        fill_held(b)
        check_attention(qdq, b, lists=random_lists(b, 7, b["rng"]))
