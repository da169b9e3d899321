"""The paged attention's softmax weights: any finite scale, the bits that the weights keep, their range.

* Scales. The tolerance is test_gpu_serving's. At scale 0 every position weighs the same.
* Bits. A weight in two terms of the pools' type is off by half a step of half a step, so that an
  fp32 result is left with the fp32 scores' and sums' error: 2 D 2^-24 reach at the worst, some
  1e-6 of the result at these sizes, against 2^-11 / sqrt(3) (fp16) or 2^-8 / sqrt(3) (bf16) of a
  weight rounded once. Root mean square errors are compared: an eighth of those of weights rounded
  once, computed on the CPU from the same inputs, is far from both.
* Range. fp16 weights are kept times 2^7, in steps of 2^-24 below 2^-14: half a step is 2^-32 of the
  largest weight, so n of them are off by n 2^-32 max|v|. (bf16 has fp32's range; its two terms leave
  2^-17 of a weight.) Sums: at most 16 additions to the accumulator a key tile, 64 and one to the
  weights' sum, a factor and an addition for each of the parts that are joined, each off by at most
  2^-23 relative to sums of positive terms.
"""
import math

import numpy as np
import pytest

from tests.test_gpu_serving import DT, batch_of, check_attention, f64, fill_held, make, qdq, sv  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

MIXED = [(37, 0), (1, 200), (70, 61), (1, 0)]


@pytest.mark.parametrize("dtype,dim", [("f16", 64), ("bf16", 64), ("f16", 128), ("bf16", 128)])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45, -1e-45, -0.02, -0.15])
@pytest.mark.parametrize("window", [0, 30])
def test_attention_of_any_scale(qdq, dtype, dim, scale, window):  # noqa: F811
    b = make(qdq, MIXED, 8, 2, dim, 16, dtype, seed=41)
    fill_held(b)
    check_attention(qdq, b, scale=scale, window=window)


def test_attention_of_scale_zero_over_a_cut_sequence(qdq):  # noqa: F811
    """Parts that several CTAs hold, one of them without any position of the pools."""
    b = make(qdq, [(1, 2500), (1, 700)], 8, 2, 128, 32, "f16", seed=42)
    b["table"][0, 30:60] = -1
    b["batch"] = batch_of(qdq, b)
    fill_held(b)
    check_attention(qdq, b, scale=0.0)


def test_attention_refuses_scales_that_overflow(qdq):  # noqa: F811
    b = make(qdq, [(3, 0)], 4, 2, 64, 16, "f16")
    q, out = (torch.zeros(3, 256, dtype=torch.float16, device="cuda") for _ in range(2))
    for scale in (3e38, -3e38, float("inf"), float("nan")):
        with pytest.raises(qdq.QdqError) as e:
            b["cache"].attention(0, b["batch"], q, out, scale=scale)
        assert e.value.rc == -2
    b["cache"].attention(0, b["batch"], q, out, scale=2e38)


def rounded_once(q, b, scale):
    """The attention with each weight rounded to the pools' type once, everything else in float64."""
    K, V = (f64(b["pools"][i, 0]) for i in (0, 1))
    T, H, D = q.shape
    out = np.zeros((T, H, D))
    for t, s, p in sv.tokens_of(b["q_start"], b["kv_len"], T):
        pg, rw = np.array([sv.row_of(b["table"], b["n_pages"], b["page"], s, j) for j in range(p + 1)]).T
        for h in range(H):
            g = h // (H // b["kv"])
            x = K[pg, rw, g] @ q[t, h] * scale
            w = np.exp(x - x.max())
            out[t, h] = f64(torch.from_numpy(w).to(DT[b["dtype"]])) @ V[pg, rw, g] / w.sum()
    return out


@pytest.mark.parametrize("dtype,dim", [("f16", 64), ("bf16", 64), ("f16", 128), ("bf16", 128)])
@pytest.mark.parametrize("lens", [[(1, 90)], [(1, 700)], [(1, 300), (3, 500), (1, 64)], [(90, 200)], [(5, 9), (140, 60)]])
def test_attention_keeps_what_the_rounding_of_weights_leaves(qdq, dtype, dim, lens):  # noqa: F811
    """Whatever the type, the head dims, the rows of a block and its key tiles."""
    b = make(qdq, lens, 8, 2, dim, 16, dtype, seed=31)
    fill_held(b)
    T, scale = b["tokens"], dim ** -0.5
    q = torch.from_numpy(b["rng"].standard_normal((T, 8 * dim)) * 1.5).to(DT[dtype]).cuda()
    out = torch.full((T, 8 * dim), 7.0, device="cuda")
    b["cache"].attention(0, b["batch"], q, out, scale=scale)
    assert qdq.get_device_status() == 0
    q = f64(q).reshape(T, 8, dim)
    ref = sv.attention(q, f64(b["pools"][0, 0]), f64(b["pools"][1, 0]), b["q_start"], b["kv_len"], b["table"], scale)[0]
    rms = lambda x: math.sqrt(np.mean(np.square(x)))
    once = rms(rounded_once(q, b, scale) - ref)
    assert once > 2.0 ** -16 * rms(ref), "the inputs show the rounding"
    assert rms(f64(out).reshape(ref.shape) - ref) <= once / 8


@pytest.mark.parametrize("dtype,dim", [("f16", 64), ("bf16", 64), ("f16", 128), ("bf16", 128)])
@pytest.mark.parametrize("lens", [[(1, 90)] * 6, [(1, 700), (2, 800)], [(3, 500), (1, 64), (2, 0)]])
def test_attention_of_few_rows_is_off_by_the_results_rounding(qdq, dtype, dim, lens):  # noqa: F811
    """16-bit results: the root mean square error is that of the exact result's rounding. (What two
    terms leave adds less than 1 % to it, weights rounded once up to 37 %.)"""
    b = make(qdq, lens, 8, 2, dim, 16, dtype, seed=37)
    fill_held(b)
    T, scale = b["tokens"], dim ** -0.5
    q = torch.from_numpy(b["rng"].standard_normal((T, 8 * dim)) * 1.5).to(DT[dtype]).cuda()
    out = torch.zeros_like(q)
    b["cache"].attention(0, b["batch"], q, out, scale=scale)
    q = f64(q).reshape(T, 8, dim)
    ref = sv.attention(q, f64(b["pools"][0, 0]), f64(b["pools"][1, 0]), b["q_start"], b["kv_len"], b["table"], scale)[0]
    rms = lambda x: math.sqrt(np.mean(np.square(x)))
    rounding = rms(f64(torch.from_numpy(ref).to(DT[dtype])) - ref)
    assert rms(f64(out).reshape(ref.shape) - ref) <= 1.05 * rounding


@pytest.mark.parametrize("dtype,dim", [("f16", 64), ("bf16", 64), ("f16", 128), ("bf16", 128)])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("gap", [9.0, 12.0, 15.0, 17.4, 19.0])
def test_attention_of_one_large_weight_over_many_small_ones(qdq, dtype, dim, new, gap):  # noqa: F811
    """Position 3 scores `gap` more than 131000 others, and its value is zero: the result is what
    the small weights leave. As many sequences (over the same pages) as there are SMs, so that
    each is one CTA's and no part of it has a maximum of its own."""
    page, n = 256, 131000
    S, pages = qdq.device_sm_count(), -(-n // 256)
    pools = torch.zeros(2, 1, pages, page, 1, dim, dtype=DT[dtype], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(7)
    pools[1] = (torch.rand(pools[1].shape, generator=gen, device="cuda") + 0.5).to(DT[dtype])
    pools[0, 0, 0, 3, 0, 0] = 4.0
    pools[1, 0, 0, 3] = 0.0
    cache = qdq.PagedCache(pools[0], pools[1], 2)
    i32 = lambda x: x.to(torch.int32).cuda()
    batch = qdq.PagedBatch(i32(torch.arange(S + 1) * new), i32(torch.full((S,), n)),
                           i32(torch.arange(pages)[None].expand(S, pages).contiguous()), S * new)
    q = torch.zeros(S * new, 2 * dim, dtype=DT[dtype], device="cuda")
    q[:, ::dim] = 4.0
    out = torch.full((S * new, 2 * dim), 7.0, device="cuda")
    lse = torch.empty(S * new, 2, device="cuda")
    cache.attention(0, batch, q, out, scale=gap / 16, lse=lse)
    assert qdq.get_device_status() == 0
    got, got_lse = f64(out).reshape(S, new, 2, dim), f64(lse).reshape(S, new, 2)
    v = f64(pools[1, 0]).reshape(-1, dim)
    sums, w = np.cumsum(v, 0), math.exp(-float(np.float32(gap / 16)) * 16)
    tiles = -(-n // 128) + 1
    for i in range(new):
        m = n - new + i + 1  # positions that this token attends to
        whole = 1 + (m - 1) * w
        ref = w * sums[m - 1] / whole
        # (the small weights' exponent: gap times 2^-23 from the rounded scale, 2^-22 from the exponential)
        rel = 2.0 ** -23 * (16 * tiles + 65 * tiles + 160) + 2.0 ** -17 + 2.0 ** -22 * (1 + gap)
        tol = rel * ref + (m * 2.0 ** -32 * v.max() / whole if dtype == "f16" else 0.0)
        assert (np.abs(got[:, i] - ref) <= tol).all(), (i, np.abs(got[:, i] / ref - 1).max(), (tol / ref).max())
        assert np.abs(got_lse[:, i] - gap - math.log(whole)).max() <= rel + 2.0 ** -22 * gap
    cache.close()
