"""The serving calls without a GPU: argument checks that answer before any device work, and the
oracle's own meaning of bad pages, empty rows and ties (oracle/serving.py)."""
import ctypes

import numpy as np
import pytest

from oracle import serving as sv


@pytest.fixture(scope="module")
def qdq():
    from quant_dequant_gemv_gb300 import build, qdq
    build.build()
    return qdq


GOOD = dict(type=2, n_layers=1, n_pages=4, page_size=16, n_heads=4, n_kv_heads=2, head_dim=64, rope_dim=64,
            rope_interleaved=1, rope_base=10000.0)


@pytest.mark.parametrize("change,code", [
    (dict(type=1), -1), (dict(type=0), -1), (dict(n_layers=0), -2), (dict(n_pages=0), -2), (dict(page_size=8), -2),
    (dict(page_size=48), -2), (dict(page_size=512), -2), (dict(n_heads=5), -2), (dict(n_heads=0), -2),
    (dict(n_heads=66), -2), (dict(head_dim=96), -2), (dict(rope_dim=4), -2), (dict(rope_dim=72), -2),
    (dict(rope_dim=-8), -2), (dict(rope_interleaved=2), -2), (dict(rope_base=1.0), -2),
    (dict(rope_base=float("nan")), -2), (dict(rope_base=float("inf")), -2), (dict(n_pages=1 << 27, page_size=16), -8)])
def test_create_refuses_a_bad_geometry(qdq, change, code):
    out = ctypes.c_void_p(12345)
    cfg = qdq.PagedConfig(**{**GOOD, **change})
    assert qdq.lib().qdq_paged_create(ctypes.byref(cfg), 0, 0, ctypes.byref(out)) == code
    assert out.value is None


def test_null_handles_and_sampling_arguments(qdq):
    L = qdq.lib()
    assert L.qdq_paged_create(None, 0, 0, None) == -4
    batch = qdq.PagedBatchDesc()
    assert L.qdq_paged_append(None, 0, ctypes.byref(batch), 1, 0, 0, 0, 0, 0, 0, 0, 0, 1e-5, 0, 0) == -4
    assert L.qdq_paged_attention(None, 0, ctypes.byref(batch), 0, 0, 2, 0, 0, 1.0, 0, 0, 0) == -4
    L.qdq_paged_destroy(None)

    def sample(type=1, stride=100, rows=1, vocab=100):
        return L.qdq_sample(type, 0, stride, rows, vocab, 0, 0, 0, 0, 0, 0, 0, 0)

    assert sample(type=0) == -1 and sample(type=4) == -1
    assert sample(rows=-1) == -2 and sample(vocab=0) == -2 and sample(rows=2, stride=99) == -2
    assert sample(vocab=(1 << 18) + 1, stride=1 << 20) == -8
    assert sample(rows=0) == 0


def test_the_binding_checks_what_it_reads_off_the_tensors(qdq):
    torch = pytest.importorskip("torch")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError):
        qdq.PagedBatch(i32(3), i32(2), i32(3, 4), 2)            # a table of another number of sequences
    with pytest.raises(ValueError):
        qdq.PagedBatch(i32(2), i32(2), i32(2, 4), 2)            # q_start too short
    with pytest.raises(ValueError):
        qdq.PagedBatch(i32(3).long(), i32(2), i32(2, 4), 2)     # another type
    with pytest.raises(ValueError):
        qdq.PagedCache(torch.zeros(2, 16, 2, 64), torch.zeros(2, 16, 2, 64), 4)
    with pytest.raises(ValueError):
        qdq.sample(torch.zeros(2, 8).t(), torch.zeros(8), torch.zeros(8, dtype=torch.int64))


def test_oracle_absent_positions_are_not_attended():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 5, 4, 1, 8))
    q = rng.standard_normal((1, 2, 8))
    table = np.array([[3, -1, 1]])
    out, lse, _, _ = sv.attention(q, k, v, [0, 1], [10], table, 0.5)
    # positions 4..7 have no page: the same as a sequence of the other six
    kk, vv = np.concatenate([k[3], k[1, :2]]), np.concatenate([v[3], v[1, :2]])
    for h in range(2):
        w = np.exp(kk[:, 0] @ q[0, h] * 0.5)
        assert np.allclose(out[0, h], w @ vv[:, 0] / w.sum()) and np.isclose(lse[0, h], np.log(w.sum()))
    # no page at all, and positions before the first: empty rows
    out, lse, _, _ = sv.attention(q, k, v, [0, 1], [10], np.array([[9, 5, -7]]), 0.5)
    assert (out == 0).all() and (lse == -np.inf).all()
    out, lse, _, _ = sv.attention(np.repeat(q, 3, 0), k, v, [0, 3], [1], table, 0.5)
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all() and (lse[2] > -np.inf).all()


def test_oracle_sampling_ties_and_empty_rows():
    x = np.array([1.0, 3.0, 3.0, 3.0, -np.inf, np.nan])
    assert sv.sample(x, 0.99, temperature=0.0) == (1, 0.0)
    assert sv.sample(x, 0.99, top_k=2)[0] == 2                  # ties: lowest indices kept
    assert sv.sample(x, 0.0, top_k=3)[0] == 1 and sv.sample(x, 0.999, top_p=0.0)[0] == 1
    assert sv.sample(x, 0.999, top_p=1 / 3, top_k=3)[0] == 1    # the mass before the second is not below
    assert sv.sample(np.full(3, -np.inf), 0.5)[0] == -1 and sv.sample(np.full(3, np.nan), 0.5)[0] == -1
    assert sv.sample(x, 0.0, min_p=0.5)[0] == 1 and sv.sample(x, 1.0)[0] == 3


def test_attention_work_split(tmp_path):
    """The kernel's own work split, compiled for the host (tests/attend_plan_check.cpp)."""
    import subprocess
    from pathlib import Path
    root = Path(__file__).resolve().parents[1]
    exe = tmp_path / "attend_plan_check"
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{root / 'quant_dequant_gemv_gb300' / 'csrc'}",
                    str(root / "tests" / "attend_plan_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
