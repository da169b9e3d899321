"""The calls over e4m3 caches and chosen pages without a GPU: argument checks that answer before any
device work, the oracle's own meaning (oracle/serving.py), rules read off the sources, and the work
split of the kernel of few rows."""
import ctypes
import re
import subprocess
from pathlib import Path

import numpy as np
import pytest

from oracle import serving as sv
from tests.test_serving_host import GOOD, qdq  # noqa: F401
from tests.test_serving_rules import CSRC, body

ROOT = Path(__file__).resolve().parents[1]


@pytest.mark.parametrize("change,code", [
    (dict(type=1), -1), (dict(type=2), -1), (dict(type=3), -1), (dict(type=0), -1), (dict(n_layers=0), -2), (dict(page_size=8), -2),
    (dict(page_size=512), -2), (dict(n_heads=5), -2), (dict(n_heads=66), -2), (dict(head_dim=96), -2), (dict(rope_dim=4), -2),
    (dict(rope_base=1.0), -2), (dict(n_pages=1 << 27, page_size=16), -8)])
def test_create_refuses_a_bad_geometry(qdq, change, code):
    out = ctypes.c_void_p(12345)
    cfg = qdq.PagedConfig(**{**GOOD, "type": 4, **change})
    assert qdq.lib().qdq_paged_create_e4m3(ctypes.byref(cfg), 0, 0, 0, 0, ctypes.byref(out)) == code
    assert out.value is None


def test_sixteen_bit_create_refuses_e4m3_and_null_handles(qdq):
    L, out = qdq.lib(), ctypes.c_void_p(12345)
    assert L.qdq_paged_create(ctypes.byref(qdq.PagedConfig(**{**GOOD, "type": 4})), 0, 0, ctypes.byref(out)) == -1
    assert L.qdq_paged_create_e4m3(None, 0, 0, 0, 0, None) == -4
    batch = qdq.PagedBatchDesc()
    ref = ctypes.byref(batch)
    assert L.qdq_paged_key_bounds(None, 0, ref, 0, 0, 0) == -4
    assert L.qdq_paged_select_pages(None, 0, ref, 0, 0, 0, 0, 4, 1, 1, 0, 0) == -4
    assert L.qdq_paged_select_pages(None, 0, ref, 0, 0, 0, 0, 0, 0, 0, 0, 0) == -2
    assert L.qdq_paged_attention_pages(None, 0, ref, 0, 0, 0, 4, 1, 0, 0, 1.0, 0, 0) == -4
    assert L.qdq_paged_attention_pages(None, 0, ref, 0, 0, 0, 0, 1, 0, 0, 1.0, 0, 0) == -2


def test_the_binding_checks_pools_and_scales(qdq):
    torch = pytest.importorskip("torch")
    pool = torch.zeros(1, 2, 4, 32, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.zeros(1, 2, 4, 2, dtype=torch.uint8)
    for args in (dict(), dict(k_scales=scale), dict(k_scales=scale, v_scales=scale[..., :1]),
                 dict(k_scales=scale, v_scales=scale.short()), dict(k_scales=scale[:, :, ::2], v_scales=scale)):
        with pytest.raises(ValueError):
            qdq.PagedCache(pool, pool, 8, **args)
    half = torch.zeros(1, 2, 32, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        qdq.PagedCache(half, half, 8, k_scales=scale, v_scales=scale)


def test_oracle_e4m3_values_and_scales():
    assert sv.E4M3[0x7E] == 448 and sv.E4M3[1] == 2.0 ** -9 and sv.E4M3[0x88] == -(2.0 ** -6) and np.isnan(sv.E4M3[0xFF])
    x = sv.E4M3[np.r_[0:127, 128:255]]
    assert np.array_equal(sv.E4M3[sv.e4m3_byte(x)], x)
    assert np.array_equal(sv.E4M3[sv.e4m3_byte(np.array([17.0, 19.0, -1e9, 465.0, 2.0 ** -10, 1.5 * 2.0 ** -9]))],
                          [16, 20, -448, 448, 0, 2 * 2.0 ** -9])     # ties to the even one, the largest beyond it
    assert [sv.least_exponent(a, 448.0, -40, 40) for a in (448, 449, 0, 1e-30, 1e30, 224)] == [0, 1, -40, -40, 40, -1]


def test_oracle_append_rescales_a_block_that_grows():
    codes, scales = np.zeros((1, 1, 16, 4), np.uint8), np.zeros((1, 1, 1), np.uint8)
    table = np.array([[0]])
    x = np.array([[[1.0, -2.0, 3.0, 448.0]], [[1.0, 0.1, 0.0, 1700.0]]])
    codes, scales, _ = sv.append_e4m3(x[:1], codes, scales, [0, 1], [1], table, 1)
    assert scales[0, 0, 0] == 127 and np.array_equal(sv.E4M3[codes[0, 0, 0]], [1, -2, 3, 448])
    codes, scales, _ = sv.append_e4m3(x[1:], codes, scales, [0, 1], [2], table, 1)
    assert scales[0, 0, 0] == 129                               # 1700 <= 448 * 4
    assert np.array_equal(sv.E4M3[codes[0, 0, 0]] * 4, [1, -2, 3, 448])
    assert np.array_equal(sv.E4M3[codes[0, 0, 1]] * 4, [1, 0.1015625, 0, 1664])
    assert not codes[0, 0, 2:].any()


def test_oracle_bounds_hold_and_rank():
    rng = np.random.default_rng(0)
    k = rng.standard_normal((3, 16, 1, 8)) * 3
    table, kv_len = np.array([[2, 0, 1]]), [40]
    b, e = sv.key_bounds(k, np.zeros((3, 1, 2, 8), np.int8), np.zeros((3, 1), np.uint8), [0, 40], kv_len, table, 40)
    q = rng.standard_normal((1, 2, 8))
    lists = sv.select_pages(q, b, e, [0, 1], kv_len, table, 16, 1, 0, 0)
    for j in range(3):
        rows = k[table[0, j], : 16 if j < 2 else 8, 0]
        unit = 2.0 ** (int(e[table[0, j], 0]) - 127)
        assert (rows <= b[table[0, j], 0, 0] * unit).all() and (rows >= b[table[0, j], 0, 1] * unit).all()
    assert lists.shape == (1, 1, 1) and 0 <= lists[0, 0, 0] < 3
    assert (sv.select_pages(q, b, e, [0, 1], kv_len, table, 16, 5, 1, 1) == [[[0, 1, 2, -1, -1]]]).all()
    table[0, 1] = -1
    assert (sv.select_pages(q, b, e, [0, 1], kv_len, table, 16, 5, 1, 1) == [[[0, 2, -1, -1, -1]]]).all()


def test_scores_reach_another_cta_only_once_it_runs():
    """Distributed shared memory may be accessed only while its CTA runs."""
    kernel = body("qdq_pages.cu", "select_kernel(const PagesArgs a)")
    assert kernel.index("cluster_sync()") < kernel.index("store_to_rank0") < kernel.rindex("cluster_sync()")
    assert "return;" not in kernel[:kernel.rindex("cluster_sync()")], "every thread passes both barriers"


def test_the_workspace_is_ready_when_create_returns():
    create = body("qdq_paged.cu", "int qdq_paged_create(")
    assert "cudaMemset(" in body("qdq_attend_rows.cu", "int rows_create(")
    assert create.index("rows_create(") < create.index("cudaStreamSynchronize(nullptr)")


def test_register_shares_of_the_widening_kernel():
    from quant_dequant_gemv_gb300 import build
    text = (CSRC / "qdq_attend.cu").read_text()
    inc, dec = (sorted(int(x) for x in re.findall(r"setmaxnreg\.%s\S* (\d+);" % way, text))[0] for way in ("inc", "dec"))
    assert 2 * inc + 2 * dec == 4 * build.REGISTERS_E4M3["qdq_attend.cu"][1]
    with pytest.raises(RuntimeError):
        build.check_registers("qdq_attend.cu", "", build.REGISTERS_E4M3)


def test_rows_work_split(tmp_path):
    """The kernel's own work split, compiled for the host (tests/rows_plan_check.cpp)."""
    exe = tmp_path / "rows_plan_check"
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{CSRC}", str(ROOT / "tests" / "rows_plan_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
