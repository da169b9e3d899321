"""The serving kernels built with -DQDQ_DEBUG: checks (QDQ_CHECK) of the rows, pages and alignment of
the append; of the attention's page-table entries, tensor-copy coordinates and ring places, zeroed rows
of values, output rows, partial results and counters; of sampling's slices, bins, list and tokens. Each
records QDQ_ERR_BOUNDS and skips the access."""
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

import pytest

from quant_dequant_gemv_gb300 import build

ROOT = Path(__file__).resolve().parents[1]
UNITS = ["qdq_paged.cu", "qdq_attend.cu", "qdq_sample.cu", "qdq_api.cu"]


@pytest.mark.skipif(shutil.which("nvcc") is None and not Path("/usr/local/cuda/bin/nvcc").exists(),
                    reason="no CUDA toolkit")
def test_debug_units_compile(tmp_path):
    def one(src):
        return subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-DQDQ_DEBUG", "-Xptxas=-v", "-c",
                               str(build.CSRC / src), "-o", str(tmp_path / (src + ".o"))], capture_output=True, text=True)

    with ThreadPoolExecutor(len(UNITS)) as ex:
        results = dict(zip(UNITS, ex.map(one, UNITS)))
    for src, r in results.items():
        assert r.returncode == 0, r.stderr[-3000:]
        if src in build.REGISTERS:
            build.check_registers(src, r.stdout + r.stderr)


@pytest.mark.gpu
def test_serving_calls_without_a_check_firing():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, QDQ_BUILD_DIR=str(ROOT / "quant_dequant_gemv_gb300" / "_build" / "debug"),
               QDQ_EXTRA_NVCC_FLAGS="-DQDQ_DEBUG", PYTHONPATH=str(ROOT) + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, str(ROOT / "tests" / "debug_serving_run.py")], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "no check fired" in r.stdout
