"""The kernels of e4m3 caches and of chosen pages built with -DQDQ_DEBUG: checks (QDQ_CHECK) of tokens,
pages, lists, copies' places, partial results, output rows and scores. Each records QDQ_ERR_BOUNDS and
skips the access."""
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

import pytest

from quant_dequant_gemv_gb300 import build

ROOT = Path(__file__).resolve().parents[1]
UNITS = ["qdq_append8.cu", "qdq_attend_rows.cu", "qdq_pages.cu"]


@pytest.mark.skipif(shutil.which("nvcc") is None and not Path("/usr/local/cuda/bin/nvcc").exists(),
                    reason="no CUDA toolkit")
def test_debug_units_compile(tmp_path):
    def one(src):
        return subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-DQDQ_DEBUG", "-c", str(build.CSRC / src), "-o",
                               str(tmp_path / (src + ".o"))], capture_output=True, text=True)

    with ThreadPoolExecutor(len(UNITS)) as ex:
        for r in ex.map(one, UNITS):
            assert r.returncode == 0, r.stderr[-3000:]


@pytest.mark.gpu
def test_the_calls_without_a_check_firing():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, QDQ_BUILD_DIR=str(ROOT / "quant_dequant_gemv_gb300" / "_build" / "debug"),
               QDQ_EXTRA_NVCC_FLAGS="-DQDQ_DEBUG", PYTHONPATH=str(ROOT) + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, str(ROOT / "tests" / "debug_more_serving_run.py")], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "no check fired" in r.stdout
