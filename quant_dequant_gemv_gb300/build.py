"""Builds libqdq.so in-tree (quant_dequant_gemv_gb300/_build/) with nvcc for sm_103a.

The translation units compile in parallel; the shared library is relinked only
when a source or header changed (content hash).
"""
from __future__ import annotations

import hashlib
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD = Path(os.environ.get("QDQ_BUILD_DIR", PKG / "_build"))
LIB = BUILD / "libqdq.so"
SOURCES = ["qdq_api.cu", "qdq_dequant.cu", "qdq_stream.cu", "qdq_stream1.cu", "qdq_mma.cu", "qdq_noalloc.cu",
           "qdq_llama.cu", "qdq_quantize.cu", "qdq_gemv_more.cu", "qdq_paged.cu", "qdq_attend.cu", "qdq_sample.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              f"-I{INCLUDE}", f"-I{CSRC}"] + os.environ.get("QDQ_EXTRA_NVCC_FLAGS", "").split()


# Kernels that move registers between their warps: the shares add up to what the launch has only
# with this many a thread, and a kernel that asked for more would wait for ever.
REGISTERS = {"qdq_attend.cu": ("attend_kernel", 168)}


def check_registers(src: str, ptxas: str) -> None:
    """Raises if a kernel of REGISTERS[src] was given another number of registers (ptxas -v's report)."""
    name, want = REGISTERS[src]
    got = re.findall(r"Compiling entry function '(\w*%s\w*)'.*?Used (\d+) registers" % name, ptxas, re.S)
    bad = sorted({int(n) for _, n in got if int(n) != want})
    if not got or bad:
        raise RuntimeError(f"{src}: {name} has {bad or 'no'} registers a thread, and its setmaxnreg shares need {want}: "
                           "built with another toolkit or other flags (QDQ_EXTRA_NVCC_FLAGS), they have to be set anew")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqdq")


def _digest() -> str:
    h = hashlib.sha256()
    for p in sorted(list(CSRC.glob("*")) + list(INCLUDE.glob("*.h"))):
        h.update(p.name.encode())
        h.update(p.read_bytes())
    h.update(" ".join(ARCH + NVCC_FLAGS).encode())
    return h.hexdigest()[:16]


def build(verbose: bool = False, force: bool = False) -> Path:
    BUILD.mkdir(parents=True, exist_ok=True)
    stamp = BUILD / "stamp"
    tag = _digest()
    if not force and LIB.exists() and stamp.exists() and stamp.read_text() == tag:
        return LIB
    cc = nvcc()

    def compile_one(src: str) -> Path:
        obj = BUILD / (Path(src).stem + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", str(CSRC / src), "-o", str(obj)]
        if verbose or src in REGISTERS:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if src in REGISTERS:
            check_registers(src, r.stdout + r.stderr)
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = BUILD / "libqdq.so.tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", str(tmp), *map(str, objs)], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    stamp.write_text(tag)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, force=True))
