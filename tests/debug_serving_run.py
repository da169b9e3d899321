"""Serving calls against the library built with -DQDQ_DEBUG (device-side index and alignment checks
that record QDQ_ERR_BOUNDS and skip the access instead of trapping).

Run as a separate process by tests/test_debug_serving.py, with QDQ_BUILD_DIR and
QDQ_EXTRA_NVCC_FLAGS set, so that the debug library is the one loaded. Every case must match the
oracle as in tests/test_gpu_serving.py, which also reads the device status, and leave it at 0."""
import sys

import numpy as np
import torch

from quant_dequant_gemv_gb300 import build, qdq
from tests import test_gpu_serving as t


def main():
    path = build.build()
    assert "QDQ_DEBUG" in " ".join(build.NVCC_FLAGS), "not a debug build"
    torch.cuda.set_device(0)
    print("library", path)
    # append: both pair layouts, norms, strided rows, one token, many sequences, absent pages
    for i, (dtype, in_dtype, dim, heads, kv, inter) in enumerate([("f16", "f32", 64, 4, 2, True), ("bf16", "bf16", 128, 7, 7, False),
                                                                 ("bf16", "f32", 128, 32, 1, False)]):
        b = t.make(qdq, [(1, 0), (5, 30), (0, 12), (33, 0), (1, 77)], heads, kv, dim, 16, dtype, rope_dim=dim // (1 + i % 2),
                   interleaved=inter, seed=i, extra_tokens=2)
        t.check_append(qdq, b, in_dtype, i != 1, dim // (1 + i % 2), inter, fused=i > 0)
    lens = [(int(n), int(x)) for n, x in np.random.default_rng(5).integers(0, 3, (700, 2))]
    t.check_append(qdq, t.make(qdq, lens, 2, 1, 64, 16, "bf16", seed=3, interleaved=False), "f32", True, 64, False, fused=True)
    t.test_append_bad_pages_and_negative_positions(qdq)
    t.test_append_far_positions(qdq)
    # attention: single tokens, chunks and both, every page size, cut items, windows, empty rows
    for i, (dtype, dim, heads, kv, page) in enumerate([("f16", 64, 8, 2, 16), ("bf16", 128, 6, 2, 32), ("f16", 128, 32, 1, 256),
                                                       ("bf16", 64, 5, 1, 128), ("f16", 128, 8, 1, 64)]):
        for lens in ([(1, 0)], [(1, 130), (1, 0), (1, 257), (0, 9), (1, 15)], [(37, 0), (1, 200), (70, 61)], [(150, 150)]):
            b = t.make(qdq, lens, heads, kv, dim, page, dtype, seed=i, extra_tokens=1, layers=2)
            t.fill_held(b, layer=1)
            t.check_attention(qdq, b, layer=1, window=(0, 100)[i % 2], out_dtype=("f32", None)[i % 2], pad=(0, 64)[i % 2])
    t.test_attention_bad_pages_and_empty_rows(qdq)
    t.test_attention_kv_len_past_the_table(qdq)
    t.test_attention_long_single_tokens(qdq, 4097)
    t.test_attention_without_any_page(qdq)
    # sampling: one CTA to eight a row, lists, wide cuts, ties, empty rows
    for vocab in (1, 31, 4097, 32000, 262144):
        t.test_sample(qdq, "f32" if vocab != 4097 else "bf16", vocab)
    t.test_sample_ties_and_extremes(qdq)
    t.test_sample_rows_with_nothing(qdq)
    t.test_sample_wide_cuts(qdq, "bf16", 50000)
    t.test_sample_extreme_parameters(qdq)
    rc = qdq.get_device_status()
    if rc != 0:
        raise SystemExit(f"device status {rc} ({qdq.status_string(rc)})")
    print("debug build, serving calls: every case within the bound, no check fired")


if __name__ == "__main__":
    sys.exit(main())
