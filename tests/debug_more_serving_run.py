"""The calls over e4m3 caches and over chosen pages against the library built with -DQDQ_DEBUG (device-side
index and alignment checks that record QDQ_ERR_BOUNDS and skip the access instead of trapping).

Run as a separate process by tests/test_debug_more_serving.py, with QDQ_BUILD_DIR and
QDQ_EXTRA_NVCC_FLAGS set, so that the debug library is the one loaded. Every case must match the
oracle as in tests/test_gpu_more_serving.py, which also reads the device status, and leave it at 0."""
import sys

import torch

from quant_dequant_gemv_gb300 import build, qdq
from tests import test_gpu_more_serving as t


def main():
    path = build.build()
    assert "QDQ_DEBUG" in " ".join(build.NVCC_FLAGS), "not a debug build"
    torch.cuda.set_device(0)
    print("library", path)
    # append: pair layouts, norms, windows of tokens, growing scales, absent pages
    for in_dtype, dim, heads, kv, page, inter, norm in (("f32", 64, 4, 2, 16, True, True), ("bf16", 128, 32, 1, 64, False, True),
                                                        ("f16", 64, 7, 7, 256, False, False)):
        t.test_append(qdq, in_dtype, dim, heads, kv, page, inter, 1, norm)
    t.test_append_many_sequences_and_a_long_prompt(qdq)
    t.test_append_token_by_token(qdq, 128, 1)
    t.test_append_bad_pages_and_negative_positions(qdq)
    # attention: few rows and many, every page size, cut items, windows, empty rows
    for dim, heads, kv, page in ((64, 4, 4, 16), (128, 8, 1, 64), (128, 6, 2, 16), (64, 12, 1, 128), (128, 32, 1, 256)):
        for lens in ([(1, 130), (1, 0), (1, 257), (0, 9), (1, 15)], [(37, 0), (1, 200), (70, 61)], [(150, 150)]):
            t.test_attention(qdq, "bf16" if dim == 64 else "f32", dim, heads, kv, page, lens)
    t.test_attention_window(qdq, 100, [(90, 200), (1, 128), (260, 0)])
    t.test_attention_bad_pages_and_empty_rows(qdq)
    t.test_attention_kv_len_past_the_table_and_no_table(qdq)
    t.test_attention_long_single_tokens(qdq, 4097, 8)
    t.test_attention_many_sequences(qdq)
    # bounds, selection, lists
    for dtype in ("e4m3", "bf16"):
        t.test_bounds(qdq, dtype, 128, 3, 256)
        t.test_bounds_of_many_tokens(qdq, dtype)
        t.test_select(qdq, dtype, 64, 32, 1, 4, 1, 2)
        t.test_attention_pages(qdq, dtype, 128, 6, 2, 16, 24)
        t.test_attention_pages(qdq, dtype, 64, 48, 2, 256, 5)
        t.test_a_decode_step_over_chosen_pages(qdq, dtype)
    t.test_select_one_token_over_many_pages(qdq)
    t.test_select_ties_and_absent_pages(qdq)
    t.test_attention_pages_odd_lists(qdq, "e4m3")
    rc = qdq.get_device_status()
    if rc != 0:
        raise SystemExit(f"device status {rc} ({qdq.status_string(rc)})")
    print("debug build, e4m3 caches and chosen pages: every case within the bound, no check fired")


if __name__ == "__main__":
    sys.exit(main())
