"""Rules of the serving kernels and their host code whose breach a GPU may not show (or may only show
by faulting), read off the sources."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "quant_dequant_gemv_gb300" / "csrc"


def body(source: str, head: str) -> str:
    """The braces that follow the first `head` in a file, without comments."""
    text = re.sub(r"//[^\n]*", "", (CSRC / source).read_text())
    at = text.index("{", text.index(head))
    depth = 0
    for end in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return text[at:end + 1]
    raise AssertionError(f"{head} in {source} has no end")


def test_sampling_reaches_other_ctas_only_once_all_have_started():
    """Distributed shared memory may be accessed only while its CTA runs: the barrier of the cluster's
    start is passed before the first call that stores to, or reads from, another CTA."""
    kernel = body("qdq_sample.cu", "sample_kernel(const SampleArgs a)")
    arrive, wait = kernel.index("cluster_started_arrive()"), kernel.index("cluster_started_wait()")
    first = min(m.start() for m in re.finditer(r"send<|gather_|first_counts<|finish<|resolve|narrow<|remote|mapa|"
                                               r"cluster_sync", kernel))
    assert arrive < wait < first
    assert "return;" not in kernel[:wait], "every thread passes the barrier"


def test_a_cache_is_ready_on_every_stream_when_create_returns():
    """The handle's table and counters are written in the default stream, which streams created as
    non-blocking do not follow: create waits for it after the last of those writes."""
    create = body("qdq_paged.cu", "int qdq_paged_create(")
    copy, clear = create.index("cudaMemcpy("), create.index("attend_create(")
    assert "cudaMemset(" in body("qdq_attend.cu", "int attend_create(")
    wait = create.index("cudaStreamSynchronize(nullptr)")
    assert copy < clear < wait < create.index("*out = c;")


def test_a_plan_and_a_model_are_ready_on_every_stream_when_create_returns():
    """The same for a plan's counters, and for a model, whose memory is cleared before its plan is made."""
    create = body("qdq_api.cu", "static int plan_create(")
    assert create.rindex("cudaMemset(") < create.index("cudaStreamSynchronize(nullptr)") < create.index("*plan_out = p;")
    model = body("qdq_llama.cu", "int qdq_llama_create(")
    assert model.rindex("cudaMemset(") < model.index("plan_create_with_attention(")


def test_the_build_refuses_other_register_counts():
    from quant_dequant_gemv_gb300 import build
    entry = "ptxas info    : Compiling entry function '_ZN3qdq{}ILi64EEE' for 'sm_103a'\nptxas info    : Used {} registers, used 1 barriers\n"
    build.check_registers("qdq_attend.cu", entry.format("13attend_kernel", 168) + entry.format("5other", 40))
    for text in (entry.format("13attend_kernel", 168) + entry.format("13attend_kernel", 160), entry.format("5other", 168), ""):
        with pytest.raises(RuntimeError, match="qdq_attend.cu"):
            build.check_registers("qdq_attend.cu", text)
    inc, dec = (int(re.search(r"setmaxnreg\.%s\S* (\d+);" % way, (CSRC / "qdq_attend.cu").read_text()).group(1))
                for way in ("inc", "dec"))
    assert 2 * inc + dec == 3 * build.REGISTERS["qdq_attend.cu"][1]
