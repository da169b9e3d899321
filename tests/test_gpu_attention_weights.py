"""The paged attention's softmax weights: any finite scale.

* Scales. The tolerance is test_gpu_serving's. At scale 0 every position weighs the same.
"""
import pytest

from tests.test_gpu_serving import batch_of, check_attention, fill_held, make, qdq  # noqa: F401

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
