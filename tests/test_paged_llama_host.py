"""PagedLlama's bookkeeping without a GPU: the library's calls replaced by recorders that can refuse."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

from quant_dequant_gemv_gb300 import paged_llama, qdq, synth  # noqa: E402

VOCAB, DIM, PAGES = 50, 256, 6


class Refused(RuntimeError):
    pass


@pytest.fixture
def model(monkeypatch):
    """A model of no layers over recorders; `refuse` names the call that raises next."""
    m = paged_llama.PagedLlama.__new__(paged_llama.PagedLlama)
    m.calls, m.refuse, m.drawn = [], None, list(range(paged_llama.ROWS))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "cuda", lambda t, *a, **k: t)

    def recorder(name):
        def call(*a, **k):
            if m.refuse == name:
                raise Refused(name)
            m.calls.append((name, a, k))
            if name == "sample":
                a[2].copy_(torch.tensor(m.drawn))
        return call

    monkeypatch.setattr(qdq, "dequant", recorder("dequant"))
    monkeypatch.setattr(qdq, "sample", recorder("sample"))
    R = paged_llama.ROWS
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    m.__dict__.update(
        dim=DIM, vocab=VOCAB, page_size=4, max_pages=3, max_seqs=3,
        embd=(synth.Q4_K, torch.zeros(VOCAB * DIM // 256 * 144, dtype=torch.uint8)),
        h=torch.zeros(R, DIM), q=None, k=None, v=None, q16=None, att=None, logits=torch.zeros(R, VOCAB), _before=[],
        _after=[], _head=types.SimpleNamespace(run=recorder("head")), cache=None, q_start=i32(4), kv_len=i32(3),
        table=i32(3, 3) - 1, batch=None, tokens=torch.zeros(R, dtype=torch.int64), logprobs=torch.zeros(R),
        _free=list(range(PAGES)), _pages=[[], [], []], lengths=[0, 0, 0])
    return m


U = torch.full((8,), 0.5)


def state(m):
    return sorted(m._free), [list(p) for p in m._pages], list(m.lengths)


def test_a_step_advances_what_it_ran(model):
    assert model.step({0: [1, 2, 3, 4, 5], 2: [49]}, U) == {0: (4, 4), 2: (5, 5)}
    assert model.lengths == [5, 0, 1] and [len(p) for p in model._pages] == [2, 0, 1] and len(model._free) == 3
    model.step({0: [7]}, U)
    assert model.lengths == [6, 0, 1] and model.kv_len.tolist() == [6, 0, 1] and model.q_start.tolist() == [0, 1, 1, 1]
    assert model.table[0, :2].tolist() == model._pages[0] and model.table[2, 0] == model._pages[2][0]
    model.release(0)
    assert model.lengths == [0, 0, 1] and len(model._free) == 5


@pytest.mark.parametrize("tokens", [[-1], [VOCAB], [3, -1], [2 ** 40], [1.5], ["a"], [None]])
def test_a_step_refuses_what_is_no_token(model, tokens):
    """-1 is what sampling answers for a row without any logit; it is no word to go on with."""
    model.step({1: [5]}, U)
    before, calls = state(model), len(model.calls)
    with pytest.raises(ValueError):
        model.step({0: [4], 1: tokens}, U)
    assert state(model) == before and len(model.calls) == calls


def test_tokens_of_any_integer_type_are_taken(model):
    np = pytest.importorskip("numpy")
    model.step({0: [np.int64(3), torch.tensor(4)], 1: [5]}, U)
    rows = [a[1].numel() for n, a, _ in model.calls if n == "dequant"]
    assert rows == [(VOCAB - t) * 144 for t in (3, 4, 5)]


@pytest.mark.parametrize("call", ["dequant", "head", "sample"])
def test_a_refused_step_leaves_the_sequences_as_they_were(model, call):
    """The caller mends the argument and runs the same tokens again, at the same positions."""
    model.step({0: [1, 2, 3], 1: [9]}, U)
    before = state(model)
    model.refuse = call
    with pytest.raises(Refused):
        model.step({0: [4, 5], 2: [6]}, U)
    assert state(model) == before
    model.refuse = None
    assert model.step({0: [4, 5], 2: [6]}, U) == {0: (1, 1), 2: (2, 2)}
    assert model.lengths == [5, 1, 1] and model.kv_len.tolist() == [5, 1, 1]
    assert model.table[0, :2].tolist() == model._pages[0] and model.table[2, 0] == model._pages[2][0]
    held = [p for pages in model._pages for p in pages] + model._free
    assert sorted(held) == list(range(PAGES))


def test_a_sampling_argument_that_qdq_sample_refuses(model, monkeypatch):
    real = []
    monkeypatch.setattr(qdq, "sample", lambda *a, **k: real.append(1) or (_ for _ in ()).throw(ValueError("top_k")))
    with pytest.raises(ValueError):
        model.step({0: [1]}, U, top_k=torch.zeros(8))
    assert real and state(model) == (list(range(PAGES)), [[], [], []], [0, 0, 0])
