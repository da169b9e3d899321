"""The paged model over an e4m3 cache and over chosen pages: it runs, and where the choice holds every
page its results are those of attention over all of them (the weights have two terms and the results
32 bits on both paths, 2^-16 of an attention output; 1e-3 of the largest logit allows for two layers)."""
import numpy as np
import pytest

from quant_dequant_gemv_gb300 import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

CFG = dict(dim=256, hidden=512, n_layers=2, n_heads=4, n_kv_heads=2, vocab=300)


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quant_dequant_gemv_gb300 import build, paged_llama
    build.build()
    torch.cuda.set_device(0)
    return paged_llama


def texts(lib, m, steps=40, **options):
    """The logits of a prompt's pieces and then single tokens of two sequences, with the same tokens throughout."""
    model = lib.PagedLlama(**CFG, **lib.device_model(m), n_pages=20, max_seqs=3, max_pages=8, **options)
    rng = np.random.default_rng(3)
    words = [[int(t) for t in rng.integers(0, CFG["vocab"], 90)] for _ in range(2)]
    u = torch.full((lib.ROWS,), 0.37, device="cuda")
    out, at = [], [0, 0]
    for i in range(steps):
        work = {s: words[s][at[s]:at[s] + (4 - s if i < 10 else 1)] for s in range(2)}
        drawn = model.step(work, u)
        for s in range(2):
            at[s] += len(work[s])
            out.append(model.logits[drawn[s][0]].clone())
    from quant_dequant_gemv_gb300 import qdq
    assert qdq.get_device_status() == 0
    model.release(0)
    model.step({2: words[0][:5]}, u)                     # pages that another sequence has used
    model.close()
    return torch.stack(out)


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_a_choice_of_every_page_changes_nothing(lib, cache):
    m = synth.gen_llama_model(seed=31, norm_scale=0.02, **CFG)
    all_, chosen = (texts(lib, m, cache=cache, select=n) for n in (0, 8))
    assert torch.isfinite(all_).all()
    assert (all_ - chosen).abs().max() <= 1e-3 * all_.abs().max()
    few = texts(lib, m, cache=cache, select=3)
    assert torch.isfinite(few).all()
    assert (few[:36] - all_[:36]).abs().max() <= 1e-3 * all_.abs().max()     # 48 tokens: three pages, every one
    assert not torch.equal(few[-2:], all_[-2:])


def test_options_are_checked(lib):
    for options in (dict(cache="int4"), dict(select=2), dict(select=-1)):
        with pytest.raises(ValueError):
            lib.PagedLlama(**CFG, embd=None, layers=[], output_norm=None, output=None, n_pages=4, **options)
