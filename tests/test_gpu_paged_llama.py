"""Several sequences through the paged model against the float64 oracle's forward pass of each.

Every cached row lies within one fp16 step of the oracle's key or value (plus 1e-3 of the row's
largest entry from the second layer on: the layers before it saw rounded queries and weights); the
oracle then takes the GPU's rows (oracle/decode_step.py). Queries and attention weights are rounded
to fp16, 2^-11 each, which with scores of order one moves an attention output by about 4 x 2^-11 of
its values; two layers of that, within 4e-3 of the head row's sum |w x|, bound the logits. Draws
follow from the GPU's own logits.
"""
import numpy as np
import pytest

import oracle
from oracle import decode_step as ds
from oracle import serving as sv
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


def test_sequences_match_the_oracle(lib):
    m = synth.gen_llama_model(seed=31, norm_scale=0.02, **CFG)
    model = lib.PagedLlama(**CFG, **lib.device_model(m), n_pages=12, page_size=16, max_seqs=3, max_pages=4)
    w = ds.from_blocks(ds.LlamaConfig(max_seq=64, **CFG), m)
    rng = np.random.default_rng(3)
    texts = {s: [int(t) for t in rng.integers(0, CFG["vocab"], n)] for s, n in ((0, 21), (1, 9), (2, 18))}
    caches = {s: ds.new_cache(w.cfg) for s in texts}
    at = {s: 0 for s in texts}
    u = torch.full((lib.ROWS,), 0.37, device="cuda")
    top_k = torch.full((lib.ROWS,), 20, dtype=torch.int32, device="cuda")
    while any(at[s] < len(t) for s, t in texts.items()):
        work, room = {}, lib.ROWS
        for s in rng.permutation(3):
            n = min(int(rng.integers(1, 6)), room, len(texts[s]) - at[s])
            if n > 0:
                work[int(s)], room = texts[s][at[s]:at[s] + n], room - n
        drawn = model.step(work, u, top_k=top_k)
        pools = model.pools.cpu().numpy()
        for s, tokens in work.items():
            kc, vc = caches[s]
            for tok in tokens:
                pos = at[s]
                page = model._pages[s][pos // 16]
                kg, vg = pools[:, :, page, pos % 16].reshape(2, CFG["n_layers"], -1)
                tr = {}
                ref = ds.forward(w, kc, vc, tok, pos, trace=tr, rows={"k": kg, "v": vg})
                for l in range(CFG["n_layers"]):
                    for got, want in ((kg[l], tr["k"][l]), (vg[l], tr["v"][l])):
                        step = np.abs(np.spacing(want.astype(np.float16)).astype(np.float64))
                        slack = (1e-5 if l == 0 else 1e-3) * np.abs(want).max()
                        assert np.all(np.abs(got.astype(np.float64) - want) <= step + slack), (s, pos, l)
                at[s] += 1
            row, token = drawn[s]
            logits = model.logits[row].cpu().numpy()
            ot, orows, ocols, ob = m["output"]
            _, S = oracle.gemv(ot, ob, orows, ocols, tr["hn"].astype(np.float32)[None, :])
            assert np.all(np.abs(logits.astype(np.float64) - ref) <= 4e-3 * S[0] + 1e-6), (s, at[s])
            near = [sv.sample(logits, 0.37 + d, top_k=20)[0] for d in (0, -1e-5, 1e-5)]
            assert token in near
    from quant_dequant_gemv_gb300 import qdq
    assert qdq.get_device_status() == 0
    model.release(0)
    assert len(model._free) == 12 - len(model._pages[1]) - len(model._pages[2])
    with pytest.raises(RuntimeError):
        for _ in range(20):  # page tables of four pages
            model.step({1: [1] * 8}, u)
    with pytest.raises(ValueError):
        model.step({0: [1] * 9}, u)
    model.close()


def test_example_runs(lib, capsys):
    lib.main()
    lines = capsys.readouterr().out.strip().splitlines()
    assert len(lines) == 3 and all("->" in x for x in lines)
