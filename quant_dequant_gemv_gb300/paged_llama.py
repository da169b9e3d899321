"""A Llama-architecture model over block-quantised weights that serves several sequences at once.

Up to eight token rows a step, of any sequences: prompt pieces and single tokens mix freely. Per
layer the rows go through two plans (rmsnorm + q/k/v; o, gate/up, down with the residuals), and
between them the cache append and the attention over the paged cache; the head's logits go to
sampling. The weights are multiplied once for all rows of a step.

    python -m quant_dequant_gemv_gb300.paged_llama        # a few sequences of a random small model
"""
from __future__ import annotations

import operator

from . import qdq, synth

ROWS = 8  # plans take at most eight columns


class PagedLlama:
    """embd, output: (type, W); layers: per layer a dict of q k v o gate up down -> (type, W) and
    attn_norm, ffn_norm -> fp32 tensors (as for qdq.Llama); head dims of 64 or 128. The tensors
    must outlive the model."""

    def __init__(self, dim, hidden, n_layers, n_heads, n_kv_heads, vocab, embd, layers, output_norm, output,
                 n_pages: int, page_size: int = 16, max_seqs: int = ROWS, max_pages: int = 64, rope_base=10000.0,
                 norm_eps=1e-5):
        import torch
        self.dim, self.vocab, self.embd, self.page_size, self.max_pages = dim, vocab, embd, page_size, max_pages
        kv = n_kv_heads * (dim // n_heads)
        new = lambda n, t=torch.float32: torch.zeros(ROWS, n, dtype=t, device="cuda")
        self.h, self.q, self.k, self.v = new(dim), new(dim), new(kv), new(kv)
        self.att, self.gate, self.up, self.logits = new(dim), new(hidden), new(hidden), new(vocab)
        self.q16 = new(dim, torch.float16)
        pools = torch.zeros(2, n_layers, n_pages, page_size, n_kv_heads, dim // n_heads, dtype=torch.float16,
                            device="cuda")
        self.pools = pools
        self.cache = qdq.PagedCache(pools[0], pools[1], n_heads, rope_base=rope_base)
        norm = lambda w: {"x_op": qdq.X_RMSNORM, "norm_w": w, "eps": norm_eps}
        self._before, self._after = [], []
        for w in layers:
            self._before.append(qdq.Plan(
                [(*w["q"], dim, dim, self.h, self.q), (*w["k"], kv, dim, self.h, self.k),
                 (*w["v"], kv, dim, self.h, self.v)], [0, 0, 0], ROWS, opts=[norm(w["attn_norm"])] * 3))
            self._after.append(qdq.Plan(
                [(*w["o"], dim, dim, self.att, self.h), (*w["gate"], hidden, dim, self.h, self.gate),
                 (*w["up"], hidden, dim, self.h, self.up), (*w["down"], dim, hidden, self.gate, self.h)],
                [0, 1, 1, 2], ROWS,
                opts=[{"y_op": qdq.Y_ADD}, norm(w["ffn_norm"]), norm(w["ffn_norm"]),
                      {"x_op": qdq.X_SWIGLU, "x2": self.up, "y_op": qdq.Y_ADD}]))
        self._head = qdq.Plan([(*output, vocab, dim, self.h, self.logits)], [0], ROWS, opts=[norm(output_norm)])
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        # every step has max_seqs sequences, those without new tokens among them, so the batch's
        # arrays and their sizes never change
        self.max_seqs = max_seqs
        self.q_start, self.kv_len, self.table = i32(max_seqs + 1), i32(max_seqs), i32(max_seqs, max_pages) - 1
        self.batch = qdq.PagedBatch(self.q_start, self.kv_len, self.table, ROWS)
        self.tokens = torch.zeros(ROWS, dtype=torch.int64, device="cuda")
        self.logprobs = torch.zeros(ROWS, device="cuda")
        self._free = list(range(n_pages))
        self._pages: list[list[int]] = [[] for _ in range(max_seqs)]
        self.lengths = [0] * max_seqs

    def release(self, seq: int) -> None:
        """Ends a sequence: its pages are free again."""
        self._free += self._pages[seq]
        self._pages[seq] = []
        self.lengths[seq] = 0

    def _word(self, token) -> int:
        try:
            word = operator.index(token)
        except TypeError:
            word = -1
        if not 0 <= word < self.vocab:  # (-1 is what sampling draws from a row of nothing)
            raise ValueError(f"tokens 0 to {self.vocab - 1} are needed, not {token!r}")
        return word

    def step(self, work: dict[int, list[int]], u, stream=None, **sampling) -> dict[int, tuple[int, int]]:
        """Runs the new tokens of each sequence in `work` (at most eight in all) and draws the next
        token of each with the random numbers u [8] and sampling's per-row tensors (temperature,
        top_k, top_p, min_p: see qdq.sample). Returns {sequence: (row, next token)}; `logits` and
        `logprobs` hold the rows'. A step that raises leaves the sequences as they were."""
        import torch
        rows = sum(len(t) for t in work.values())
        if not 1 <= rows <= ROWS or any(not 0 <= s < self.max_seqs or not t for s, t in work.items()):
            raise ValueError(f"1 to {ROWS} tokens of sequences 0 to {self.max_seqs - 1}")
        order = sorted(work)
        words = [self._word(t) for s in order for t in work[s]]
        need = {s: -(-(self.lengths[s] + len(work[s])) // self.page_size) - len(self._pages[s]) for s in order}
        if sum(need.values()) > len(self._free) or \
                any(len(self._pages[s]) + need[s] > self.max_pages for s in order):
            raise RuntimeError("the page pool, or a sequence's page table, is full")
        # what the sequences hold after the step: theirs once it has run whole, so that one that is
        # refused on the way (a sampling argument, say) can be run again
        free, pages, lengths = list(self._free), {}, list(self.lengths)
        for s in order:
            pages[s] = self._pages[s] + [free.pop() for _ in range(need[s])]
            lengths[s] += len(work[s])
        starts, last, at = [0], {}, 0
        for s in range(self.max_seqs):
            at += len(work.get(s, ()))
            starts.append(at)
            if s in work:
                last[s] = at - 1
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            self.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
            self.kv_len.copy_(torch.tensor(lengths, dtype=torch.int32))
            for s in order:
                if need[s]:
                    self.table[s, :len(pages[s])] = torch.tensor(pages[s], dtype=torch.int32).cuda()
            kind, W = self.embd
            row = self.dim // qdq.block_weights(kind) * qdq.block_bytes(kind)
            self.h[rows:].zero_()
            for r, token in enumerate(words):
                qdq.dequant(kind, W.view(-1)[token * row:], self.dim, self.h[r])
            for l, (before, after) in enumerate(zip(self._before, self._after)):
                before.run()
                self.cache.append(l, self.batch, self.q, self.k, self.v, self.q16)
                self.cache.attention(l, self.batch, self.q16, self.att)
                after.run()
            self._head.run()
            qdq.sample(self.logits, u, self.tokens, logprobs=self.logprobs, **sampling)
            drawn = self.tokens.tolist()
        self._free, self.lengths = free, lengths
        for s in order:
            self._pages[s] = pages[s]
        return {s: (r, drawn[r]) for s, r in last.items()}

    def close(self) -> None:
        for plan in (*self._before, *self._after, self._head):
            plan.close()
        self.cache.close()


def device_model(m: dict) -> dict:
    """synth.gen_llama_model's tensors on the GPU, as PagedLlama (and qdq.Llama) take them."""
    import numpy as np
    import torch
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    layers = [{**{k: (w[k][0], dev(w[k][3])) for k in synth.LAYER_TENSORS}, "attn_norm": dev(w["attn_norm"]),
               "ffn_norm": dev(w["ffn_norm"])} for w in m["layers"]]
    return dict(embd=(m["token_embd"][0], dev(m["token_embd"][3])), layers=layers, output_norm=dev(m["output_norm"]),
                output=(m["output"][0], dev(m["output"][3])))


def main() -> None:
    import torch
    cfg = dict(dim=512, hidden=1024, n_layers=2, n_heads=8, n_kv_heads=2, vocab=1000)
    model = PagedLlama(**cfg, **device_model(synth.gen_llama_model(seed=1, norm_scale=0.02, **cfg)), n_pages=32)
    gen = torch.Generator(device="cuda").manual_seed(0)
    prompts = {0: [5, 17, 300, 2, 41], 1: [7], 2: [900, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10]}
    text = {s: list(p) for s, p in prompts.items()}
    waiting = {s: list(p) for s, p in prompts.items()}
    knobs = dict(temperature=torch.full((ROWS,), 0.8, device="cuda"), top_p=torch.full((ROWS,), 0.95, device="cuda"),
                 top_k=torch.full((ROWS,), 40, dtype=torch.int32, device="cuda"))
    while any(len(t) < len(prompts[s]) + 12 for s, t in text.items()):
        work, room = {}, ROWS
        for s in sorted(waiting, key=lambda s: len(waiting[s])):  # single tokens first, then prompt pieces
            piece = waiting[s][:room]
            if piece:
                work[s], room = piece, room - len(piece)
        drawn = model.step(work, torch.rand(ROWS, generator=gen, device="cuda"), **knobs)
        for s, (_, token) in drawn.items():
            del waiting[s][:len(work[s])]
            if not waiting[s]:  # the whole text has been read: the drawn token goes on
                text[s].append(token)
                waiting[s] = [token]
    for s, t in text.items():
        print(f"sequence {s}: {t[:len(prompts[s])]} -> {t[len(prompts[s]):]}")
    model.close()


if __name__ == "__main__":
    main()
