"""Plain NumPy references, in float64, of the serving calls: the append of new tokens to a paged
cache, attention over it, and sampling. Written from the definitions; loops over tokens and heads.

Arrays are float64 holding the values of whatever type the device tensors have; nothing here
rounds to 16 bits (the tests count that rounding)."""
from __future__ import annotations

import numpy as np


def tokens_of(q_start, kv_len, n_tokens):
    """(token, sequence, position) of every row that belongs to a sequence."""
    out = []
    for s in range(len(kv_len)):
        a, b = int(q_start[s]), int(q_start[s + 1])
        for t in range(a, b):
            out.append((t, s, int(kv_len[s]) - (b - a) + (t - a)))
    assert all(t < n_tokens for t, _, _ in out)
    return out


def row_of(page_table, n_pages, page_size, s, j):
    """(page, row) of position j of sequence s, or None where it is absent."""
    if j < 0 or j // page_size >= page_table.shape[1]:
        return None
    page = int(page_table[s, j // page_size])
    return (page, j % page_size) if 0 <= page < n_pages else None


def head_norm(x, w, eps):
    return x if w is None else x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w


def rotate(x, pos, rope_dim, interleaved, base):
    """x [heads, dim] turned at position pos."""
    y = x.copy()
    i = np.arange(rope_dim // 2)
    angle = pos * base ** (-2.0 * i / max(rope_dim, 1))
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rope_dim // 2)
    y[:, a] = x[:, a] * np.cos(angle) - x[:, b] * np.sin(angle)
    y[:, b] = x[:, a] * np.sin(angle) + x[:, b] * np.cos(angle)
    return y


def append(q, k, v, q_start, kv_len, page_table, n_pages, page_size, dim, rope_dim, interleaved, base=10000.0,
           q_norm=None, k_norm=None, eps=1e-5):
    """{token: q row [heads, dim]}, {(page, row): (k [kv, dim], v [kv, dim])}."""
    q_out, cache = {}, {}
    for t, s, p in tokens_of(q_start, kv_len, len(q)):
        qh = head_norm(q[t].reshape(-1, dim), q_norm, eps)
        q_out[t] = rotate(qh, p, rope_dim, interleaved, base) if p >= 0 else np.zeros_like(qh)
        at = row_of(page_table, n_pages, page_size, s, p)
        if at is not None:
            kh = head_norm(k[t].reshape(-1, dim), k_norm, eps)
            cache[at] = (rotate(kh, p, rope_dim, interleaved, base), v[t].reshape(-1, dim))
    return q_out, cache


def attention(q, k_pages, v_pages, q_start, kv_len, page_table, scale, window=0):
    """out [tokens, heads, dim], lse [tokens, heads] and, for error bounds, sum_j a_j |v_j| and
    the largest sum_d |q_d k_jd| of a row; rows of no sequence are NaN.
    q: [tokens, heads, dim]; pages: [n_pages, page_size, kv, dim]."""
    n_pages, page_size, kv, dim = k_pages.shape
    T, H, _ = q.shape
    out, spread = np.full((T, H, dim), np.nan), np.zeros((T, H, dim))
    lse, reach = np.full((T, H), np.nan), np.zeros((T, H))
    for t, s, p in tokens_of(q_start, kv_len, T):
        at = [row_of(page_table, n_pages, page_size, s, j) for j in range(max(0, p - window + 1) if window else 0, p + 1)]
        at = [x for x in at if x is not None]
        out[t], lse[t] = 0.0, -np.inf
        if not at:
            continue
        pg, rw = np.array(at).T
        for h in range(H):
            K, V = k_pages[pg, rw, h // (H // kv)], v_pages[pg, rw, h // (H // kv)]
            x = K @ q[t, h] * scale
            m = x.max()
            w = np.exp(x - m)
            out[t, h] = w @ V / w.sum()
            spread[t, h] = w @ np.abs(V) / w.sum()
            lse[t, h] = m + np.log(w.sum())
            reach[t, h] = (np.abs(K) @ np.abs(q[t, h])).max() * abs(scale)
    return out, lse, spread, reach


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log of its share of the kept mass) of one row."""
    x = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    if not (x > -np.inf).any():
        return -1, -np.inf
    order = np.argsort(-x, kind="stable")
    if not temperature > 0:
        return int(order[0]), 0.0
    order = order[x[order] > -np.inf]
    w = np.exp((x - x[order[0]]) / temperature)
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        before = np.cumsum(w[order]) - w[order]
        order = order[: max(1, int((before < top_p * w[order].sum()).sum()))]
    order = np.sort(order[w[order] >= min(min_p, 1.0)])
    mass = np.cumsum(w[order])
    at = min(int((mass <= u * mass[-1]).sum()), len(order) - 1)
    share = w[order[at]] / mass[-1]
    return int(order[at]), float(np.log(share)) if share > 0 else -np.inf
