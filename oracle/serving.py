"""Plain NumPy references, in float64, of the serving calls: the append of new tokens to a paged
cache (16-bit, or e4m3 with scales), attention over it and over chosen pages, and sampling. Written from the definitions; loops over tokens and heads.

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


# ---- a cache of e4m3 values ----------------------------------------------------------------
E4M3 = np.array([(-1.0) ** (b >> 7) * (2.0 ** -9 * (b & 7) if b >> 3 & 15 == 0 else 2.0 ** ((b >> 3 & 15) - 7) * (1 + (b & 7) / 8))
                 if b & 127 != 127 else np.nan for b in range(256)])
_BY_SIZE = np.array([E4M3[b] for b in range(127)])  # 0 .. 448, rising


def e4m3_byte(x):
    """The bytes of the e4m3 values nearest to x (ties to the even byte, 448 beyond it)."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_BY_SIZE, a), 1, 126)
    lo = hi - 1
    up, down = _BY_SIZE[hi] - a, a - _BY_SIZE[lo]
    b = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    b = np.where(np.isnan(x), 127, b)
    return (b + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def least_exponent(amax, most, lo, hi):
    """The least e in lo..hi with amax <= most * 2^e."""
    e = lo
    while e < hi and amax > most * 2.0 ** e:
        e += 1
    return e


def append_e4m3(x, codes, scales, q_start, kv_len, page_table, n_tokens):
    """Stores the rows x [tokens, kv, dim] (float64, turned) in copies of codes [n_pages, kv, page, dim] and
    scales [n_pages, kv, page / 16] (bytes). Also the unrounded new values in units of their scales, by
    (page, head, row)."""
    codes, scales, exact = codes.copy(), scales.copy(), {}
    n_pages, kv, page, _ = codes.shape
    blocks = {}
    for t, s, p in tokens_of(q_start, kv_len, n_tokens):
        at = row_of(page_table, n_pages, page, s, p)
        if at is not None:
            blocks.setdefault((at[0], at[1] // 16, s), []).append((at[1], t))
    for (pg, b, _), rows in blocks.items():
        for g in range(kv):
            v = np.abs(x[[t for _, t in rows], g])
            amax = np.max(v, initial=0.0, where=np.isfinite(v))
            e, first = least_exponent(amax, 448.0, -40, 40), rows[0][0] % 16
            if first:
                old = int(np.clip(int(scales[pg, g, b]) - 127, -40, 40))
                e = max(e, old)
                for r in range(16 * b, 16 * b + first):
                    codes[pg, g, r] = e4m3_byte(E4M3[codes[pg, g, r]] * 2.0 ** (old - e))
            scales[pg, g, b] = e + 127
            for r, t in rows:
                exact[pg, g, r] = x[t, g] * 2.0 ** -e
                codes[pg, g, r] = e4m3_byte(exact[pg, g, r])
    return codes, scales, exact


def values_e4m3(codes, scales):
    """Pools [n_pages, kv, page, dim] of bytes as values [n_pages, page, kv, dim], as `attention` takes them."""
    e = np.clip(scales.astype(np.int64) - 127, -40, 40)
    return (E4M3[codes] * 2.0 ** np.repeat(e, 16, axis=2)[..., None]).transpose(0, 2, 1, 3)


# ---- pages chosen by bounds of their keys ----------------------------------------------------
def quantised(x):
    """x in units of 2^e with the least e in -100 .. 121 that brings it to 127 at most (121 if there is
    none), and e."""
    v = np.abs(x)
    e = least_exponent(np.max(v, initial=0.0, where=~np.isnan(v)), 127.0, -100, 121)
    return np.nan_to_num(x, posinf=3e38 * 10, neginf=-3e38 * 10) * 2.0 ** -e, e


def key_bounds(k_pages, bounds, scales, q_start, kv_len, page_table, n_tokens):
    """Copies of bounds [n_pages, kv, 2, dim] and scales [n_pages, kv] with the touched pages' new ones;
    k_pages [n_pages, page, kv, dim]."""
    bounds, scales = bounds.copy(), scales.copy()
    n_pages, page, kv, _ = k_pages.shape
    for _, s, p in tokens_of(q_start, kv_len, n_tokens):
        at = row_of(page_table, n_pages, page, s, p)
        if at is None:
            continue
        rows = k_pages[at[0], : min(page, int(kv_len[s]) - p // page * page)]
        for g in range(kv):
            x, e = quantised(np.stack([np.nanmax(rows[:, g], 0), np.nanmin(rows[:, g], 0)]))
            bounds[at[0], g] = np.clip([np.ceil(x[0]), np.floor(x[1])], -127, 127)
            scales[at[0], g] = e + 127
    return bounds, scales


def select_pages(q, bounds, scales, q_start, kv_len, page_table, page_size, n_select, n_first, n_last):
    """[tokens, kv, n_select] page numbers; rows of no sequence are -2. q: [tokens, heads, dim]."""
    n_pages, kv, _, _ = bounds.shape
    T, H, _ = q.shape
    out = np.full((T, kv, n_select), -2)
    b, e = bounds.astype(np.int64), scales.astype(int) - 127
    for t, s, p in tokens_of(q_start, kv_len, T):
        out[t] = -1
        have = [j for j in range(min(p // page_size + 1, page_table.shape[1]) if p >= 0 else 0)
                if 0 <= page_table[s, j] < n_pages]
        for g in range(kv):
            heads = [quantised(q[t, h]) for h in range(g * (H // kv), (g + 1) * (H // kv))]
            rank = []
            for j in have:
                pg = page_table[s, j]
                best = -np.inf
                for x, eq in heads:
                    x = np.rint(x).astype(np.int64)
                    total = int((x * np.where(x >= 0, b[pg, g, 0], b[pg, g, 1])).sum())
                    best = max(best, total * 2.0 ** int(np.clip(eq + e[pg, g], -100, 100)))
                forced = j < n_first or j > p // page_size - n_last
                rank.append((0 if forced else 1, -best, j))
            chosen = sorted(j for _, _, j in sorted(rank)[:n_select])
            out[t, g, : len(chosen)] = chosen
    return out


def attention_pages(q, k_pages, v_pages, lists, q_start, kv_len, page_table, scale):
    """As `attention`, over the positions in the listed pages: lists [tokens, kv, n]."""
    n_pages, page_size, kv, dim = k_pages.shape
    T, H, _ = q.shape
    out, spread = np.full((T, H, dim), np.nan), np.zeros((T, H, dim))
    lse, reach = np.full((T, H), np.nan), np.zeros((T, H))
    for t, s, p in tokens_of(q_start, kv_len, T):
        out[t], lse[t] = 0.0, -np.inf
        for g in range(kv):
            x = lists[t, g]
            use = [int(j) for i, j in enumerate(x) if j >= 0 and (i == 0 or j > x[i - 1])]
            at = [row_of(page_table, n_pages, page_size, s, r) for j in use
                  for r in range(j * page_size, min((j + 1) * page_size, p + 1))]
            at = [y for y in at if y is not None]
            if not at:
                continue
            pg, rw = np.array(at).T
            K, V = k_pages[pg, rw, g], v_pages[pg, rw, g]
            for h in range(g * (H // kv), (g + 1) * (H // kv)):
                x_h = K @ q[t, h] * scale
                w = np.exp(x_h - x_h.max())
                out[t, h] = w @ V / w.sum()
                spread[t, h] = w @ np.abs(V) / w.sum()
                lse[t, h] = x_h.max() + np.log(w.sum())
                reach[t, h] = (np.abs(K) @ np.abs(q[t, h])).max() * abs(scale)
    return out, lse, spread, reach
