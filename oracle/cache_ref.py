"""Plain numpy restatement of the cache's own operators, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Rotary positions with several axes and the append, the score modifiers (soft
cap, distance bias, window, documents, prefix), the key weights and the
eviction, each written from its definition in loops over sequences, heads and
tokens; nothing here is shared with the CUDA path.  e4m3 and bf16 roundings
are left to the caller where a comparison wants the value before them.
"""

from __future__ import annotations

import numpy as np

from . import e4m3_table

E4M3_MAX = 448.0


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value of float64 x, ties to even, saturating (NaN stays)."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(np.where(np.isfinite(x), x, 1.0))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.rint(x / step) * step, -E4M3_MAX, E4M3_MAX)


def rotate(x, pos, cos_sin, freq_axis, rot_dim, interleaved):
    """Head rows x (tokens, heads, d) turned by pos (axes, tokens) through the
    table cos_sin (max_pos, rot_dim): pair by pair."""
    half = rot_dim // 2
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        row = cos_sin[pos[freq_axis[i]]].astype(np.float64)
        c, s = row[:, i][:, None], row[:, half + i][:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def append_slots(seq_lens, cu_tokens, num_tokens, block_table, page_size):
    """(token, sequence, index among its new tokens, slot, page, row) of every
    token that has a cache row."""
    out = []
    for b in range(len(seq_lens)):
        n = int(cu_tokens[b + 1]) - int(cu_tokens[b])
        for i in range(n):
            slot = int(seq_lens[b]) - n + i
            if slot >= 0:
                out.append((int(cu_tokens[b]) + i, b, i, slot, int(block_table[b, slot // page_size]), slot % page_size))
    return out


def visible(L, q_len, causal, window=0, key_begin=None, key_end=None, prefix=0):
    """bool (q_len, L): which keys each query token of one sequence sees."""
    see = np.zeros((q_len, max(L, 0)), dtype=bool)
    for i in range(q_len):
        pos = L - q_len + i
        for j in range(L):
            if j < prefix:
                see[i, j] = True
                continue
            ok = j <= pos if causal else True
            if window > 0:
                ok = ok and j >= pos - window + 1
            if key_begin is not None:
                ok = ok and j >= key_begin[i]
            if key_end is not None:
                ok = ok and j < key_end[i]
            see[i, j] = ok
    return see


def cache_rows(cache_values, block_table_row, L, page_size, g):
    """(L, d) rows of one sequence and kv head from a (pages, ps, h_k, d) array of values."""
    j = np.arange(L)
    return cache_values[block_table_row[j // page_size], j % page_size, g]


def logits(q, k, scale, softcap, slopes, L, q_len, h_r):
    """Modified logits (rows, L) of one (sequence, kv head): q (rows, d) packed
    rows, k (L, d), slopes (h_r,) or None."""
    z = scale * (q @ k.T)
    if softcap > 0:
        z = softcap * np.tanh(z / softcap)
    if slopes is not None:
        row = np.arange(q.shape[0])
        pos = L - q_len + row // h_r
        z = z - np.asarray(slopes, dtype=np.float64)[row % h_r][:, None] * np.abs(pos[:, None] - np.arange(L)[None])
    return z


def softmax_rows(z, see):
    """(weights, lse) over the keys each row sees; a row that sees none has
    zero weights and lse -inf."""
    w = np.zeros_like(z)
    lse = np.full(z.shape[0], -np.inf)
    for n in range(z.shape[0]):
        if see[n].any():
            m = z[n, see[n]].max()
            lse[n] = m + np.log(np.exp(z[n, see[n]] - m).sum())
            w[n, see[n]] = np.exp(z[n, see[n]] - lse[n])
    return w, lse


def evict_slots(weights, pos, L, budget, end, keep_first, keep_last):
    """Where each kept slot comes from: source slot of every slot below
    min(L, budget), for one (sequence, kv head)."""
    new = min(L, budget)

    def rank(j):
        if pos[j] < keep_first or pos[j] >= end - keep_last:
            return (0, 0.0, j)
        w = float(weights[j])
        return (2, 0.0, j) if np.isnan(w) else (1, -w + 0.0, j)

    kept = set(sorted(range(L), key=rank)[:new])
    movers = [j for j in range(new, L) if j in kept]
    src = []
    for j in range(new):
        src.append(j if j in kept else movers.pop(0))
    assert not movers
    return np.asarray(src, dtype=np.int64)


def values_of(codes: np.ndarray) -> np.ndarray:
    """float64 values of e4m3 codes (NaN codes are NaN)."""
    return np.asarray(e4m3_table(), dtype=np.float64)[codes]
