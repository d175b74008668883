"""Plain restatements of the page and tree operators (whole numbers and byte
moves), one element at a time, and the mask of a tree from its parents."""

from __future__ import annotations

import numpy as np

INVALID, CAPACITY = 1, 3


def reserve(seq_lens, new_tokens, free_pages, num_free, table, page, num_tokens):
    """(table, seq_lens, num_free, cu_tokens, positions, slots, status)."""
    num_pages, max_len = len(free_pages), table.shape[1] * page
    table = table.copy()
    status = set()
    if not 0 <= num_free <= num_pages:
        num_free = 0
        status.add(INVALID)
    out, cu, pos, slots = [], [0], [], []
    asked = taken = 0  # pages wanted so far, and given
    for b, (n, m) in enumerate(zip(map(int, seq_lens), map(int, new_tokens))):
        ok = n >= 0 and m >= 0
        count = m if ok else 0
        if ok and n + m > max_len:
            ok = False
        if not ok:
            status.add(INVALID)
        held, want = -(-max(n, 0) // page), -(-(max(n, 0) + count) // page)
        need = want - held if ok else 0
        if need:
            asked += need
            if asked > num_free:
                ok = False
                status.add(CAPACITY)
            else:
                for j in range(need):
                    table[b, held + j] = free_pages[num_free - 1 - (asked - need + j)]
                taken = asked
        for t in range(count):
            pos.append(n + t if ok else 0)
            slots.append(int(table[b, (n + t) // page]) * page + (n + t) % page if ok else -1)
        cu.append(len(pos))
        out.append(n + count if ok else n)
    if len(pos) > num_tokens:
        status.add(INVALID)
    pos, slots = (pos + [0] * num_tokens)[:num_tokens], (slots + [-1] * num_tokens)[:num_tokens]
    return (table, np.array(out, np.int32), num_free - taken, np.array(cu, np.int32), np.array(pos, np.int32),
            np.array(slots, np.int64), INVALID if INVALID in status else CAPACITY if status else 0)


def release(seq_lens, keep_lens, free_pages, num_free, table, page):
    """(free_pages, num_free, status)."""
    free_pages, max_len = free_pages.copy(), table.shape[1] * page
    status = 0
    if not 0 <= num_free <= len(free_pages):
        num_free, status = 0, INVALID
    for b, (n, keep) in enumerate(zip(map(int, seq_lens), map(int, keep_lens))):
        if not 0 <= keep <= n <= max_len:
            status = status or INVALID
            continue
        for j in range(-(-keep // page), -(-n // page)):
            if num_free == len(free_pages):
                status = CAPACITY
                continue
            free_pages[num_free] = table[b, j]
            num_free += 1
    return free_pages, num_free, status


def commit(rows, ctx, path):
    """A sequence's rows (slots, ...) after the nodes of `path` moved to the front of its tree."""
    out = rows.copy()
    for i, node in enumerate(path):
        out[ctx + i] = rows[ctx + node]
    return out


def tree_mask(parents, words):
    """(nodes, words) uint32: each node's ancestors and itself."""
    bits = np.zeros((len(parents), words * 32), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            bits[i] = bits[p]
        bits[i, i] = True
    return np.packbits(bits.astype(np.uint8), axis=-1, bitorder="little").view(np.uint32)
