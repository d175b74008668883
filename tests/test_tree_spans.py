"""The spans of drafted trees on the host, against the keys their nodes see one
by one; what the call refuses (CPU only)."""

import ctypes

import numpy as np
import pytest

import paged_fp8_kv_gb300 as mj

BAD, UNSUP = mj.MJ_ERR_INVALID_ARG, mj.MJ_ERR_UNSUPPORTED


def _seen(L, nodes, begin, prefix):
    """Keys that any of a sequence's nodes may see: the tree's, and context keys by the nodes' ranges."""
    nodes = max(0, min(nodes, len(begin), L))
    j, ctx = np.arange(L), L - nodes
    keep = j >= ctx
    for i in range(nodes):
        keep |= (j >= begin[i]) & (j < ctx)
        if prefix is not None:
            keep |= j < min(prefix, ctx)
    return keep


def _covers(span, keep):
    j = np.arange(len(keep))
    return not (keep & ~((j < span[0]) | ((j >= span[1]) & (j < span[2])))).any()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_len", [1, 4, 16, 61, 70])
def test_spans_hold_what_the_nodes_see(q_len, causal):
    rng = np.random.default_rng(q_len)
    for case in range(60):
        nb = int(rng.integers(1, 6))
        p = mj.make_params(nb, q_len, 2, 4, 16, 40, 100, causal=causal)
        lens = rng.integers(0, 641, nb).astype(np.int32)
        nodes = rng.integers(-2, q_len + 3, nb).astype(np.int32)
        held = np.clip(nodes, 0, np.minimum(q_len, lens))
        # windows from one key to wider than the tree; rows without a node hold anything
        begin = (lens - held)[:, None] + rng.integers(0, 5, (nb, q_len)) - rng.integers(1, 100, (nb, 1))
        begin = begin.astype(np.int32)
        for b in range(nb):
            begin[b, held[b] :] = rng.choice([-(2**31), 2**31 - 1, 0, int(lens[b])])
        prefix = rng.integers(-3, 700, nb).astype(np.int32) if case % 2 else None
        spans, plan = mj.tree_spans(p, mj.ScoreMod(key_begin=begin, prefix=prefix), lens, nodes)
        for b in range(nb):
            keep = _seen(int(lens[b]), int(nodes[b]), begin[b], None if prefix is None else int(prefix[b]))
            assert _covers(spans[b], keep), (case, b)
            if held[b] == 0:
                assert spans[b].tolist() == [0, 0, 0, 0] and plan[b] == 0
                continue
            ctx = int(lens[b] - held[b])
            pfx = 0 if prefix is None else int(np.clip(prefix[b], 0, ctx))
            first = max(pfx, min(max(0, int(begin[b, : held[b]].min())), ctx))
            assert spans[b].tolist() == [pfx, first, lens[b], 0]  # and no more than that
            assert -(-int(plan[b]) // 128) == max(1, -(-pfx // 128) + -(-int(lens[b]) // 128) - max(first // 128, -(-pfx // 128)))


def test_short_windows_of_a_small_tree():
    """Four nodes of 64 rows under a window of 16 keys, rows without a node at the context's end: a row's place among
    the rows says nothing about where its context ends."""
    begin = np.full((1, 64), 2996, np.int32)
    begin[0, :4] = [2981, 2982, 2983, 2984]
    for causal in (True, False):
        p = mj.make_params(1, 64, 2, 4, 16, 200, 300, causal=causal)
        spans, plan = mj.tree_spans(p, mj.ScoreMod(key_begin=begin), [3000], [4])
        assert spans.tolist() == [[0, 2981, 3000, 0]] and plan.tolist() == [3000 - 128 * 23]


def test_refused():
    p = mj.make_params(2, 8, 2, 4, 16, 8, 20)
    x = np.zeros(64, np.int32).ctypes.data
    call = mj.lib().mj_tree_spans
    t, m = mj.TreeArgs(None, 0, x), mj.ScoreModArgs()
    args = [ctypes.byref(p), ctypes.byref(t), ctypes.byref(m), x, x + 64, x + 128]
    for i in (0, 1, 3, 4, 5):
        bad = list(args)
        bad[i] = None
        assert call(*bad) == BAD
    for field, value in (("window", 5), ("alibi_slopes", x), ("key_end", x)):
        good = getattr(m, field)
        setattr(m, field, value)
        assert call(*args) == UNSUP
        assert mj.lib().mj_tree_spans_device(*args[:3], x, x, x, None) == UNSUP
        setattr(m, field, good)
    t.tree_lens = x + 2
    assert call(*args) == BAD and mj.lib().mj_tree_spans_device(*args[:3], x, x, x, None) == BAD
    t.tree_lens = x
    device = [*args[:3], 1 << 20, 1 << 20, 1 << 20, None]
    for i, value in ((0, None), (1, None), (3, None), (4, None), (5, None), (3, (1 << 20) + 2), (4, (1 << 20) + 8), (5, (1 << 20) + 1)):
        bad = list(device)
        bad[i] = value
        assert mj.lib().mj_tree_spans_device(*bad) == BAD
    for lens in ([129, 0], [-1, 0]):
        with pytest.raises(mj.MjError):
            mj.tree_spans(p, None, lens)
    with pytest.raises(ValueError):
        mj.tree_spans(p, None, [1, 2], [1, 2, 3])
