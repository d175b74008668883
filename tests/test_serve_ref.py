"""The restatements of the page and tree operators, on examples worked by hand."""

import numpy as np

from oracle import serve_ref


def test_reserve_by_hand():
    # pages of 16; the list holds 7, 3, 9, 4 (4 is given first); sequence 0 grows from 15 to 17 tokens (one page more),
    # 1 from 0 to 1 (its first), 2 from 16 to 30 (needs one), 3 stays within its page
    table = np.full((4, 3), -5, dtype=np.int32)
    table[0, 0], table[2, 0], table[3, 0] = 20, 22, 23
    free = np.array([7, 3, 9, 4, -1, -1], dtype=np.int32)
    t, lens, n, cu, pos, slots, st = serve_ref.reserve([15, 0, 16, 2], [2, 1, 14, 1], free, 4, table, 16, 20)
    assert (t[0].tolist(), t[1].tolist(), t[2].tolist(), t[3].tolist()) == ([20, 4, -5], [9, -5, -5], [22, 3, -5], [23, -5, -5])
    assert lens.tolist() == [17, 1, 30, 3] and n == 1 and cu.tolist() == [0, 2, 3, 17, 18] and st == 0
    assert pos.tolist() == [15, 16, 0] + list(range(16, 30)) + [2, 0, 0]
    assert slots.tolist() == [20 * 16 + 15, 4 * 16, 9 * 16] + [3 * 16 + i for i in range(14)] + [23 * 16 + 2, -1, -1]


def test_reserve_leaves_out_what_does_not_fit():
    table = np.full((4, 2), 1, dtype=np.int32)
    free = np.array([5, 6, 0, 0, 0, 0, 0, 0], dtype=np.int32)
    # sequence 1 would need the third page of two; 2 needs none; 3 comes after it and is left out too
    t, lens, n, cu, pos, slots, st = serve_ref.reserve([0, 0, 3, 16], [16, 32, 2, 1], free, 2, table, 16, 51)
    assert t[0].tolist() == [6, 1] and n == 1 and lens.tolist() == [16, 0, 5, 16] and st == serve_ref.CAPACITY
    assert cu.tolist() == [0, 16, 48, 50, 51] and set(slots[16:48]) == {-1} and slots[48:].tolist() == [16 + 3, 16 + 4, -1]
    # more tokens than the table holds, and negative counts
    t, lens, n, cu, _, _, st = serve_ref.reserve([0, -1, 5, 3], [33, 1, -2, 1], free, 2, table, 16, 40)
    assert st == serve_ref.INVALID and cu.tolist() == [0, 33, 33, 33, 34] and lens.tolist() == [0, -1, 5, 4] and n == 2


def test_release_is_reserve_backwards():
    table = np.array([[4, 8, 2], [9, 1, 0]], dtype=np.int32)
    free = np.zeros(10, dtype=np.int32)
    out, n, st = serve_ref.release([40, 17], [16, 0], free, 0, table, 16)
    assert out[:n].tolist() == [8, 2, 9, 1] and st == 0
    out, n, st = serve_ref.release([40, 17], [41, 0], free, 9, table, 16)
    assert out[9] == 9 and n == 10 and st == serve_ref.CAPACITY


def test_commit_and_mask():
    rows = np.arange(10)[:, None] * np.ones((1, 2))
    assert serve_ref.commit(rows, 4, [0, 2, 5])[:, 0].tolist() == [0, 1, 2, 3, 4, 6, 9, 7, 8, 9]
    m = serve_ref.tree_mask([-1, 0, 0, 1, 3] + [4] * 30, 2)
    assert m[0].tolist() == [1, 0] and m[2].tolist() == [0b101, 0] and m[4].tolist() == [0b11011, 0]
    assert m[34].tolist() == [0b11011, 1 << 2]
