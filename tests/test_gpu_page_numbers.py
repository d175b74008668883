"""Pages outside the pool, in the free list and in block tables: neither given
out nor taken back, and reported."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import serve_ref
from tests.serving_helpers import I32

pytestmark = pytest.mark.gpu
INVALID, CAPACITY = mj.MJ_ERR_INVALID_ARG, mj.MJ_ERR_CAPACITY


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _reserve(lens, news, page, blocks, free, table, tokens):
    n = len(lens)
    d = dict(seq_lens_out=torch.full((n,), -7, **I32), num_free_out=torch.full((1,), -7, **I32), block_table=_dev(table),
             cu_tokens=torch.full((n + 1,), -7, **I32), positions=torch.full((tokens,), -7, **I32),
             slots=torch.full((tokens,), -7, dtype=torch.int64, device="cuda"), granted=torch.full((n,), -7, **I32),
             status=torch.zeros(1, **I32))
    mj.pages_reserve(mj.make_page_params(n, page, blocks, len(free)), seq_lens=_dev(np.asarray(lens, np.int32)),
                     new_tokens=_dev(np.asarray(news, np.int32)), free_pages=_dev(free), num_free=torch.tensor([len(free)], **I32), **d)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in d.items()}


@pytest.mark.parametrize("seqs,tokens", [(5, 300), (40, 9000), (1100, 40000)])  # one CTA, a cluster, sequences in two turns
@pytest.mark.parametrize("bad", [-1, -(2**31), 2**31 - 1, None])
def test_a_bad_page_ends_the_list(seqs, tokens, bad):
    rng = np.random.default_rng(seqs)
    page, blocks = 16, 64
    lens = rng.integers(0, 30, seqs).astype(np.int32)
    news = rng.integers(0, max(2, 2 * tokens // seqs - 30), seqs).astype(np.int32)
    tokens = int(news.sum()) + 9
    held = -(-lens // page)
    need = int((-(-(lens + news) // page) - held).sum())
    pages = int(held.sum()) + need + 4
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((seqs, blocks), -5, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at : at + h]
        at += h
    bad = pages if bad is None else bad  # the first number that is none
    for place in (0, 3, need // 2, need - 1, need, None):  # pages given before it (need: it is not reached)
        free = np.concatenate([perm[at:], perm[:at]])[::-1].copy()
        n = len(free)
        if place is not None:
            free[n - 1 - place] = bad
        got = _reserve(lens, news, page, blocks, free, table, tokens)
        reached = place is not None and place < need
        below = n - place if reached else 0  # entries at the bad one and below it
        want = serve_ref.reserve(lens, news, free[below:], n - below, table, page, tokens)
        names = ("block_table", "seq_lens_out", None, "cu_tokens", "positions", "slots")
        for name, x in zip(names, want):
            assert name is None or np.array_equal(got[name], x), (name, place)
        assert got["num_free_out"][0] == want[2] + below and got["status"][0] == (INVALID if reached else want[6])
        assert np.array_equal(got["granted"], want[1] - lens)


def test_a_bad_page_that_a_sequence_holds():
    table = np.array([[7, -5], [-1, -5], [3, -5], [99, 2], [100, -5]], np.int32)
    free = np.array([11, 12, 13] + [0] * 97, np.int32)
    free[3:] = np.arange(3, 100)
    got = _reserve([3, 3, 3, 15, 3], [2, 2, 14, 2, 1], 16, 2, free, table, 21)
    assert got["status"][0] == INVALID and got["seq_lens_out"].tolist() == [5, 5, 17, 17, 4] and got["granted"].tolist() == [2, 2, 14, 2, 1]
    assert got["slots"].tolist() == [115, 116, -1, -1] + list(range(51, 64)) + [99 * 16] + [99 * 16 + 15, 98 * 16] + [-1]
    # and too few pages in the same call: what is wrong is what is reported
    got = _reserve([3, 3, 3, 15, 3], [2, 2, 31, 18, 1], 16, 4, free[:100], np.pad(table, ((0, 0), (0, 2))), 54)
    assert got["status"][0] == INVALID


def _release(lens, keep, page, table, free, n_free, in_place):
    seqs, d = len(lens), {}
    if not in_place:
        d["num_free_out"] = torch.full((1,), -7, **I32)
    d.update(free_pages=_dev(free), num_free=torch.tensor([n_free], **I32), status=torch.zeros(1, **I32))
    mj.pages_release(mj.make_page_params(seqs, page, table.shape[1], len(free)), seq_lens=_dev(lens), keep_lens=_dev(keep),
                     block_table=_dev(table), **d)
    torch.cuda.synchronize()
    n = int(d.get("num_free_out", d["num_free"]).item())
    return d["free_pages"][:n].tolist(), int(d["status"].item())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seqs,blocks", [(3, 8), (60, 100), (1500, 12)])
def test_bad_pages_are_not_given_back(seqs, blocks, in_place):
    rng = np.random.default_rng(seqs)
    page = 16
    lens = rng.integers(0, blocks * page + 1, seqs).astype(np.int32)
    keep = (lens * rng.random(seqs) * 0.5).astype(np.int32)
    lens[0], keep[0] = blocks * page, 1
    pages = int((-(-lens // page)).sum()) + 7
    perm = rng.permutation(pages).astype(np.int32)
    at, table = 0, rng.integers(-9, -1, (seqs, blocks)).astype(np.int32)
    for b, n in enumerate(-(-lens // page)):
        table[b, :n] = perm[at : at + n]
        at += n
    start = perm[at:]  # seven pages in the list
    back = [(b, j) for b in range(seqs) for j in range(-(-int(keep[b]) // page), -(-int(lens[b]) // page))]
    for which in ([], [0], [len(back) - 1], list(range(0, len(back), 3)), list(range(len(back)))):
        t, lost = table.copy(), set()
        for i in which:
            t[back[i]] = (-1, pages, 2**31 - 1, -(2**31))[i % 4]
            lost.add(back[i])
        free = np.concatenate([start, np.full(pages - 7, -3, np.int32)])
        got, status = _release(lens, keep, page, t, free, 7, in_place)
        assert got == start.tolist() + [int(t[x]) for x in back if x not in lost]
        assert status == (INVALID if which else 0)


def test_bad_pages_and_a_full_list():
    table = np.array([[0, 1, 2, 3], [4, -1, 5, 6], [9, 7, 8, 1]], np.int32)
    lens, keep = np.array([64, 64, 64], np.int32), np.array([0, 16, 32], np.int32)
    free = np.arange(100, 110).astype(np.int32) % 10
    for n_free, want, status in ((1, [0, 0, 1, 2, 3, 5, 6, 8, 1], INVALID), (2, [0, 1, 0, 1, 2, 3, 5, 6, 8, 1], INVALID),
                                 (3, [0, 1, 2, 0, 1, 2, 3, 5, 6, 8], CAPACITY), (6, [0, 1, 2, 3, 4, 5, 0, 1, 2, 3], CAPACITY)):
        assert _release(lens, keep, 16, table, free, n_free, False) == (want, status)


@pytest.mark.parametrize("outputs", [("positions",), ("slots",), ("positions", "slots"), ()])
@pytest.mark.parametrize("new", [0, 3])
def test_no_entries_for_new_tokens(outputs, new):
    """Outputs of no entries are given all the same: tokens that they do not hold are reported."""
    d = {name: torch.zeros(0, dtype=torch.int64 if name == "slots" else torch.int32, device="cuda") for name in outputs}
    status, lens = torch.zeros(1, **I32), torch.zeros(2, **I32)
    mj.pages_reserve(mj.make_page_params(2, 16, 4, 9), seq_lens=lens, new_tokens=torch.tensor([0, new], **I32),
                     free_pages=torch.arange(9, **I32), num_free=torch.tensor([9], **I32), block_table=torch.zeros(2, 4, **I32),
                     status=status, **d)
    assert int(status.item()) == (INVALID if outputs and new else 0) and lens.tolist() == [0, new]
