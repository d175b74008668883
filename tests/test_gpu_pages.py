"""Pages reserved and released on the GPU: equal to the plain restatement, entry
by entry."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import serve_ref

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _case(seqs, page, blocks, lens, news, seed, spare=3, num_free=None):
    """A table with the pages the sequences hold, and a list of the others."""
    rng = np.random.default_rng(seed)
    held = [-(-max(0, int(n)) // page) for n in lens]
    need = sum(max(0, -(-(int(n) + int(m)) // page) - h) for n, m, h in zip(lens, news, held) if n >= 0 and m >= 0)
    pages = max(1, sum(min(h, blocks) for h in held) + need + spare)
    perm = rng.permutation(pages).astype(np.int32)
    table = rng.integers(-9, -1, (seqs, blocks)).astype(np.int32)
    at = 0
    for b, h in enumerate(held):
        h = min(h, blocks)
        table[b, :h] = perm[at : at + h]
        at += h
    free = np.concatenate([perm[at:], np.full(at, -3, np.int32)])
    return table, free, pages - at if num_free is None else num_free


def _reserve(seqs, page, blocks, lens, news, seed=0, spare=3, num_free=None, tokens=None, q_len=None, in_place=False, outputs=True,
             expect=0):
    lens, news = np.asarray(lens, np.int32), np.asarray(news, np.int32)
    table, free, n_free = _case(seqs, page, blocks, lens, news, seed, spare, num_free)
    total = int(news.clip(0).astype(np.int64).sum()) if tokens is None else tokens
    want = serve_ref.reserve(lens, news, free, n_free, table, page, total)
    d = dict(seq_lens=_dev(lens), free_pages=_dev(free), num_free=_dev(np.array([n_free], np.int32)), block_table=_dev(table))
    if not in_place:
        d.update(seq_lens_out=torch.full((seqs,), -7, dtype=torch.int32, device="cuda"),
                 num_free_out=torch.full((1,), -7, dtype=torch.int32, device="cuda"))
    if outputs:
        d.update(cu_tokens=torch.full((seqs + 1,), -7, dtype=torch.int32, device="cuda"),
                 positions=torch.full((total,), -7, dtype=torch.int32, device="cuda"),
                 slots=torch.full((total,), -7, dtype=torch.int64, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = dict(new_tokens=_dev(news)) if q_len is None else dict(q_len=q_len)
    mj.pages_reserve(mj.make_page_params(seqs, page, blocks, len(free)), status=status, **d, **new)
    torch.cuda.synchronize()
    got = [d["block_table"], d.get("seq_lens_out", d["seq_lens"]), d.get("num_free_out", d["num_free"])]
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert int(got[2].item()) == want[2]
    assert np.array_equal(d["free_pages"].cpu().numpy(), free)
    if not in_place:
        assert np.array_equal(d["seq_lens"].cpu().numpy(), lens) and int(d["num_free"].item()) == n_free
    if outputs:
        for name, x in zip(("cu_tokens", "positions", "slots"), want[3:6]):
            assert np.array_equal(d[name].cpu().numpy(), x), name
    assert int(status.item()) == want[6] == expect


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("seqs,hi,new", [(1, 0, 1), (1, 300, 77), (7, 200, 1), (33, 500, 40), (1025, 100, 3)])
def test_reserve(seqs, hi, new, page):
    rng = np.random.default_rng(seqs + page)
    _reserve(seqs, page, -(-(hi + new) // page) + 1, rng.integers(0, hi + 1, seqs), rng.integers(0, new + 1, seqs))


def test_reserve_many_tokens():
    rng = np.random.default_rng(5)
    _reserve(33, 64, 70, np.zeros(33), rng.integers(0, 4001, 33), tokens=70001)  # 8 CTAs, padding behind
    _reserve(3000, 16, 40, rng.integers(0, 300, 3000), rng.integers(0, 30, 3000), in_place=True)
    _reserve(16384, 16, 3, rng.integers(0, 40, 16384), np.ones(16384), q_len=1)  # the most sequences
    _reserve(1, 16, 8192, [0], [131072])


@pytest.mark.parametrize("in_place", [False, True])
def test_reserve_forms(in_place):
    lens, news = [15, 0, 16, 31, 100], [2, 1, 0, 1, 20]
    _reserve(5, 16, 8, lens, news, in_place=in_place)
    _reserve(5, 16, 8, lens, news, in_place=in_place, outputs=False)
    _reserve(5, 16, 8, lens, [1] * 5, in_place=in_place, q_len=1)
    _reserve(5, 16, 8, lens, news, in_place=in_place, tokens=30)
    _reserve(5, 16, 8, lens, [0] * 5, in_place=in_place, tokens=0)
    _reserve(5, 16, 8, lens, news, in_place=in_place, spare=0)  # the list ends empty


def test_reserve_leaves_out():
    lens, news = [15, 0, 16, 31, 100], [2, 40, 0, 1, 20]
    for n in range(6):
        _reserve(5, 16, 8, lens, news, num_free=n, expect=0 if n >= 5 else mj.MJ_ERR_CAPACITY)
    _reserve(3, 16, 2, [0, 30, 5], [33, 1, 3], expect=mj.MJ_ERR_INVALID_ARG)  # past the table
    _reserve(4, 16, 2, [0, -1, 5, 3], [1, 1, -2, 1], expect=mj.MJ_ERR_INVALID_ARG)
    _reserve(2, 16, 4, [3, 4], [5, 6], tokens=7, expect=mj.MJ_ERR_INVALID_ARG)  # more tokens than entries
    for n in (-1, 1000):
        _reserve(2, 16, 4, [3, 4], [5, 30], num_free=n, expect=mj.MJ_ERR_INVALID_ARG)


def _release(seqs, page, blocks, lens, keep, num_free=None, in_place=False, expect=0):
    lens, keep = np.asarray(lens, np.int32), np.asarray(keep, np.int32)
    table, free, n_free = _case(seqs, page, blocks, lens, np.zeros(seqs, np.int32), seqs, 3, num_free)
    want = serve_ref.release(lens, keep, free, n_free, table, page)
    d = dict(seq_lens=_dev(lens), keep_lens=_dev(keep), free_pages=_dev(free), num_free=_dev(np.array([n_free], np.int32)),
             block_table=_dev(table))
    if not in_place:
        d["num_free_out"] = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mj.pages_release(mj.make_page_params(seqs, page, blocks, len(free)), status=status, **d)
    torch.cuda.synchronize()
    assert np.array_equal(d["free_pages"].cpu().numpy(), want[0])
    assert int(d.get("num_free_out", d["num_free"]).item()) == want[1]
    assert np.array_equal(d["block_table"].cpu().numpy(), table)
    assert int(status.item()) == want[2] == expect


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("seqs,hi", [(1, 1), (1, 5000), (64, 8192), (1500, 200)])
def test_release(seqs, hi, page, in_place):
    rng = np.random.default_rng(seqs + hi)
    lens = rng.integers(0, hi + 1, seqs)
    _release(seqs, page, -(-hi // page) + 2, lens, rng.integers(0, lens + 1), in_place=in_place)
    _release(seqs, page, -(-hi // page) + 2, lens, np.zeros(seqs), in_place=in_place)
    _release(seqs, page, -(-hi // page) + 2, lens, lens, in_place=in_place)


def test_release_reports():
    _release(3, 16, 8, [100, 20, 7], [101, 3, 0], expect=mj.MJ_ERR_INVALID_ARG)
    _release(3, 16, 8, [100, 20, 7], [-1, 3, 0], expect=mj.MJ_ERR_INVALID_ARG)
    _release(3, 16, 2, [100, 20, 7], [1, 3, 0], expect=mj.MJ_ERR_INVALID_ARG)  # longer than the table
    _release(3, 16, 8, [100, 20, 7], [1, 3, 0], num_free=10, expect=mj.MJ_ERR_CAPACITY)  # given back before
    _release(3, 16, 8, [100, 20, 7], [1, 3, 0], num_free=-5, expect=mj.MJ_ERR_INVALID_ARG)


def test_reserve_then_release_gives_every_page_back():
    rng = np.random.default_rng(1)
    seqs, page, blocks, pages = 40, 16, 40, 900
    p = mj.make_page_params(seqs, page, blocks, pages)
    d = dict(seq_lens=torch.zeros(seqs, dtype=torch.int32, device="cuda"), free_pages=_dev(rng.permutation(pages).astype(np.int32)),
             num_free=_dev(np.array([pages], np.int32)), block_table=torch.full((seqs, blocks), -1, dtype=torch.int32, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = np.zeros(seqs, np.int64)
    for step in range(12):
        new = rng.integers(0, 60, seqs).astype(np.int32)
        mj.pages_reserve(p, new_tokens=_dev(new), status=status, **d)
        lens += new
        keep = (lens * rng.random(seqs)).astype(np.int32)
        mj.pages_release(p, keep_lens=_dev(keep), status=status, **d)
        d["seq_lens"].copy_(_dev(keep))
        lens = keep.astype(np.int64)
        used = [d["block_table"][b, : -(-int(n) // page)].tolist() for b, n in enumerate(lens)]
        free = d["free_pages"][: int(d["num_free"].item())].tolist()
        assert sorted(sum(used, []) + free) == list(range(pages)) and int(status.item()) == 0


def test_reserve_behind_impossible_demands():
    """More tokens in all than an int32 counts, of sequences left out: those behind them get theirs."""
    most = 2**31 - 1
    d = dict(seq_lens=_dev(np.array([0, 7, 3, 16], np.int32)), free_pages=_dev(np.arange(4, dtype=np.int32)),
             num_free=_dev(np.array([2], np.int32)), block_table=torch.full((4, 3), -1, dtype=torch.int32, device="cuda"),
             seq_lens_out=torch.zeros(4, dtype=torch.int32, device="cuda"), cu_tokens=torch.zeros(5, dtype=torch.int32, device="cuda"))
    d["block_table"][2, 0] = 3
    d["block_table"][3, 0] = 2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mj.pages_reserve(mj.make_page_params(4, 16, 3, 4), new_tokens=_dev(np.array([most, most, 14, 1], np.int32)), status=status, **d)
    assert d["seq_lens_out"].tolist() == [0, 7, 17, 17]
    assert d["block_table"].tolist() == [[-1] * 3, [-1] * 3, [3, 1, -1], [2, 0, -1]]
    assert d["cu_tokens"].tolist() == [0, most, most, most, most] and d["num_free"].item() == 0
    assert int(status.item()) == mj.MJ_ERR_INVALID_ARG
