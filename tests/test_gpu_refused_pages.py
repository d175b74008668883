"""Steps whose pages run out: what was left out keeps its keys and its length,
through the append, the attention, the commit and the release, eagerly and as
one replayed graph; the others go on."""

import ctypes

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import serve_ref
from tests.serving_helpers import I32, SPLIT_P
from tests.test_gpu_serving_chain import D, Server

CAPACITY, INVALID = mj.MJ_ERR_CAPACITY, mj.MJ_ERR_INVALID_ARG


def test_granted_pointers_refused():
    """Misaligned, or over an input or another output (CPU only: aligned pointers that nothing reads)."""
    at = iter(range(1 << 20, 1 << 60, 1 << 32))
    p, a = mj.make_page_params(3, 16, 8, 40), mj.ReserveArgs()
    for f in ("seq_lens", "new_tokens", "free_pages", "num_free", "num_free_out", "block_table", "seq_lens_out", "cu_tokens"):
        setattr(a, f, next(at))
    for bad in (next(at) + 2, a.seq_lens, a.new_tokens, a.seq_lens_out + 4, a.cu_tokens, a.block_table + 8, a.free_pages):
        a.granted = ctypes.cast(bad, mj._pi32)
        assert mj.lib().mj_pages_reserve(ctypes.byref(p), ctypes.byref(a), None) == INVALID
    r = mj.make_rope_params(3, 1, 1, 4, 16, 8, 40, max_pos=9)
    a = mj.RopeArgs()
    for f in ("q", "k", "v", "positions", "cos_sin", "q_out", "k_cache", "v_cache", "block_table", "seq_lens", "k_descale", "v_descale"):
        setattr(a, f, next(at))
    a.q_tok = a.k_tok = a.v_tok = a.q_out_stride = 4 * D
    a.q_head = a.k_head_in = a.v_head_in = D
    a.num_tokens, a.k_page, a.k_row, a.k_head, a.v_page, a.v_row, a.v_head = 3, 16 * D, D, D, 16 * D, D, D
    a.granted = ctypes.cast(next(at) + 2, mj._pi32)
    assert mj.lib().mj_rope_append(ctypes.byref(r), ctypes.byref(a), None) == INVALID


class Short(Server):
    """A server whose steps pass on what the reservation granted."""

    def __init__(self, *args):
        super().__init__(*args)
        self.granted = torch.full((4,), -7, **I32)

    def reserve(self, **kw):
        super().reserve(granted=self.granted, **kw)

    def append(self, x, positions, q_out, cu_tokens=None, q_len=1):
        hq = self.h_k * self.h_r
        p = mj.make_rope_params(4, q_len, self.h_k, self.h_r, self.page, self.blocks, self.pages, max_pos=800)
        mj.rope_append(p, q=x[:, :hq], k=x[:, hq : hq + self.h_k], v=x[:, hq + self.h_k :], positions=positions, cos_sin=self.cos_sin,
                       q_out=q_out, k_cache=self.k, v_cache=self.v, block_table=self.table, seq_lens=self.lens, k_descale=self.kd,
                       v_descale=self.vd, cu_tokens=cu_tokens, status=self.status, granted=self.granted)


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_a_steps_refusal_leaves_the_cache(captured):
    h_k, h_r, page, q_len = 2, 4, 16, 6
    s = Short(h_k, h_r, page, q_len)
    first = torch.full((160, h_k * h_r, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 42, 70, 101, 160], **I32)
    s.reserve(new_tokens=torch.tensor([42, 28, 31, 59], **I32))
    s.append(s.projection(160), torch.cat([torch.arange(n, **I32) for n in (42, 28, 31, 59)]), first, cu_tokens=cu)
    params = mj.make_params(4, q_len, h_k, h_r, page, s.blocks, s.pages, max_splits=4)
    x = torch.zeros(4 * q_len, h_k * (h_r + 2), D, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4 * q_len, **I32)
    mask = torch.from_numpy(np.tile(serve_ref.tree_mask(list(range(-1, q_len - 1)), 1).view(np.int32), (4, 1, 1))).cuda()
    path = torch.arange(q_len, **I32).repeat(4, 1)
    count = torch.full((4,), q_len, **I32)
    held = torch.zeros(4, **I32)
    q = torch.empty(4, h_k, q_len * h_r, D, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    pad = mj.decode_plan_max_items(params)
    work, n_splits = torch.zeros(pad, 4, **I32), torch.zeros(4, **I32)
    ws = torch.empty(mj.workspace_bytes(params), dtype=torch.uint8, device="cuda")
    stages = [torch.zeros(1, **I32) for _ in range(2)]  # the status after the reservation, and after the append

    def step():
        s.status.zero_()
        s.reserve(q_len=q_len)
        stages[0].copy_(s.status)
        s.append(x, pos, q, q_len=q_len)
        stages[1].copy_(s.status)
        mj.decode_plan_device(params, s.lens, work, n_splits, pad_to=pad, status=s.status)
        mj.decode_attn_tree(params, tree_mask=mask, tree_lens=s.granted, q=q, k_cache=s.k, v_cache=s.v, block_table=s.table,
                            seq_lens=s.lens, work=work, n_splits=n_splits, q_descale=s.one, k_descale=s.kd, v_descale=s.vd, o=o,
                            lse=lse, workspace=ws, softmax_scale=D**-0.5, status=s.status)
        held.copy_(s.lens)
        mj.tree_commit(params, k_cache=s.k, v_cache=s.v, block_table=s.table, seq_lens=s.lens, tree_lens=s.granted, accepted=path,
                       num_accepted=count, status=s.status)
        mj.pages_release(s.page_params, seq_lens=held, keep_lens=s.lens, free_pages=s.free, num_free=s.num_free, block_table=s.table,
                         status=s.status)

    graph = None
    if captured:
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
        torch.cuda.synchronize()
    lens = [42, 28, 31, 59]  # pages of 16: the first has room for 6 more, 28 and 59 need a page, 31 needs one
    for free in (0, 1, 2, 50):
        need = [-(-(n + 6) // page) - -(-n // page) for n in lens]
        left, want = free, []
        for n in need:  # in order, and none behind one that found too few
            left -= n
            want.append(6 if n == 0 or left >= 0 else 0)
        listed = s.free[: int(s.num_free.item())].clone()
        away = len(listed) - free  # pages held elsewhere meanwhile
        s.free[:free] = listed[away:]
        s.num_free.fill_(free)
        before = [s.rows(b, n) for b, n in enumerate(lens)]
        x.copy_(torch.randn(x.shape, generator=s.gen, device="cuda"))
        pos.copy_(torch.tensor([n + i for n in lens for i in range(q_len)], **I32))
        count.fill_(q_len)
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert s.granted.tolist() == want, free
        refused = 0 in want
        assert int(stages[0].item()) == int(stages[1].item()) == (CAPACITY if refused else 0)
        assert int(s.status.item()) == (INVALID if refused else 0)  # the commit of nodes that are not there
        rest = int(s.num_free.item())
        assert rest == free - sum(n for n, w in zip(need, want) if w)
        s.free[: away + rest] = torch.cat([listed[:away], s.free[:rest].clone()])
        s.num_free.fill_(away + rest)
        for b in range(4):
            n = lens[b] + want[b]
            assert int(s.lens[b].item()) == n
            now = s.rows(b, n)
            assert torch.equal(now[: lens[b]], before[b]), b
            if not want[b]:
                assert (o[b] == 0).all() and torch.isneginf(lse[b]).all()
                continue
            seen = torch.arange(n, device="cuda") <= torch.arange(lens[b], n, device="cuda")[:, None]
            un = lambda t: t[b].view(h_k, q_len, h_r, -1).permute(1, 0, 2, 3).reshape(q_len, h_k * h_r, -1)  # noqa: E731
            s.check_attention(b, un(q), un(o), un(lse[..., None])[..., 0], now, seen, SPLIT_P, q[b].double().abs().amax((1, 2)))
            lens[b] = n
        s.pages_whole(lens)


@pytest.mark.gpu
def test_prompts_that_get_no_pages_are_not_appended():
    """Tokens by cu_tokens, a sequence whose tokens do not fit the table among them; positions' planes too; a number that is
    not the sequence's is reported."""
    s = Short(2, 4, 16, 1)
    hq = 8
    news = [20, 33, 0, 701]
    s.lens.copy_(torch.tensor([0, 0, 5, 9], **I32))
    s.table[2, 0], s.table[3, 0] = 3, 4
    cu = torch.zeros(5, **I32)
    s.reserve(new_tokens=torch.tensor(news, **I32), cu_tokens=cu)
    assert s.granted.tolist() == [20, 33, 0, 0] and int(s.status.item()) == INVALID and s.lens.tolist() == [20, 33, 5, 9]
    s.status.zero_()
    total = sum(news)
    before = [s.k.clone(), s.v.clone()]
    planes = torch.full((4, 2, s.blocks * 16), -5, **I32)
    x, pos = s.projection(total), torch.cat([torch.arange(n, **I32) % 700 for n in news])
    p = mj.make_rope_params(4, 1, 2, 4, 16, s.blocks, s.pages, max_pos=800)
    q = torch.full((total, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")

    def append():
        mj.rope_append(p, q=x[:, :hq], k=x[:, hq : hq + 2], v=x[:, hq + 2 :], positions=pos, cos_sin=s.cos_sin, q_out=q, k_cache=s.k,
                       v_cache=s.v, block_table=s.table, seq_lens=s.lens, k_descale=s.kd, v_descale=s.vd, cu_tokens=cu,
                       key_pos=planes, status=s.status, granted=s.granted)
        torch.cuda.synchronize()

    append()
    assert int(s.status.item()) == 0 and not torch.isnan(q).any()
    assert (planes[2:] == -5).all() and planes[0, 1, :20].tolist() == list(range(20)) and planes[1, 0, :33].tolist() == list(range(33))
    for b in (2, 3):  # nothing of what they held moved
        pg = int(s.table[b, 0].item())
        assert torch.equal(s.k[pg], before[0][pg]) and torch.equal(s.v[pg], before[1][pg])
    for b in (0, 1):
        assert not (s.rows(b, news[b]) == 0x7F).all(-1).any()
    s.k.copy_(before[0])
    s.v.copy_(before[1])
    s.granted.copy_(torch.tensor([19, 33, 0, 0], **I32))
    append()
    assert int(s.status.item()) == INVALID
    pages = s.table[0, :2].long()
    assert torch.equal(s.k[pages], before[0][pages]) and not (s.rows(1, 33) == 0x7F).all(-1).any()
