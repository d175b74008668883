"""Drafted trees under spans, on the GPU: short windows of small trees among many
rows, by every row count's kernel; spans that leave out what a node sees are
reported."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from tests.serving_helpers import I32
from tests.test_gpu_tree import D, Tree

pytestmark = pytest.mark.gpu
ROWS = [(4, 2), (4, 4), (16, 1), (8, 4), (16, 4), (31, 4), (61, 4)]  # 8 and 16 rows, 32, 64, 128, above


class Windowed(Tree):
    """Trees whose node i sees `window` keys of its path and context; rows without a node hold `idle` as their first key."""

    def __init__(self, lens, nodes, q_len, h_r, window, idle, force_splits=0, **kw):
        super().__init__(lens, nodes, q_len, 2, h_r, 16, begin=True, **kw)
        for b, (n, t) in enumerate(zip(lens, nodes)):
            depth = self.see[b].sum(1) - 1
            self.begin[b, :t] = np.maximum(n - t + depth - window + 1, 0)
            self.begin[b, t:] = n - t if idle is None else idle
        self.mod = mj.ScoreMod(softcap=self.softcap, key_begin=torch.from_numpy(self.begin).cuda(),
                               prefix=None if self.prefix is None else torch.from_numpy(self.prefix).cuda())
        self.force_splits = force_splits

    def attend(self, spans, plan_lens):
        c = self.c
        plan = mj.decode_plan(self.params, plan_lens, force_splits=self.force_splits)
        self.o.fill_(float("nan"))
        self.lse.fill_(float("nan"))
        mj.decode_attn_tree(
            self.params, self.mod, spans=torch.from_numpy(spans).cuda(), tree_mask=self.mask, tree_lens=self.tree_lens, q=self.q,
            k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=c.seq_lens, work=torch.from_numpy(plan.work).cuda(),
            n_splits=torch.from_numpy(plan.n_splits).cuda(), q_descale=self.qd, k_descale=c.kd, v_descale=c.vd, o=self.o,
            lse=self.lse, workspace=torch.empty(mj.workspace_bytes(self.params), dtype=torch.uint8, device="cuda"),
            softmax_scale=D**-0.5, scale_o=0.75, status=self.status, max_n_splits=plan.max_n_splits)
        torch.cuda.synchronize()
        return int(self.status.item())


@pytest.mark.parametrize("q_len,h_r", ROWS)
@pytest.mark.parametrize("window,idle,kw", [(2, None, {}), (16, None, {}), (16, 2**31 - 1, {}), (3, -5, dict(force_splits=2)),
                                            (9, None, dict(prefix=True, softcap=20.0)), (300, None, dict(e4m3=True))])
def test_short_windows(q_len, h_r, window, idle, kw):
    nodes = [max(1, q_len // 8), q_len, 1, 0, max(1, q_len // 2), 1]
    t = Windowed([900, 517, 257, 140, 64 + q_len, 1], nodes, q_len, h_r, window, idle, **kw)
    spans, plan_lens = mj.tree_spans(t.params, t.mod, t.c.lens, t.tree_lens)
    got, lens = torch.full((6, 4), -7, **I32), torch.full((6,), -7, **I32)
    mj.tree_spans_device(t.params, t.mod, t.c.seq_lens, got, lens, t.tree_lens)
    assert np.array_equal(got.cpu().numpy(), spans) and np.array_equal(lens.cpu().numpy(), plan_lens)
    assert t.attend(spans, plan_lens) == 0
    t.check()


@pytest.mark.parametrize("q_len,h_r", ROWS)
def test_spans_without_a_nodes_keys_are_reported(q_len, h_r):
    """mj_score_spans takes row i's context to end at L - q_len + i; a tree's ends at L - n."""
    t = Windowed([900, 517], [1, q_len], q_len, h_r, 2, None)
    spans, plan_lens = mj.score_spans(t.params, t.mod, t.c.lens)
    assert spans[0].tolist() == [0, 899, 900, 0]  # key 898 is the one context key of the single node
    assert t.attend(spans, plan_lens) == mj.MJ_ERR_INVALID_ARG
    t.status.zero_()
    # the tree's last keys, or the prefix, left out
    spans, plan_lens = mj.tree_spans(t.params, t.mod, t.c.lens, t.tree_lens)
    spans[1, 2] -= 1
    assert t.attend(spans, plan_lens) == mj.MJ_ERR_INVALID_ARG
    t.status.zero_()
    t.mod.prefix = torch.tensor([10, 0], **I32)
    assert t.attend(*mj.tree_spans(t.params, mj.ScoreMod(key_begin=t.mod.key_begin), t.c.lens, t.tree_lens)) == mj.MJ_ERR_INVALID_ARG
    t.status.zero_()
    assert t.attend(*mj.tree_spans(t.params, t.mod, t.c.lens, t.tree_lens)) == 0


@pytest.mark.parametrize("q_len,h_r", ROWS)
def test_keys_outside_the_spans_may_hold_anything(q_len, h_r):
    """NaN codes of K and V between the prefix and the first key, and pages of the table that no key of the spans lies in."""
    nodes = [max(1, q_len // 8), q_len, 0]
    t = Windowed([1500, 517, 300], nodes, q_len, h_r, 20, None, prefix=True)
    spans, plan_lens = mj.tree_spans(t.params, t.mod, t.c.lens, t.tree_lens)
    assert t.attend(spans, plan_lens) == 0
    want = t.o.clone(), t.lse.clone()
    t.check()
    for b in range(3):
        for j in range(int(spans[b][0]), int(spans[b][1])):
            at = t.c.table_host[b, j // 16], j % 16
            t.c.k[at], t.c.v[at] = 0x7F, 0x7F
        for blk in range(-(-int(spans[b][0]) // 16), int(spans[b][1]) // 16):
            t.c.table[b, blk] = (-1, 2**31 - 1, t.c.num_pages)[blk % 3]
    assert t.attend(spans, plan_lens) == 0
    assert torch.equal(t.o, want[0]) and torch.equal(t.lse, want[1])


def test_spans_follow_the_lengths_in_a_graph():
    """Spans, plan and attention captured together; lengths, trees and first keys change in their buffers."""
    q_len, h_r = 16, 4
    t = Windowed([900, 517, 260], [16, 5, 1], q_len, h_r, 4, None)
    c, p = t.c, t.params
    pad = mj.decode_plan_max_items(p)
    work, n_splits = torch.zeros(pad, 4, **I32), torch.zeros(3, **I32)
    spans, lens = torch.zeros(3, 4, **I32), torch.zeros(3, **I32)
    ws = torch.empty(mj.workspace_bytes(p), dtype=torch.uint8, device="cuda")
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        mj.tree_spans_device(p, t.mod, c.seq_lens, spans, lens, t.tree_lens)
        mj.decode_plan_device(p, lens, work, n_splits, pad_to=pad, status=t.status)
        mj.decode_attn_tree(p, t.mod, spans=spans, tree_mask=t.mask, tree_lens=t.tree_lens, q=t.q, k_cache=c.k, v_cache=c.v,
                            block_table=c.table, seq_lens=c.seq_lens, work=work, n_splits=n_splits, q_descale=t.qd, k_descale=c.kd,
                            v_descale=c.vd, o=t.o, lse=t.lse, workspace=ws, softmax_scale=D**-0.5, scale_o=0.75, status=t.status)
    for lens_now, nodes in (([900, 517, 260], [16, 5, 1]), ([800, 16, 100], [2, 5, 0]), ([17, 500, 1], [16, 1, 1])):
        c.lens, t.nodes = lens_now, [min(n, k.shape[0]) for n, k in zip(nodes, t.see)]
        see, t.see = t.see, [k[:n, :n] for n, k in zip(t.nodes, t.see)]
        for b, n in enumerate(t.nodes):
            t.begin[b, :] = lens_now[b] - n
            t.begin[b, :n] = np.maximum(lens_now[b] - n + t.see[b].sum(1) - 4, 0)
        t.mod.key_begin.copy_(torch.from_numpy(t.begin))
        c.seq_lens.copy_(torch.tensor(lens_now, **I32))
        t.tree_lens.copy_(torch.tensor(t.nodes, **I32))
        t.o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert int(t.status.item()) == 0
        t.check()
        t.see = see
