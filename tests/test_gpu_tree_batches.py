"""Batches of trees as a server's slots hold them: slots without keys, trees
without nodes, work lists of the device's plan padded far past their items,
captured and replayed while lengths and trees change; by every row count's
kernel."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from tests.serving_helpers import HALF_P, I32, SPLIT_P
from tests.test_gpu_tree import D, Tree
from tests.test_gpu_tree_kernels import check

pytestmark = pytest.mark.gpu
ROWS = [(4, 2), (4, 4), (8, 4), (16, 4), (31, 4), (61, 4), (70, 5)]


def _check(t):
    check(t, *((HALF_P, True) if t.q_len * t.h_r > 128 else (SPLIT_P, False)))


@pytest.mark.parametrize("q_len,h_r", ROWS)
@pytest.mark.parametrize("kw", [{}, dict(e4m3=True), dict(force_splits=2), dict(max_splits=1), dict(prefix=True, begin=True)])
def test_slots_without_keys(q_len, h_r, kw):
    Tree([0, 300, 0, q_len, 77, 0], [0, q_len, 0, q_len, 0, 0], q_len, 2, h_r, 32, **kw).run()
    t = Tree([0, 0], [0, 0], q_len, 1, h_r, 16, **kw).run()
    assert (t.o == 0).all() and torch.isneginf(t.lse).all()
    _check(Tree([0, 300, 0, q_len, 77, 0], [0, q_len, 0, q_len, 0, 0], q_len, 2, h_r, 32, **kw).run())


@pytest.mark.parametrize("q_len,h_r", ROWS)
@pytest.mark.parametrize("max_splits,force_splits", [(1, 0), (16, 0), (16, 3)])
def test_padded_plans_replayed(q_len, h_r, max_splits, force_splits):
    """One graph of plan and attention; most of the work list is padding."""
    t = Tree([2000, 600, 300, 64 + q_len], [q_len, q_len // 2, 1, q_len], q_len, 2, h_r, 16, max_splits=max_splits)
    c, p = t.c, t.params
    pad = mj.decode_plan_max_items(p) + 37
    work, n_splits = torch.full((pad, 4), -7, **I32), torch.zeros(4, **I32)
    ws = torch.full((mj.workspace_bytes(p) // 4 + 4,), float("nan"), device="cuda").view(torch.uint8)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        mj.decode_plan_device(p, c.seq_lens, work, n_splits, pad_to=pad, status=t.status, force_splits=force_splits)
        mj.decode_attn_tree(p, tree_mask=t.mask, tree_lens=t.tree_lens, q=t.q, k_cache=c.k, v_cache=c.v, block_table=c.table,
                            seq_lens=c.seq_lens, work=work, n_splits=n_splits, q_descale=t.qd, k_descale=c.kd, v_descale=c.vd, o=t.o,
                            lse=t.lse, workspace=ws, softmax_scale=D**-0.5, scale_o=0.75, status=t.status)
    see = t.see
    for lens, nodes in ((c.lens, t.nodes), ([130, 0, 5, 1], [q_len // 2, 0, 0, 1]), ([q_len, 600, 0, 2], [q_len, 0, 0, 1]),
                        ([2000, 599, 300, 64], [1, 1, 1, 1])):
        c.lens, t.nodes = list(lens), [min(n, x.shape[0]) for n, x in zip(nodes, see)]
        t.see = [x[:n, :n] for n, x in zip(t.nodes, see)]
        c.seq_lens.copy_(torch.tensor(c.lens, **I32))
        t.tree_lens.copy_(torch.tensor(t.nodes, **I32))
        t.o.fill_(float("nan"))
        t.lse.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert int(t.status.item()) == 0
        _check(t)
