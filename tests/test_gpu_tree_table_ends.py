"""Trees whose device length passes their block table (reported by the device's
plan): what lies behind a sequence's row of the table, the last one's among
them, is not looked up, by any row count's kernel."""

import pytest
import torch

import paged_fp8_kv_gb300 as mj
from tests.serving_helpers import I32

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("q_len,h_r", [(4, 2), (4, 4), (8, 4), (16, 4), (31, 4), (61, 4)])
@pytest.mark.parametrize("page,blocks", [(16, 17), (64, 3)])
def test_entries_behind_the_table(q_len, h_r, page, blocks):
    h_k, pages, nb = 2, 40, 2
    gen = torch.Generator("cuda").manual_seed(q_len)
    k, v = (torch.randn(pages, page, h_k, D, generator=gen, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    p = mj.make_params(nb, q_len, h_k, h_r, page, blocks, pages, max_splits=4)
    table = torch.randint(0, pages, ((nb + 2) * blocks,), generator=gen, device="cuda", dtype=torch.int32)
    q = torch.randn(nb, h_k, q_len * h_r, D, generator=gen, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([blocks * page - 9, blocks * page + 300], **I32)
    pad = mj.decode_plan_max_items(p)
    work, n_splits, status = torch.zeros(pad, 4, **I32), torch.zeros(nb, **I32), torch.zeros(1, **I32)
    mj.decode_plan_device(p, lens, work, n_splits, pad_to=pad, status=status)
    assert int(status.item()) == mj.MJ_ERR_INVALID_ARG
    one = torch.ones(nb, h_k, device="cuda")
    mask = torch.full((nb, q_len, -(-q_len // 32)), -1, **I32)
    outs = []
    for behind in (3, 17, -1, pages):
        table[nb * blocks :] = behind
        o = torch.full_like(q, float("nan"))
        lse = torch.full(q.shape[:3], float("nan"), device="cuda")
        mj.decode_attn_tree(p, tree_mask=mask, q=q, k_cache=k, v_cache=v, block_table=table[: nb * blocks].view(nb, blocks), seq_lens=lens,
                            work=work, n_splits=n_splits, q_descale=one, k_descale=one, v_descale=one, o=o, lse=lse,
                            workspace=torch.empty(mj.workspace_bytes(p), dtype=torch.uint8, device="cuda"), softmax_scale=D**-0.5)
        torch.cuda.synchronize()
        outs.append((o, lse))
    for o, lse in outs:
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
