"""Attention over whole prompts on the GPU against the float64 definition."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from tests.serving_helpers import HALF_P, I32, Cache, attend, check_rows, value_of

pytestmark = pytest.mark.gpu
D = 128


class Prompt:
    """A batch of prompts: `news` query tokens at the end of `lens` keys each."""

    def __init__(self, lens, news, h_k, h_r, page, causal=True, window=0, softcap=0.0, e4m3=False, pad=0, max_splits=256,
                 seed=0, extra_blocks=0, q_slice=False, spread=1.0, first=0, lse=True):
        self.c = c = Cache(lens, h_k, page, seed, extra_blocks, spread)
        self.news, self.h_k, self.h_r, self.causal, self.window, self.softcap, self.e4m3 = news, h_k, h_r, causal, window, softcap, e4m3
        self.params = mj.make_params(len(lens), 1, h_k, h_r, page, c.max_blocks, c.num_pages, causal=causal,
                                     q_dtype=mj.MJ_E4M3 if e4m3 else mj.MJ_BF16, max_splits=max_splits)
        self.first, total = first, sum(news)  # the first sequence's tokens may lie behind others'
        tokens = first + total + pad
        h_q = h_k * h_r
        if q_slice:  # the query heads of a projection that holds keys and values behind them
            self.q = c.queries((tokens, h_q + 2 * h_k, D), e4m3)[:, :h_q]
        else:
            self.q = c.queries((tokens, h_q, D), e4m3)
        self.qd = torch.rand(len(lens), h_k, generator=c.gen, device="cuda") + 0.5 if e4m3 else torch.ones(len(lens), h_k, device="cuda")
        self.cu = torch.tensor(first + np.concatenate([[0], np.cumsum(news)]), **I32)
        self.o = torch.full((tokens, h_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((tokens, h_q), float("nan"), device="cuda") if lse else None
        self.status = torch.zeros(1, **I32)
        self.plan = torch.randint(0, 256, (mj.prompt_plan_bytes(self.params, tokens),), dtype=torch.uint8, device="cuda")
        self.ws = torch.full((mj.prompt_workspace_bytes(self.params) // 4 + 4,), float("nan"), device="cuda").view(torch.uint8)
        self.make_plan = mj.PromptPlan(self.params, cu_tokens=self.cu, seq_lens=c.seq_lens, num_tokens=tokens, window=window,
                                       plan=self.plan, status=self.status)
        self.call = mj.PromptAttn(self.params, q=self.q, k_cache=c.k, v_cache=c.v, block_table=c.table, plan=self.plan,
                                  q_descale=self.qd, k_descale=c.kd, v_descale=c.vd, o=self.o, lse=self.lse, workspace=self.ws,
                                  softmax_scale=D**-0.5, softcap=softcap, window=window, scale_o=0.75, status=self.status)

    def run(self):
        self.make_plan()
        self.call()
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        return self

    def plan_head(self):
        return self.plan[:16].view(torch.int32).tolist()  # items, merges, parts, chunk

    def check(self):
        c, t0 = self.c, self.first
        for b, (n, L) in enumerate(zip(self.news, c.lens)):
            k, v = c.rows(c.k, b), c.rows(c.v, b)
            pos = torch.arange(L - n, L, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")[None]
            seen = (j <= pos) if self.causal else torch.ones(n, L, dtype=torch.bool, device="cuda")
            if self.window:
                seen = seen & (j > pos - self.window)
            for h in range(self.h_k * self.h_r):
                g = h // self.h_r
                scale = float(self.qd[b, g].double() * c.kd[b, g].double()) * D**-0.5
                ref = attend(value_of(self.q[t0 : t0 + n, h]), k[g], v[g] * c.vd[b, g].double() * 0.75, scale, seen, self.softcap, HALF_P)
                check_rows(self.o[t0 : t0 + n, h], None if self.lse is None else self.lse[t0 : t0 + n, h], ref, f"sequence {b}, head {h}")
            t0 += n
        for x in (self.o, self.lse):  # padding, left as it was
            if x is not None:
                assert torch.isnan(x[: self.first]).all() and torch.isnan(x[t0:]).all()
        return self


@pytest.mark.parametrize("n,h_k,h_r,page", [(1, 1, 1, 16), (37, 1, 8, 16), (128, 2, 1, 128), (129, 1, 4, 64), (256, 1, 2, 32),
                                            (300, 3, 5, 16)])
def test_one_prompt(n, h_k, h_r, page):
    Prompt([n], [n], h_k, h_r, page).run().check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("h_k,h_r,page", [(2, 4, 16), (1, 16, 128)])
def test_packed_prompts(h_k, h_r, page, causal, e4m3):
    """Sequences of no, one and many tokens, with and without keys ahead, and padding behind."""
    news = [0, 1, 127, 64, 333, 1, 90, 0]
    ctx = [5, 0, 1, 1000, 0, 700, 129, 0]
    Prompt([a + b for a, b in zip(ctx, news)], news, h_k, h_r, page, causal=causal, e4m3=e4m3, pad=7, first=3).run().check()
