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


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(window=100), dict(window=1), dict(window=129, softcap=20.0), dict(window=5000),
                                dict(q_slice=True), dict(lse=False), dict(extra_blocks=5), dict(softcap=2.0, causal=False)])
def test_modifiers_and_forms(kw, e4m3):
    news = [300, 1, 64, 517]
    ctx = [0, 900, 257, 130]
    Prompt([a + b for a, b in zip(ctx, news)], news, 2, 4, 32, e4m3=e4m3, pad=5, **kw).run().check()


@pytest.mark.parametrize("n,ctx", [(1, 0), (1, 127), (1, 128), (2, 126), (63, 65), (64, 64), (65, 63), (128, 0), (129, 127), (257, 255)])
def test_borders(n, ctx):
    """Tokens and keys at, before and behind the borders of tiles, halves and row groups."""
    for h_r in (1, 4):
        Prompt([n + ctx] * 2, [n, n], 1, h_r, 16, seed=n + ctx).run().check()


def test_many_groups():
    """More query heads than a row group holds tokens for: heads 128 and 200 a group, a tile of one or two tokens."""
    Prompt([40, 7], [40, 7], 1, 128, 16).run().check()
    Prompt([30], [13], 1, 200, 16).run().check()


@pytest.mark.parametrize("max_splits", [1, 2, 256])
@pytest.mark.parametrize("e4m3", [False, True])
def test_long_cache_before_few_tokens(max_splits, e4m3):
    """A few tokens before long caches: their keys are cut into parts and merged."""
    p = Prompt([9000, 5000, 3], [1, 5, 3], 1, 8, 64, max_splits=max_splits, e4m3=e4m3).run().check()
    items, merges, parts, chunk = p.plan_head()
    if max_splits == 1:
        assert merges == 0 and parts == 0
    else:
        assert merges == 2 and parts <= 2 * 152 and items == parts + 1
    # windows cut what is read, and what is cut
    Prompt([9000, 5000], [1, 5], 1, 8, 64, max_splits=max_splits, window=3000, e4m3=e4m3).run().check()
    Prompt([6000, 5000], [3, 40], 2, 16, 128, max_splits=max_splits, softcap=10.0, causal=False, e4m3=e4m3).run().check()


def test_rows_that_see_nothing():
    """Sequences with fewer keys than tokens (none at all among them): O = 0 and LSE = -inf."""
    Prompt([5, 0, 140, 1], [9, 300, 150, 3], 2, 4, 16).run().check()
    Prompt([5, 0, 140], [9, 300, 150], 2, 4, 16, causal=False).run().check()
    Prompt([5, 0, 300], [9, 4, 310], 1, 2, 16, window=7).run().check()


def test_rising_scores():
    """Scores that grow along the keys move every row's reference again and again."""
    p = Prompt([1500], [1500], 1, 2, 16, spread=1.0)
    c = p.c
    j = torch.arange(1500, device="cuda")
    pages = torch.from_numpy(c.table_host[0].astype(np.int64)).cuda()[j // 16]
    k = torch.zeros(1500, 128, device="cuda")
    k[:, 0] = (j // 100).float() * 4.0  # up to 56
    c.k[pages, j % 16, 0] = k.to(torch.float8_e4m3fn).view(torch.uint8)
    p.q.zero_()
    p.q[:, :, 0] = 3.0
    p.run().check()


def test_large_and_small_queries():
    """Rows of very different magnitudes side by side, a row of zeros, the smallest and large values."""
    p = Prompt([200], [200], 1, 4, 16)
    scale = torch.tensor([1.0, 1e-30, 0.0, 40.0], device="cuda").view(1, 4, 1)
    p.q.copy_((p.q.float() * scale).to(torch.bfloat16))
    p.q[7, 0] = 2.0**-126
    p.run().check()


def test_no_tokens():
    p = Prompt([40, 7], [0, 0], 1, 4, 16, pad=3).run().check()
    assert p.plan_head()[0] == 0
    Prompt([40], [0], 1, 4, 16).run()


def test_padded_batches_replayed():
    """One graph of plan and attention, replayed while the batch changes inside its buffers."""
    p = Prompt([900, 700, 300, 400], [60, 1, 300, 400], 2, 4, 16, pad=39, extra_blocks=4)
    p.run().check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            p.make_plan()
            p.call()
    torch.cuda.synchronize()
    c = p.c
    for news in ([60, 1, 300, 400], [0, 0, 1, 0], [1, 1, 1, 1], [400, 0, 300, 100], [0, 700, 0, 0]):
        p.news = news
        p.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(news)]), **I32))
        p.o.fill_(float("nan"))
        p.lse.fill_(float("nan"))
        p.ws.view(torch.float32).fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert int(p.status.item()) == 0
        p.check()
    del c


def test_repeats_are_the_same_bytes():
    p = Prompt([3000, 50, 700], [40, 50, 1], 1, 8, 16).run()
    o, lse = p.o.clone(), p.lse.clone()
    for _ in range(5):
        p.o.fill_(float("nan"))
        p.run()
        assert torch.equal(o.view(torch.int16), p.o.view(torch.int16)) and torch.equal(lse, p.lse)


def test_what_is_reported():
    """Tokens out of order or range leave O alone; lengths out of range are taken as the nearest; a plan of another shape is refused."""
    for bad in ([0, 5, 3, 20], [-1, 5, 9, 20], [0, 5, 9, 21], [0, 2**31 - 1, 9, 20], [7, 5, 3, 1]):
        p = Prompt([100, 90, 80], [5, 4, 11], 2, 4, 16)
        p.cu.copy_(torch.tensor(bad, **I32))
        p.make_plan()
        p.call()
        torch.cuda.synchronize()
        assert int(p.status.item()) == mj.MJ_ERR_INVALID_ARG and torch.isnan(p.o).all() and torch.isnan(p.lse).all()
    p = Prompt([96, 40, 96], [5, 4, 11], 2, 4, 16)
    p.c.seq_lens.copy_(torch.tensor([2**30, -5, 96], **I32))
    p.make_plan()
    p.call()
    torch.cuda.synchronize()
    assert int(p.status.item()) == mj.MJ_ERR_INVALID_ARG and (p.o[5:9] == 0).all() and not torch.isnan(p.o).any()
    p = Prompt([100, 90], [5, 4], 2, 4, 16).run()
    p.o.fill_(float("nan"))
    other = mj.make_params(2, 1, 1, 8, 16, p.c.max_blocks, p.c.num_pages, max_splits=256)
    plan = torch.zeros(mj.prompt_plan_bytes(other, 9) + 65536, dtype=torch.uint8, device="cuda")
    for made in (None, other):  # nothing in it, and a plan for other heads
        if made is not None:
            mj.prompt_plan(made, cu_tokens=p.cu, seq_lens=p.c.seq_lens, num_tokens=9, plan=plan)
        p.status.zero_()
        mj.prompt_attn(p.params, q=p.q, k_cache=p.c.k, v_cache=p.c.v, block_table=p.c.table, plan=plan, q_descale=p.qd,
                       k_descale=p.c.kd, v_descale=p.c.vd, o=p.o, lse=p.lse, workspace=p.ws, softmax_scale=0.1, status=p.status)
        torch.cuda.synchronize()
        assert int(p.status.item()) == mj.MJ_ERR_INVALID_ARG and torch.isnan(p.o).all()


def test_pools_in_other_layouts():
    """Heads outermost in a page, K and V interleaved in one buffer: the same bytes."""
    p = Prompt([300, 170], [300, 20], 2, 4, 32).run().check()
    o = p.o.clone()
    c = p.c
    hnd = [x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (c.k, c.v)]
    both = torch.stack([c.k, c.v], 1).contiguous()
    for k, v in (hnd, (both[:, 0], both[:, 1])):
        p.o.fill_(float("nan"))
        mj.prompt_attn(p.params, q=p.q, k_cache=k, v_cache=v, block_table=c.table, plan=p.plan, q_descale=p.qd, k_descale=c.kd,
                       v_descale=c.vd, o=p.o, lse=p.lse, workspace=p.ws, softmax_scale=D**-0.5, scale_o=0.75, status=p.status)
        torch.cuda.synchronize()
        assert torch.equal(o, p.o)


def test_long_items():
    """Items of many tiles, several to a CTA: rings, phases and buffers come round."""
    Prompt([20000, 9000], [700, 30], 1, 4, 128, max_splits=1).run().check()


def test_two_streams():
    """Two batches at once on two streams, each with its own plan and workspace."""
    ps = [Prompt([3000, 800], [200, 800], 2, 4, 16, seed=s, q_slice=bool(s)) for s in (0, 1)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(4):
        for p, s in zip(ps, streams):
            p.make_plan(s)
            p.call(s)
    torch.cuda.synchronize()
    for p in ps:
        assert int(p.status.item()) == 0
        p.check()


def test_bad_tensors_refused():
    p = Prompt([100], [5], 2, 4, 16)
    good = dict(q=p.q, k_cache=p.c.k, v_cache=p.c.v, block_table=p.c.table, plan=p.plan, q_descale=p.qd, k_descale=p.c.kd,
                v_descale=p.c.vd, o=p.o, lse=p.lse, workspace=p.ws, softmax_scale=0.1)
    for name, x in [("q", p.q.float()), ("q", p.q[:, :4]), ("q", p.q.cpu()), ("o", p.o[:, :4]), ("lse", p.lse[:4]),
                    ("block_table", p.c.table[:, :-1]), ("k_cache", p.c.k[:, :8]), ("plan", p.plan.view(torch.int32)), ("lse", p.lse.half())]:
        with pytest.raises(ValueError):
            mj.PromptAttn(p.params, **{**good, name: x})
    with pytest.raises(mj.MjError):
        mj.prompt_attn(p.params, **{**good, "plan": p.plan[:64]})
    with pytest.raises(mj.MjError):
        mj.prompt_attn(p.params, **{**good, "workspace": None})


@pytest.mark.parametrize("page,fewer", [(16, 1), (32, 0)])
def test_plan_of_other_tables_refused(page, fewer):
    """A plan for longer tables or other pages names keys that this call's table does not list."""
    p = Prompt([90, 33], [40, 33], 1, 4, 16, extra_blocks=2)
    c = p.c
    blocks = c.max_blocks - fewer if page == 16 else c.max_blocks
    params = mj.make_params(2, 1, 1, 4, page, blocks, c.num_pages, max_splits=256)
    assert mj.prompt_plan_bytes(params, 73) == p.plan.numel()
    p.make_plan()
    k, v = (x if page == 16 else x[: c.num_pages // 2 * 2].view(-1, page, 1, D) for x in (c.k, c.v))
    if page != 16:
        params.num_pages = k.shape[0]
    mj.prompt_attn(params, q=p.q, k_cache=k, v_cache=v, block_table=c.table[:, :blocks].contiguous(), plan=p.plan, q_descale=p.qd,
                   k_descale=c.kd, v_descale=c.vd, o=p.o, lse=p.lse, workspace=p.ws, softmax_scale=D**-0.5, status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == mj.MJ_ERR_INVALID_ARG
    assert torch.isnan(p.o).all() and torch.isnan(p.lse).all()


@pytest.mark.parametrize("h_k,h_r", [(1, 4), (2, 8)])
def test_shared_rows_before_short_items(h_k, h_r):
    """Items whose rows both row groups hold, an odd number of tiles, and behind them on the same CTA items in which the
    second group has no tile: its rows' statistics of the first kind must outlive the second."""
    lens = [300] * 200 + [60] * 200 + [0, 5]
    news = [1] * 400 + [0, 1]
    Prompt(lens, news, h_k, h_r, 64).run().check()
    p = Prompt([300] * 200 + [20] * 20, [1] * 200 + [129 // h_r + 31] * 20, h_k, h_r, 64, seed=1)  # tokens ahead of any key
    p.run().check()


def test_more_items_than_are_ordered():
    """Over 8192 work items: the list stays in the sequences' order; sequences without tokens between."""
    rng = np.random.default_rng(0)
    news = rng.integers(0, 3, 12500)
    lens = news + rng.integers(0, 40, 12500)
    p = Prompt(lens.tolist(), news.tolist(), 1, 2, 16)
    p.run()
    assert p.plan_head()[0] > 8192
    keep = rng.choice(np.nonzero(news)[0], 400, replace=False)
    at = np.concatenate([[0], np.cumsum(news)])
    c, sel = p.c, sorted(keep.tolist())
    for b in sel:
        n, L, t0 = int(news[b]), c.lens[b], int(at[b])
        k, v = c.rows(c.k, b), c.rows(c.v, b)
        seen = torch.arange(L, device="cuda")[None] <= torch.arange(L - n, L, device="cuda")[:, None]
        for h in range(2):
            scale = float(c.kd[b, 0].double()) * D**-0.5
            ref = attend(value_of(p.q[t0 : t0 + n, h]), k[0], v[0] * c.vd[b, 0].double() * 0.75, scale, seen, 0.0, HALF_P)
            check_rows(p.o[t0 : t0 + n, h], p.lse[t0 : t0 + n, h], ref, f"sequence {b}, head {h}")
    assert not torch.isnan(p.o).any()
