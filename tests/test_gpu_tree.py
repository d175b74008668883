"""Attention of drafted trees, and the accepted branch moved to the front, on the
GPU against plain definitions."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import e4m3_table, serve_ref
from oracle.narrow_ref import pack_bits, to_e4m3_codes
from tests.serving_helpers import I32, SPLIT_P, Cache, attend, check_rows, value_of

pytestmark = pytest.mark.gpu
D = 128
QROWS = mj.MJ_KERNEL_TENSOR_CORE_QROWS


class Tree:
    """Trees of `nodes` tokens (of q_len) at the end of `lens` keys; mask rows of
    tokens without a node, and bits past the tree, hold ones."""

    def __init__(self, lens, nodes, q_len, h_k, h_r, page, kernel=mj.MJ_KERNEL_AUTO, e4m3=False, softcap=0.0, begin=False,
                 prefix=False, spans=False, force_splits=0, max_splits=16, seed=0, words=None, chain=False, full=False, empty=False):
        self.c = c = Cache(lens, h_k, page, seed)
        self.q_len, self.h_r, self.nodes, self.softcap = q_len, h_r, nodes, softcap
        nb, rows = len(lens), q_len * h_r
        self.params = mj.make_params(nb, q_len, h_k, h_r, page, c.max_blocks, c.num_pages, max_splits=max_splits, kernel=kernel,
                                     q_dtype=mj.MJ_E4M3 if e4m3 else mj.MJ_BF16)
        words = words or -(-q_len // 32)
        mask = np.full((nb, q_len, words), 0xFFFFFFFF, dtype=np.uint32)
        self.see = []
        for b, t in enumerate(nodes):
            parents = [i - 1 if chain else (-1 if i == 0 else int(c.rng.integers(max(0, i - 9), i))) for i in range(t)]
            m = serve_ref.tree_mask(parents, words)
            if empty and t > 1:
                m[1] = 0  # a node that sees no node, not even itself
            see = np.unpackbits(m.view(np.uint8), axis=-1, bitorder="little")[:, :t].astype(bool)
            mask[b, :t] = m if full else m | (0xFFFFFFFF << np.clip(t - 32 * np.arange(words), 0, 32)).astype(np.uint64).astype(np.uint32)
            self.see.append(see)
        self.mask = torch.from_numpy(mask.view(np.int32)).cuda()
        self.tree_lens = None if full else torch.tensor(nodes, **I32)
        ctx = np.array(lens) - np.array(nodes)
        self.begin = (c.rng.random((nb, q_len)) * (ctx[:, None] + 1)).astype(np.int32) if begin else None
        if begin and empty:
            self.begin[:, 1] = ctx  # nothing at all
        self.prefix = np.minimum(c.rng.integers(0, 200, nb), np.array(lens)).astype(np.int32) if prefix else None
        dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
        mod = mj.ScoreMod(softcap=softcap, key_begin=dev(self.begin), prefix=dev(self.prefix))
        self.q = c.queries((nb, h_k, rows, D), e4m3)
        self.qd = torch.rand(nb, h_k, generator=c.gen, device="cuda") + 0.5 if e4m3 else torch.ones(nb, h_k, device="cuda")
        sp, plan_lens = (None, lens)
        if spans:
            sp, plan_lens = mj.score_spans(self.params, mod, lens)
            sp = torch.from_numpy(sp).cuda()
        plan = mj.decode_plan(self.params, plan_lens, force_splits=force_splits)
        self.o = torch.full((nb, h_k, rows, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((nb, h_k, rows), float("nan"), device="cuda")
        self.status = torch.zeros(1, **I32)
        ws = torch.full((mj.workspace_bytes(self.params) // 4 + 4,), float("nan"), device="cuda").view(torch.uint8)
        self.call = mj.DecodeAttnTree(
            self.params, mod, spans=sp, tree_mask=self.mask, tree_lens=self.tree_lens, q=self.q, k_cache=c.k, v_cache=c.v,
            block_table=c.table, seq_lens=c.seq_lens, work=torch.from_numpy(plan.work).cuda(),
            n_splits=torch.from_numpy(plan.n_splits).cuda(), q_descale=self.qd, k_descale=c.kd, v_descale=c.vd, o=self.o,
            lse=self.lse, workspace=ws, softmax_scale=D**-0.5, scale_o=0.75, status=self.status, max_n_splits=plan.max_n_splits)

    def run(self):
        self.call()
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        return self

    def check(self):
        c = self.c
        for b, (L, t) in enumerate(zip(c.lens, self.nodes)):
            ctx = L - t
            see = np.zeros((self.q_len, L), dtype=bool)
            j = np.arange(ctx)
            for i in range(t):
                see[i, :ctx] = j >= (0 if self.begin is None else self.begin[b, i])
                if self.prefix is not None:
                    see[i, :ctx] |= j < self.prefix[b]
                see[i, ctx:] = self.see[b][i]
            seen = torch.from_numpy(np.repeat(see, self.h_r, axis=0)).cuda()
            k, v = c.rows(c.k, b), c.rows(c.v, b)
            for g in range(c.h_k):
                q = value_of(self.q[b, g])
                scale = float(self.qd[b, g].double() * c.kd[b, g].double()) * D**-0.5
                ref = attend(q, k[g], v[g] * c.vd[b, g].double() * 0.75, scale, seen, self.softcap, SPLIT_P, q.abs().max())
                check_rows(self.o[b, g], self.lse[b, g], ref, f"sequence {b}, head {g}")
        return self


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_len,h_r", [(1, 8), (4, 2), (4, 4), (16, 1), (5, 3), (8, 4), (16, 4), (13, 5), (61, 1), (31, 8), (61, 4), (70, 5)])
def test_tree_rows(q_len, h_r, e4m3):
    """Every row count's kernel: 8 and 16 rows, 32 and 64 (copies), 128, pairs, more than one CTA."""
    nodes = [q_len, max(1, q_len // 2), q_len, 1, 0]
    lens = [q_len, 128 + q_len // 2, 700, 129, 64]
    Tree([max(a, t) for a, t in zip(lens, nodes)], nodes, q_len, 2, h_r, 16, e4m3=e4m3).run().check()


@pytest.mark.parametrize("q_len,h_r", [(4, 4), (16, 4), (61, 4)])
@pytest.mark.parametrize("ctx", [0, 1, 96, 100, 127, 128, 129, 255, 300])
def test_tree_borders(ctx, q_len, h_r):
    """Trees that begin at, before and behind the borders of tiles and mask words."""
    Tree([ctx + q_len] * 2, [q_len, q_len], q_len, 1, h_r, 32, seed=ctx, full=True).run().check()


@pytest.mark.parametrize("q_len,h_r", [(4, 4), (8, 4), (16, 4), (25, 4), (61, 4)])
@pytest.mark.parametrize("kw", [dict(softcap=20.0), dict(begin=True), dict(begin=True, spans=True), dict(prefix=True, begin=True, spans=True),
                                dict(prefix=True), dict(force_splits=3), dict(begin=True, empty=True), dict(words=5), dict(chain=True)])
def test_tree_modifiers(kw, q_len, h_r):
    nodes = [q_len, max(1, q_len - 3), 2]
    Tree([900, 517, 260], nodes, q_len, 2, h_r, 64, **kw).run().check()


@pytest.mark.parametrize("kernel", [mj.MJ_KERNEL_AUTO, QROWS])
def test_chain_is_causal(kernel):
    """A tree of one branch sees what the causal tail sees: the same bytes as the plain call on modified scores."""
    t = Tree([700, 300], [4, 4], 4, 2, 4, 16, chain=True, full=True, kernel=kernel).run()
    o, lse, c = t.o.clone(), t.lse.clone(), t.c
    plan = mj.decode_plan(t.params, c.lens)
    mj.decode_attn_mod(t.params, mj.ScoreMod(), q=t.q, k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=c.seq_lens,
                       work=torch.from_numpy(plan.work).cuda(), n_splits=torch.from_numpy(plan.n_splits).cuda(), q_descale=t.qd,
                       k_descale=c.kd, v_descale=c.vd, o=t.o, lse=t.lse, softmax_scale=D**-0.5, scale_o=0.75,
                       workspace=torch.empty(mj.workspace_bytes(t.params), dtype=torch.uint8, device="cuda"),
                       max_n_splits=plan.max_n_splits)
    assert torch.equal(o, t.o) and torch.equal(lse, t.lse)


def test_tree_lens_are_clamped():
    """More nodes than rows or keys, or fewer than none, are taken as the nearest there is."""
    t = Tree([40, 7, 40], [6, 6, 0], 6, 1, 2, 16)
    t.tree_lens.copy_(torch.tensor([50, 6, -3], **I32))
    t.run().check()
    t.tree_lens.copy_(torch.tensor([6, 6, -(2**31)], **I32))
    t.run().check()


# ------------------------------------------------------------------ commit


def _path(rng, nodes, n):
    return np.sort(rng.choice(nodes, n, replace=False)).astype(np.int32)


@pytest.mark.parametrize("kv", ["e4m3", "e3m2", "e2m1", "nvfp4"])
@pytest.mark.parametrize("h_k,page,pos", [(1, 16, "heads"), (3, 32, "one"), (8, 128, None)])
def test_commit(h_k, page, pos, kv):
    rng = np.random.default_rng(h_k)
    q_len, most = 80, 70
    nodes = [80, 5, 1, 0, 64, 20, 33]
    lens = [80, 300, 129, 50, 64, 1000, 47]
    counts = [70, 3, 1, 0, 0, 20, 9]
    row = {"e4m3": 128, "e3m2": 96, "e2m1": 64, "nvfp4": 64}[kv]
    need = [-(-n // page) for n in lens]
    blocks, pages = max(need) + 1, sum(need) + 2
    perm = rng.permutation(pages)
    table, at = np.full((7, blocks), -9, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at : at + n]
        at += n
    gen = torch.Generator("cuda").manual_seed(0)
    pools = [torch.randint(0, 256, (pages, page, h_k, row), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2)]
    scales = [torch.randint(0, 256, (pages, h_k, page, 8), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2)]
    key_pos = None
    if pos:
        planes = torch.randint(0, 9999, (7, h_k if pos == "heads" else 1, blocks * page), generator=gen, device="cuda", dtype=torch.int32)
        key_pos = planes if pos == "heads" else planes.expand(7, h_k, blocks * page)
    path = np.zeros((7, most), np.int32)
    for b, n in enumerate(counts):
        path[b, :n] = _path(rng, nodes[b], n)
    before = [x.cpu().numpy().copy() for x in pools + scales] + ([planes.cpu().numpy().copy()] if pos else [])
    params = mj.make_params(7, q_len, h_k, 4, page, blocks, pages, kv_format=mj.KV_FORMATS[kv])
    status, new = torch.zeros(1, **I32), torch.full((7,), -1, **I32)
    d = dict(k_cache=pools[0], v_cache=pools[1], block_table=torch.from_numpy(table).cuda(), seq_lens=torch.tensor(lens, **I32),
             tree_lens=torch.tensor(nodes, **I32), accepted=torch.from_numpy(path).cuda(), num_accepted=torch.tensor(counts, **I32),
             key_pos=key_pos, status=status)
    if kv == "nvfp4":
        d.update(k_scales=scales[0], v_scales=scales[1])
    mj.tree_commit(params, new_lens=new, **d)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert new.tolist() == [n - t + c for n, t, c in zip(lens, nodes, counts)]
    want = [x.copy() for x in before]
    for b, n in enumerate(lens):
        j = np.arange(n)
        pg, r = table[b, j // page], j % page
        ctx, p = n - nodes[b], path[b, : counts[b]]
        for i in range(2):
            want[i][pg, r] = serve_ref.commit(before[i][pg, r], ctx, p)
            if kv == "nvfp4":
                want[2 + i][pg, :, r] = serve_ref.commit(before[2 + i][pg, :, r], ctx, p)
        if pos:
            want[4][b, :, :n] = serve_ref.commit(before[4][b, :, :n].T, ctx, p).T
    got = pools + scales + ([planes] if pos else [])
    for i, (x, y) in enumerate(zip(got, want)):
        assert np.array_equal(x.cpu().numpy(), y), i
    # the lengths in place
    for x, y in zip(got, before):
        x.copy_(torch.from_numpy(y).cuda())
    mj.tree_commit(params, **d)
    assert torch.equal(d["seq_lens"], new)
    for i, (x, y) in enumerate(zip(got, want)):
        assert np.array_equal(x.cpu().numpy(), y), i


@pytest.mark.parametrize("path,count,length,bad_page", [
    ([0, 2, 2], 3, 40, False), ([0, 3, 1], 3, 40, False), ([0, 8], 2, 40, False), ([-1, 1], 2, 40, False), ([0, 1], -1, 40, False),
    ([0, 1], 9, 40, False), ([0, 5], 2, 5, False), ([0, 1], 2, -3, False), ([0, 1], 2, 99, False), ([3, 5], 2, 40, True),
])
def test_commit_reports(path, count, length, bad_page):
    """What is wrong is not moved: the sequence's pools and length stay."""
    table = torch.arange(5, **I32)[None].contiguous()
    if bad_page:
        table[0] = torch.tensor([0, 1, 77, -4, 0], **I32)
    pools = [torch.randint(0, 256, (5, 16, 2, 128), device="cuda", dtype=torch.uint8) for _ in range(2)]
    before = [x.clone() for x in pools]
    lens, new, status = torch.tensor([length], **I32), torch.zeros(1, **I32), torch.zeros(1, **I32)
    params = mj.make_params(1, 8, 2, 4, 16, 5, 5)
    mj.tree_commit(params, k_cache=pools[0], v_cache=pools[1], block_table=table, seq_lens=lens, num_accepted=torch.tensor([count], **I32),
                   accepted=torch.tensor([path + [0] * (8 - len(path))], **I32), new_lens=new, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == mj.MJ_ERR_INVALID_ARG
    assert all(torch.equal(x, y) for x, y in zip(pools, before))
    assert new.item() == (34 if bad_page else length)


@pytest.mark.parametrize("kv", ["e2m1", "e2m3", "e3m2"])
@pytest.mark.parametrize("q_len,h_r", [(4, 2), (4, 4), (8, 4), (13, 4), (31, 4), (61, 4)])
def test_tree_over_narrow_pools(q_len, h_r, kv):
    """Codes of a narrow format, by every row count's kernel, against the e4m3 codes of equal value."""
    nodes = [q_len, max(1, q_len // 2), 1]
    t = Tree([400, 128 + q_len, 61], nodes, q_len, 2, h_r, 32, seed=q_len)
    c, bits = t.c, 4 if kv == "e2m1" else 6
    codes = [c.rng.integers(0, 2**bits, (c.num_pages, c.page, 2, D)).astype(np.uint8) for _ in range(2)]
    for pool, x in zip((c.k, c.v), codes):
        pool.copy_(torch.from_numpy(to_e4m3_codes(x, kv, e4m3_table())))
    k, v = (torch.from_numpy(pack_bits(x, bits)).cuda() for x in codes)
    p = mj.make_params(3, q_len, 2, h_r, 32, c.max_blocks, c.num_pages, max_splits=16, kv_format=mj.KV_FORMATS[kv])
    plan = mj.decode_plan(p, c.lens)
    mj.decode_attn_tree(p, tree_mask=t.mask, tree_lens=t.tree_lens, q=t.q, k_cache=k, v_cache=v, block_table=c.table,
                        seq_lens=c.seq_lens, work=torch.from_numpy(plan.work).cuda(), n_splits=torch.from_numpy(plan.n_splits).cuda(),
                        q_descale=t.qd, k_descale=c.kd, v_descale=c.vd, o=t.o, lse=t.lse, softmax_scale=D**-0.5, scale_o=0.75,
                        workspace=torch.empty(mj.workspace_bytes(p), dtype=torch.uint8, device="cuda"), status=t.status,
                        max_n_splits=plan.max_n_splits)
    assert int(t.status.item()) == 0
    t.check()
