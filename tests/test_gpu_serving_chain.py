"""The serving operators as a step uses them, one after another over one cache:
pages reserved, rotary positions and the cache write, prompts attended whole,
trees drafted, attended and committed, pages given back; against a plain
restatement of the sequences, eagerly and as replayed graphs."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import serve_ref
from tests.serving_helpers import HALF_P, I32, SPLIT_P, attend, check_rows

pytestmark = pytest.mark.gpu
D = 128


class Server:
    """Four sequences over a pool whose pages a free list holds."""

    def __init__(self, h_k, h_r, page, q_len, seed=0):
        self.h_k, self.h_r, self.page, self.q_len, self.n = h_k, h_r, page, q_len, 4
        self.blocks, self.pages = -(-700 // page), 4 * -(-700 // page) + 5
        self.rng, self.gen = np.random.default_rng(seed), torch.Generator("cuda").manual_seed(seed)
        self.k, self.v = (torch.full((self.pages, page, h_k, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.table = torch.full((4, self.blocks), -1, **I32)
        self.lens = torch.zeros(4, **I32)
        self.free = torch.from_numpy(self.rng.permutation(self.pages).astype(np.int32)).cuda()
        self.num_free = torch.tensor([self.pages], **I32)
        self.kd = torch.rand(4, h_k, generator=self.gen, device="cuda") * 0.02 + 0.01
        self.vd = torch.rand(4, h_k, generator=self.gen, device="cuda") * 0.02 + 0.01
        self.one = torch.ones(4, h_k, device="cuda")
        angle = torch.outer(torch.arange(800, device="cuda"), 10000.0 ** (-torch.arange(64, device="cuda") / 64))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
        self.page_params = mj.make_page_params(4, page, self.blocks, self.pages)
        self.status = torch.zeros(1, **I32)
        self.slots_of = [[] for _ in range(4)]  # the sequences as they should be: codes of each token's K and V rows

    def reserve(self, **kw):
        mj.pages_reserve(self.page_params, seq_lens=self.lens, free_pages=self.free, num_free=self.num_free, block_table=self.table,
                         status=self.status, **kw)

    def append(self, x, positions, q_out, cu_tokens=None, q_len=1):
        hq = self.h_k * self.h_r
        p = mj.make_rope_params(4, q_len, self.h_k, self.h_r, self.page, self.blocks, self.pages, max_pos=800)
        mj.rope_append(p, q=x[:, :hq], k=x[:, hq : hq + self.h_k], v=x[:, hq + self.h_k :], positions=positions, cos_sin=self.cos_sin,
                       q_out=q_out, k_cache=self.k, v_cache=self.v, block_table=self.table, seq_lens=self.lens, k_descale=self.kd,
                       v_descale=self.vd, cu_tokens=cu_tokens, status=self.status)

    def projection(self, tokens):
        return torch.randn(tokens, self.h_k * (self.h_r + 2), D, generator=self.gen, device="cuda").to(torch.bfloat16)

    def rows(self, b, n):
        """The first n rows of a sequence's K and V in the pool, codes (n, 2, h_k, 128)."""
        t = self.table[b].cpu().numpy()
        j = np.arange(n)
        at = torch.from_numpy(t[j // self.page].astype(np.int64) * self.page + j % self.page).cuda()
        return torch.stack([p.view(-1, self.h_k, D)[at] for p in (self.k, self.v)], 1)

    def pages_whole(self, lens):
        """Every page is in one sequence's table or the free list, once."""
        t = self.table.cpu().numpy()
        used = sum((t[b, : -(-n // self.page)].tolist() for b, n in enumerate(lens)), [])
        free = self.free[: int(self.num_free.item())].tolist()
        assert sorted(used + free) == list(range(self.pages))

    def check_attention(self, b, q, o, lse, keys, seen, bounds, amax=None):
        """q (rows, heads, 128) against the sequence's codes."""
        for h in range(self.h_k * self.h_r):
            g = h // self.h_r
            k, v = (keys[:, i, g].view(torch.float8_e4m3fn).double() for i in (0, 1))
            ref = attend(q[:, h].double(), k, v * self.vd[b, g].double(), float(self.kd[b, g].double()) * D**-0.5, seen, 0.0, bounds,
                         None if amax is None else amax[g])
            check_rows(o[:, h], lse[:, h], ref, f"sequence {b}, head {h}")


@pytest.mark.parametrize("h_k,h_r,page,q_len", [(2, 4, 16, 4), (1, 8, 32, 13), (2, 5, 64, 33)])
def test_serving_loop(h_k, h_r, page, q_len):
    s = Server(h_k, h_r, page, q_len)
    hq, lens = h_k * h_r, np.zeros(4, np.int64)
    # ---- prompts, in two chunks of different lengths
    params = mj.make_params(4, 1, h_k, h_r, page, s.blocks, s.pages, max_splits=16)
    for news in ([150, 0, 33, 1], [7, 200, 1, 64]):
        total, pad = sum(news), 5
        cu, pos = torch.zeros(5, **I32), torch.zeros(total + pad, **I32)
        slots = torch.zeros(total + pad, dtype=torch.int64, device="cuda")
        s.reserve(new_tokens=torch.tensor(news, **I32), cu_tokens=cu, positions=pos, slots=slots)
        lens += news
        x = s.projection(total + pad)
        q = torch.full((total + pad, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        s.append(x, pos, q, cu_tokens=cu)
        plan = torch.empty(mj.prompt_plan_bytes(params, total + pad), dtype=torch.uint8, device="cuda")
        mj.prompt_plan(params, cu_tokens=cu, seq_lens=s.lens, num_tokens=total + pad, plan=plan, status=s.status)
        o, lse = torch.full_like(q, float("nan")), torch.full((total + pad, hq), float("nan"), device="cuda")
        mj.prompt_attn(params, q=q, k_cache=s.k, v_cache=s.v, block_table=s.table, plan=plan, q_descale=s.one, k_descale=s.kd,
                       v_descale=s.vd, o=o, lse=lse, softmax_scale=D**-0.5, status=s.status,
                       workspace=torch.empty(mj.prompt_workspace_bytes(params), dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0 and s.lens.tolist() == lens.tolist()
        s.pages_whole(lens)
        assert torch.isnan(o[total:]).all() and (slots[total:] == -1).all()
        t0 = 0
        for b, n in enumerate(news):
            L = int(lens[b])
            keys = s.rows(b, L)
            # the rows written are where the slot map says
            flat = torch.stack([p.view(-1, h_k, D)[slots[t0 : t0 + n]] for p in (s.k, s.v)], 1)
            assert torch.equal(keys[L - n :], flat)
            if s.slots_of[b] != []:
                assert torch.equal(keys[: L - n], s.slots_of[b])  # and the earlier ones stayed
            s.slots_of[b] = keys
            at = torch.arange(L - n, L, device="cuda")[:, None]
            if n:
                s.check_attention(b, q[t0 : t0 + n], o[t0 : t0 + n], lse[t0 : t0 + n], keys, torch.arange(L, device="cuda") <= at, HALF_P)
            t0 += n
    # ---- trees: draft, attend, commit, give pages back
    params = mj.make_params(4, q_len, h_k, h_r, page, s.blocks, s.pages, max_splits=16)
    words = -(-q_len // 32)
    for step in range(3):
        parents = [[-1 if i == 0 else int(s.rng.integers(max(0, i - 5), i)) for i in range(q_len)] for _ in range(4)]
        masks = [serve_ref.tree_mask(p, words) for p in parents]
        see = [np.unpackbits(m.view(np.uint8), axis=-1, bitorder="little")[:, :q_len].astype(bool) for m in masks]
        ctx = lens.copy()
        depth = np.stack([v.sum(1) - 1 for v in see])
        s.reserve(q_len=q_len)
        lens = lens + q_len
        x = s.projection(4 * q_len)
        q = torch.empty(4, h_k, q_len * h_r, D, dtype=torch.bfloat16, device="cuda")
        pos = torch.from_numpy((ctx[:, None] + depth).astype(np.int32).reshape(-1)).cuda()
        s.append(x, pos, q, q_len=q_len)
        mask = torch.from_numpy(np.stack(masks).view(np.int32)).cuda()
        plan = mj.decode_plan(params, lens.tolist())
        o, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
        mj.decode_attn_tree(params, tree_mask=mask, q=q, k_cache=s.k, v_cache=s.v, block_table=s.table, seq_lens=s.lens,
                            work=torch.from_numpy(plan.work).cuda(), n_splits=torch.from_numpy(plan.n_splits).cuda(), q_descale=s.one,
                            k_descale=s.kd, v_descale=s.vd, o=o, lse=lse, softmax_scale=D**-0.5, max_n_splits=plan.max_n_splits,
                            workspace=torch.empty(mj.workspace_bytes(params), dtype=torch.uint8, device="cuda"), status=s.status)
        path = np.zeros((4, q_len), np.int32)
        count = np.zeros(4, np.int32)
        for b in range(4):
            node, branch = int(s.rng.integers(0, q_len)), []
            while node >= 0:
                branch.insert(0, node)
                node = parents[b][node]
            path[b, : len(branch)], count[b] = branch, len(branch)
        torch.cuda.synchronize()
        drafted = [s.rows(b, int(lens[b])) for b in range(4)]
        for b in range(4):
            seen = torch.zeros(q_len, int(lens[b]), dtype=torch.bool, device="cuda")
            seen[:, : ctx[b]] = True
            seen[:, ctx[b] :] = torch.from_numpy(see[b]).cuda()
            un = lambda t: t[b].view(h_k, q_len, h_r, -1).permute(1, 0, 2, 3).reshape(q_len, hq, -1)  # noqa: E731
            amax = q[b].double().abs().amax((1, 2))
            s.check_attention(b, un(q), un(o), un(lse[..., None])[..., 0], drafted[b], seen, SPLIT_P, amax)
        held = s.lens.clone()
        mj.tree_commit(params, k_cache=s.k, v_cache=s.v, block_table=s.table, seq_lens=s.lens, accepted=torch.from_numpy(path).cuda(),
                       num_accepted=torch.from_numpy(count).cuda(), status=s.status)
        mj.pages_release(s.page_params, seq_lens=held, keep_lens=s.lens, free_pages=s.free, num_free=s.num_free, block_table=s.table,
                         status=s.status)
        torch.cuda.synchronize()
        lens = ctx + count
        assert int(s.status.item()) == 0 and s.lens.tolist() == lens.tolist()
        s.pages_whole(lens)
        for b in range(4):
            keys = s.rows(b, int(lens[b]))
            assert torch.equal(keys[: ctx[b]], s.slots_of[b])
            assert torch.equal(keys[ctx[b] :], drafted[b][[int(ctx[b]) + int(m) for m in path[b, : count[b]]]])
            s.slots_of[b] = keys


def test_captured_step_equals_the_eager_one():
    """Reserve, append, attend a tree, commit and release in one graph, replayed
    over steps, beside the same steps run eagerly on a copy: the same bytes."""
    h_k, h_r, page, q_len = 2, 4, 16, 6
    runs = []
    for captured in (False, True):
        s = Server(h_k, h_r, page, q_len, seed=3)
        s.lens.copy_(torch.tensor([0, 0, 0, 0], **I32))
        s.reserve(q_len=40)
        s.append(s.projection(160), torch.arange(40, **I32).repeat(4), torch.empty(4, h_k, 40 * h_r, D, dtype=torch.bfloat16, device="cuda"), q_len=40)
        params = mj.make_params(4, q_len, h_k, h_r, page, s.blocks, s.pages, max_splits=4)
        x = torch.zeros(4 * q_len, h_k * (h_r + 2), D, dtype=torch.bfloat16, device="cuda")
        pos, mask = torch.zeros(4 * q_len, **I32), torch.zeros(4, q_len, 1, **I32)
        path, count, held = torch.zeros(4, q_len, **I32), torch.zeros(4, **I32), torch.zeros(4, **I32)
        q = torch.empty(4, h_k, q_len * h_r, D, dtype=torch.bfloat16, device="cuda")
        o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        pad = mj.decode_plan_max_items(params)
        work, n_splits = torch.zeros(pad, 4, **I32), torch.zeros(4, **I32)
        ws = torch.empty(mj.workspace_bytes(params), dtype=torch.uint8, device="cuda")

        def step():
            s.reserve(q_len=q_len)
            s.append(x, pos, q, q_len=q_len)
            mj.decode_plan_device(params, s.lens, work, n_splits, pad_to=pad, status=s.status)
            mj.decode_attn_tree(params, tree_mask=mask, q=q, k_cache=s.k, v_cache=s.v, block_table=s.table, seq_lens=s.lens, work=work,
                                n_splits=n_splits, q_descale=s.one, k_descale=s.kd, v_descale=s.vd, o=o, lse=lse, workspace=ws,
                                softmax_scale=D**-0.5, status=s.status)
            held.copy_(s.lens)
            mj.tree_commit(params, k_cache=s.k, v_cache=s.v, block_table=s.table, seq_lens=s.lens, accepted=path, num_accepted=count, status=s.status)
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
        rng, lens, seen = np.random.default_rng(8), np.full(4, 40), []
        for _ in range(6):
            parents = [[-1] + [int(rng.integers(0, i)) for i in range(1, q_len)] for _ in range(4)]
            m = np.stack([serve_ref.tree_mask(p, 1) for p in parents])
            depth = np.unpackbits(m.view(np.uint8), axis=-1).sum(-1) - 1
            n = rng.integers(0, 3, 4)
            take = np.zeros((4, q_len), np.int32)
            take[:, 1] = 3
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32)).cuda())
            pos.copy_(torch.from_numpy((lens[:, None] + depth).astype(np.int32).reshape(-1)))
            mask.copy_(torch.from_numpy(m.view(np.int32)))
            path.copy_(torch.from_numpy(take))
            count.copy_(torch.from_numpy(n.astype(np.int32)))
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            assert int(s.status.item()) == 0
            lens = lens + n
            assert s.lens.tolist() == lens.tolist()
            seen += [o.clone(), lse.clone(), s.table.clone(), s.free.clone(), s.k.clone(), s.v.clone()]
        runs.append(seen)
    for a, b in zip(*runs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
