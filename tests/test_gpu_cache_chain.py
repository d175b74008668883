"""The cache operators as a serving loop uses them: ragged prompts appended,
then decode steps (append, attention on capped scores, key weights), with the
caches cut whenever they pass the budget, all on one stream with no host
synchronisation inside a step.  A host mirror of every cache follows the rows
(codes, weights, positions) and gives each step's float64 reference."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import cache_ref

pytestmark = pytest.mark.gpu

H_K, H_R, PS, CAP, BUDGET, SLACK = 2, 4, 16, 12.0, 48, 8
SCALE = 128**-0.5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_serving_loop():
    rng = np.random.default_rng(0)
    gen = torch.Generator("cuda").manual_seed(1)
    prompts = [37, 1, 70]
    b, h_q, max_blocks = len(prompts), H_K * H_R, 8
    pages = b * max_blocks + 1
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.from_numpy(rng.permutation(pages)[: b * max_blocks].reshape(b, max_blocks).astype(np.int32)).cuda()
    kc = torch.full((pages, PS, H_K, 128), 0x7F, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    kd, vd = torch.rand(b, H_K, generator=gen, device="cuda") * 0.02 + 0.01, torch.rand(b, H_K, generator=gen, device="cuda") * 0.02 + 0.01
    qd = torch.ones(1, device="cuda")
    acc = torch.full((b, H_K, max_blocks * PS), float("nan"), device="cuda")
    key_pos = torch.full(acc.shape, -1, **i32)
    ang = np.outer(np.arange(400), 10000.0 ** (-np.arange(64) / 64))
    cos_sin = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    lens = torch.tensor(prompts, **i32)
    new_lens, next_pos = torch.zeros(b, **i32), torch.tensor(prompts, **i32)
    status = torch.zeros(1, **i32)
    mirror = {(i, g): [] for i in range(b) for g in range(H_K)}  # rows (k codes, v codes, position)

    def qkv(n):
        return (2 * torch.randn(n, h_q + 2 * H_K, 128, generator=gen, device="cuda")).to(torch.bfloat16)

    def collect(news):
        """The rows the append wrote, read back slot by slot."""
        k, v, t, ls, kp = kc.cpu().numpy(), vc.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy(), key_pos.cpu().numpy()
        for i, n in enumerate(news):
            for slot in range(ls[i] - n, ls[i]):
                for g in range(H_K):
                    pg, r = t[i, slot // PS], slot % PS
                    mirror[i, g].append((k[pg, r, g], v[pg, r, g], int(kp[i, g, slot])))

    # ---- prompts, ragged
    x = qkv(sum(prompts))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), **i32)
    pos = torch.from_numpy(np.concatenate([np.arange(n) for n in prompts]).astype(np.int32)).cuda()
    rp = mj.make_rope_params(b, 1, H_K, H_R, PS, max_blocks, pages, max_pos=400)
    mj.rope_append(rp, q=x[:, :h_q], k=x[:, h_q : h_q + H_K], v=x[:, h_q + H_K :], positions=pos, cos_sin=cos_sin, q_out=x[:, :h_q],
                   k_cache=kc, v_cache=vc, block_table=table, seq_lens=lens, k_descale=kd, v_descale=vd, cu_tokens=cu,
                   key_pos=key_pos, status=status)
    torch.cuda.synchronize()
    collect(prompts)
    # nothing has weighed the prompt yet
    acc.zero_()

    params = mj.make_params(b, 1, H_K, H_R, PS, max_blocks, pages, max_splits=4, kernel=mj.MJ_KERNEL_TENSOR_CORE_QROWS)
    mod = mj.ScoreMod(softcap=CAP)
    pad = mj.decode_plan_max_items(params)
    work, n_splits = torch.zeros(pad, 4, **i32), torch.zeros(b, **i32)
    ws = torch.empty(mj.workspace_bytes(params), dtype=torch.uint8, device="cuda")
    ews = torch.empty(mj.evict_workspace_bytes(params, BUDGET), dtype=torch.uint8, device="cuda")
    q = torch.empty(b, H_K, H_R, 128, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(b, H_K, H_R, device="cuda")
    want_acc = {key: np.zeros(len(rows)) for key, rows in mirror.items()}
    cuts = 0
    for step in range(30):
        x = qkv(b)
        lens += 1
        mj.rope_append(rp, q=x[:, :h_q], k=x[:, h_q : h_q + H_K], v=x[:, h_q + H_K :], positions=next_pos.clone(), cos_sin=cos_sin,
                       q_out=q, k_cache=kc, v_cache=vc, block_table=table, seq_lens=lens, k_descale=kd, v_descale=vd,
                       key_pos=key_pos, status=status)
        next_pos += 1
        mj.decode_plan_device(params, lens, work, n_splits, pad, status=status)
        mj.decode_attn_mod(params, mod, q=q, k_cache=kc, v_cache=vc, block_table=table, seq_lens=lens, work=work, n_splits=n_splits,
                           q_descale=qd, k_descale=kd, v_descale=vd, o=o, lse=lse, softmax_scale=SCALE, workspace=ws,
                           status=status, max_n_splits=4)
        mj.key_weights(params, mod, q=q, k_cache=kc, block_table=table, seq_lens=lens, work=work, q_descale=qd, k_descale=kd,
                       lse=lse, acc=acc, softmax_scale=SCALE, fresh=1, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        collect([1] * b)
        # ---- the step's reference over the mirror's rows
        qh, oh, lh, ah = (t.float().cpu().numpy().astype(np.float64) for t in (q, o, lse, acc))
        kdh, vdh = kd.cpu().numpy().astype(np.float64), vd.cpu().numpy().astype(np.float64)
        for (i, g), rows in mirror.items():
            assert len(rows) == int(lens[i])
            k = np.stack([cache_ref.values_of(r[0]) for r in rows])
            v = np.stack([cache_ref.values_of(r[1]) for r in rows]) * vdh[i, g]
            z = cache_ref.logits(qh[i, g], k, SCALE * kdh[i, g], CAP, None, len(rows), 1, H_R)
            w, l = cache_ref.softmax_rows(z, np.ones(z.shape, dtype=bool))
            assert np.abs(lh[i, g] - l).max() <= 2e-3
            want = w @ v
            assert (np.abs(oh[i, g] - want) <= 2e-2 + 2e-2 * np.abs(want)).all()
            want_acc[i, g] = np.append(want_acc[i, g], 0.0) + w.sum(0)
            # a weight is off by its logit's and the LSE's error, at most 2e-3 of it together a step
            assert (np.abs(ah[i, g, : len(rows)] - want_acc[i, g]) <= 2e-3 * want_acc[i, g] + 1e-6).all()
        # ---- the cut
        if int(lens.max()) > BUDGET + SLACK:
            before, kp, L = acc.cpu().numpy(), key_pos.cpu().numpy(), lens.cpu().numpy()
            mj.evict(params, k_cache=kc, v_cache=vc, block_table=table, seq_lens=lens, acc=acc, key_pos=key_pos, next_pos=next_pos,
                     new_lens=new_lens, budget=BUDGET, keep_first=2, keep_last=6, workspace=ews, status=status)
            lens.copy_(new_lens)
            torch.cuda.synchronize()
            assert int(status.item()) == 0
            cuts += 1
            for (i, g), rows in mirror.items():
                src = cache_ref.evict_slots(before[i, g], kp[i, g], int(L[i]), BUDGET, int(next_pos[i]), 2, 6)
                mirror[i, g] = [rows[s] for s in src]
                want_acc[i, g] = want_acc[i, g][src]
                got = key_pos[i, g, : len(src)].cpu().numpy()
                assert got.tolist() == [r[2] for r in mirror[i, g]]
                newest = set(range(max(0, int(next_pos[i]) - 6), int(next_pos[i])))
                assert newest <= set(got.tolist())  # the newest six are still there
    assert cuts >= 2


class Loop:
    """A decode step of every operator, budget 40, on state of its own, whose
    pages are the pool's from `base` on."""

    def __init__(self, base=0):
        gen = torch.Generator("cuda").manual_seed(3)
        i32 = dict(dtype=torch.int32, device="cuda")
        lens, b, max_blocks = [33, 1, 40], 3, 4
        pages, h_q = b * max_blocks, H_K * H_R
        rand = lambda *shape: torch.rand(*shape, generator=gen, device="cuda")  # noqa: E731
        self.base, pools = base, torch.empty(2, base + pages, PS, H_K, 128, dtype=torch.uint8, device="cuda")
        for pool in pools:
            pool[base:] = torch.randint(0, 0x7F, (pages, PS, H_K, 128), generator=gen, device="cuda").to(torch.uint8)
        self.kc, self.vc = pools
        table = (base + torch.randperm(pages, generator=gen, device="cuda")).reshape(b, max_blocks).to(torch.int32)
        pages += base
        kd, vd, qd = rand(b, H_K) * 1e-3 + 1e-3, rand(b, H_K) * 1e-3 + 1e-3, torch.ones(1, device="cuda")
        self.acc = rand(b, H_K, max_blocks * PS)
        self.key_pos = torch.arange(max_blocks * PS, **i32).expand(b, H_K, -1).contiguous()
        self.lens, self.next_pos = torch.tensor(lens, **i32), torch.tensor(lens, **i32)
        self.new_lens, self.status = torch.zeros(b, **i32), torch.zeros(1, **i32)
        ang = torch.outer(torch.arange(100.0, device="cuda"), 10000.0 ** (-torch.arange(64.0, device="cuda") / 64))
        cos_sin = torch.cat([ang.cos(), ang.sin()], 1)
        self.x = torch.empty(b, h_q + 2 * H_K, 128, dtype=torch.bfloat16, device="cuda")
        q = torch.empty(b, H_K, H_R, 128, dtype=torch.bfloat16, device="cuda")
        self.o, self.lse = torch.zeros_like(q), torch.zeros(b, H_K, H_R, device="cuda")
        self.params = params = mj.make_params(b, 1, H_K, H_R, PS, max_blocks, pages, max_splits=4)
        self.mod = mj.ScoreMod(softcap=CAP)
        self.pad = pad = mj.decode_plan_max_items(params)
        self.work, self.all_work = torch.zeros(pad, 4, **i32), torch.zeros(pad, 4, **i32)
        self.n_splits, self.spans, self.plan_lens = torch.zeros(b, **i32), torch.zeros(b, 4, **i32), torch.zeros(b, **i32)
        self.ws = torch.empty(mj.workspace_bytes(params), dtype=torch.uint8, device="cuda")
        self.ews = torch.empty(mj.evict_workspace_bytes(params, 40), dtype=torch.uint8, device="cuda")
        cache = dict(block_table=table, seq_lens=self.lens, status=self.status)
        self.append = mj.RopeAppend(
            mj.make_rope_params(b, 1, H_K, H_R, PS, max_blocks, pages, max_pos=100), q=self.x[:, :h_q],
            k=self.x[:, h_q : h_q + H_K], v=self.x[:, h_q + H_K :], positions=self.next_pos, cos_sin=cos_sin, q_out=q,
            k_cache=self.kc, v_cache=self.vc, k_descale=kd, v_descale=vd, key_pos=self.key_pos, **cache)
        self.attn = mj.DecodeAttnMod(params, self.mod, q=q, k_cache=self.kc, v_cache=self.vc, work=self.work, n_splits=self.n_splits,
                                     q_descale=qd, k_descale=kd, v_descale=vd, o=self.o, lse=self.lse, softmax_scale=SCALE,
                                     workspace=self.ws, spans=self.spans, max_n_splits=4, **cache)
        self.weigh = mj.KeyWeights(params, self.mod, q=q, k_cache=self.kc, work=self.all_work, q_descale=qd, k_descale=kd, lse=self.lse,
                                   acc=self.acc, softmax_scale=SCALE, decay=0.9, fresh=1, **cache)
        self.cut = mj.Evict(params, k_cache=self.kc, v_cache=self.vc, acc=self.acc, key_pos=self.key_pos, next_pos=self.next_pos,
                            new_lens=self.new_lens, budget=40, keep_first=1, keep_last=4, workspace=self.ews, **cache)

    def step(self):
        self.lens += 1
        self.append()
        self.next_pos += 1
        mj.score_spans_device(self.params, self.mod, self.lens, self.spans, self.plan_lens)
        mj.decode_plan_device(self.params, self.plan_lens, self.work, self.n_splits, self.pad, status=self.status)
        self.attn()
        mj.decode_plan_device(self.params, self.lens, self.all_work, self.plan_lens, self.pad, status=self.status)
        self.weigh()
        self.cut()
        self.lens.copy_(self.new_lens)

    def state(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.kc[self.base :], self.vc[self.base :], self.acc, self.key_pos, self.lens, self.next_pos, self.o, self.lse, self.status)]


def test_captured_steps_give_the_eager_steps_bytes():
    """Two graphs of the same step, which share its workspaces, replayed in
    turn while the caches grow to the budget and are cut at every step."""
    gen = torch.Generator("cuda").manual_seed(5)
    xs = torch.randn(16, 3, (H_R + 2) * H_K, 128, generator=gen, device="cuda").to(torch.bfloat16)
    eager, replayed = Loop(), Loop()
    graphs = []
    side = torch.cuda.Stream()
    start = [t.clone() for t in (replayed.lens, replayed.next_pos)]
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            replayed.step()
        graphs.append(graph)
    assert torch.equal(replayed.lens, start[0]) and torch.equal(replayed.next_pos, start[1])  # capture ran nothing
    for i, x in enumerate(xs):
        eager.x.copy_(x)
        eager.step()
        replayed.x.copy_(x)
        graphs[i % 2].replay()
    got, want = replayed.state(), eager.state()
    assert int(want[-1].item()) == 0 and want[4].tolist() == [40, 17, 40]
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_pools_past_32_bits():
    """The same steps on pages at byte offsets beyond 2^32 of each pool."""
    gen = torch.Generator("cuda").manual_seed(6)
    near, far = Loop(), Loop(base=2**32 // (PS * H_K * 128) + 12345)
    for _ in range(10):
        x = torch.randn(near.x.shape, generator=gen, device="cuda").to(torch.bfloat16)
        for loop in (near, far):
            loop.x.copy_(x)
            loop.step()
    want, got = near.state(), far.state()
    assert int(want[-1].item()) == 0
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
