"""The serving operators where offsets pass 32 bits, and calls that share what they
only read."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import serve_ref
from tests.serving_helpers import I32, Cache
from tests.test_gpu_prompt import Prompt
from tests.test_gpu_tree import Tree

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture
def far(monkeypatch):
    """Pools of over 2^32 bytes (pages of 64 x 2 x 128) with the sequences at their end."""
    monkeypatch.setattr(Cache, "ahead", (1 << 18) + 99)
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompts_in_a_far_pool(far, e4m3):
    Prompt([700, 129, 1], [300, 1, 1], 2, 4, 64, e4m3=e4m3).run().check()


@pytest.mark.parametrize("q_len,h_r", [(5, 2), (12, 4), (70, 4)])
def test_trees_in_a_far_pool(far, q_len, h_r):
    """By each of the kernels that trees take."""
    Tree([700, 129, q_len], [q_len, 3, q_len], q_len, 2, h_r, 64).run().check()


def test_commit_in_a_far_pool(far):
    c = Cache([300, 129, 70], 2, 64)
    before = [[c.rows(pool, b) for b in range(3)] for pool in (c.k, c.v)]
    paths, nodes = [[1, 2, 60, 69], [0, 5], [9]], [70, 6, 70]
    accepted = torch.tensor([p + [0] * (4 - len(p)) for p in paths], **I32)
    status, new = torch.zeros(1, **I32), torch.zeros(3, **I32)
    mj.tree_commit(mj.make_params(3, 70, 2, 1, 64, c.max_blocks, c.num_pages), k_cache=c.k, v_cache=c.v, block_table=c.table,
                   seq_lens=c.seq_lens, accepted=accepted, num_accepted=torch.tensor([4, 2, 1], **I32),
                   tree_lens=torch.tensor(nodes, **I32), new_lens=new, status=status)
    assert int(status.item()) == 0 and new.tolist() == [234, 125, 1]
    for pool, rows in zip((c.k, c.v), before):
        for b in range(3):
            want = [serve_ref.commit(x.cpu().numpy(), c.lens[b] - nodes[b], np.array(paths[b], np.int32)) for x in rows[b]]
            assert np.array_equal(c.rows(pool, b).cpu().numpy(), np.stack(want))


def test_queries_and_results_far_apart():
    """Tokens 2^26 elements apart: Q and O pass 2^32 bytes and 2^31 elements."""
    n, h_q = 41, 8
    p = Prompt([200], [n], 2, 4, 16)
    q, o = (torch.empty((n << 26) // 2, dtype=torch.int32, device="cuda").view(torch.bfloat16).as_strided((n, h_q, D), (1 << 26, D, 1))
            for _ in range(2))
    q.copy_(p.q)
    o.fill_(float("nan"))
    p.make_plan()
    mj.prompt_attn(p.params, q=q, k_cache=p.c.k, v_cache=p.c.v, block_table=p.c.table, plan=p.plan, q_descale=p.qd, k_descale=p.c.kd,
                   v_descale=p.c.vd, o=o, lse=p.lse, workspace=p.ws, softmax_scale=D**-0.5, scale_o=0.75, status=p.status)
    p.o.copy_(o)
    assert int(p.status.item()) == 0
    p.check()
    del q, o
    torch.cuda.empty_cache()


def test_layers_share_a_plan():
    """Two layers' attention at once on two streams by one plan, each with a workspace of its own, and again as two graphs."""
    p = Prompt([3000, 700], [40, 300], 2, 4, 16)
    p.run()
    want, lse = p.o.clone(), p.lse.clone()
    outs = [(torch.full_like(p.o, float("nan")), torch.full_like(p.lse, float("nan")), torch.empty_like(p.ws)) for _ in range(2)]
    calls = [mj.PromptAttn(p.params, q=p.q, k_cache=p.c.k, v_cache=p.c.v, block_table=p.c.table, plan=p.plan, q_descale=p.qd,
                           k_descale=p.c.kd, v_descale=p.c.vd, o=o, lse=x, workspace=ws, softmax_scale=D**-0.5, scale_o=0.75,
                           status=p.status) for o, x, ws in outs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, call in zip(streams, calls):
        call(s)
    torch.cuda.synchronize()
    for o, x, _ in outs:
        assert torch.equal(o, want) and torch.equal(x, lse)
        o.fill_(float("nan"))
    graphs = []
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, x, _ in outs:
            assert torch.equal(o, want) and torch.equal(x, lse)
            o.fill_(float("nan"))
    assert int(p.status.item()) == 0


def test_pages_captured_and_on_two_streams():
    """Two pools' steps at once on two streams, as graphs replayed while demands and lengths change in their buffers."""
    rng = np.random.default_rng(3)
    seqs, page, blocks, pages = 20, 16, 30, 700
    params = mj.make_page_params(seqs, page, blocks, pages)
    sides = []
    for _ in range(2):
        d = dict(seq_lens=torch.zeros(seqs, **I32), free_pages=torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda(),
                 num_free=torch.full((1,), pages, **I32), block_table=torch.full((seqs, blocks), -1, **I32))
        more = dict(new_tokens=torch.zeros(seqs, **I32), cu_tokens=torch.zeros(seqs + 1, **I32), positions=torch.zeros(9000, **I32),
                    slots=torch.zeros(9000, dtype=torch.int64, device="cuda"), status=torch.zeros(1, **I32))
        keep = torch.zeros(seqs, **I32)
        side = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            mj.pages_reserve(params, **d, **more)
            mj.pages_release(params, keep_lens=keep, status=more["status"], **d)
            d["seq_lens"].copy_(keep)
        host = [x.cpu().numpy().copy() for x in (d["seq_lens"], d["free_pages"], d["block_table"])] + [pages]
        sides.append((d, more, keep, side, g, host))
    for _ in range(5):
        for d, more, keep, side, g, host in sides:
            lens, free, table, n = host
            new = rng.integers(0, 90, seqs).astype(np.int32)
            want = serve_ref.reserve(lens, new, free, n, table, page, 9000)
            held = np.asarray(want[1], np.int32)
            kept = rng.integers(0, held + 1).astype(np.int32)
            out = serve_ref.release(held, kept, free, want[2], want[0], page)
            assert want[6] == out[2] == 0
            with torch.cuda.stream(side):
                more["new_tokens"].copy_(torch.from_numpy(new))
                keep.copy_(torch.from_numpy(kept))
                g.replay()
            host[:] = [kept, out[0], want[0], out[1]]
            host.append(want)
        torch.cuda.synchronize()
        for d, more, keep, side, g, host in sides:
            want = host.pop()
            assert np.array_equal(d["block_table"].cpu().numpy(), host[2]) and d["num_free"].item() == host[3]
            assert np.array_equal(d["free_pages"].cpu().numpy(), host[1])
            for name, x in zip(("cu_tokens", "positions", "slots"), want[3:6]):
                assert np.array_equal(more[name].cpu().numpy(), x), name
            assert int(more["status"].item()) == 0
