"""GPU parity of the eviction (mj_evict): the kept set, its order, the moved
rows and planes, byte for byte, against the plain rule."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import cache_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Case:
    def __init__(self, lens, budget, h_k=2, page_size=16, first=0, last=0, pos=False, in_place=False, fmt="e4m3", layout="nhd",
                 weights="mixed", seed=0):
        rng = np.random.default_rng(seed)
        self.__dict__.update(locals())
        self.b = b = len(lens)
        need = [-(-L // page_size) for L in lens]
        self.max_blocks = max(need + [1]) + 1
        pages = sum(need) + 2
        perm = rng.permutation(pages)
        self.bt = np.full((b, self.max_blocks), -1, dtype=np.int32)
        at = 0
        for i, m in enumerate(need):
            self.bt[i, :m] = perm[at : at + m]
            at += m
        bits = {"e4m3": 8, "e3m2": 6, "e2m3": 6, "e2m1": 4, "nvfp4": 4}[fmt]
        rb = 16 * bits
        kv = torch.from_numpy(rng.integers(0, 256, (2, pages, page_size, h_k, rb)).astype(np.uint8)).cuda()
        if layout == "hnd":
            buf = kv.permute(1, 0, 3, 2, 4).contiguous()
            self.k, self.v = buf[:, 0].transpose(1, 2), buf[:, 1].transpose(1, 2)
        else:
            self.k, self.v = kv[0], kv[1]
        self.scales = [torch.from_numpy(rng.integers(0, 256, (pages, h_k, page_size, 8)).astype(np.uint8)).cuda() for _ in range(2)] if fmt == "nvfp4" else [None, None]
        slots = self.max_blocks * page_size
        acc = rng.exponential(1.0, (b, h_k, slots)).astype(np.float32)
        if weights == "mixed":
            acc = np.where(rng.random(acc.shape) < 0.4, np.round(acc * 2) / 2, acc).astype(np.float32)
            acc[rng.random(acc.shape) < 0.05] = -0.0
        elif weights == "equal":
            acc[:] = 0.25
        elif weights == "wild":
            special = np.asarray([np.nan, np.inf, -np.inf, -1.0, 0.0, -0.0, 1e-42, -1e-42, 3e38], dtype=np.float32)
            acc = special[rng.integers(0, len(special), acc.shape)]
        self.acc_host = acc
        self.acc = torch.from_numpy(acc.copy()).cuda()
        self.pos_host = rng.integers(0, 2 * slots, acc.shape).astype(np.int32) if pos else np.broadcast_to(np.arange(slots, dtype=np.int32), acc.shape)
        self.pos = torch.from_numpy(self.pos_host.copy()).cuda() if pos else None
        self.next = np.asarray(lens, dtype=np.int32) + (slots if pos else 0)
        self.acc_out = self.acc if in_place else torch.full_like(self.acc, -77.0)
        self.pos_out = None if not pos else (self.pos if in_place else torch.full_like(self.pos, -77))
        self.new_lens = torch.full((b,), -1, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.params = mj.make_params(b, 1, h_k, 1, page_size, self.max_blocks, pages, kv_format=mj.KV_FORMATS[fmt],
                                     q_dtype=mj.MJ_E4M3 if fmt == "nvfp4" else mj.MJ_BF16)
        self.ws = torch.full((mj.evict_workspace_bytes(self.params, budget),), 0xA5, dtype=torch.uint8, device="cuda")
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.table = torch.from_numpy(self.bt).cuda()
        self.host = [x.cpu().numpy().copy() for x in (self.k, self.v)] + [None if s is None else s.cpu().numpy().copy() for s in self.scales]

    def call(self):
        return mj.Evict(self.params, k_cache=self.k, v_cache=self.v, block_table=self.table, seq_lens=self.seq_lens, acc=self.acc,
                        acc_out=self.acc_out, key_pos=self.pos, key_pos_out=self.pos_out,
                        next_pos=torch.from_numpy(self.next).cuda() if self.pos is not None else None, new_lens=self.new_lens,
                        budget=self.budget, keep_first=self.first, keep_last=self.last, workspace=self.ws, status=self.status,
                        k_scales=self.scales[0], v_scales=self.scales[1])

    def check(self, status=0, skip=()):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        pools = [None if x is None else x.copy() for x in self.host]
        acc = self.acc_host.copy() if self.in_place else np.full_like(self.acc_host, -77.0)
        pos = self.pos_host.copy() if self.in_place else np.full(self.pos_host.shape, -77, dtype=np.int32)
        ps = self.page_size
        for b, L in enumerate(self.lens):
            for g in range(self.h_k):
                src = cache_ref.evict_slots(self.acc_host[b, g], self.pos_host[b, g], L, self.budget, int(self.next[b]), self.first, self.last)
                acc[b, g, : len(src)] = self.acc_host[b, g, src]
                pos[b, g, : len(src)] = self.pos_host[b, g, src]
                for dst, s in enumerate(src):
                    if s == dst or (b, dst // ps) in skip or (b, s // ps) in skip:
                        continue
                    dp, sp = self.bt[b, dst // ps], self.bt[b, s // ps]
                    for i in (0, 1):
                        pools[i][dp, dst % ps, g] = self.host[i][sp, s % ps, g]
                        if pools[2 + i] is not None:
                            pools[2 + i][dp, g, dst % ps] = self.host[2 + i][sp, g, s % ps]
        assert np.array_equal(self.new_lens.cpu().numpy(), np.minimum(self.lens, self.budget))
        for x, want in zip((self.k, self.v, *self.scales), pools):
            if x is not None:
                assert np.array_equal(x.cpu().numpy(), want)
        assert np.array_equal(self.acc_out.cpu().numpy(), acc, equal_nan=True)
        if self.pos is not None:
            assert np.array_equal(self.pos_out.cpu().numpy(), pos)


LENS = [0, 1, 63, 64, 65, 100, 128, 700, 1025]


@pytest.mark.parametrize("budget", [1, 63, 64, 65, 500, 1024, 1025, 4000])
@pytest.mark.parametrize("weights", ["mixed", "equal", "wild"])
def test_budgets_and_ties(budget, weights):
    c = Case(LENS, budget, weights=weights, seed=budget)
    c.call()()
    c.check()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("first,last", [(0, 0), (4, 0), (0, 40), (4, 60), (32, 32)])
@pytest.mark.parametrize("pos", [False, True])
def test_protection_and_positions(in_place, first, last, pos):
    c = Case(LENS, 64, first=first, last=last, pos=pos, in_place=in_place, seed=first + last)
    c.call()()
    c.check()


@pytest.mark.parametrize("fmt", ["e4m3", "e3m2", "e2m3", "e2m1", "nvfp4"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_pool_formats(fmt, layout):
    c = Case([300, 90], 70, h_k=4 if fmt != "e4m3" else 3, page_size=32, fmt=fmt, layout=layout, pos=True, last=5)
    c.call()()
    c.check()


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
def test_long_sequences(page_size):
    c = Case([20011, 5, 9000], 6001, h_k=1, page_size=page_size, first=4, last=300, seed=page_size)
    c.call()()
    c.check()


def test_one_sequence_longer_than_shared_memory_holds():
    c = Case([300001], 100000, h_k=1, page_size=128, first=10, last=5000, pos=True)
    c.call()()
    c.check()


def test_runs_too_long_for_shared_memory():
    """Every CTA's run is read again from the weights in each pass."""
    c = Case([500003], 250000, h_k=1, page_size=128, first=3, last=1000, weights="mixed")
    c.call()()
    c.check()


def test_more_groups_than_the_gpu_holds():
    rng = np.random.default_rng(8)
    c = Case(rng.integers(0, 700, 90).tolist(), 150, h_k=8, first=2, last=20, pos=True)
    c.call()()
    c.check()


@pytest.mark.parametrize("b", [305, 512, 513])
def test_many_sequences(b):
    """Around the number up to which the longest are taken first; equal
    lengths among them."""
    rng = np.random.default_rng(b)
    c = Case(rng.integers(0, 60, b).tolist(), 20, h_k=1, first=1, last=4)
    c.call()()
    c.check()


def test_everything_protected_in_excess_keeps_the_lowest_slots():
    """More slots hold a protected position than the budget: the lowest stay."""
    c = Case([200], 50, h_k=1, pos=True, last=50)
    c.pos_host = np.full(c.pos_host.shape, int(c.next[0]) - 1, dtype=np.int32)
    c.pos.copy_(torch.from_numpy(c.pos_host))
    c.call()()
    c.check()


def test_bad_pages_are_not_moved():
    for entry in (-1, -2, 2**31 - 1):
        c = Case([300, 200], 64, h_k=2, seed=5)
        c.table[0, 2] = entry
        c.table[0, 10] = entry
        c.call()()
        c.check(status=mj.MJ_ERR_INVALID_ARG, skip=((0, 2), (0, 10)))


def test_length_past_the_table_is_reported():
    c = Case([40, 30], 16)
    c.seq_lens[1] = c.max_blocks * 16 + 1
    call = c.call()
    c.bt[1] = c.bt[0]  # every block it may touch names a page
    c.table[1] = 0
    call()
    torch.cuda.synchronize()
    assert int(c.status.item()) == mj.MJ_ERR_INVALID_ARG


def test_again_on_the_same_inputs_is_the_same():
    """With separate outputs a second call finds its sources unchanged."""
    c = Case(LENS, 64, first=3, last=20, pos=True)
    call = c.call()
    call()
    call()
    c.check()


def test_graph_and_stream():
    c = Case(LENS, 64, first=3, last=20)
    call = c.call()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call(side)
    graph.replay()
    c.check()


def test_binding_refuses():
    c = Case([40, 30], 16, pos=True)
    with pytest.raises(ValueError):
        mj.Evict(c.params, k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=c.seq_lens, acc=c.acc[:, :, :16],
                 new_lens=c.new_lens, budget=16, workspace=c.ws)
    with pytest.raises(ValueError):
        mj.Evict(c.params, k_cache=c.k, v_cache=c.v[:1], block_table=c.table, seq_lens=c.seq_lens, acc=c.acc, new_lens=c.new_lens,
                 budget=16, workspace=c.ws)
    with pytest.raises(TypeError):
        mj.Evict(c.params, k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=c.seq_lens, acc=c.acc, new_lens=c.new_lens,
                 budget=16, workspace=c.ws, key_pos=c.pos)  # no next_pos
    with pytest.raises(mj.MjError):
        mj.evict(c.params, k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=c.seq_lens, acc=c.acc, new_lens=c.seq_lens,
                 budget=16, workspace=c.ws)
    with pytest.raises(mj.MjError):
        mj.evict(c.params, k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=c.seq_lens, acc=c.acc, new_lens=c.new_lens,
                 budget=16, workspace=c.ws[:16])
    with pytest.raises(ValueError):
        mj.Evict(c.params, k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=c.seq_lens, acc=c.acc, new_lens=c.new_lens,
                 budget=16, workspace=c.ws, k_scales=c.k, v_scales=c.v)
