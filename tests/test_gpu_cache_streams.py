"""GPU: two batches' cache operators in flight at once, each on its own stream
with buffers of its own, give the bytes that they give one after the other."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from paged_fp8_kv_gb300 import synthetic as syn
from tests.cache_helpers import ModStep, make_mod
from tests.test_gpu_evict import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Batch:
    """Attention, key weights and an eviction whose outputs are apart from
    their inputs, so that a second run gives the same."""

    def __init__(self, lens, q_len, h_k, h_r, seed):
        w = syn.make_workload("two", lens, q_len, h_k, h_r, 16, seed=seed, max_splits=4)
        mod, _ = make_mod(w, np.random.default_rng(seed), softcap=15.0, alibi=True, window=700, prefix=50)
        self.step = ModStep(w, mod)
        s = self.s = self.step.s
        self.acc = torch.empty(w.num_seqs, h_k, w.max_blocks * 16, device="cuda")
        self.work = torch.from_numpy(mj.decode_plan(s.params, w.seq_lens).work).cuda()
        self.weights = mj.KeyWeights(
            s.params, mod, q=s.q_packed, k_cache=s.k_cache, block_table=s.block_table, seq_lens=s.seq_lens, work=self.work,
            q_descale=s.q_descale, k_descale=s.k_descale, lse=s.lse, acc=self.acc, softmax_scale=w.softmax_scale, decay=0.0,
            status=self.step.status)
        self.case = Case(lens, 200, h_k=h_k, first=2, last=30, pos=True, seed=seed)
        self.evict = self.case.call()

    def clear(self):
        for x in (self.s.o_packed, self.s.lse, self.acc):
            x.fill_(float("nan"))

    def run(self, stream):
        self.step.call(stream)
        self.weights(stream)
        self.evict(stream)

    def bytes(self):
        assert int(self.step.status.item()) == 0
        return [x.cpu().numpy().copy() for x in (self.s.o_packed.view(torch.int16), self.s.lse, self.acc)]


@pytest.mark.parametrize("shapes", [((1, 8, 4), (4, 2, 8)), ((2, 4, 8), (9, 2, 16)), ((1, 4, 4), (8, 3, 8))],
                         ids=["r4_r32", "r16_r144", "r4_r64"])
def test_two_streams(shapes):
    rng = np.random.default_rng(5)
    batches = [Batch(rng.integers(1, 2500, 12).tolist(), *shape, seed=11 + i) for i, shape in enumerate(shapes)]
    streams = [torch.cuda.Stream() for _ in batches]
    alone = []
    for x in batches:
        x.clear()
        x.run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        alone.append(x.bytes())
    for x in batches:
        x.clear()
    torch.cuda.synchronize()
    for _ in range(20):
        for x, stream in zip(batches, streams):
            x.run(stream)
    torch.cuda.synchronize()
    for x, want in zip(batches, alone):
        for got, ref in zip(x.bytes(), want):
            assert np.array_equal(got, ref, equal_nan=got.dtype == np.float32)
        x.case.check()
