"""GPU parity of the accumulated key weights (mj_key_weights) against the
float64 reference: rows from 1 to 600 (one to three launches), modifiers,
pool formats, decay and fresh keys, slots that are left alone, rows without
keys, determinism, graphs."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from paged_fp8_kv_gb300 import synthetic as syn
from tests.cache_helpers import ModStep, Reference, make_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


LENS = [0, 1, 100, 127, 128, 129, 300, 1000]


class Weights:
    def __init__(self, w, kw, decay=1.0, fresh=0, force_splits=0, kv_layout="nhd", seed=0, with_mod=True):
        rng = np.random.default_rng(seed)
        mod, host = make_mod(w, rng, **kw)
        self.ref = Reference(w, host)
        st = ModStep(w, mod, spans=False, force_splits=force_splits, kv_layout=kv_layout)
        s = self.s = st.s
        slots = w.max_blocks * w.page_size
        self.old = rng.random((w.num_seqs, w.h_k, slots)).astype(np.float32)
        self.acc = torch.from_numpy(self.old.copy()).cuda()
        self.lse = torch.from_numpy(self.ref.lse.astype(np.float32)).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.w, self.decay, self.fresh = w, decay, fresh
        self.call = mj.KeyWeights(s.params, mod if with_mod else None, q=s.q_packed, k_cache=s.k_cache, block_table=s.block_table,
                                  seq_lens=s.seq_lens, work=s.work, q_descale=s.q_descale, k_descale=s.k_descale, lse=self.lse,
                                  acc=self.acc, softmax_scale=w.softmax_scale, decay=decay, fresh=fresh, status=self.status)

    def check(self):
        self.call()
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        got = self.acc.cpu().numpy()
        for (b, g), want in self.ref.keys.items():
            L = len(want)
            old = self.decay * self.old[b, g, :L].astype(np.float64)
            old[max(0, L - self.fresh) :] = 0.0
            bound = self.ref.d_keys[b, g] + 2.0**-23 * (old + want) + 2.0**-126
            err = np.abs(got[b, g, :L] - (old + want))
            assert (err <= bound).all(), (b, g, int(np.argmax(err - bound)), err.max())
            assert np.array_equal(got[b, g, L:], self.old[b, g, L:])
        return got


@pytest.mark.parametrize("q_len,h_r", [(1, 1), (1, 4), (4, 8), (5, 9), (1, 128), (3, 48), (16, 16), (5, 64), (12, 50)],
                         ids=["r1", "r4", "r32", "r45", "r128", "r144", "r256", "r320", "r600"])
@pytest.mark.parametrize("q_is_e4m3", [False, True])
def test_rows(q_len, h_r, q_is_e4m3):
    w = syn.make_workload("kw", [2, 130, 517], q_len, 2, h_r, 32, seed=q_len + h_r, q_is_e4m3=q_is_e4m3, max_splits=4)
    Weights(w, {}, with_mod=False, force_splits=2).check()


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("decay,fresh", [(1.0, 0), (1.0, 3), (0.5, 3), (0.0, 0), (0.9, 5000)])
def test_lengths_decay_and_fresh(page_size, decay, fresh):
    w = syn.make_workload("kw", LENS, 3, 2, 4, page_size, seed=page_size, max_splits=4)
    Weights(w, {}, decay, fresh, with_mod=False).check()


@pytest.mark.parametrize("kw", [dict(softcap=9.0), dict(softcap=0.5), dict(alibi=True), dict(window=150), dict(window=60, prefix=300),
                                dict(docs=200, ends=True), dict(softcap=20.0, alibi=True, window=400, docs=300, prefix=90)],
                         ids=["cap", "cap_small", "alibi", "window", "window_prefix", "docs", "all"])
def test_modifiers(kw):
    w = syn.make_workload("kw", LENS, 3, 2, 4, 16, seed=11, max_splits=4)
    Weights(w, kw, 0.75, 3, force_splits=3).check()


@pytest.mark.parametrize("fmt", ["e3m2", "e2m3", "e2m1"])
def test_narrow_pools(fmt):
    w = syn.make_workload("kw", [64, 500, 901], 2, 2, 6, 32, seed=9, kv_format=fmt, max_splits=4)
    Weights(w, dict(softcap=8.0)).check()


@pytest.mark.parametrize("layout", ["hnd", "interleaved", "flashinfer"])
def test_layouts(layout):
    w = syn.make_workload("kw", [33, 700], 2, 3, 5, 64, seed=6, max_splits=4)
    Weights(w, {}, kv_layout=layout, with_mod=False).check()


def test_decay_zero_and_fresh_do_not_read_what_was_there():
    w = syn.make_workload("kw", [300, 40], 2, 2, 4, 16, seed=14, max_splits=2)
    for decay, fresh in ((0.0, 0), (1.0, 300)):
        x = Weights(w, {}, decay, fresh, with_mod=False)
        x.acc.fill_(float("nan"))
        x.old[:] = 0
        x.call()
        torch.cuda.synchronize()
        got = x.acc.cpu().numpy()
        for (b, g), want in x.ref.keys.items():
            assert not np.isnan(got[b, g, : len(want)]).any()
            assert np.isnan(got[b, g, len(want) :]).all()


def test_weights_of_a_step_sum_to_its_rows():
    """Rows that see keys give one each (from the decode's own LSE)."""
    w = syn.make_workload("kw", [1500, 2, 129], 4, 2, 8, 16, seed=15, max_splits=4)
    mod, _ = make_mod(w, np.random.default_rng(0), softcap=25.0)
    st = ModStep(w, mod)
    st.run()
    s = st.s
    acc = torch.full((3, 2, w.max_blocks * 16), float("nan"), device="cuda")
    s.replan(w.seq_lens)
    mj.key_weights(s.params, mod, q=s.q_packed, k_cache=s.k_cache, block_table=s.block_table, seq_lens=s.seq_lens, work=s.work,
                   q_descale=s.q_descale, k_descale=s.k_descale, lse=s.lse, acc=acc, softmax_scale=w.softmax_scale, decay=0.0)
    got = acc.cpu().numpy()
    for b, L in enumerate(w.seq_lens):
        rows = sum(1 for i in range(4) if L - 4 + i >= 0) * 8
        # the LSE's and the logits' fp32 errors, 2^-17 of a weight at most here
        assert np.allclose(got[b, :, :L].sum(-1, dtype=np.float64), rows, rtol=2.0**-14)


def test_same_bytes_in_a_graph():
    w = syn.make_workload("kw", [1500, 2, 129], 4, 2, 8, 16, seed=15, max_splits=4)
    x = Weights(w, dict(softcap=25.0), 0.5, 4)
    one = x.check()
    x.acc.copy_(torch.from_numpy(x.old))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        x.call(side)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(one, x.acc.cpu().numpy())


def test_a_plan_of_the_spans_or_of_shorter_lengths_is_reported():
    """It leaves tiles out; one made for longer lengths does not."""
    w = syn.make_workload("kw", [1500, 2, 0, 129], 2, 2, 4, 16, seed=23, max_splits=4)
    mod, _ = make_mod(w, np.random.default_rng(0), window=100)
    x = Weights(w, dict(window=100), 0.5, 2)
    x.check()
    s, lens = x.s, np.asarray(w.seq_lens)
    longer = np.minimum(lens + [0, 0, 40, 500], w.max_blocks * 16)
    for plan_lens, want in ((mj.score_spans(s.params, mod, lens)[1], mj.MJ_ERR_INVALID_ARG), (lens - [129, 0, 0, 0], mj.MJ_ERR_INVALID_ARG),
                            (lens - [0, 0, 0, 1], mj.MJ_ERR_INVALID_ARG), (longer, 0), (lens, 0)):
        work = torch.from_numpy(mj.decode_plan(s.params, plan_lens).work).cuda()
        x.status.zero_()
        mj.key_weights(s.params, mod, q=s.q_packed, k_cache=s.k_cache, block_table=s.block_table, seq_lens=s.seq_lens, work=work,
                       q_descale=s.q_descale, k_descale=s.k_descale, lse=x.lse, acc=x.acc, softmax_scale=w.softmax_scale, decay=0.5,
                       fresh=2, status=x.status)
        torch.cuda.synchronize()
        assert int(x.status.item()) == want, plan_lens
