"""GPU parity of decode attention on modified scores (mj_decode_attn_mod)
against the float64 reference, element by element: soft cap, distance bias,
window, documents, prefix and their combinations; every row-tile shape; page
sizes, pool formats and layouts; empty and short sequences; splits; NaN codes
outside the span; the device spans; determinism, graphs and streams."""

import copy
import itertools

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


LENS = [0, 1, 2, 100, 127, 128, 129, 300, 1000]

MODS = {
    "none": {},
    "cap": dict(softcap=15.0),
    "cap_small": dict(softcap=0.7),  # most scores far beyond the cap
    "alibi": dict(alibi=True),
    "window": dict(window=150),
    "window1": dict(window=1),
    "docs": dict(docs=170),
    "prefix": dict(prefix=260),
    "window_prefix": dict(window=70, prefix=200),
    "all": dict(softcap=20.0, alibi=True, window=400, docs=300, prefix=90),
}


def check(w, kw, seed=0, **step):
    """Every kernel family that takes the shape."""
    mod, host = make_mod(w, np.random.default_rng(seed), **kw)
    ref = Reference(w, host)
    for kernel in families(w):
        ref.check(*ModStep(w, mod, kernel=kernel, **step).run())


def families(w):
    return (mj.MJ_KERNEL_TENSOR_CORE_QROWS,) + ((mj.MJ_KERNEL_AUTO,) if w.q_len * w.h_r <= 16 else ())


@pytest.mark.parametrize("kw", MODS.values(), ids=MODS.keys())
@pytest.mark.parametrize("q_len,h_r", [(1, 4), (4, 8)], ids=["rows4", "rows32"])
def test_modifiers(kw, q_len, h_r):
    w = syn.make_workload("mod", LENS, q_len, 2, h_r, 16, seed=5 + h_r, max_splits=4)
    check(w, kw)
    check(w, kw, force_splits=3)


@pytest.mark.parametrize("q_len,h_r", [(1, 1), (1, 16), (5, 9), (7, 12), (1, 128), (3, 48), (16, 16), (5, 64)],
                         ids=["r1", "r16", "r45", "r84", "r128", "r144", "r256", "r320"])
@pytest.mark.parametrize("q_is_e4m3", [False, True])
def test_row_tiles(q_len, h_r, q_is_e4m3):
    w = syn.make_workload("mod", [3, 130, 700], q_len, 2, h_r, 64, seed=q_len * h_r, q_is_e4m3=q_is_e4m3, max_splits=4)
    check(w, MODS["all"], force_splits=2)
    check(w, MODS["cap_small"])


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "interleaved", "flashinfer"])
def test_pages_and_layouts(page_size, layout):
    w = syn.make_workload("mod", [5, 640, 1411], 2, 3, 5, page_size, seed=page_size, max_splits=4)
    check(w, dict(softcap=10.0, window=333, prefix=140), kv_layout=layout)


@pytest.mark.parametrize("fmt", ["e3m2", "e2m3", "e2m1"])
def test_narrow_pools(fmt):
    w = syn.make_workload("mod", [64, 500, 901], 2, 2, 6, 32, seed=9, kv_format=fmt, max_splits=4)
    check(w, dict(softcap=8.0, alibi=True, window=300))


def test_noncausal_documents_and_prefix():
    w = syn.make_workload("mod", [7, 400, 901], 5, 2, 4, 32, seed=19, causal=False, max_splits=4)
    check(w, dict(docs=130, ends=True, alibi=True))
    check(w, dict(docs=130, ends=True, prefix=300), force_splits=3)


def test_rows_that_see_nothing():
    """A document that begins past every key, or ends before the first."""
    w = syn.make_workload("mod", [40, 300], 3, 1, 4, 16, seed=3, max_splits=2)
    begin = np.array([[0, 400, 10], [900, 900, 900]], dtype=np.int32)
    end = np.array([[0, 500, 60], [950, 950, 950]], dtype=np.int32)
    host = dict(softcap=0.0, window=0, slopes=None, begin=begin, end=end, prefix=None)
    mod = mj.ScoreMod(key_begin=torch.from_numpy(begin).cuda(), key_end=torch.from_numpy(end).cuda())
    ref = Reference(w, host)
    for spans, kernel in itertools.product((True, False), families(w)):
        st = ModStep(w, mod, spans=spans, kernel=kernel)
        o, lse = st.run()
        assert np.isneginf(lse[1]).all() and np.isneginf(lse[0, 0, :8]).all()
        ref.check(o, lse)


def test_without_spans_all_keys_are_read():
    w = syn.make_workload("mod", LENS, 2, 2, 4, 16, seed=8, max_splits=4)
    check(w, MODS["window_prefix"], spans=False, force_splits=2)


def test_nan_outside_the_span_and_in_masked_keys():
    """Keys no row sees may hold NaN in K and V, also inside a tile that is
    read, and their table entries may point anywhere; keys some row sees and
    another does not may hold NaN in K of the masked row's tile only where no
    row sees them."""
    w = copy.deepcopy(syn.make_workload("mod", [1000, 555], 2, 2, 4, 16, seed=21, max_splits=4))
    kw = dict(window=200, prefix=40)
    mod, host = make_mod(w, np.random.default_rng(1), **kw)
    ref = Reference(w, host)  # before the poison
    p = mj.make_params(2, 2, 2, 4, 16, w.max_blocks, w.num_pages, kernel=mj.MJ_KERNEL_TENSOR_CORE_QROWS)
    spans, _ = mj.score_spans(p, mod, w.seq_lens)
    w.k_cache, w.v_cache, w.block_table = w.k_cache.copy(), w.v_cache.copy(), w.block_table.copy()
    for b in range(2):
        for j in range(int(spans[b][0]), int(spans[b][1])):
            page, r = w.block_table[b, j // 16], j % 16
            w.k_cache[page, r] = 0x7F
            w.v_cache[page, r] = 0x7F
        # blocks wholly between prefix and window: entries that name no page
        for blk in range(-(-int(spans[b][0]) // 16), int(spans[b][1]) // 16):
            w.block_table[b, blk] = (-1, 2**31 - 1)[blk % 2]
    for kernel in families(w):
        ref.check(*ModStep(w, mod, kernel=kernel).run())
        ref.check(*ModStep(w, mod, force_splits=4, kernel=kernel).run())


def test_wide_window_matches_plain_decode_bits():
    """Modifiers that change nothing give the plain kernel's LSE to fp32
    rounding and its O to the bf16 step."""
    w = syn.make_workload("mod", [700, 90], 1, 2, 8, 16, seed=2, max_splits=1)
    mod, _ = make_mod(w, np.random.default_rng(0), window=10000)
    st = ModStep(w, mod, kernel=mj.MJ_KERNEL_AUTO)
    o, lse = st.run()
    st.s.decode()
    torch.cuda.synchronize()
    assert np.abs(lse - st.s.lse_host()).max() <= 2.0**-18 * (1 + np.abs(lse).max())
    o2 = st.s.o_host()
    assert (np.abs(o - o2) <= 2.0**-7 * np.abs(o2) + 2.0**-7 * np.abs(o2).max() * 0.1).all()


@pytest.mark.parametrize("q_len", [1, 5])
def test_device_spans_match_host(q_len):
    rng = np.random.default_rng(q_len)
    w = syn.make_workload("mod", LENS, q_len, 1, 2, 16, seed=1, max_splits=4)
    for kw in MODS.values():
        mod, _ = make_mod(w, rng, **kw)
        p = mj.make_params(w.num_seqs, q_len, 1, 2, 16, w.max_blocks, w.num_pages, kernel=mj.MJ_KERNEL_TENSOR_CORE_QROWS)
        want = mj.score_spans(p, mod, w.seq_lens)
        spans = torch.full((w.num_seqs, 4), -7, dtype=torch.int32, device="cuda")
        lens = torch.full((w.num_seqs,), -7, dtype=torch.int32, device="cuda")
        mj.score_spans_device(p, mod, torch.from_numpy(np.asarray(w.seq_lens)).cuda(), spans, lens)
        assert np.array_equal(spans.cpu().numpy(), want[0]) and np.array_equal(lens.cpu().numpy(), want[1])


@pytest.mark.parametrize("kernel", [mj.MJ_KERNEL_AUTO, mj.MJ_KERNEL_TENSOR_CORE_QROWS])
def test_graph_of_spans_plan_and_decode_follows_the_lengths(kernel):
    """One captured step, replayed while the lengths change."""
    w = syn.make_workload("mod", [900, 700, 64], 2, 2, 4, 16, seed=31, max_splits=8)
    mod, host = make_mod(w, np.random.default_rng(0), softcap=12.0, window=260)
    st = ModStep(w, mod, kernel=kernel)
    s = st.s
    pad = mj.decode_plan_max_items(s.params)
    work = torch.zeros(pad, 4, dtype=torch.int32, device="cuda")
    n_splits = torch.zeros(3, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    call = mj.DecodeAttnMod(
        s.params, mod, spans=st.spans, q=s.q_packed, k_cache=s.k_cache, v_cache=s.v_cache, block_table=s.block_table,
        seq_lens=s.seq_lens, work=work, n_splits=n_splits, q_descale=s.q_descale, k_descale=s.k_descale,
        v_descale=s.v_descale, o=s.o_packed, lse=s.lse, workspace=s.workspace, softmax_scale=w.softmax_scale,
        status=st.status, max_n_splits=8)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        mj.score_spans_device(s.params, mod, s.seq_lens, st.spans, lens, stream=side)
        mj.decode_plan_device(s.params, lens, work, n_splits, pad, stream=side)
        call(side)
    for new in ([900, 700, 64], [33, 700, 2], [0, 1, 500]):
        w2 = copy.copy(w)
        w2.seq_lens = np.minimum(np.asarray(new, dtype=np.int32), w.seq_lens)
        s.seq_lens.copy_(torch.from_numpy(w2.seq_lens))
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.status.item()) == 0
        Reference(w2, host).check(s.o_host(), s.lse_host())


def test_same_bytes_again_and_on_another_stream():
    w = syn.make_workload("mod", [800, 3, 401], 3, 2, 8, 32, seed=77, max_splits=4)
    mod, _ = make_mod(w, np.random.default_rng(0), **MODS["all"])
    st = ModStep(w, mod, force_splits=3)
    a = st.run()
    st.s.fill_workspace(1.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    st.call(side)
    torch.cuda.synchronize()
    assert np.array_equal(a[0], st.s.o_host()) and np.array_equal(a[1], st.s.lse_host())


def test_long_sequence_splits():
    w = syn.make_workload("mod", [20011, 600], 1, 1, 16, 128, seed=4, max_splits=32)
    check(w, dict(softcap=30.0, alibi=True))
    check(w, dict(softcap=30.0, window=9000, prefix=700))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_len,h_r", [(2, 8), (5, 8), (3, 48)], ids=["r16", "r40", "r144"])
def test_slopes_of_either_sign(q_len, h_r, causal):
    """Biases that grow with the distance, that leave a row one key, and none:
    the running maximum moves both ways along the keys."""
    w = syn.make_workload("mod", [2, 500, 1300], q_len, 1, h_r, 16, seed=41, causal=causal, max_splits=4)
    mod, host = make_mod(w, np.random.default_rng(0), softcap=30.0)
    slopes = np.resize(np.float32([-0.5, 3.0, 0.0, -0.001, 100.0]), h_r)
    host["slopes"], mod.alibi_slopes = slopes, torch.from_numpy(slopes).cuda()
    ref = Reference(w, host)
    for kernel, splits in itertools.product(families(w), (0, 3)):
        ref.check(*ModStep(w, mod, kernel=kernel, force_splits=splits).run())
