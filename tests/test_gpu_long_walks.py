"""GPU: the cache operators' kernels in steady state, against the float64
reference.  Key-weights CTAs that walk many tiles over many segments (the K
ring, the S buffers, the segments' Q and row buffers and the block-table
window all come round again, with segments that no row sees between others),
and modified attention on items of up to 47 tiles in one CTA, with the jump
over unseen tiles inside an item.  Bounds as in tests.cache_helpers."""

import copy

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import cache_ref
from paged_fp8_kv_gb300 import synthetic as syn
from tests.cache_helpers import ModStep, Reference, make_mod, q_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ------------------------------------------------------------- key weights

H_K, HEADS = 38, (0, 17, 37)  # the heads' CTAs walk alike: the reference takes three
RING = 8  # K stages of a CTA, at most


def some_heads(w, heads):
    """The workload of these kv heads alone."""
    x = copy.copy(w)
    h = list(heads)
    x.h_k = len(h)
    x.k_cache, x.v_cache = w.k_cache[:, :, h], w.v_cache[:, :, h]
    x.q = w.q.reshape(-1, w.h_k, w.h_r, 128)[:, h].reshape(-1, len(h) * w.h_r, 128)
    for name in ("q_descale", "k_descale", "v_descale"):
        setattr(x, name, getattr(w, name)[:, h])
    return x


def middle_cap(w):
    """A cap that about half of the (32 keys, all rows) score blocks pass the
    polynomial's range of: a warp then changes forms along its tiles."""
    x, q, tops = some_heads(w, HEADS), None, []
    q = q_rows(x)
    kv = cache_ref.values_of(x.k_cache)
    for b, L in enumerate(x.seq_lens):
        for g in range(x.h_k):
            k = cache_ref.cache_rows(kv, x.block_table[b], int(L), x.page_size, g)
            z = np.abs(q[b, g] @ k.T).max(0) * (w.softmax_scale * float(x.q_descale[b, g]) * float(x.k_descale[b, g]))
            tops += [z[j : j + 32].max() for j in range(0, int(L), 32)]
    cap = float(np.float32(np.median(tops) / 0.6))
    passed = np.mean(np.asarray(tops) > 0.6 * cap)
    assert 0.3 < passed < 0.7
    return cap


@pytest.mark.parametrize("kind", ["plain", "gaps", "cap", "all"])
@pytest.mark.parametrize("q_len,h_r", [(1, 4), (2, 8), (4, 8), (8, 8), (16, 8), (16, 16)],
                         ids=["r4", "r16", "r32", "r64", "r128", "r256"])
@pytest.mark.parametrize("q_is_e4m3", [False, True], ids=["bf16", "e4m3"])
def test_key_weights_over_many_segments(q_is_e4m3, q_len, h_r, kind):
    rng = np.random.default_rng(7)
    lens = np.concatenate([rng.integers(1, 1500, 22), [0, 1, 128, 5000]])
    w = syn.make_workload("walk", lens.tolist(), q_len, H_K, h_r, 16, seed=q_len * h_r, q_is_e4m3=q_is_e4m3, max_splits=3)
    b = w.num_seqs
    kw = {"plain": {}, "gaps": dict(window=150, prefix=200), "cap": dict(softcap=middle_cap(w)),
          "all": dict(softcap=middle_cap(w), alibi=True, window=400, prefix=100)}[kind]
    mod, host = make_mod(w, rng, **kw)
    if kind in ("gaps", "all"):  # every third sequence's rows see no key but a prefix, which every sixth has not
        begin = np.zeros((b, q_len), dtype=np.int32)
        begin[1::3] = 1 << 20
        host["prefix"][1::6] = 0
        host["begin"], mod.key_begin = begin, torch.from_numpy(begin).cuda()
        mod.prefix = torch.from_numpy(host["prefix"]).cuda()
    part = dict(host, slopes=None if host["slopes"] is None else host["slopes"].reshape(H_K, h_r)[list(HEADS)].reshape(-1))
    ref = Reference(some_heads(w, HEADS), part)
    s = ModStep(w, mod, spans=False).s
    # tiles and segments a CTA (an item costs three tiles besides its own)
    rows, sms = q_len * h_r, torch.cuda.get_device_properties(0).multi_processor_count
    shares = sms * (2 if rows <= 64 else 1) // H_K
    launches = -(-rows // (256 if q_is_e4m3 else 128))
    work = s.plan.work.reshape(-1, 4)
    assert (work[:, 2] - work[:, 1]).sum() >= 2 * RING * shares and len(work) >= 3 * shares
    slots = w.max_blocks * w.page_size
    old = rng.random((b, H_K, slots)).astype(np.float32)
    acc = torch.from_numpy(old.copy()).cuda()
    full = torch.full((b, H_K, rows), float("nan"), device="cuda")
    full[:, list(HEADS)] = torch.from_numpy(ref.lse.astype(np.float32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mj.key_weights(s.params, None if kind == "plain" else mod, q=s.q_packed, k_cache=s.k_cache, block_table=s.block_table,
                   seq_lens=s.seq_lens, work=s.work, q_descale=s.q_descale, k_descale=s.k_descale, lse=full, acc=acc,
                   softmax_scale=w.softmax_scale, decay=0.75, fresh=q_len, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = acc.cpu().numpy()
    for (i, g), want in ref.keys.items():
        L, head = len(want), HEADS[g]
        kept = 0.75 * old[i, head, :L].astype(np.float64)
        kept[max(0, L - q_len) :] = 0.0
        # decay times the old value is rounded once, then every launch's sum
        # with what it finds, each by half a step of a value up to the result
        bound = ref.d_keys[i, g] + (1 + launches) * 2.0**-24 * (kept + want) + 2.0**-126
        err = np.abs(got[i, head, :L] - (kept + want))
        assert (err <= bound).all(), (i, head, np.argwhere(err > bound)[:4].tolist(), err.max())
    for i, L in enumerate(w.seq_lens):
        assert np.array_equal(got[i, :, L:], old[i, :, L:])


# ------------------------------------------------------- modified attention


@pytest.mark.parametrize("kind", ["jump", "whole", "cap"])
@pytest.mark.parametrize("page_size", [16, 128])
@pytest.mark.parametrize("q_len,h_r", [(1, 4), (2, 8), (4, 8), (8, 8), (16, 8), (16, 16), (20, 16)],
                         ids=["r4", "r16", "r32", "r64", "r128", "r256", "r320"])
@pytest.mark.parametrize("q_is_e4m3", [False, True], ids=["bf16", "e4m3"])
def test_attention_over_long_items(q_is_e4m3, q_len, h_r, page_size, kind):
    w = syn.make_workload("long", [6001, 3300, 517], q_len, 1, h_r, page_size, seed=q_len * h_r, q_is_e4m3=q_is_e4m3, max_splits=1)
    kw = {"jump": dict(window=2600, prefix=900), "whole": {}, "cap": dict(softcap=4.0, window=5000, prefix=700)}[kind]
    mod, host = make_mod(w, np.random.default_rng(3), **kw)
    # biases that fall and that grow with the distance: the maxima move along all of an item
    slopes = np.resize(np.float32([0.004, -0.002, 0.0, 0.05, -0.03]), h_r)
    host["slopes"], mod.alibi_slopes = slopes, torch.from_numpy(slopes).cuda()
    if host["prefix"] is not None:
        host["prefix"][0] = kw["prefix"]
        mod.prefix = torch.from_numpy(host["prefix"]).cuda()
    ref = Reference(w, host)
    for kernel in (mj.MJ_KERNEL_TENSOR_CORE_QROWS,) + ((mj.MJ_KERNEL_AUTO,) if q_len * h_r <= 16 else ()):
        for spans in (True, False):
            st = ModStep(w, mod, kernel=kernel, spans=spans)
            work = st.s.plan.work.reshape(-1, 4)
            assert len(work) == 3 and (work[:, 2] - work[:, 1]).max() >= 26
            ref.check(*st.run())
