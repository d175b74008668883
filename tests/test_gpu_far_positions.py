"""GPU: the distance bias at positions past 2^24, where neighbouring integers
share an fp32 value.  Under a window the logits depend on distances alone, so
a sequence moved by a whole number of tiles gives the same attention, bit for
bit, as the short one it was made from, which is compared with the float64
reference.  The blocks ahead of the tail share one page."""

import copy

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from paged_fp8_kv_gb300 import synthetic as syn
from tests.cache_helpers import ModStep, Reference, make_mod

pytestmark = pytest.mark.gpu

SHIFT = (1 << 25) + 128 * 3  # neighbouring fp32 values here are 4 apart


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def moved(w):
    """The same last keys, SHIFT positions further on."""
    far = copy.copy(w)
    far.seq_lens = (np.asarray(w.seq_lens) + SHIFT).astype(np.int32)
    ahead = np.repeat(w.block_table[:, :1], SHIFT // w.page_size, axis=1)
    far.block_table = np.ascontiguousarray(np.concatenate([ahead, w.block_table], axis=1))
    return far


def problem(q_len, h_r, softcap):
    w = syn.make_workload("far", [901], q_len, 1, h_r, 128, seed=q_len + h_r, max_splits=1)
    mod, host = make_mod(w, np.random.default_rng(0), softcap=softcap, window=333)
    slopes = np.resize(np.float32([0.5, -0.02, 2.0, 0.0]), h_r)
    host["slopes"], mod.alibi_slopes = slopes, torch.from_numpy(slopes).cuda()
    return w, mod, host


@pytest.mark.parametrize("softcap", [0.0, 9.0])
@pytest.mark.parametrize("q_len,h_r", [(1, 4), (3, 5), (4, 8), (7, 8), (7, 16), (9, 16)],
                         ids=["r4", "r15", "r32", "r56", "r112", "r144"])
def test_attention(q_len, h_r, softcap):
    w, mod, host = problem(q_len, h_r, softcap)
    ref = Reference(w, host)
    for kernel in (mj.MJ_KERNEL_TENSOR_CORE_QROWS,) + ((mj.MJ_KERNEL_AUTO,) if q_len * h_r <= 16 else ()):
        near = ModStep(w, mod, kernel=kernel).run()
        far = ModStep(moved(w), mod, kernel=kernel).run()
        ref.check(*near)
        ref.check(*far)
        assert np.array_equal(near[0], far[0]) and np.array_equal(near[1], far[1])


@pytest.mark.parametrize("softcap", [0.0, 9.0])
@pytest.mark.parametrize("q_len,h_r", [(1, 4), (4, 8), (9, 16)], ids=["r4", "r32", "r144"])
def test_key_weights(q_len, h_r, softcap):
    w, mod, host = problem(q_len, h_r, softcap)
    ref = Reference(w, host)
    lse = torch.from_numpy(ref.lse.astype(np.float32)).cuda()
    got = []
    for x in (w, moved(w)):
        s = ModStep(x, mod, spans=False).s
        acc = torch.ones(1, 1, x.max_blocks * x.page_size, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mj.key_weights(s.params, mod, q=s.q_packed, k_cache=s.k_cache, block_table=s.block_table, seq_lens=s.seq_lens, work=s.work,
                       q_descale=s.q_descale, k_descale=s.k_descale, lse=lse, acc=acc, softmax_scale=w.softmax_scale, decay=0.5,
                       status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        L = int(x.seq_lens[0])
        assert bool((acc[0, 0, : L - 901] == 0.5).all()) and bool((acc[0, 0, L:] == 1.0).all())
        got.append(acc[0, 0, L - 901 : L].cpu().numpy())
    want = 0.5 + ref.keys[0, 0]
    bound = ref.d_keys[0, 0] + 2.0**-23 * want
    for x in got:
        assert (np.abs(x - want) <= bound).all(), np.abs(x - want).max()
    assert np.array_equal(got[0], got[1])
