"""Refusals of the cache operators' entry points, on the host, before anything
is launched (CPU only; the pointers are aligned and never dereferenced)."""

import ctypes

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj

BAD, UNSUP, CAP = mj.MJ_ERR_INVALID_ARG, mj.MJ_ERR_UNSUPPORTED, mj.MJ_ERR_CAPACITY
PTR = iter(range(1 << 20, 1 << 60, 1 << 30))


def _ptr():
    return next(PTR)


def _set(obj, **kw):
    for k, v in kw.items():
        setattr(obj, k, v)
    return obj


# ------------------------------------------------------------------- rope


def _rope():
    p = mj.make_rope_params(2, 3, 2, 4, 16, 8, 20, rot_dim=64, n_axes=2, max_pos=100)
    a = mj.RopeArgs()
    for f in ("q", "k", "v", "positions", "cos_sin", "q_out", "k_cache", "v_cache", "block_table", "seq_lens", "k_descale", "v_descale"):
        setattr(a, f, _ptr())
    _set(a, q_tok=8 * 128, q_head=128, k_tok=2 * 128, k_head_in=128, v_tok=2 * 128, v_head_in=128, num_tokens=6, pos_axis=6,
         q_packed=1, q_out_stride=2 * 12 * 128, k_page=16 * 256, k_row=256, k_head=128, v_page=16 * 256, v_row=256, v_head=128)
    return p, a


def _rope_status(p, a):
    return mj.lib().mj_rope_append(ctypes.byref(p), ctypes.byref(a), None)


@pytest.mark.parametrize("field,value,want", [
    ("head_dim", 64, UNSUP), ("page_size", 24, UNSUP), ("rot_dim", 0, UNSUP), ("rot_dim", 24, UNSUP), ("rot_dim", 144, UNSUP),
    ("n_axes", 0, UNSUP), ("n_axes", 5, UNSUP), ("interleaved", 2, BAD), ("max_pos", 0, BAD), ("num_seqs", 0, BAD),
    ("q_len", 0, BAD), ("h_k", 0, BAD), ("h_r", -1, BAD), ("max_blocks", 0, BAD), ("num_pages", 0, BAD),
    ("max_blocks", 1 << 30, UNSUP), ("h_r", 5000, UNSUP),
])
def test_rope_params_refused(field, value, want):
    p, a = _rope()
    setattr(p, field, value)
    assert _rope_status(p, a) == want


@pytest.mark.parametrize("field", ["q", "k", "v", "positions", "cos_sin", "q_out", "k_cache", "v_cache", "block_table", "seq_lens",
                                   "k_descale", "v_descale"])
def test_rope_null_and_misaligned_refused(field):
    p, a = _rope()
    good = getattr(a, field)
    setattr(a, field, None)
    assert _rope_status(p, a) == BAD
    setattr(a, field, good + 2)
    assert _rope_status(p, a) == BAD


@pytest.mark.parametrize("field,value", [
    ("q_tok", 1028), ("q_head", -128), ("k_tok", 12), ("v_head_in", 4), ("k_page", 0), ("k_row", 100), ("v_head", -16),
    ("num_tokens", 5), ("num_tokens", -1), ("q_packed", 2), ("q_out_stride", 2 * 12 * 128 - 8), ("q_out_stride", 2 * 12 * 128 + 4),
    ("kd_seq", -1), ("kp_seq", -1), ("pos_axis", -6),
])
def test_rope_args_refused(field, value):
    p, a = _rope()
    setattr(a, field, value)
    assert _rope_status(p, a) == BAD


def test_rope_layout_and_axes_refused():
    p, a = _rope()
    axes = np.zeros(32, np.uint8)
    axes[7] = 2  # only axes 0 and 1 exist
    a.freq_axis = axes.ctypes.data
    assert _rope_status(p, a) == BAD
    axes[7] = 1
    a.pos_axis = 5  # axis 1 would overlap axis 0
    assert _rope_status(p, a) == BAD
    p, a = _rope()
    a.cu_tokens = _ptr()  # ragged tokens have no packed rows
    assert _rope_status(p, a) == BAD
    p, a = _rope()
    _set(a, q_packed=0, q_out_stride=8 * 128, q_out=a.q + 256)  # shifted over its input
    assert _rope_status(p, a) == BAD
    p, a = _rope()
    a.q_out = a.q  # packed over the token layout
    assert _rope_status(p, a) == BAD
    p, a = _rope()
    a.q_out = a.k
    assert _rope_status(p, a) == BAD
    assert mj.lib().mj_rope_append(None, ctypes.byref(a), None) == BAD
    assert mj.lib().mj_rope_append(ctypes.byref(p), None, None) == BAD
    p, a = _rope()
    a.cu_tokens, a.q_packed, a.q_out_stride, a.num_tokens = _ptr(), 0, 8 * 128, 0
    assert _rope_status(p, a) == mj.MJ_OK  # nothing to do, nothing launched
    a.q = a.k = a.v = a.positions = a.q_out = None  # an empty tensor has no address
    assert _rope_status(p, a) == mj.MJ_OK


@pytest.mark.parametrize("field", ["q_tok", "k_tok", "v_tok", "q_out_stride"])
def test_rope_offsets_past_any_memory_refused(field):
    p, a = _rope()
    _set(a, cu_tokens=_ptr(), q_packed=0, q_out_stride=8 * 128, num_tokens=1 << 30, pos_axis=1 << 30)
    setattr(a, field, (1 << 40) - 16)
    assert _rope_status(p, a) == BAD


def test_rope_in_place_refuses_k_or_v_under_the_output():
    rows = 8 + 2 + 2  # heads of one projection's token
    for name, tok, head in (("k", "k_tok", "k_head_in"), ("v", "v_tok", "v_head_in")):
        for at, step in ((0, rows * 128), (7 * 128, rows * 128), (11 * 128, rows * 128), (-128, rows * 128),
                         (8 * 128, 2 * 128), (8 * 128, rows * 256)):
            p, a = _rope()
            a.cu_tokens = _ptr()
            _set(a, q_packed=0, q_tok=rows * 128, q_out_stride=rows * 128, q_out=a.q)
            _set(a, **{name: a.q + 2 * at, tok: step})
            assert _rope_status(p, a) == BAD, (name, at, step)


# ---------------------------------------------------------- modified scores


def _attn(kernel=mj.MJ_KERNEL_TENSOR_CORE_QROWS, causal=True, kv_format=0, q_dtype=0):
    p = mj.make_params(2, 1, 1, 4, 16, 64, 1000, causal, q_dtype, 4, kernel=kernel, kv_format=kv_format)
    a = mj.DecodeArgs()
    for f in ("q", "k", "v", "block_table", "seq_lens", "work", "n_splits", "q_descale", "k_descale", "v_descale", "o", "lse"):
        setattr(a, f, _ptr())
    _set(a, q_seq_stride=4 * 128, o_seq_stride=4 * 128, k_page=16 * 128, k_row=128, k_head=128, v_page=16 * 128, v_row=128,
         v_head=128, num_work=2, softmax_scale=0.09, scale_o=1.0, workspace=_ptr(), workspace_bytes=1 << 30)
    return p, a


def _mod_status(p, m, a, spans=None):
    return mj.lib().mj_decode_attn_mod(ctypes.byref(p), ctypes.byref(m), spans, ctypes.byref(a), None)


def test_decode_attn_mod_refused():
    inf = float("inf")
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=inf), dict(softcap=1e-40), dict(softcap=1e38),
                dict(window=-1), dict(alibi_slopes=_ptr() + 2),
                dict(key_begin=_ptr() + 1), dict(key_end=_ptr() + 2), dict(prefix=_ptr() + 3)):
        p, a = _attn()
        assert _mod_status(p, _set(mj.ScoreModArgs(), **bad), a) == BAD, bad
    p, a = _attn(causal=False)
    assert _mod_status(p, _set(mj.ScoreModArgs(), window=5), a) == BAD
    p, a = _attn()
    assert _mod_status(p, mj.ScoreModArgs(), a, spans=_ptr() + 4) == BAD  # spans are 16-byte rows
    p, a = _attn(kernel=mj.MJ_KERNEL_CUDA_CORE)
    assert _mod_status(p, mj.ScoreModArgs(), a) == UNSUP
    p, a = _attn(kernel=mj.MJ_KERNEL_TENSOR_CORE_GROUPED)
    assert _mod_status(p, mj.ScoreModArgs(), a) == UNSUP
    p, a = _attn(kernel=mj.MJ_KERNEL_TENSOR_CORE)
    p.h_r = 17  # past the swap-AB instances
    assert _mod_status(p, mj.ScoreModArgs(), a) == UNSUP
    p, a = _attn(kernel=mj.MJ_KERNEL_AUTO, kv_format=mj.MJ_KV_NVFP4, q_dtype=mj.MJ_E4M3)
    assert _mod_status(p, mj.ScoreModArgs(), a) == UNSUP
    p, a = _attn()
    L = mj.lib()
    assert L.mj_decode_attn_mod(ctypes.byref(p), None, None, ctypes.byref(a), None) == BAD
    assert L.mj_decode_attn_mod(ctypes.byref(p), ctypes.byref(mj.ScoreModArgs()), None, None, None) == BAD
    for field, value, want in (("lse", None, BAD), ("num_work", 0, BAD), ("q_seq_stride", 4 * 128 - 8, BAD),
                               ("workspace_bytes", 16, CAP), ("softmax_scale", 0.0, BAD)):
        p, a = _attn()
        setattr(a, field, value)
        assert _mod_status(p, mj.ScoreModArgs(), a) == want, field


def test_score_spans_device_refused():
    L, m = mj.lib(), mj.ScoreModArgs()
    p, _ = _attn()
    f = L.mj_score_spans_device
    assert f(ctypes.byref(p), None, _ptr(), _ptr(), _ptr(), None) == BAD
    assert f(ctypes.byref(p), ctypes.byref(m), None, _ptr(), _ptr(), None) == BAD
    assert f(ctypes.byref(p), ctypes.byref(m), _ptr(), _ptr() + 8, _ptr(), None) == BAD
    assert f(ctypes.byref(p), ctypes.byref(m), _ptr(), _ptr(), _ptr() + 2, None) == BAD
    p.head_dim = 64
    assert f(ctypes.byref(p), ctypes.byref(m), _ptr(), _ptr(), _ptr(), None) == UNSUP


# -------------------------------------------------------------- key weights


def _kw_status(p, a, acc=1 << 21, seq=1024, head=1024, decay=1.0, fresh=0, mod=None):
    return mj.lib().mj_key_weights(ctypes.byref(p), None if mod is None else ctypes.byref(mod), ctypes.byref(a), acc, seq, head,
                                   decay, fresh, None)


def test_key_weights_refused():
    for kw in (dict(acc=None), dict(acc=(1 << 21) + 2), dict(seq=-1), dict(head=-4), dict(decay=-0.1), dict(decay=1.5),
               dict(decay=float("nan")), dict(fresh=-1), dict(mod=_set(mj.ScoreModArgs(), softcap=-2.0))):
        p, a = _attn()
        assert _kw_status(p, a, **kw) == BAD, kw
    for field, value in (("q", None), ("k", None), ("lse", None), ("work", None), ("work", _ptr() + 4), ("k_row", 100),
                         ("q_seq_stride", 4 * 128 - 8), ("num_work", 0), ("softmax_scale", -1.0), ("kd_seq", -1)):
        p, a = _attn()
        setattr(a, field, value)
        assert _kw_status(p, a) == BAD, field
    p, a = _attn(kernel=mj.MJ_KERNEL_AUTO, kv_format=mj.MJ_KV_NVFP4, q_dtype=mj.MJ_E4M3)
    assert _kw_status(p, a) == UNSUP
    p, a = _attn()
    assert mj.lib().mj_key_weights(ctypes.byref(p), None, None, 1 << 21, 1, 1, 1.0, 0, None) == BAD


# -------------------------------------------------------------------- evict


def _evict(budget=100, kv_format=0):
    p = mj.make_params(2, 1, 2, 1, 16, 64, 1000, kv_format=kv_format, kernel=0,
                       q_dtype=mj.MJ_E4M3 if kv_format == mj.MJ_KV_NVFP4 else 0)
    a = mj.EvictArgs()
    for f in ("k", "v", "block_table", "seq_lens", "acc", "new_lens", "workspace"):
        setattr(a, f, _ptr())
    _set(a, acc_out=a.acc, k_page=16 * 256, k_row=256, k_head=128, v_page=16 * 256, v_row=256, v_head=128, acc_seq=2048,
         acc_head=1024, budget=budget, workspace_bytes=mj.evict_workspace_bytes(p, budget))
    return p, a


def _evict_status(p, a):
    return mj.lib().mj_evict(ctypes.byref(p), ctypes.byref(a), None)


@pytest.mark.parametrize("field,value,want", [
    ("k", None, BAD), ("v", None, BAD), ("acc", None, BAD), ("acc_out", None, BAD), ("new_lens", None, BAD),
    ("block_table", None, BAD), ("seq_lens", None, BAD), ("k", (1 << 20) + 8, BAD), ("k_row", 24, BAD), ("v_page", -16, BAD),
    ("budget", 0, BAD), ("keep_first", -1, BAD), ("keep_last", 101, BAD), ("acc_seq", -1, BAD), ("workspace", None, BAD),
    ("workspace", (1 << 20) + 8, BAD), ("workspace_bytes", 8, CAP), ("key_pos", 1 << 22, BAD), ("acc", (1 << 20) + 1, BAD),
])
def test_evict_refused(field, value, want):
    p, a = _evict()
    setattr(a, field, value)
    assert _evict_status(p, a) == want


def test_evict_aliases_and_planes_refused():
    p, a = _evict()
    a.new_lens = a.seq_lens  # other heads still read the old lengths
    assert _evict_status(p, a) == BAD
    p, a = _evict()
    _set(a, key_pos=_ptr(), key_pos_out=_ptr(), next_pos=a.new_lens)
    assert _evict_status(p, a) == BAD
    p, a = _evict()
    a.acc_out = a.acc + 4  # neither acc itself nor apart from it
    assert _evict_status(p, a) == BAD
    p, a = _evict()
    key_pos = _ptr()
    _set(a, key_pos=key_pos, key_pos_out=key_pos + 64, next_pos=_ptr())
    assert _evict_status(p, a) == BAD
    p, a = _evict(kv_format=mj.MJ_KV_NVFP4)  # no scale planes given
    assert _evict_status(p, a) == BAD
    p, a = _evict()
    p.num_seqs, a.acc_seq = 1 << 22, (1 << 40) - 16  # past any memory
    a.workspace_bytes = mj.evict_workspace_bytes(p, 100)
    assert _evict_status(p, a) == BAD
    p, a = _evict()
    _set(a, keep_first=60, keep_last=41)
    assert _evict_status(p, a) == BAD
    assert mj.lib().mj_evict_workspace_bytes(ctypes.byref(p), 0) == 0
    with pytest.raises(mj.MjError):
        mj.evict_workspace_bytes(p, 0)


# --------------------------------- offsets past any memory, whatever they index


FAR = (1 << 40) - 32


@pytest.mark.parametrize("field", ["kp_seq", "kp_head", "kd_seq", "kd_head", "vd_seq", "vd_head", "k_page", "v_page", "k_head", "v_head"])
def test_rope_planes_descales_and_pools_past_any_memory_refused(field):
    p, a = _rope()
    p.num_seqs, p.h_k, p.h_r, p.num_pages = 1 << 20, 1024, 1, 1 << 20
    _set(a, cu_tokens=_ptr(), q_packed=0, q_tok=1024 * 128, q_out_stride=1024 * 128, key_pos=_ptr())
    setattr(a, field, FAR)
    assert _rope_status(p, a) == BAD


@pytest.mark.parametrize("field", ["k_page", "v_page", "k_head", "v_head", "ks_page", "vs_page", "ks_head", "vs_head"])
def test_evict_pools_past_any_memory_refused(field):
    p, a = _evict(kv_format=mj.MJ_KV_NVFP4)
    p.h_k, p.num_pages = 1024, 1 << 20
    _set(a, k_scales=_ptr(), v_scales=_ptr(), ks_page=128 * 1024, ks_head=128, vs_page=128 * 1024, vs_head=128, acc_seq=1 << 20,
         acc_out=a.acc, workspace_bytes=mj.evict_workspace_bytes(p, 100))
    assert _evict_status(p, a) != BAD
    setattr(a, field, FAR)
    assert _evict_status(p, a) == BAD


@pytest.mark.parametrize("field", ["qd_seq", "kd_seq", "q_seq_stride"])
def test_key_weights_descales_and_rows_past_any_memory_refused(field):
    p, a = _attn()
    p.num_seqs = 1 << 20
    setattr(a, field, FAR)
    assert _kw_status(p, a) == BAD


# ------------------------------------------------- planes of slots that coincide


@pytest.mark.parametrize("seq,head,apart", [
    (2048, 1024, True), (1024, 2048, True), (1024 + 1024, 1500, False), (1024, 1024, False), (1500, 1024, False),
    (1024, 1500, False), (2524, 1500, True), (1024, 2047, False),
])
def test_planes_of_two_heads_that_share_slots_refused(seq, head, apart):
    """Two sequences, two heads, 1024 slots: each plane's slots are its own."""
    p, a = _attn()
    p.h_k, a.q_seq_stride = 2, 2 * 4 * 128
    assert (_kw_status(p, a, seq=seq, head=head) != BAD) == apart
    p, a = _evict()
    _set(a, acc_seq=seq, acc_head=head)
    assert (_evict_status(p, a) != BAD) == apart


# ---------------------------------------------------------- binding's checks


def test_binding_refuses_host_tensors():
    """Every tensor has to be on the current CUDA device."""
    p = mj.make_params(1, 1, 1, 4, 16, 4, 8, kernel=mj.MJ_KERNEL_TENSOR_CORE_QROWS)
    t = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16)
    pool = torch.zeros(8, 16, 1, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        mj.KeyWeights(p, None, q=t, k_cache=pool, block_table=torch.zeros(1, 4, dtype=torch.int32),
                      seq_lens=torch.zeros(1, dtype=torch.int32), work=torch.zeros(1, 4, dtype=torch.int32),
                      q_descale=torch.ones(1), k_descale=torch.ones(1), lse=torch.zeros(1, 1, 4), acc=torch.zeros(1, 1, 64),
                      softmax_scale=0.1)
    with pytest.raises(TypeError):
        mj.Evict(p, k_cache=np.zeros(4), v_cache=pool, block_table=None, seq_lens=None, acc=None, new_lens=None, budget=1,
                 workspace=None)
