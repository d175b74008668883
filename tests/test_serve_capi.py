"""Refusals of the serving operators' entry points, on the host, before anything
is launched (CPU only; the pointers are aligned and never dereferenced)."""

import ctypes

import pytest

import paged_fp8_kv_gb300 as mj

BAD, UNSUP, CAP = mj.MJ_ERR_INVALID_ARG, mj.MJ_ERR_UNSUPPORTED, mj.MJ_ERR_CAPACITY
PTR = iter(range(1 << 20, 1 << 60, 1 << 32))


def _ptr():
    return next(PTR)


def _set(obj, **kw):
    for k, v in kw.items():
        setattr(obj, k, v)
    return obj


def _refused(call, obj, field, value, want):
    good = getattr(obj, field)
    setattr(obj, field, value)
    assert call() == want, (field, value)
    setattr(obj, field, good)


# ------------------------------------------------------------------ pages


def _reserve():
    p = mj.make_page_params(3, 16, 8, 40)
    a = mj.ReserveArgs()
    for f in ("seq_lens", "new_tokens", "free_pages", "num_free", "num_free_out", "block_table", "seq_lens_out", "cu_tokens",
              "positions", "slots", "status"):
        setattr(a, f, _ptr())
    a.num_tokens = 5
    return p, a, lambda: mj.lib().mj_pages_reserve(ctypes.byref(p), ctypes.byref(a), None)


def _release():
    p = mj.make_page_params(3, 16, 8, 40)
    a = mj.ReleaseArgs()
    for f in ("seq_lens", "keep_lens", "free_pages", "num_free", "num_free_out", "block_table", "status"):
        setattr(a, f, _ptr())
    return p, a, lambda: mj.lib().mj_pages_release(ctypes.byref(p), ctypes.byref(a), None)


@pytest.mark.parametrize("make", [_reserve, _release])
def test_page_params_refused(make):
    p, a, call = make()
    for field, value, want in [("num_seqs", 0, BAD), ("max_blocks", 0, BAD), ("num_pages", 0, BAD), ("page_size", 24, UNSUP),
                               ("page_size", 256, UNSUP), ("num_seqs", 16385, UNSUP), ("max_blocks", (1 << 26) + 1, UNSUP),
                               ("num_pages", (1 << 30) + 1, UNSUP)]:
        _refused(call, p, field, value, want)


@pytest.mark.parametrize("make,needed", [
    (_reserve, ("seq_lens", "free_pages", "num_free", "num_free_out", "block_table", "seq_lens_out")),
    (_release, ("seq_lens", "keep_lens", "free_pages", "num_free", "num_free_out", "block_table")),
])
def test_page_pointers_refused(make, needed):
    p, a, call = make()
    for f in needed:
        _refused(call, a, f, None, BAD)
    for f, t in a._fields_:
        if t is ctypes.c_void_p and f not in needed + ("status",) or f in needed:
            _refused(call, a, f, getattr(a, f) + 2, BAD)


def test_reserve_counts_and_overlaps_refused():
    p, a, call = _reserve()
    a.new_tokens = None
    for q_len in (0, -1):
        _refused(call, a, "q_len", q_len, BAD)
    a.q_len = 1
    _refused(call, a, "num_tokens", -1, BAD)
    _refused(call, a, "num_tokens", (1 << 30) + 1, UNSUP)
    _refused(call, a, "slots", a.slots + 4, BAD)  # 64-bit entries
    for out in ("seq_lens_out", "block_table", "positions", "cu_tokens"):
        _refused(call, a, out, a.free_pages + 4, BAD)
    _refused(call, a, "seq_lens_out", a.seq_lens + 4, BAD)  # itself is fine, a shifted one is not
    _refused(call, a, "cu_tokens", a.seq_lens, BAD)
    _refused(call, a, "positions", a.slots, BAD)
    _refused(call, a, "num_free_out", a.block_table + 8, BAD)


def test_release_overlaps_refused():
    p, a, call = _release()
    for f in ("seq_lens", "keep_lens", "block_table", "num_free", "num_free_out"):
        _refused(call, a, f, a.free_pages + 16, BAD)
    _refused(call, a, "num_free_out", a.keep_lens + 4, BAD)


# ----------------------------------------------------------------- prompts


def _prompt():
    p = mj.make_params(3, 1, 2, 4, 16, 8, 20, max_splits=8)
    a = mj.PromptArgs()
    for f in ("q", "o", "lse", "k", "v", "block_table", "plan", "q_descale", "k_descale", "v_descale", "workspace", "status"):
        setattr(a, f, _ptr())
    _set(a, q_tok=12 * 128, q_head=128, o_tok=8 * 128, num_tokens=30, k_page=16 * 256, k_row=256, k_head=128, v_page=16 * 256,
         v_row=256, v_head=128, plan_bytes=1 << 20, softmax_scale=0.1, scale_o=1.0, workspace_bytes=1 << 40)
    return p, a, lambda: mj.lib().mj_prompt_attn(ctypes.byref(p), ctypes.byref(a), None)


def test_prompt_sizes():
    p, _, _ = _prompt()
    size = mj.lib().mj_prompt_plan_bytes
    assert size(ctypes.byref(p), 0) > 0 and size(ctypes.byref(p), 100_000) > size(ctypes.byref(p), 10)
    assert size(ctypes.byref(p), -1) == 0 and size(ctypes.byref(p), 1 << 28) == 0  # over 2^30 rows
    ws = mj.lib().mj_prompt_workspace_bytes
    assert ws(ctypes.byref(p)) > 0
    p.max_splits = 1
    assert ws(ctypes.byref(p)) == 0
    p.q_len, p.kernel, p.l2_prefetch = 0, 77, -9  # not looked at
    assert size(ctypes.byref(p), 5) > 0


@pytest.mark.parametrize("field,value,want", [
    ("num_seqs", 0, BAD), ("h_k", 0, BAD), ("h_r", 0, BAD), ("max_blocks", 0, BAD), ("num_pages", 0, BAD), ("causal", 2, BAD),
    ("max_splits", 0, BAD), ("max_splits", 257, BAD), ("head_dim", 64, UNSUP), ("page_size", 8, UNSUP), ("q_dtype", 2, UNSUP),
    ("kv_format", mj.MJ_KV_E2M1, UNSUP), ("kv_format", 9, BAD), ("num_seqs", 16385, UNSUP), ("h_r", 4000, UNSUP),
])
def test_prompt_params_refused(field, value, want):
    p, a, call = _prompt()
    _refused(call, p, field, value, want)
    plan = lambda: mj.lib().mj_prompt_plan(ctypes.byref(p), _ptr(), _ptr(), 30, 0, _ptr(), 1 << 20, None, None)  # noqa: E731
    _refused(plan, p, field, value, want)


def test_prompt_plan_refused():
    p, _, _ = _prompt()
    good = [_ptr(), _ptr(), 30, 0, _ptr(), 1 << 20, _ptr()]

    def call(i, value):
        x = list(good)
        x[i] = value
        return mj.lib().mj_prompt_plan(ctypes.byref(p), *x, None)

    for i in (0, 1, 4):
        assert call(i, None) == BAD
    for i, off in ((0, 2), (1, 2), (4, 8), (6, 1)):
        assert call(i, good[i] + off) == BAD
    assert call(2, -1) == BAD and call(3, -1) == BAD
    assert call(5, 64) == CAP
    p.causal = 0
    assert call(3, 5) == BAD  # a window is causal


@pytest.mark.parametrize("field", ["q", "o", "k", "v", "block_table", "plan", "q_descale", "k_descale", "v_descale", "workspace"])
def test_prompt_null_and_misaligned_refused(field):
    p, a, call = _prompt()
    _refused(call, a, field, None, BAD)
    _refused(call, a, field, getattr(a, field) + 2, BAD)


@pytest.mark.parametrize("field,value,want", [
    ("num_tokens", -1, BAD), ("q_tok", -8, BAD), ("q_tok", 12, BAD), ("q_head", 4, BAD), ("q_tok", 1 << 40, BAD),
    ("o_tok", 8 * 128 - 8, BAD), ("o_tok", 8 * 128 + 4, BAD), ("o_tok", 1 << 40, BAD), ("k_row", 8, BAD), ("k_page", -16, BAD),
    ("v_head", 1 << 44, BAD), ("qd_seq", -1, BAD), ("kd_head", -1, BAD), ("vd_seq", 1 << 43, BAD),
    ("softmax_scale", 0.0, BAD), ("softmax_scale", float("nan"), BAD), ("scale_o", float("nan"), BAD), ("softcap", -1.0, BAD),
    ("softcap", 2.0**-21, BAD), ("softcap", 2.0**61, BAD), ("softcap", float("nan"), BAD), ("window", -1, BAD),
    ("plan_bytes", 10, CAP), ("workspace_bytes", 10, CAP),
])
def test_prompt_args_refused(field, value, want):
    p, a, call = _prompt()
    _refused(call, a, field, value, want)


def test_prompt_overlaps_refused():
    p, a, call = _prompt()
    _refused(call, a, "o", a.q, BAD)
    _refused(call, a, "o", a.q + 16, BAD)
    _refused(call, a, "lse", a.o + 16, BAD)
    _refused(call, a, "lse", a.q + 4, BAD)
    p.causal = 0
    _refused(call, a, "window", 4, BAD)


# ------------------------------------------------------------------- trees


def _tree():
    p = mj.make_params(2, 20, 2, 4, 16, 8, 20, max_splits=4)
    a = mj.DecodeArgs()
    for f in ("q", "k", "v", "block_table", "seq_lens", "work", "n_splits", "q_descale", "k_descale", "v_descale", "o", "lse",
              "workspace"):
        setattr(a, f, _ptr())
    rows = 2 * 80 * 128
    _set(a, q_seq_stride=rows, o_seq_stride=rows, num_work=2, k_page=16 * 256, k_row=256, k_head=128, v_page=16 * 256, v_row=256,
         v_head=128, softmax_scale=0.1, scale_o=1.0, workspace_bytes=1 << 40)
    t = mj.TreeArgs(_ptr(), 1, _ptr())
    m = mj.ScoreModArgs()
    return p, a, t, m, lambda: mj.lib().mj_decode_attn_tree(ctypes.byref(p), ctypes.byref(t), ctypes.byref(m), None, ctypes.byref(a), None)


def test_tree_refused():
    p, a, t, m, call = _tree()
    _refused(call, t, "mask", None, BAD)
    _refused(call, t, "mask", t.mask + 2, BAD)
    _refused(call, t, "tree_lens", t.tree_lens + 1, BAD)
    _refused(call, t, "mask_words", 0, BAD)
    p.q_len = 33
    assert call() == BAD  # two words a row
    p.q_len = 20
    for field, value in [("window", 5), ("alibi_slopes", _ptr()), ("key_end", _ptr())]:
        _refused(call, m, field, value, UNSUP)
    _refused(call, m, "softcap", -1.0, BAD)
    _refused(call, m, "key_begin", _ptr() + 2, BAD)
    for kernel in (mj.MJ_KERNEL_CUDA_CORE, mj.MJ_KERNEL_TENSOR_CORE_GROUPED, mj.MJ_KERNEL_TENSOR_CORE):  # 80 rows
        _refused(call, p, "kernel", kernel, UNSUP)
    _refused(call, a, "q", None, BAD)
    _refused(call, a, "workspace_bytes", 16, CAP)
    assert mj.lib().mj_decode_attn_tree(ctypes.byref(p), None, None, None, ctypes.byref(a), None) == BAD


def _commit():
    p = mj.make_params(2, 20, 2, 4, 16, 8, 20)
    a = mj.CommitArgs()
    for f in ("k", "v", "block_table", "seq_lens", "tree_lens", "accepted", "num_accepted", "new_lens", "key_pos", "status"):
        setattr(a, f, _ptr())
    _set(a, max_accept=5, k_page=16 * 256, k_row=256, k_head=128, v_page=16 * 256, v_row=256, v_head=128, kp_seq=256, kp_head=128)
    return p, a, lambda: mj.lib().mj_tree_commit(ctypes.byref(p), ctypes.byref(a), None)


def test_commit_refused():
    p, a, call = _commit()
    for f in ("k", "v", "block_table", "seq_lens", "accepted", "num_accepted", "new_lens"):
        _refused(call, a, f, None, BAD)
    for f in ("k", "block_table", "seq_lens", "tree_lens", "accepted", "num_accepted", "new_lens", "key_pos", "status"):
        _refused(call, a, f, getattr(a, f) + 2, BAD)
    for field, value, want in [("max_accept", 0, BAD), ("k_row", 24, BAD), ("v_page", 1 << 44, BAD), ("kp_seq", 200, BAD),
                               ("kp_head", 100, BAD), ("kp_head", -1, BAD), ("kp_seq", 1 << 41, BAD)]:
        _refused(call, a, field, value, want)
    _refused(call, a, "new_lens", a.seq_lens + 4, BAD)
    _refused(call, a, "new_lens", a.num_accepted, BAD)
    _refused(call, a, "new_lens", a.accepted + 8, BAD)
    _refused(call, a, "new_lens", a.block_table + 8, BAD)
    for field, value, want in [("num_seqs", 0, BAD), ("q_len", 0, BAD), ("h_k", 0, BAD), ("page_size", 48, UNSUP),
                               ("head_dim", 96, UNSUP), ("kv_format", 7, BAD)]:
        _refused(call, p, field, value, want)
    p.kv_format = mj.MJ_KV_NVFP4  # without its scale planes
    assert call() == BAD
