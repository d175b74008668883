"""Paged fp8-KV split-KV decode attention for GB300 (sm_103a).

A thin ctypes binding over the C ABI of ``libmj.so`` (declared in
``include/mj.h``): argument marshalling only.  Every step of the decode path
runs in the library's CUDA kernels; there is no Python or CPU fallback, and
loading fails loudly when the library has not been built
(``python -m paged_fp8_kv_gb300.build``).

PyTorch is used only for device memory, streams and events.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmj.so")

MJ_OK = 0
MJ_ERR_INVALID_ARG = 1
MJ_ERR_UNSUPPORTED = 2
MJ_ERR_CAPACITY = 3
MJ_ERR_CUDA = 4
MJ_ERR_TIMEOUT = 5

MJ_BF16 = 0
MJ_E4M3 = 1

MJ_KV_E4M3 = 0
MJ_KV_E3M2 = 1
MJ_KV_E2M3 = 2
MJ_KV_E2M1 = 3
MJ_KV_NVFP4 = 4
KV_FORMATS = {"e4m3": MJ_KV_E4M3, "e3m2": MJ_KV_E3M2, "e2m3": MJ_KV_E2M3, "e2m1": MJ_KV_E2M1, "nvfp4": MJ_KV_NVFP4}

MJ_KERNEL_AUTO = 0
MJ_KERNEL_CUDA_CORE = 1
MJ_KERNEL_TENSOR_CORE = 2
MJ_KERNEL_TENSOR_CORE_GROUPED = 3
MJ_KERNEL_TENSOR_CORE_QROWS = 4


class MjError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class DecodeParams(ctypes.Structure):
    _fields_ = [
        (name, ctypes.c_int32)
        for name in (
            "num_seqs",
            "q_len",
            "h_k",
            "h_r",
            "head_dim",
            "page_size",
            "max_blocks",
            "num_pages",
            "causal",
            "q_dtype",
            "max_splits",
            "kernel",
            "l2_prefetch",
            "kv_evict_first",
            "kv_format",
        )
    ]


class PlanOpts(ctypes.Structure):
    _fields_ = [
        (name, ctypes.c_int32)
        for name in ("sm_count", "ctas_per_sm", "n_q_tiles", "force_splits", "min_chunk_tiles", "pad_to")
    ]


_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_pi32 = ctypes.POINTER(ctypes.c_int32)


class DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("q", _vp),
        ("q_seq_stride", _i64),
        ("k", _vp),
        ("v", _vp),
        ("k_page", _i64),
        ("k_row", _i64),
        ("k_head", _i64),
        ("v_page", _i64),
        ("v_row", _i64),
        ("v_head", _i64),
        ("block_table", _vp),
        ("seq_lens", _vp),
        ("work", _vp),
        ("n_splits", _vp),
        ("num_work", ctypes.c_int32),
        ("q_descale", _vp),
        ("k_descale", _vp),
        ("v_descale", _vp),
        ("qd_seq", _i64),
        ("qd_head", _i64),
        ("kd_seq", _i64),
        ("kd_head", _i64),
        ("vd_seq", _i64),
        ("vd_head", _i64),
        ("softmax_scale", ctypes.c_float),
        ("scale_o", ctypes.c_float),
        ("o", _vp),
        ("o_seq_stride", _i64),
        ("lse", _vp),
        ("workspace", _vp),
        ("workspace_bytes", ctypes.c_size_t),
        ("status", _vp),
        ("max_n_splits", ctypes.c_int32),
        ("timing_events", _vp),
        ("k_scales", _vp),
        ("v_scales", _vp),
        ("ks_page", _i64),
        ("ks_head", _i64),
        ("vs_page", _i64),
        ("vs_head", _i64),
    ]


class RopeParams(ctypes.Structure):
    _fields_ = [
        (name, ctypes.c_int32)
        for name in (
            "num_seqs",
            "q_len",
            "h_k",
            "h_r",
            "head_dim",
            "page_size",
            "max_blocks",
            "num_pages",
            "rot_dim",
            "n_axes",
            "interleaved",
            "max_pos",
        )
    ]


class RopeArgs(ctypes.Structure):
    _fields_ = [
        ("q", _vp),
        ("k", _vp),
        ("v", _vp),
        ("q_tok", _i64),
        ("q_head", _i64),
        ("k_tok", _i64),
        ("k_head_in", _i64),
        ("v_tok", _i64),
        ("v_head_in", _i64),
        ("num_tokens", ctypes.c_int32),
        ("positions", _vp),
        ("pos_axis", _i64),
        ("cos_sin", _vp),
        ("freq_axis", _vp),
        ("cu_tokens", _vp),
        ("q_out", _vp),
        ("q_packed", ctypes.c_int32),
        ("q_out_stride", _i64),
        ("k_cache", _vp),
        ("v_cache", _vp),
        ("k_page", _i64),
        ("k_row", _i64),
        ("k_head", _i64),
        ("v_page", _i64),
        ("v_row", _i64),
        ("v_head", _i64),
        ("block_table", _vp),
        ("seq_lens", _vp),
        ("k_descale", _vp),
        ("v_descale", _vp),
        ("kd_seq", _i64),
        ("kd_head", _i64),
        ("vd_seq", _i64),
        ("vd_head", _i64),
        ("key_pos", _vp),
        ("kp_seq", _i64),
        ("kp_head", _i64),
        ("status", _vp),
        ("granted", _pi32),
    ]


class ScoreModArgs(ctypes.Structure):
    _fields_ = [
        ("softcap", ctypes.c_float),
        ("window", ctypes.c_int32),
        ("alibi_slopes", _vp),
        ("key_begin", _vp),
        ("key_end", _vp),
        ("prefix", _vp),
    ]


class EvictArgs(ctypes.Structure):
    _fields_ = [
        ("k", _vp),
        ("v", _vp),
        ("k_page", _i64),
        ("k_row", _i64),
        ("k_head", _i64),
        ("v_page", _i64),
        ("v_row", _i64),
        ("v_head", _i64),
        ("block_table", _vp),
        ("seq_lens", _vp),
        ("acc", _vp),
        ("acc_out", _vp),
        ("acc_seq", _i64),
        ("acc_head", _i64),
        ("key_pos", _vp),
        ("key_pos_out", _vp),
        ("next_pos", _vp),
        ("new_lens", _vp),
        ("budget", ctypes.c_int32),
        ("keep_first", ctypes.c_int32),
        ("keep_last", ctypes.c_int32),
        ("workspace", _vp),
        ("workspace_bytes", ctypes.c_size_t),
        ("status", _vp),
        ("k_scales", _vp),
        ("v_scales", _vp),
        ("ks_page", _i64),
        ("ks_head", _i64),
        ("vs_page", _i64),
        ("vs_head", _i64),
    ]


class PageParams(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in ("num_seqs", "page_size", "max_blocks", "num_pages")]


class ReserveArgs(ctypes.Structure):
    _fields_ = [
        ("seq_lens", _vp),
        ("new_tokens", _vp),
        ("q_len", ctypes.c_int32),
        ("free_pages", _vp),
        ("num_free", _vp),
        ("num_free_out", _vp),
        ("block_table", _vp),
        ("seq_lens_out", _vp),
        ("cu_tokens", _vp),
        ("positions", _vp),
        ("slots", _vp),
        ("num_tokens", ctypes.c_int32),
        ("status", _vp),
        ("granted", _pi32),
    ]


class ReleaseArgs(ctypes.Structure):
    _fields_ = [
        (name, _vp) for name in ("seq_lens", "keep_lens", "free_pages", "num_free", "num_free_out", "block_table", "status")
    ]


class PromptArgs(ctypes.Structure):
    _fields_ = [
        ("q", _vp),
        ("q_tok", _i64),
        ("q_head", _i64),
        ("o", _vp),
        ("o_tok", _i64),
        ("lse", _vp),
        ("num_tokens", ctypes.c_int32),
        ("k", _vp),
        ("v", _vp),
        ("k_page", _i64),
        ("k_row", _i64),
        ("k_head", _i64),
        ("v_page", _i64),
        ("v_row", _i64),
        ("v_head", _i64),
        ("block_table", _vp),
        ("plan", _vp),
        ("plan_bytes", ctypes.c_size_t),
        ("q_descale", _vp),
        ("k_descale", _vp),
        ("v_descale", _vp),
        ("qd_seq", _i64),
        ("qd_head", _i64),
        ("kd_seq", _i64),
        ("kd_head", _i64),
        ("vd_seq", _i64),
        ("vd_head", _i64),
        ("softmax_scale", ctypes.c_float),
        ("scale_o", ctypes.c_float),
        ("softcap", ctypes.c_float),
        ("window", ctypes.c_int32),
        ("workspace", _vp),
        ("workspace_bytes", ctypes.c_size_t),
        ("status", _vp),
    ]


class TreeArgs(ctypes.Structure):
    _fields_ = [("mask", _vp), ("mask_words", ctypes.c_int32), ("tree_lens", _vp)]


class CommitArgs(ctypes.Structure):
    _fields_ = [
        ("k", _vp),
        ("v", _vp),
        ("k_page", _i64),
        ("k_row", _i64),
        ("k_head", _i64),
        ("v_page", _i64),
        ("v_row", _i64),
        ("v_head", _i64),
        ("block_table", _vp),
        ("seq_lens", _vp),
        ("tree_lens", _vp),
        ("accepted", _vp),
        ("max_accept", ctypes.c_int32),
        ("num_accepted", _vp),
        ("new_lens", _vp),
        ("key_pos", _vp),
        ("kp_seq", _i64),
        ("kp_head", _i64),
        ("status", _vp),
        ("k_scales", _vp),
        ("v_scales", _vp),
        ("ks_page", _i64),
        ("ks_head", _i64),
        ("vs_page", _i64),
        ("vs_head", _i64),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmj.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m paged_fp8_kv_gb300.build` "
                "(there is no fallback implementation)"
            )
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        L.mj_decode_plan.restype = ctypes.c_int
        L.mj_decode_plan.argtypes = [P(DecodeParams), P(PlanOpts), _vp, _vp, ctypes.c_int32, _vp, _vp, _vp]
        L.mj_decode_workspace_bytes.restype = ctypes.c_size_t
        L.mj_decode_workspace_bytes.argtypes = [P(DecodeParams)]
        L.mj_decode_attn.restype = ctypes.c_int
        L.mj_decode_attn.argtypes = [P(DecodeParams), P(DecodeArgs), _vp]
        L.mj_pack_q.restype = ctypes.c_int
        L.mj_pack_q.argtypes = [_vp, _vp] + [ctypes.c_int32] * 6 + [_vp]
        L.mj_decode_plan_max_items.restype = ctypes.c_int32
        L.mj_decode_plan_max_items.argtypes = [_vp, _vp]
        L.mj_decode_plan_device.restype = ctypes.c_int
        L.mj_decode_plan_device.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
        L.mj_check_preconditions.restype = ctypes.c_int
        L.mj_check_preconditions.argtypes = [P(DecodeParams), _vp, _vp, _vp, _vp, _vp] + [_i64] * 6 + [_vp]
        L.mj_check_gather_kv.restype = ctypes.c_int
        L.mj_check_gather_kv.argtypes = [P(DecodeParams), P(DecodeArgs), ctypes.c_int32, _vp, ctypes.c_int32, _vp]
        L.mj_check_dequant_e4m3.restype = ctypes.c_int
        L.mj_check_dequant_e4m3.argtypes = [_vp, _vp]
        L.mj_check_bounded_wait.restype = ctypes.c_int
        L.mj_check_bounded_wait.argtypes = [_vp, _vp, ctypes.c_int32, _vp]
        L.mj_quantize_pack_q.restype = ctypes.c_int
        L.mj_quantize_pack_q.argtypes = [_vp, _vp, _vp] + [ctypes.c_int32] * 5 + [_vp]
        L.mj_unpack_o.restype = ctypes.c_int
        L.mj_unpack_o.argtypes = [_vp, _vp] + [ctypes.c_int32] * 5 + [_vp]
        L.mj_status_string.restype = ctypes.c_char_p
        L.mj_status_string.argtypes = [ctypes.c_int]
        L.mj_rope_append.restype = ctypes.c_int
        L.mj_rope_append.argtypes = [P(RopeParams), P(RopeArgs), _vp]
        L.mj_score_spans.restype = ctypes.c_int
        L.mj_score_spans.argtypes = [P(DecodeParams), P(ScoreModArgs), _vp, _vp, _vp]
        L.mj_score_spans_device.restype = ctypes.c_int
        L.mj_score_spans_device.argtypes = [P(DecodeParams), P(ScoreModArgs), _vp, _vp, _vp, _vp]
        L.mj_decode_attn_mod.restype = ctypes.c_int
        L.mj_decode_attn_mod.argtypes = [P(DecodeParams), P(ScoreModArgs), _vp, P(DecodeArgs), _vp]
        L.mj_key_weights.restype = ctypes.c_int
        L.mj_key_weights.argtypes = [P(DecodeParams), P(ScoreModArgs), P(DecodeArgs), _vp, _i64, _i64, ctypes.c_float,
                                     ctypes.c_int32, _vp]
        L.mj_evict_workspace_bytes.restype = ctypes.c_size_t
        L.mj_evict_workspace_bytes.argtypes = [P(DecodeParams), ctypes.c_int32]
        L.mj_evict.restype = ctypes.c_int
        L.mj_evict.argtypes = [P(DecodeParams), P(EvictArgs), _vp]
        L.mj_pages_reserve.restype = ctypes.c_int
        L.mj_pages_reserve.argtypes = [P(PageParams), P(ReserveArgs), _vp]
        L.mj_pages_release.restype = ctypes.c_int
        L.mj_pages_release.argtypes = [P(PageParams), P(ReleaseArgs), _vp]
        L.mj_prompt_plan_bytes.restype = ctypes.c_size_t
        L.mj_prompt_plan_bytes.argtypes = [P(DecodeParams), ctypes.c_int32]
        L.mj_prompt_plan.restype = ctypes.c_int
        L.mj_prompt_plan.argtypes = [P(DecodeParams), _vp, _vp, ctypes.c_int32, ctypes.c_int32, _vp, ctypes.c_size_t, _vp, _vp]
        L.mj_prompt_workspace_bytes.restype = ctypes.c_size_t
        L.mj_prompt_workspace_bytes.argtypes = [P(DecodeParams)]
        L.mj_prompt_attn.restype = ctypes.c_int
        L.mj_prompt_attn.argtypes = [P(DecodeParams), P(PromptArgs), _vp]
        L.mj_decode_attn_tree.restype = ctypes.c_int
        L.mj_decode_attn_tree.argtypes = [P(DecodeParams), P(TreeArgs), P(ScoreModArgs), _vp, P(DecodeArgs), _vp]
        L.mj_tree_spans.restype = ctypes.c_int
        L.mj_tree_spans.argtypes = [P(DecodeParams), P(TreeArgs), P(ScoreModArgs), _vp, _vp, _vp]
        L.mj_tree_spans_device.restype = ctypes.c_int
        L.mj_tree_spans_device.argtypes = [P(DecodeParams), P(TreeArgs), P(ScoreModArgs), _vp, _vp, _vp, _vp]
        L.mj_tree_commit.restype = ctypes.c_int
        L.mj_tree_commit.argtypes = [P(DecodeParams), P(CommitArgs), _vp]
        L.mj_kernel_name.restype = ctypes.c_int
        L.mj_kernel_name.argtypes = [P(DecodeParams), ctypes.c_char_p, ctypes.c_int32]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().mj_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != MJ_OK:
        raise MjError(status, what)


def make_params(
    num_seqs: int,
    q_len: int,
    h_k: int,
    h_r: int,
    page_size: int,
    max_blocks: int,
    num_pages: int,
    causal: bool = True,
    q_dtype: int = MJ_BF16,
    max_splits: int = 16,
    head_dim: int = 128,
    kernel: int = MJ_KERNEL_AUTO,
    l2_prefetch: int = 0,
    kv_evict_first: int = 0,
    kv_format: int = MJ_KV_E4M3,
) -> DecodeParams:
    return DecodeParams(
        num_seqs,
        q_len,
        h_k,
        h_r,
        head_dim,
        page_size,
        max_blocks,
        num_pages,
        int(causal),
        q_dtype,
        max_splits,
        kernel,
        l2_prefetch,
        kv_evict_first,
        kv_format,
    )


@dataclass
class Plan:
    work: np.ndarray  # int32 (num_work, 4)
    n_splits: np.ndarray  # int32 (num_seqs,)
    chunk_tiles: int
    opts: PlanOpts

    @property
    def num_work(self) -> int:
        return int(self.work.shape[0])

    @property
    def max_n_splits(self) -> int:
        return int(self.n_splits.max())


def decode_plan(
    params: DecodeParams,
    seq_lens: Sequence[int],
    sm_count: int = 0,
    ctas_per_sm: int = 0,
    n_q_tiles: int = 0,
    force_splits: int = 0,
    min_chunk_tiles: int = 0,
    pad_to: int = 0,
) -> Plan:
    """mj_decode_plan on host seq_lens."""
    sl = np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
    opts = PlanOpts(sm_count, ctas_per_sm, n_q_tiles, force_splits, min_chunk_tiles, pad_to)
    cap = max(pad_to, int(params.num_seqs) * int(params.max_splits), 1)
    work = np.zeros((cap, 4), dtype=np.int32)
    n_splits = np.zeros(int(params.num_seqs), dtype=np.int32)
    num_work = ctypes.c_int32(0)
    chunk = ctypes.c_int32(0)
    st = lib().mj_decode_plan(
        ctypes.byref(params),
        ctypes.byref(opts),
        sl.ctypes.data,
        work.ctypes.data,
        cap,
        ctypes.addressof(num_work),
        n_splits.ctypes.data,
        ctypes.addressof(chunk),
    )
    _check(st, "mj_decode_plan")
    return Plan(work[: num_work.value].copy(), n_splits, chunk.value, opts)


def workspace_bytes(params: DecodeParams) -> int:
    return int(lib().mj_decode_workspace_bytes(ctypes.byref(params)))


def kernel_name(params: DecodeParams) -> str:
    buf = ctypes.create_string_buffer(64)
    _check(lib().mj_kernel_name(ctypes.byref(params), buf, 64), "mj_kernel_name")
    return buf.value.decode()


# ------------------------------------------------------------ torch glue


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _i32_ptr(t):
    """_ptr for a field of type _pi32."""
    return None if t is None else ctypes.cast(_ptr(t), _pi32)


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch

        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def descale_strides(t, num_seqs: int, h_k: int) -> Tuple[int, int]:
    """(seq, head) element strides of a descale tensor: one element is a
    per-tensor scale, (h_k,) per head, (b, h_k) per sequence and head."""
    if t.numel() == 1:
        return (0, 0)
    if t.dim() == 1:
        if t.shape[0] != h_k:
            raise ValueError(f"descale shape {tuple(t.shape)}")
        return (0, int(t.stride(0)))
    if t.dim() != 2 or t.shape[1] != h_k or t.shape[0] != num_seqs:
        raise ValueError(f"descale shape {tuple(t.shape)}")
    return (int(t.stride(0)), int(t.stride(1)))


def kv_strides(t) -> Tuple[int, int, int]:
    """(page, row, head) strides of a (num_pages, PS, h_k, d) byte view."""
    if t.element_size() != 1 or t.stride(3) != 1:
        raise ValueError("KV cache must be a 1-byte view with d contiguous")
    return (int(t.stride(0)), int(t.stride(1)), int(t.stride(2)))


def _decode_args(
    params, *, q, k_cache, v_cache, block_table, seq_lens, work, n_splits, q_descale, k_descale, v_descale, o, lse,
    workspace, softmax_scale, scale_o, status, max_n_splits,
) -> DecodeArgs:
    a = DecodeArgs()
    a.q = _ptr(q)
    a.q_seq_stride = int(q.stride(0))
    a.k, a.v = _ptr(k_cache), _ptr(v_cache)
    a.k_page, a.k_row, a.k_head = kv_strides(k_cache)
    a.v_page, a.v_row, a.v_head = kv_strides(v_cache)
    a.block_table, a.seq_lens = _ptr(block_table), _ptr(seq_lens)
    a.work, a.n_splits = _ptr(work), _ptr(n_splits)
    a.num_work = int(work.shape[0])
    nb, hk = int(params.num_seqs), int(params.h_k)
    a.q_descale, a.k_descale, a.v_descale = _ptr(q_descale), _ptr(k_descale), _ptr(v_descale)
    a.qd_seq, a.qd_head = descale_strides(q_descale, nb, hk)
    a.kd_seq, a.kd_head = descale_strides(k_descale, nb, hk)
    a.vd_seq, a.vd_head = descale_strides(v_descale, nb, hk)
    a.softmax_scale, a.scale_o = float(softmax_scale), float(scale_o)
    a.o = _ptr(o)
    a.o_seq_stride = int(o.stride(0))
    a.lse = _ptr(lse)
    a.workspace = _ptr(workspace)
    a.workspace_bytes = 0 if workspace is None else int(workspace.numel() * workspace.element_size())
    a.status = _ptr(status)
    a.max_n_splits = int(max_n_splits)
    return a


def decode_attn(
    params: DecodeParams,
    *,
    q,
    k_cache,
    v_cache,
    block_table,
    seq_lens,
    work,
    n_splits,
    q_descale,
    k_descale,
    v_descale,
    o,
    lse,
    workspace=None,
    softmax_scale: float,
    scale_o: float = 1.0,
    status=None,
    max_n_splits: int = 0,
    timing_events=None,
    stream=None,
    k_scales=None,
    v_scales=None,
) -> None:
    """mj_decode_attn on device tensors.

    q / o are packed (b, h_k, n_q, d) views (rows contiguous, sequence stride
    free); k_cache / v_cache are (num_pages, PS, h_k, d) 1-byte views of any
    physical layout with d contiguous."""
    a = _decode_args(
        params, q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, seq_lens=seq_lens, work=work,
        n_splits=n_splits, q_descale=q_descale, k_descale=k_descale, v_descale=v_descale, o=o, lse=lse,
        workspace=workspace, softmax_scale=softmax_scale, scale_o=scale_o, status=status, max_n_splits=max_n_splits,
    )
    ev_arr = None
    if timing_events is not None:
        handles = [int(e.cuda_event) for e in timing_events]
        if len(handles) != 3 or not all(handles):
            raise ValueError("timing_events: three created CUDA events (record each once first)")
        ev_arr = (ctypes.c_void_p * 3)(*handles)
        a.timing_events = ctypes.cast(ev_arr, ctypes.c_void_p)
    _set_scales(a, k_scales, v_scales)
    st = lib().mj_decode_attn(ctypes.byref(params), ctypes.byref(a), _stream_handle(stream))
    _check(st, "mj_decode_attn")


def scale_strides(t) -> Tuple[int, int]:
    """(page, head) byte strides of an nvfp4 scale plane viewed as
    (num_pages, h_k, page_size, d / 16) uint8 (rows 8 bytes apart)."""
    if t.dim() != 4 or t.element_size() != 1 or t.stride(3) != 1 or t.stride(2) != t.shape[3]:
        raise ValueError("scale plane: (pages, h_k, page_size, d/16) bytes with contiguous rows")
    return int(t.stride(0)), int(t.stride(1))


def _set_scales(a, k_scales, v_scales) -> None:
    if k_scales is None or v_scales is None:
        return
    a.k_scales, a.v_scales = _ptr(k_scales), _ptr(v_scales)
    a.ks_page, a.ks_head = scale_strides(k_scales)
    a.vs_page, a.vs_head = scale_strides(v_scales)


def pack_q(q_vllm, q_packed, num_seqs: int, q_len: int, h_k: int, h_r: int, stream=None) -> None:
    """mj_pack_q: (b*q_len, h_k*h_r, d) -> (b, h_k, q_len*h_r, d)."""
    st = lib().mj_pack_q(
        _ptr(q_vllm),
        _ptr(q_packed),
        int(q_vllm.element_size()),
        num_seqs,
        q_len,
        h_k,
        h_r,
        int(q_vllm.shape[-1]),
        _stream_handle(stream),
    )
    _check(st, "mj_pack_q")


def check_preconditions(params: DecodeParams, block_table, seq_lens, q_descale, k_descale, v_descale):
    """mj_check_preconditions on host (numpy) copies; returns (status, first
    offending sequence or -1)."""
    bt = np.ascontiguousarray(block_table, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    nb, hk = int(params.num_seqs), int(params.h_k)
    # the C checker reads num_seqs rows of max_blocks entries and num_seqs
    # lengths: refuse arrays of another shape instead of reading past them
    if bt.shape != (nb, int(params.max_blocks)):
        raise ValueError(f"block_table shape {bt.shape}, expected {(nb, int(params.max_blocks))}")
    if sl.shape != (nb,):
        raise ValueError(f"seq_lens shape {sl.shape}, expected {(nb,)}")
    ds = [np.ascontiguousarray(d, dtype=np.float32) for d in (q_descale, k_descale, v_descale)]

    def strides(d):  # the element strides descale_strides gives a tensor
        if d.size == 1:
            return (0, 0)
        if d.ndim == 1 and d.shape[0] == hk:
            return (0, 1)
        if d.ndim == 2 and d.shape == (nb, hk):
            return (hk, 1)
        raise ValueError(f"descale shape {d.shape}")

    st_ = [strides(d) for d in ds]
    bad = ctypes.c_int32(0)
    st = lib().mj_check_preconditions(
        ctypes.byref(params),
        bt.ctypes.data,
        sl.ctypes.data,
        ds[0].ctypes.data,
        ds[1].ctypes.data,
        ds[2].ctypes.data,
        *st_[0],
        *st_[1],
        *st_[2],
        ctypes.addressof(bad),
    )
    return int(st), int(bad.value)


def check_gather_kv(params: DecodeParams, k_cache, v_cache, block_table, seq_lens, values: bool, out,
                    stream=None, k_scales=None, v_scales=None) -> None:
    """mj_check_gather_kv: the decode path's K (values False) or V rows of
    every (sequence, kv head) into out (b, h_k, out_rows, 128) uint8 (for an
    nvfp4 pool, the e4m3 rows its conversion gives)."""
    a = DecodeArgs()
    a.k, a.v = _ptr(k_cache), _ptr(v_cache)
    a.k_page, a.k_row, a.k_head = kv_strides(k_cache)
    a.v_page, a.v_row, a.v_head = kv_strides(v_cache)
    a.block_table, a.seq_lens = _ptr(block_table), _ptr(seq_lens)
    _set_scales(a, k_scales, v_scales)
    st = lib().mj_check_gather_kv(
        ctypes.byref(params), ctypes.byref(a), int(bool(values)), _ptr(out), int(out.shape[2]), _stream_handle(stream)
    )
    _check(st, "mj_check_gather_kv")


def check_dequant_e4m3(out, stream=None) -> None:
    """mj_check_dequant_e4m3: out (256,) float32 = the CUDA-core kernel's
    value of every e4m3 code."""
    _check(lib().mj_check_dequant_e4m3(_ptr(out), _stream_handle(stream)), "mj_check_dequant_e4m3")


def check_bounded_wait(status, waited_ns=None, limit_us: int = 1000, stream=None) -> None:
    """mj_check_bounded_wait: one warp waits limit_us on an mbarrier that
    never completes, then writes MJ_ERR_TIMEOUT to status (device int32) and
    the time waited to waited_ns (device int64, optional)."""
    _check(
        lib().mj_check_bounded_wait(_ptr(status), _ptr(waited_ns), int(limit_us), _stream_handle(stream)),
        "mj_check_bounded_wait",
    )


def decode_plan_max_items(
    params: DecodeParams,
    sm_count: int = 0,
    ctas_per_sm: int = 0,
    n_q_tiles: int = 0,
    force_splits: int = 0,
    min_chunk_tiles: int = 0,
) -> int:
    """mj_decode_plan_max_items: the tightest pad_to for the device plan."""
    opts = PlanOpts(sm_count, ctas_per_sm, n_q_tiles, force_splits, min_chunk_tiles, 0)
    n = int(lib().mj_decode_plan_max_items(ctypes.byref(params), ctypes.byref(opts)))
    if n < 0:
        raise MjError(MJ_ERR_INVALID_ARG, "mj_decode_plan_max_items")
    return n


def decode_plan_device(
    params: DecodeParams,
    seq_lens,
    work,
    n_splits,
    pad_to: int,
    sm_count: int = 0,
    ctas_per_sm: int = 0,
    n_q_tiles: int = 0,
    force_splits: int = 0,
    min_chunk_tiles: int = 0,
    chunk_tiles=None,
    status=None,
    stream=None,
) -> PlanOpts:
    """mj_decode_plan_device on device seq_lens (int32 (b,)) into device work
    (int32 (pad_to, 4)) and n_splits (int32 (b,)); returns the options used."""
    opts = PlanOpts(sm_count, ctas_per_sm, n_q_tiles, force_splits, min_chunk_tiles, pad_to)
    st = lib().mj_decode_plan_device(
        ctypes.byref(params),
        ctypes.byref(opts),
        _ptr(seq_lens),
        _ptr(work),
        _ptr(n_splits),
        _ptr(chunk_tiles),
        _ptr(status),
        _stream_handle(stream),
    )
    _check(st, "mj_decode_plan_device")
    return opts


def quantize_pack_q(q_vllm, q_packed, q_descale, num_seqs: int, q_len: int, h_k: int, h_r: int, stream=None) -> None:
    """mj_quantize_pack_q: bf16 (b*q_len, h_k*h_r, d) -> e4m3 codes
    (b, h_k, q_len*h_r, d) and fp32 descales (b, h_k)."""
    st = lib().mj_quantize_pack_q(
        _ptr(q_vllm),
        _ptr(q_packed),
        _ptr(q_descale),
        num_seqs,
        q_len,
        h_k,
        h_r,
        int(q_vllm.shape[-1]),
        _stream_handle(stream),
    )
    _check(st, "mj_quantize_pack_q")


def unpack_o(o_packed, o_vllm, num_seqs: int, q_len: int, h_k: int, h_r: int, stream=None) -> None:
    """mj_unpack_o: (b, h_k, q_len*h_r, d) -> (b*q_len, h_k*h_r, d), bf16."""
    st = lib().mj_unpack_o(
        _ptr(o_packed), _ptr(o_vllm), num_seqs, q_len, h_k, h_r, int(o_packed.shape[-1]), _stream_handle(stream)
    )
    _check(st, "mj_unpack_o")


# ------------------------------------------- the cache's own operators
#
# A call of these is an object: its tensors are checked and marshalled once,
# it holds them, and calling it (with an optional stream; torch's current one
# otherwise) launches the operator on whatever they hold then.  A serving loop
# makes one per set of buffers; ``rope_append`` and the like make one and call
# it.


def _tensor(name, t, dtypes, shape=None, strided=False):
    """Refuse a tensor the library would misread: its type, its shape (None:
    any extent), its device, and (unless strided) its contiguity."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: a torch tensor, got {type(t).__name__}")
    if t.device.type != "cuda" or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: on {t.device}, expected the current CUDA device")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and (t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape))):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple('*' if n is None else n for n in shape)}")
    if not strided and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t


def _dtypes():
    import torch

    return torch.bfloat16, torch.float32, torch.int32, (torch.uint8, torch.int8, torch.float8_e4m3fn)


def _check_descale(name, t, num_seqs, h_k):
    import torch

    _tensor(name, t, (torch.float32,), strided=True)
    descale_strides(t, num_seqs, h_k)


def _check_pools(params, k_cache, v_cache, row_bytes=128):
    codes = _dtypes()[3]
    shape = (int(params.num_pages), int(params.page_size), int(params.h_k), row_bytes)
    _tensor("k_cache", k_cache, codes, shape, strided=True)
    if v_cache is not None:
        _tensor("v_cache", v_cache, codes, shape, strided=True)


def _row_bytes(params) -> int:
    return {MJ_KV_E4M3: 128, MJ_KV_E3M2: 96, MJ_KV_E2M3: 96}.get(int(params.kv_format), 64)


def _check_tables(params, block_table, seq_lens):
    i32 = _dtypes()[2]
    _tensor("block_table", block_table, (i32,), (int(params.num_seqs), int(params.max_blocks)))
    _tensor("seq_lens", seq_lens, (i32,), (int(params.num_seqs),))


def _check_status(status):
    if status is not None:
        t = _tensor("status", status, (_dtypes()[2],))
        if t.numel() < 1:
            raise ValueError("status: one int32")


def _per_slot(name, t, dtype, params):
    """A (num_seqs, h_k, slots) tensor with contiguous slots, one for each
    the block table covers."""
    _tensor(name, t, (dtype,), (int(params.num_seqs), int(params.h_k), None), strided=True)
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: slots must be contiguous")
    if t.shape[2] < int(params.max_blocks) * int(params.page_size):
        raise ValueError(f"{name}: {t.shape[2]} slots, expected max_blocks*page_size")
    return int(t.stride(0)), int(t.stride(1))


class _Call:
    """A marshalled call: ``call(stream=None)`` launches it."""

    _name = ""

    @staticmethod
    def _own(params):
        """A copy: the caller may change its own for the next call."""
        return type(params).from_buffer_copy(params)

    def _bind(self, fn, args, keep) -> None:
        import torch

        self._fn, self._args, self._keep = fn, args, keep  # keep: the tensors behind the pointers
        self._device, self._current_device = torch.cuda.current_device(), torch.cuda.current_device
        # the current stream's handle without a Stream object around it (3 us of a call that takes 6)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._raw_stream = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)

    def __call__(self, stream=None) -> None:
        if self._current_device() != self._device:
            raise ValueError(f"{self._name}: its tensors are on CUDA device {self._device}, which is not the current one")
        st = self._fn(*self._args, self._raw_stream(self._device) if stream is None else stream.cuda_stream)
        if st != MJ_OK:
            raise MjError(st, self._name)


def make_rope_params(
    num_seqs: int,
    q_len: int,
    h_k: int,
    h_r: int,
    page_size: int,
    max_blocks: int,
    num_pages: int,
    *,
    rot_dim: int = 128,
    n_axes: int = 1,
    interleaved: bool = False,
    max_pos: int,
    head_dim: int = 128,
) -> RopeParams:
    return RopeParams(num_seqs, q_len, h_k, h_r, head_dim, page_size, max_blocks, num_pages, rot_dim, n_axes,
                      int(interleaved), max_pos)


class RopeAppend(_Call):
    """mj_rope_append on device tensors.

    q (tokens, h_k*h_r, 128), k and v (tokens, h_k, 128) are bf16 and may be
    slices of one projection's output; positions (n_axes, tokens) or (tokens,)
    int32; cos_sin (max_pos, rot_dim) float32; freq_axis a host sequence of
    rot_dim/2 axes (None: axis 0).  q_out is the packed (num_seqs, h_k,
    q_len*h_r, 128) or the token layout (tokens, h_k*h_r, 128), which may be q.
    cu_tokens (num_seqs + 1,) int32 gives the sequences their tokens where
    they differ in number.  key_pos (num_seqs, h_k, slots) int32 is optional;
    granted (num_seqs,) int32 of pages_reserve keeps the tokens of sequences
    that it left out from the cache."""

    _name = "mj_rope_append"

    def __init__(self, params: RopeParams, *, q, k, v, positions, cos_sin, q_out, k_cache, v_cache, block_table, seq_lens,
                 k_descale, v_descale, freq_axis=None, cu_tokens=None, key_pos=None, status=None, granted=None):
        params = self._own(params)
        bf16, f32, i32, _ = _dtypes()
        nb, hk, hq = int(params.num_seqs), int(params.h_k), int(params.h_k) * int(params.h_r)
        n = int(q.shape[0])
        for name, t, heads in (("q", q, hq), ("k", k, hk), ("v", v, hk)):
            _tensor(name, t, (bf16,), (n, heads, 128), strided=True)
            if t.stride(2) != 1:
                raise ValueError(f"{name}: the head dimension must be contiguous")
        _tensor("positions", positions, (i32,), strided=True)
        if positions.dim() == 1:
            positions = positions[None]
        if positions.dim() != 2 or tuple(positions.shape) != (int(params.n_axes), n) or (n > 1 and positions.stride(1) != 1):
            raise ValueError(f"positions: shape {tuple(positions.shape)}, expected {(int(params.n_axes), n)}, tokens contiguous")
        _tensor("cos_sin", cos_sin, (f32,), (int(params.max_pos), int(params.rot_dim)))
        _tensor("q_out", q_out, (bf16,), strided=True)
        packed = q_out.dim() == 4
        want = (nb, hk, int(params.q_len) * int(params.h_r), 128) if packed else (n, hq, 128)
        if tuple(q_out.shape) != want or any(
            q_out.shape[i] > 1 and q_out.stride(i) != int(np.prod(want[i + 1 :])) for i in range(1, len(want))
        ):
            raise ValueError(f"q_out: shape {tuple(q_out.shape)}, expected {want} with contiguous rows")
        _check_pools(params, k_cache, v_cache)
        _check_tables(params, block_table, seq_lens)
        _check_descale("k_descale", k_descale, nb, hk)
        _check_descale("v_descale", v_descale, nb, hk)
        if cu_tokens is not None:
            _tensor("cu_tokens", cu_tokens, (i32,), (nb + 1,))
        if granted is not None:
            _tensor("granted", granted, (i32,), (nb,))
        axes = None
        if freq_axis is not None:
            axes = np.ascontiguousarray(np.asarray(freq_axis), dtype=np.uint8)
            if axes.shape != (int(params.rot_dim) // 2,) or not np.array_equal(axes, np.asarray(freq_axis)):
                raise ValueError("freq_axis: rot_dim/2 axes")
        _check_status(status)
        a = RopeArgs()
        a.q, a.k, a.v = _ptr(q), _ptr(k), _ptr(v)
        a.q_tok, a.q_head = int(q.stride(0)), int(q.stride(1))
        a.k_tok, a.k_head_in = int(k.stride(0)), int(k.stride(1))
        a.v_tok, a.v_head_in = int(v.stride(0)), int(v.stride(1))
        a.num_tokens = n
        a.positions, a.pos_axis = _ptr(positions), int(positions.stride(0))
        a.cos_sin = _ptr(cos_sin)
        a.freq_axis = None if axes is None else axes.ctypes.data
        a.cu_tokens = _ptr(cu_tokens)
        a.q_out, a.q_packed, a.q_out_stride = _ptr(q_out), int(packed), int(q_out.stride(0))
        a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
        a.k_page, a.k_row, a.k_head = kv_strides(k_cache)
        a.v_page, a.v_row, a.v_head = kv_strides(v_cache)
        a.block_table, a.seq_lens = _ptr(block_table), _ptr(seq_lens)
        a.k_descale, a.v_descale = _ptr(k_descale), _ptr(v_descale)
        a.kd_seq, a.kd_head = descale_strides(k_descale, nb, hk)
        a.vd_seq, a.vd_head = descale_strides(v_descale, nb, hk)
        if key_pos is not None:
            a.kp_seq, a.kp_head = _per_slot("key_pos", key_pos, i32, params)
            a.key_pos = _ptr(key_pos)
        a.status, a.granted = _ptr(status), _i32_ptr(granted)
        self._bind(lib().mj_rope_append, (ctypes.byref(params), ctypes.byref(a)),
                   (params, a, axes, q, k, v, positions, cos_sin, q_out, k_cache, v_cache, block_table, seq_lens, k_descale,
                    v_descale, cu_tokens, key_pos, status, granted))


def rope_append(params: RopeParams, *, stream=None, **tensors) -> None:
    """One RopeAppend call."""
    RopeAppend(params, **tensors)(stream)


@dataclass
class ScoreMod:
    """mj_score_mod: device tensors (alibi_slopes (h_k*h_r,) float32,
    key_begin / key_end (num_seqs, q_len) int32, prefix (num_seqs,) int32) or
    None, softcap (else 2^-20 to 2^60) and window 0 = off."""

    softcap: float = 0.0
    window: int = 0
    alibi_slopes: object = None
    key_begin: object = None
    key_end: object = None
    prefix: object = None

    def _marshal(self, params) -> ScoreModArgs:
        _, f32, i32, _ = _dtypes()
        nb, ql = int(params.num_seqs), int(params.q_len)
        if self.alibi_slopes is not None:
            _tensor("alibi_slopes", self.alibi_slopes, (f32,), (int(params.h_k) * int(params.h_r),))
        for name in ("key_begin", "key_end"):
            if getattr(self, name) is not None:
                _tensor(name, getattr(self, name), (i32,), (nb, ql))
        if self.prefix is not None:
            _tensor("prefix", self.prefix, (i32,), (nb,))
        return ScoreModArgs(float(self.softcap), int(self.window), _ptr(self.alibi_slopes), _ptr(self.key_begin),
                            _ptr(self.key_end), _ptr(self.prefix))

    def _tensors(self):
        return self.alibi_slopes, self.key_begin, self.key_end, self.prefix


def score_spans(params: DecodeParams, mod: ScoreMod, seq_lens: Sequence[int]) -> Tuple[np.ndarray, np.ndarray]:
    """mj_score_spans on host seq_lens: (spans (num_seqs, 4), plan_lens
    (num_seqs,)), int32.  The modifiers' tensors are read back to the host."""
    return _spans_host(params, mod, seq_lens, None)


def _host_i32(name, t, shape):
    """A device tensor or host sequence as a host int32 array, or None."""
    if t is None:
        return None
    x = np.ascontiguousarray(t.cpu().numpy() if hasattr(t, "cpu") else np.asarray(t), dtype=np.int32)
    if x.shape != shape:
        raise ValueError(f"{name}: shape {x.shape}, expected {shape}")
    return x


def _spans_host(params, mod, seq_lens, tree):
    """mj_score_spans, or mj_tree_spans with ``tree`` = (tree_lens or None,)."""
    nb, ql = int(params.num_seqs), int(params.q_len)
    sl = np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
    if sl.shape != (nb,):
        raise ValueError(f"seq_lens shape {sl.shape}, expected {(nb,)}")
    x = [_host_i32(name, getattr(mod, name), shape) for name, shape in (("key_begin", (nb, ql)), ("key_end", (nb, ql)), ("prefix", (nb,)))]
    slopes = None if tree is None else _ptr(mod.alibi_slopes)  # (refused for trees, not looked at else)
    m = ScoreModArgs(float(mod.softcap), int(mod.window), slopes, *(None if y is None else y.ctypes.data for y in x))
    spans = np.zeros((nb, 4), dtype=np.int32)
    plan_lens = np.zeros(nb, dtype=np.int32)
    out = (sl.ctypes.data, spans.ctypes.data, plan_lens.ctypes.data)
    if tree is None:
        _check(lib().mj_score_spans(ctypes.byref(params), ctypes.byref(m), *out), "mj_score_spans")
    else:
        nodes = _host_i32("tree_lens", tree[0], (nb,))
        t = TreeArgs(None, 0, None if nodes is None else nodes.ctypes.data)
        _check(lib().mj_tree_spans(ctypes.byref(params), ctypes.byref(t), ctypes.byref(m), *out), "mj_tree_spans")
    return spans, plan_lens


def score_spans_device(params: DecodeParams, mod: ScoreMod, seq_lens, spans, plan_lens, stream=None) -> None:
    """mj_score_spans_device: spans (num_seqs, 4) and plan_lens (num_seqs,)
    int32 from device seq_lens."""
    i32, nb = _dtypes()[2], int(params.num_seqs)
    _tensor("seq_lens", seq_lens, (i32,), (nb,))
    _tensor("spans", spans, (i32,), (nb, 4))
    _tensor("plan_lens", plan_lens, (i32,), (nb,))
    m = mod._marshal(params)
    st = lib().mj_score_spans_device(ctypes.byref(params), ctypes.byref(m), _ptr(seq_lens), _ptr(spans), _ptr(plan_lens),
                                     _stream_handle(stream))
    _check(st, "mj_score_spans_device")


def tree_spans(params: DecodeParams, mod: Optional[ScoreMod], seq_lens: Sequence[int], tree_lens=None) -> Tuple[np.ndarray, np.ndarray]:
    """mj_tree_spans on host seq_lens: score_spans for DecodeAttnTree, with
    its mod and tree_lens (read back to the host)."""
    return _spans_host(params, ScoreMod() if mod is None else mod, seq_lens, (tree_lens,))


def tree_spans_device(params: DecodeParams, mod: Optional[ScoreMod], seq_lens, spans, plan_lens, tree_lens=None, stream=None) -> None:
    """mj_tree_spans_device: spans (num_seqs, 4) and plan_lens (num_seqs,)
    int32 from device seq_lens and DecodeAttnTree's mod and tree_lens."""
    i32, nb = _dtypes()[2], int(params.num_seqs)
    for name, t, shape in (("seq_lens", seq_lens, (nb,)), ("spans", spans, (nb, 4)), ("plan_lens", plan_lens, (nb,)),
                           ("tree_lens", tree_lens, (nb,))):
        if t is not None:
            _tensor(name, t, (i32,), shape)
    m = (ScoreMod() if mod is None else mod)._marshal(params)
    t = TreeArgs(None, 0, _ptr(tree_lens))
    st = lib().mj_tree_spans_device(ctypes.byref(params), ctypes.byref(t), ctypes.byref(m), _ptr(seq_lens), _ptr(spans),
                                    _ptr(plan_lens), _stream_handle(stream))
    _check(st, "mj_tree_spans_device")


def _check_queries(params, q):
    bf16, _, _, codes = _dtypes()
    import torch

    kinds = codes if int(params.q_dtype) == MJ_E4M3 else (bf16, torch.int16)
    rows = int(params.q_len) * int(params.h_r)
    _tensor("q", q, kinds, (int(params.num_seqs), int(params.h_k), rows, 128), strided=True)
    _rows_packed("q", q)


def _rows_packed(name, t):
    if not t[0].is_contiguous():
        raise ValueError(f"{name}: a sequence's rows must be contiguous")


class DecodeAttnMod(_Call):
    """mj_decode_attn_mod on device tensors: decode_attn's, a ScoreMod, and
    the spans (num_seqs, 4) whose plan_lens the plan was made from (None: a
    plan from seq_lens)."""

    _name = "mj_decode_attn_mod"

    def __init__(self, params: DecodeParams, mod: ScoreMod, *, q, k_cache, v_cache, block_table, seq_lens, work, n_splits,
                 q_descale, k_descale, v_descale, o, lse, softmax_scale: float, workspace=None, spans=None,
                 scale_o: float = 1.0, status=None, max_n_splits: int = 0):
        params = self._own(params)
        m, a, keep = self._marshal(params, mod, q, k_cache, v_cache, block_table, seq_lens, work, n_splits, q_descale,
                                   k_descale, v_descale, o, lse, softmax_scale, workspace, spans, scale_o, status, max_n_splits)
        self._bind(lib().mj_decode_attn_mod, (ctypes.byref(params), ctypes.byref(m), _ptr(spans), ctypes.byref(a)), (params, keep))

    @staticmethod
    def _marshal(params, mod, q, k_cache, v_cache, block_table, seq_lens, work, n_splits, q_descale, k_descale, v_descale, o,
                 lse, softmax_scale, workspace, spans, scale_o, status, max_n_splits):
        """The checked modifiers and arguments, and all that they point to."""
        import torch

        bf16, f32, i32, _ = _dtypes()
        nb, hk, rows = int(params.num_seqs), int(params.h_k), int(params.q_len) * int(params.h_r)
        _check_queries(params, q)
        _check_pools(params, k_cache, v_cache, _row_bytes(params))
        _check_tables(params, block_table, seq_lens)
        _tensor("work", work, (i32,), (None, 4))
        _tensor("n_splits", n_splits, (i32,), (nb,))
        for name, t in (("q_descale", q_descale), ("k_descale", k_descale), ("v_descale", v_descale)):
            _check_descale(name, t, nb, hk)
        _tensor("o", o, (bf16,), (nb, hk, rows, 128), strided=True)
        _rows_packed("o", o)
        _tensor("lse", lse, (f32,), (nb, hk, rows))
        if spans is not None:
            _tensor("spans", spans, (i32,), (nb, 4))
        if workspace is not None:
            _tensor("workspace", workspace, (torch.uint8,))
        _check_status(status)
        m = mod._marshal(params)
        a = _decode_args(
            params, q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, seq_lens=seq_lens, work=work,
            n_splits=n_splits, q_descale=q_descale, k_descale=k_descale, v_descale=v_descale, o=o, lse=lse,
            workspace=workspace, softmax_scale=softmax_scale, scale_o=scale_o, status=status, max_n_splits=max_n_splits,
        )
        return m, a, (mod._tensors(), m, a, spans, q, k_cache, v_cache, block_table, seq_lens, work, n_splits, q_descale,
                      k_descale, v_descale, o, lse, workspace, status)


def decode_attn_mod(params: DecodeParams, mod: ScoreMod, *, stream=None, **tensors) -> None:
    """One DecodeAttnMod call."""
    DecodeAttnMod(params, mod, **tensors)(stream)


class DecodeAttnTree(DecodeAttnMod):
    """mj_decode_attn_tree on device tensors: DecodeAttnMod's (mod None, or
    with softcap, key_begin and prefix alone), tree_mask (num_seqs, q_len,
    words) int32, bit m of a token's words set if it sees node m, and tree_lens
    (num_seqs,) int32 (None: q_len nodes each).  spans and the plan's lengths
    are of tree_spans."""

    _name = "mj_decode_attn_tree"

    def __init__(self, params: DecodeParams, mod: Optional[ScoreMod] = None, *, tree_mask, q, k_cache, v_cache, block_table,
                 seq_lens, work, n_splits, q_descale, k_descale, v_descale, o, lse, softmax_scale: float, tree_lens=None,
                 workspace=None, spans=None, scale_o: float = 1.0, status=None, max_n_splits: int = 0):
        params = self._own(params)
        i32 = _dtypes()[2]
        m, a, keep = self._marshal(params, ScoreMod() if mod is None else mod, q, k_cache, v_cache, block_table, seq_lens, work,
                                   n_splits, q_descale, k_descale, v_descale, o, lse, softmax_scale, workspace, spans, scale_o,
                                   status, max_n_splits)
        _tensor("tree_mask", tree_mask, (i32,), (int(params.num_seqs), int(params.q_len), None))
        if tree_lens is not None:
            _tensor("tree_lens", tree_lens, (i32,), (int(params.num_seqs),))
        t = TreeArgs(_ptr(tree_mask), int(tree_mask.shape[2]), _ptr(tree_lens))
        self._bind(lib().mj_decode_attn_tree,
                   (ctypes.byref(params), ctypes.byref(t), ctypes.byref(m), _ptr(spans), ctypes.byref(a)),
                   (params, t, tree_mask, tree_lens, keep))


def decode_attn_tree(params: DecodeParams, mod: Optional[ScoreMod] = None, *, stream=None, **tensors) -> None:
    """One DecodeAttnTree call."""
    DecodeAttnTree(params, mod, **tensors)(stream)


class KeyWeights(_Call):
    """mj_key_weights on device tensors: acc (num_seqs, h_k, slots) float32
    receives the weights of every cached key; work is of a plan made from
    seq_lens themselves (not from spans' plan_lens: status reports one that
    holds too few tiles); mod may be None."""

    _name = "mj_key_weights"

    def __init__(self, params: DecodeParams, mod: Optional[ScoreMod], *, q, k_cache, block_table, seq_lens, work, q_descale,
                 k_descale, lse, acc, softmax_scale: float, decay: float = 1.0, fresh: int = 0, status=None):
        params = self._own(params)
        _, f32, i32, _ = _dtypes()
        nb, hk, rows = int(params.num_seqs), int(params.h_k), int(params.q_len) * int(params.h_r)
        _check_queries(params, q)
        _check_pools(params, k_cache, None, _row_bytes(params))
        _check_tables(params, block_table, seq_lens)
        _tensor("work", work, (i32,), (None, 4))
        _check_descale("q_descale", q_descale, nb, hk)
        _check_descale("k_descale", k_descale, nb, hk)
        _tensor("lse", lse, (f32,), (nb, hk, rows))
        seq, head = _per_slot("acc", acc, f32, params)
        _check_status(status)
        m = None if mod is None else mod._marshal(params)
        a = DecodeArgs()
        a.q, a.q_seq_stride = _ptr(q), int(q.stride(0))
        a.k = _ptr(k_cache)
        a.k_page, a.k_row, a.k_head = kv_strides(k_cache)
        a.block_table, a.seq_lens = _ptr(block_table), _ptr(seq_lens)
        a.work, a.num_work = _ptr(work), int(work.shape[0])
        a.q_descale, a.k_descale = _ptr(q_descale), _ptr(k_descale)
        a.qd_seq, a.qd_head = descale_strides(q_descale, nb, hk)
        a.kd_seq, a.kd_head = descale_strides(k_descale, nb, hk)
        a.softmax_scale = float(softmax_scale)
        a.lse, a.status = _ptr(lse), _ptr(status)
        self._bind(lib().mj_key_weights,
                   (ctypes.byref(params), None if m is None else ctypes.byref(m), ctypes.byref(a), _ptr(acc), seq, head,
                    float(decay), int(fresh)),
                   (params, None if mod is None else mod._tensors(), m, a, q, k_cache, block_table, seq_lens, work, q_descale, k_descale, lse, acc, status))


def key_weights(params: DecodeParams, mod: Optional[ScoreMod] = None, *, stream=None, **tensors) -> None:
    """One KeyWeights call."""
    KeyWeights(params, mod, **tensors)(stream)


def evict_workspace_bytes(params: DecodeParams, budget: int) -> int:
    """mj_evict_workspace_bytes."""
    n = int(lib().mj_evict_workspace_bytes(ctypes.byref(params), int(budget)))
    if n == 0:
        raise MjError(MJ_ERR_INVALID_ARG, "mj_evict_workspace_bytes")
    return n


class Evict(_Call):
    """mj_evict on device tensors: cuts every (sequence, head) to ``budget``
    keys.  acc / acc_out (the same tensor or two of one layout), key_pos /
    key_pos_out (likewise; None: positions are slots) are (num_seqs, h_k,
    slots); new_lens (num_seqs,) int32 receives the lengths."""

    _name = "mj_evict"

    def __init__(self, params: DecodeParams, *, k_cache, v_cache, block_table, seq_lens, acc, new_lens, budget: int,
                 workspace, acc_out=None, key_pos=None, key_pos_out=None, next_pos=None, keep_first: int = 0,
                 keep_last: int = 0, status=None, k_scales=None, v_scales=None):
        import torch

        params = self._own(params)
        _, f32, i32, codes = _dtypes()
        nb, hk = int(params.num_seqs), int(params.h_k)
        _check_pools(params, k_cache, v_cache, _row_bytes(params))
        _check_tables(params, block_table, seq_lens)
        _tensor("new_lens", new_lens, (i32,), (nb,))
        acc_out = acc if acc_out is None else acc_out
        strides = _per_slot("acc", acc, f32, params)
        planes = [("acc_out", acc_out, f32)]
        if key_pos is not None:
            key_pos_out = key_pos if key_pos_out is None else key_pos_out
            planes += [("key_pos", key_pos, i32), ("key_pos_out", key_pos_out, i32)]
            _tensor("next_pos", next_pos, (i32,), (nb,))
        for name, t, dtype in planes:
            if _per_slot(name, t, dtype, params) != strides or t.shape != acc.shape:
                raise ValueError(f"{name}: the layout of acc")
        _tensor("workspace", workspace, (torch.uint8,))
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if t is not None:
                shape = (int(params.num_pages), hk, int(params.page_size), 8)
                _tensor(name, t, codes, shape, strided=True)
        _check_status(status)
        a = EvictArgs()
        a.k, a.v = _ptr(k_cache), _ptr(v_cache)
        a.k_page, a.k_row, a.k_head = kv_strides(k_cache)
        a.v_page, a.v_row, a.v_head = kv_strides(v_cache)
        a.block_table, a.seq_lens = _ptr(block_table), _ptr(seq_lens)
        a.acc, a.acc_out = _ptr(acc), _ptr(acc_out)
        a.acc_seq, a.acc_head = strides
        if key_pos is not None:
            a.key_pos, a.key_pos_out, a.next_pos = _ptr(key_pos), _ptr(key_pos_out), _ptr(next_pos)
        a.new_lens = _ptr(new_lens)
        a.budget, a.keep_first, a.keep_last = int(budget), int(keep_first), int(keep_last)
        a.workspace, a.workspace_bytes = _ptr(workspace), int(workspace.numel())
        a.status = _ptr(status)
        _set_scales(a, k_scales, v_scales)
        self._bind(lib().mj_evict, (ctypes.byref(params), ctypes.byref(a)),
                   (params, a, k_cache, v_cache, block_table, seq_lens, acc, acc_out, key_pos, key_pos_out, next_pos,
                    new_lens, workspace, status, k_scales, v_scales))


def evict(params: DecodeParams, *, stream=None, **tensors) -> None:
    """One Evict call."""
    Evict(params, **tensors)(stream)


# ------------------------------------------- a serving step's operators


def make_page_params(num_seqs: int, page_size: int, max_blocks: int, num_pages: int) -> PageParams:
    return PageParams(num_seqs, page_size, max_blocks, num_pages)


def _check_page_list(params, seq_lens, free_pages, num_free, num_free_out, block_table, status):
    i32, nb = _dtypes()[2], int(params.num_seqs)
    _tensor("seq_lens", seq_lens, (i32,), (nb,))
    _tensor("free_pages", free_pages, (i32,), (int(params.num_pages),))
    _tensor("num_free", num_free, (i32,), (1,))
    _tensor("num_free_out", num_free_out, (i32,), (1,))
    _tensor("block_table", block_table, (i32,), (nb, int(params.max_blocks)))
    _check_status(status)


class PagesReserve(_Call):
    """mj_pages_reserve on device tensors: pages from the free list
    (free_pages (num_pages,) int32, of which the first num_free (1,) int32)
    for new_tokens (num_seqs,) int32 (None: q_len each) behind seq_lens.
    seq_lens_out and num_free_out may be (and are, if None) seq_lens and
    num_free themselves; cu_tokens (num_seqs + 1,) int32, positions (tokens,)
    int32, slots (tokens,) int64 and granted (num_seqs,) int32, the tokens each
    sequence got (0: left out), are optional outputs."""

    _name = "mj_pages_reserve"

    def __init__(self, params: PageParams, *, seq_lens, free_pages, num_free, block_table, new_tokens=None, q_len: int = 1,
                 num_free_out=None, seq_lens_out=None, cu_tokens=None, positions=None, slots=None, status=None, granted=None):
        import torch

        params = self._own(params)
        i32, nb = _dtypes()[2], int(params.num_seqs)
        num_free_out = num_free if num_free_out is None else num_free_out
        seq_lens_out = seq_lens if seq_lens_out is None else seq_lens_out
        _check_page_list(params, seq_lens, free_pages, num_free, num_free_out, block_table, status)
        _tensor("seq_lens_out", seq_lens_out, (i32,), (nb,))
        if new_tokens is not None:
            _tensor("new_tokens", new_tokens, (i32,), (nb,))
        if cu_tokens is not None:
            _tensor("cu_tokens", cu_tokens, (i32,), (nb + 1,))
        if granted is not None:
            _tensor("granted", granted, (i32,), (nb,))
        n = 0
        for name, t, dtype in (("positions", positions, i32), ("slots", slots, torch.int64)):
            if t is not None:
                _tensor(name, t, (dtype,), (None,))
                n = int(t.shape[0])
        if positions is not None and slots is not None and positions.shape != slots.shape:
            raise ValueError(f"slots: {slots.shape[0]} entries, positions has {positions.shape[0]}")
        # (an empty tensor's pointer is NULL, which would say that none was given)
        positions, slots = (t.new_empty(1) if t is not None and n == 0 else t for t in (positions, slots))
        a = ReserveArgs(_ptr(seq_lens), _ptr(new_tokens), int(q_len), _ptr(free_pages), _ptr(num_free), _ptr(num_free_out),
                        _ptr(block_table), _ptr(seq_lens_out), _ptr(cu_tokens), _ptr(positions), _ptr(slots), n, _ptr(status), _i32_ptr(granted))
        self._bind(lib().mj_pages_reserve, (ctypes.byref(params), ctypes.byref(a)),
                   (params, a, seq_lens, new_tokens, free_pages, num_free, num_free_out, block_table, seq_lens_out, cu_tokens,
                    positions, slots, status, granted))


def pages_reserve(params: PageParams, *, stream=None, **tensors) -> None:
    """One PagesReserve call."""
    PagesReserve(params, **tensors)(stream)


class PagesRelease(_Call):
    """mj_pages_release on device tensors: the pages behind keep_lens
    (num_seqs,) int32 of sequences of seq_lens tokens go back to the free
    list; num_free_out None: num_free itself."""

    _name = "mj_pages_release"

    def __init__(self, params: PageParams, *, seq_lens, keep_lens, free_pages, num_free, block_table, num_free_out=None,
                 status=None):
        params = self._own(params)
        num_free_out = num_free if num_free_out is None else num_free_out
        _check_page_list(params, seq_lens, free_pages, num_free, num_free_out, block_table, status)
        _tensor("keep_lens", keep_lens, (_dtypes()[2],), (int(params.num_seqs),))
        a = ReleaseArgs(_ptr(seq_lens), _ptr(keep_lens), _ptr(free_pages), _ptr(num_free), _ptr(num_free_out),
                        _ptr(block_table), _ptr(status))
        self._bind(lib().mj_pages_release, (ctypes.byref(params), ctypes.byref(a)),
                   (params, a, seq_lens, keep_lens, free_pages, num_free, num_free_out, block_table, status))


def pages_release(params: PageParams, *, stream=None, **tensors) -> None:
    """One PagesRelease call."""
    PagesRelease(params, **tensors)(stream)


def prompt_plan_bytes(params: DecodeParams, num_tokens: int) -> int:
    """mj_prompt_plan_bytes."""
    n = int(lib().mj_prompt_plan_bytes(ctypes.byref(params), int(num_tokens)))
    if n == 0:
        raise MjError(MJ_ERR_INVALID_ARG, "mj_prompt_plan_bytes")
    return n


def prompt_workspace_bytes(params: DecodeParams) -> int:
    """mj_prompt_workspace_bytes (0 when max_splits is 1)."""
    return int(lib().mj_prompt_workspace_bytes(ctypes.byref(params)))


class PromptPlan(_Call):
    """mj_prompt_plan on device tensors: cu_tokens (num_seqs + 1,) and seq_lens
    (num_seqs,) int32 into plan (prompt_plan_bytes,) uint8."""

    _name = "mj_prompt_plan"

    def __init__(self, params: DecodeParams, *, cu_tokens, seq_lens, num_tokens: int, plan, window: int = 0, status=None):
        import torch

        params = self._own(params)
        i32, nb = _dtypes()[2], int(params.num_seqs)
        _tensor("cu_tokens", cu_tokens, (i32,), (nb + 1,))
        _tensor("seq_lens", seq_lens, (i32,), (nb,))
        _tensor("plan", plan, (torch.uint8,))
        _check_status(status)
        self._bind(lib().mj_prompt_plan,
                   (ctypes.byref(params), _ptr(cu_tokens), _ptr(seq_lens), int(num_tokens), int(window), _ptr(plan),
                    int(plan.numel()), _ptr(status)),
                   (params, cu_tokens, seq_lens, plan, status))


def prompt_plan(params: DecodeParams, *, stream=None, **tensors) -> None:
    """One PromptPlan call."""
    PromptPlan(params, **tensors)(stream)


class PromptAttn(_Call):
    """mj_prompt_attn on device tensors: q (tokens, h_k*h_r, 128) bf16, or
    e4m3 codes for params of that q_dtype (a slice of a projection's output, or
    rope_append's); o (tokens, h_k*h_r, 128) bf16 with contiguous rows; lse
    (tokens, h_k*h_r) float32 or None; plan of prompt_plan for the same params,
    tokens and window."""

    _name = "mj_prompt_attn"

    def __init__(self, params: DecodeParams, *, q, k_cache, v_cache, block_table, plan, q_descale, k_descale, v_descale, o,
                 softmax_scale: float, lse=None, softcap: float = 0.0, window: int = 0, scale_o: float = 1.0, workspace=None,
                 status=None):
        import torch

        params = self._own(params)
        bf16, f32, i32, codes = _dtypes()
        nb, hk, hq = int(params.num_seqs), int(params.h_k), int(params.h_k) * int(params.h_r)
        n = int(q.shape[0])
        _tensor("q", q, codes if int(params.q_dtype) == MJ_E4M3 else (bf16,), (n, hq, 128), strided=True)
        if q.stride(2) != 1:
            raise ValueError("q: the head dimension must be contiguous")
        _tensor("o", o, (bf16,), (n, hq, 128), strided=True)
        if n and not o[0].is_contiguous():
            raise ValueError("o: a token's rows must be contiguous")
        if lse is not None:
            _tensor("lse", lse, (f32,), (n, hq))
        _check_pools(params, k_cache, v_cache)
        _tensor("block_table", block_table, (i32,), (nb, int(params.max_blocks)))
        for name, t in (("q_descale", q_descale), ("k_descale", k_descale), ("v_descale", v_descale)):
            _check_descale(name, t, nb, hk)
        _tensor("plan", plan, (torch.uint8,))
        if workspace is not None:
            _tensor("workspace", workspace, (torch.uint8,))
        _check_status(status)
        a = PromptArgs()
        a.q, a.q_tok, a.q_head = _ptr(q), int(q.stride(0)), int(q.stride(1))
        a.o, a.o_tok = _ptr(o), int(o.stride(0))
        a.lse, a.num_tokens = _ptr(lse), n
        a.k, a.v = _ptr(k_cache), _ptr(v_cache)
        a.k_page, a.k_row, a.k_head = kv_strides(k_cache)
        a.v_page, a.v_row, a.v_head = kv_strides(v_cache)
        a.block_table = _ptr(block_table)
        a.plan, a.plan_bytes = _ptr(plan), int(plan.numel())
        a.q_descale, a.k_descale, a.v_descale = _ptr(q_descale), _ptr(k_descale), _ptr(v_descale)
        a.qd_seq, a.qd_head = descale_strides(q_descale, nb, hk)
        a.kd_seq, a.kd_head = descale_strides(k_descale, nb, hk)
        a.vd_seq, a.vd_head = descale_strides(v_descale, nb, hk)
        a.softmax_scale, a.scale_o, a.softcap, a.window = float(softmax_scale), float(scale_o), float(softcap), int(window)
        if workspace is not None:
            a.workspace, a.workspace_bytes = _ptr(workspace), int(workspace.numel())
        a.status = _ptr(status)
        self._bind(lib().mj_prompt_attn, (ctypes.byref(params), ctypes.byref(a)),
                   (params, a, q, k_cache, v_cache, block_table, plan, q_descale, k_descale, v_descale, o, lse, workspace, status))


def prompt_attn(params: DecodeParams, *, stream=None, **tensors) -> None:
    """One PromptAttn call."""
    PromptAttn(params, **tensors)(stream)


class TreeCommit(_Call):
    """mj_tree_commit on device tensors: the rows of nodes accepted (num_seqs,
    max_accept) int32, num_accepted (num_seqs,) of each, move to the front of
    their trees (tree_lens (num_seqs,) int32; None: params.q_len nodes each);
    new_lens (num_seqs,) int32, None: seq_lens itself.  key_pos (num_seqs, h_k,
    slots) int32 moves along."""

    _name = "mj_tree_commit"

    def __init__(self, params: DecodeParams, *, k_cache, v_cache, block_table, seq_lens, accepted, num_accepted, tree_lens=None,
                 new_lens=None, key_pos=None, status=None, k_scales=None, v_scales=None):
        params = self._own(params)
        i32, codes = _dtypes()[2:]
        nb = int(params.num_seqs)
        new_lens = seq_lens if new_lens is None else new_lens
        _check_pools(params, k_cache, v_cache, _row_bytes(params))
        _check_tables(params, block_table, seq_lens)
        _tensor("accepted", accepted, (i32,), (nb, None))
        for name, t in (("num_accepted", num_accepted), ("new_lens", new_lens), ("tree_lens", tree_lens)):
            if t is not None:
                _tensor(name, t, (i32,), (nb,))
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if t is not None:
                _tensor(name, t, codes, (int(params.num_pages), int(params.h_k), int(params.page_size), 8), strided=True)
        _check_status(status)
        a = CommitArgs()
        a.k, a.v = _ptr(k_cache), _ptr(v_cache)
        a.k_page, a.k_row, a.k_head = kv_strides(k_cache)
        a.v_page, a.v_row, a.v_head = kv_strides(v_cache)
        a.block_table, a.seq_lens, a.tree_lens = _ptr(block_table), _ptr(seq_lens), _ptr(tree_lens)
        a.accepted, a.max_accept, a.num_accepted = _ptr(accepted), int(accepted.shape[1]), _ptr(num_accepted)
        a.new_lens = _ptr(new_lens)
        if key_pos is not None:
            a.kp_seq, a.kp_head = _per_slot("key_pos", key_pos, i32, params)
            a.key_pos = _ptr(key_pos)
        a.status = _ptr(status)
        _set_scales(a, k_scales, v_scales)
        self._bind(lib().mj_tree_commit, (ctypes.byref(params), ctypes.byref(a)),
                   (params, a, k_cache, v_cache, block_table, seq_lens, tree_lens, accepted, num_accepted, new_lens, key_pos,
                    status, k_scales, v_scales))


def tree_commit(params: DecodeParams, *, stream=None, **tensors) -> None:
    """One TreeCommit call."""
    TreeCommit(params, **tensors)(stream)
