"""Shared pieces of the cache operators' GPU tests: workloads on the device,
and the float64 reference of a step with the bounds its roundings allow.

Bounds, per row n of one (sequence, kv head), from the arithmetic:

* a logit: the scores are exact products accumulated in fp32, but for bf16 Q's
  hi + lo e4m3 parts, which leave at most 2^-10 of a scaled element whose
  row-tile maximum is at least 128: |dq| <= 2^-17 amax(|Q tile|), so
  |ds| <= 2^-17 amax sum_d |k_d|; the fp32 sum of 128 products is within
  128 * 2^-24 of sum |q_d k_d|.  The modifiers are at most eight fp32
  operations on values up to |z| + cap + |bias| (2^-24 each), tanh to 2^-22 of
  the cap, exp2 to 2^-22:
     dz = scale (2^-17 amax sum|k| + 2^-17 sum|q k|) + 2^-20 (|z| + cap + |bias|) + 2^-21
* LSE: max over the visible keys of dz, and 2^-22 of itself.
* O: weights off by 2 dz, P as hi + lo e4m3 (2^-8 of an entry, through 11-bit
  halves: 2^-11, and e4m3's subnormal floor 2^-10 against a largest entry of
  at least 28), and the bf16 result (2^-8):
     dO = 2^-8 |O| + sum_j w_j |v_j| (2 dz + 2^-8 + 2^-10) + 2^-10/28 max_j w_j sum_j |v_j|
* a key's weight: sum_n w_nj (dz + 2^-20 (1 + |lse|)), and the sum's own
  roundings 2^-24 (rows) of it.
"""

from __future__ import annotations

import numpy as np
import torch

import paged_fp8_kv_gb300 as mj
from oracle import cache_ref
from paged_fp8_kv_gb300 import synthetic as syn
from paged_fp8_kv_gb300.session import DecodeSession
from tests.gpu_helpers import e4m3_view

QROWS = mj.MJ_KERNEL_TENSOR_CORE_QROWS


def make_mod(w, rng, softcap=0.0, alibi=False, window=0, docs=0, ends=False, prefix=0):
    """ScoreMod with device tensors, and the same on the host."""
    heads = w.h_k * w.h_r
    slopes = (2.0 ** (-8.0 * (np.arange(heads) + 1) / heads)).astype(np.float32) if alibi else None
    if alibi and heads > 1:
        slopes[0] = 0.0  # a head without a bias among the others
    begin = end = pre = None
    lens = np.asarray(w.seq_lens)[:, None]
    if docs:
        pos = np.maximum(lens - w.q_len + np.arange(w.q_len)[None], 0)
        begin = (pos // docs * docs).astype(np.int32)
        if ends:
            end = (begin + docs).astype(np.int32)
    if prefix:
        pre = rng.integers(0, prefix + 1, w.num_seqs).astype(np.int32)
    dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    mod = mj.ScoreMod(softcap=softcap, window=window, alibi_slopes=dev(slopes), key_begin=dev(begin), key_end=dev(end), prefix=dev(pre))
    host = dict(softcap=softcap, window=window, slopes=slopes, begin=begin, end=end, prefix=pre)
    return mod, host


def q_rows(w):
    """Packed Q values (b, h_k, n_q, d), float64."""
    x = cache_ref.values_of(w.q) if w.q_is_e4m3 else syn.bf16_bits_to_float(w.q).astype(np.float64)
    x = x.reshape(w.num_seqs, w.q_len, w.h_k, w.h_r, 128).transpose(0, 2, 1, 3, 4)
    return x.reshape(w.num_seqs, w.h_k, w.q_len * w.h_r, 128)


def _descale(d, b, g):
    d = np.asarray(d)
    return float(d.reshape(-1)[0]) if d.size == 1 else float(d[b, g] if d.ndim == 2 else d[g])


class Reference:
    """Float64 logits, weights, LSE and O of every (b, g), with their bounds."""

    def __init__(self, w, host):
        w = e4m3_view(w)
        kv, vv = cache_ref.values_of(w.k_cache), cache_ref.values_of(w.v_cache)
        q = q_rows(w)
        n_q = w.q_len * w.h_r
        self.o = np.zeros((w.num_seqs, w.h_k, n_q, 128))
        self.lse = np.full((w.num_seqs, w.h_k, n_q), -np.inf)
        self.d_o, self.d_lse = np.zeros_like(self.o), np.zeros((w.num_seqs, w.h_k, n_q))
        self.keys, self.d_keys = {}, {}  # (b, g) -> (L,) summed weights
        amax = np.abs(q).max(axis=(2, 3))  # >= that of any row tile of the head
        for b in range(w.num_seqs):
            L = int(w.seq_lens[b])
            arr = lambda x: None if x is None else x[b]  # noqa: E731
            see = cache_ref.visible(L, w.q_len, bool(w.causal), host["window"], arr(host["begin"]), arr(host["end"]),
                                    0 if host["prefix"] is None else int(host["prefix"][b]))
            see = np.repeat(see, w.h_r, axis=0)
            for g in range(w.h_k):
                k = cache_ref.cache_rows(kv, w.block_table[b], L, w.page_size, g)
                v = cache_ref.cache_rows(vv, w.block_table[b], L, w.page_size, g) * _descale(w.v_descale, b, g)
                scale = w.softmax_scale * _descale(w.q_descale, b, g) * _descale(w.k_descale, b, g)
                sl = None if host["slopes"] is None else host["slopes"][g * w.h_r : (g + 1) * w.h_r]
                z = cache_ref.logits(q[b, g], k, scale, host["softcap"], sl, L, w.q_len, w.h_r)
                zb = 0.0 if sl is None else z - cache_ref.logits(q[b, g], k, scale, host["softcap"], None, L, w.q_len, w.h_r)
                dz = (scale * 2.0**-17 * (amax[b, g] * np.abs(k).sum(1)[None] + np.abs(q[b, g]) @ np.abs(k).T)
                      + 2.0**-20 * (np.abs(z) + host["softcap"] + np.abs(zb)) + 2.0**-21)
                wt, lse = cache_ref.softmax_rows(z, see)
                self.lse[b, g] = lse
                fin = np.isfinite(lse)
                top = np.where(see, dz, 0.0).max(1, initial=0.0)
                self.d_lse[b, g] = top + 2.0**-22 * np.where(fin, np.abs(lse), 0.0)
                self.o[b, g] = wt @ v
                av = np.abs(v)
                self.d_o[b, g] = (2.0**-8 * np.abs(self.o[b, g]) + (wt * (2 * dz + 2.0**-8 + 2.0**-10)) @ av
                                  + 2.0**-10 / 28 * wt.max(1, initial=0.0)[:, None] * (see @ av))
                self.keys[b, g] = wt.sum(0)
                rel = dz + 2.0**-20 * (1 + np.where(fin, np.abs(lse), 0.0))[:, None] + n_q * 2.0**-24
                self.d_keys[b, g] = (wt * (rel + self.d_lse[b, g][:, None])).sum(0)

    def check(self, o, lse):
        assert not np.isnan(o).any(), "NaN in O"
        assert np.array_equal(np.isneginf(lse), np.isneginf(self.lse)), "rows without keys"
        fin = np.isfinite(self.lse)
        assert (np.abs(lse[fin] - self.lse[fin]) <= self.d_lse[fin]).all(), np.abs(lse[fin] - self.lse[fin]).max()
        bad = np.abs(o - self.o) > self.d_o
        assert not bad.any(), (np.argwhere(bad)[:4].tolist(), np.abs(o - self.o).max())
        assert (o[~fin] == 0).all()


class ModStep:
    """A workload's modified decode on the device: spans, plan and the call."""

    def __init__(self, w, mod, spans=True, force_splits=0, kv_layout="nhd", fill=float("nan"), kernel=QROWS):
        self.s = s = DecodeSession(w, kernel=kernel, kv_layout=kv_layout)
        self.w, self.mod = w, mod
        if w.q_len > 1:
            mj.pack_q(s.q_vllm, s.q_packed, w.num_seqs, w.q_len, w.h_k, w.h_r)
        self.spans, lens = None, w.seq_lens
        if spans:
            sp, lens = mj.score_spans(s.params, mod, w.seq_lens)
            self.spans = torch.from_numpy(sp).cuda()
        s.replan(lens, force_splits=force_splits)
        s.fill_workspace(fill)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        s.o_packed.fill_(float("nan"))
        s.lse.fill_(float("nan"))
        self.call = mj.DecodeAttnMod(
            s.params, mod, spans=self.spans, q=s.q_packed, k_cache=s.k_cache, v_cache=s.v_cache, block_table=s.block_table,
            seq_lens=s.seq_lens, work=s.work, n_splits=s.n_splits, q_descale=s.q_descale, k_descale=s.k_descale,
            v_descale=s.v_descale, o=s.o_packed, lse=s.lse, workspace=s.workspace, softmax_scale=w.softmax_scale,
            status=self.status, max_n_splits=s.plan.max_n_splits)

    def run(self):
        self.call()
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        return self.s.o_host(), self.s.lse_host()
