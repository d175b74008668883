"""Shared pieces of the serving operators' GPU tests: caches on the device, and
the float64 reference of an attention over them with the bounds its roundings
allow.

Bounds, per row of one (sequence, query head), from the arithmetic (2^-p is half
a step of a type with p bits):

* a logit: e4m3 codes are exact; bf16 Q is hi + lo e4m3 parts of the row (or
  row tile) scaled so that its largest element is at least 128, which leave at
  most 2^-10 of a scaled element: |dq| <= 2^-17 amax, so
  |ds| <= 2^-17 amax sum_d |k_d|; the fp32 sum of 128 products is within
  128 * 2^-24 of sum |q_d k_d|; the cap is at most eight fp32 operations on
  values up to |z| + cap (2^-24 each), tanh to 2^-22 of the cap, exp2 to 2^-22:
     dz = scale (2^-17 amax sum|k| + 2^-17 sum|q k|) + 2^-20 (|z| + cap) + 2^-21
* LSE: max over the visible keys of dz, and 2^-22 of itself.
* O: weights off by 2 dz; P rounded by ``p_rel`` of an entry, with a floor of
  ``p_floor`` of the row's largest entry; the accumulation in fp32 (2^-24 a key
  at most, of sums of |w v|: 2^-12 to 4096 keys); the bf16 result 2^-8:
     dO = 2^-8 |O| + sum_j w_j |v_j| (2 dz + p_rel + 2^-12) + p_floor max_j w_j sum_j |v_j|
  Half precision P (the prompt kernel): p_rel 2^-11, entries below 2^-21 of the
  reference keep 2^-32 of it.  Two e4m3 parts of P (the decode kernels): p_rel
  2^-8 + 2^-11, floor 2^-10 / 28.
"""

from __future__ import annotations

import numpy as np
import torch

import paged_fp8_kv_gb300 as mj

HALF_P = (2.0**-11, 2.0**-32)
SPLIT_P = (2.0**-8 + 2.0**-11, 2.0**-10 / 28)
I32 = dict(dtype=torch.int32, device="cuda")


class Cache:
    """Pools with sequences of `lens` keys on random pages; rows past each
    sequence's end and pages of no sequence hold NaN codes.  The first `ahead`
    pages are nobody's."""

    ahead = 0

    def __init__(self, lens, h_k, page, seed=0, extra_blocks=0, spread=1.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.h_k, self.page = list(lens), h_k, page
        need = [-(-n // page) for n in lens]
        self.num_pages = self.ahead + sum(need) + 3
        self.max_blocks = max(1, max(need)) + extra_blocks
        perm = self.ahead + rng.permutation(self.num_pages - self.ahead)
        table = rng.integers(-(2**31), 2**31 - 1, (len(lens), self.max_blocks)).astype(np.int32)  # never read past the end
        at = 0
        self.k, self.v = (torch.full((self.num_pages, page, h_k, 128), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        for b, n in enumerate(lens):
            table[b, : need[b]] = perm[at : at + need[b]]
            at += need[b]
            if n:
                slots = torch.arange(n, device="cuda")
                pages = torch.from_numpy(table[b].astype(np.int64)).cuda()[slots // page]
                for pool in (self.k, self.v):
                    x = spread * torch.randn(n, h_k, 128, generator=gen, device="cuda")
                    pool[pages, slots % page] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        self.table_host = table
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(self.lens, **I32)
        self.kd = torch.rand(len(lens), h_k, generator=gen, device="cuda") * 0.75 + 0.25
        self.vd = torch.rand(len(lens), h_k, generator=gen, device="cuda") * 1.5 + 0.5
        self.gen, self.rng = gen, rng

    def rows(self, pool, b):
        """(h_k, L, 128), float64."""
        n = self.lens[b]
        j = np.arange(n)
        at = torch.from_numpy(self.table_host[b, j // self.page].astype(np.int64) * self.page + j % self.page).cuda()
        return pool.view(-1, self.h_k, 128)[at].view(torch.float8_e4m3fn).double().permute(1, 0, 2)

    def queries(self, shape, e4m3, spread=1.5):
        q = spread * torch.randn(shape, generator=self.gen, device="cuda")
        return q.to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else q.to(torch.bfloat16)


def value_of(q):
    return q.view(torch.float8_e4m3fn).double() if q.dtype == torch.uint8 else q.double()


def attend(q, k, v, scale, seen, softcap, p_bounds, amax=None):
    """O, LSE of rows q (rows, 128) over k, v (keys, 128), and their bounds;
    amax: the largest |q| of the rows scaled together (None: each row's own)."""
    p_rel, p_floor = p_bounds
    raw = (q @ k.T) * scale
    z = torch.tanh(raw / softcap) * softcap if softcap else raw
    top = q.abs().amax(1) if amax is None else amax.expand(q.shape[0])
    dz = scale * 2.0**-17 * (top[:, None] * k.abs().sum(1)[None] + q.abs() @ k.abs().T)
    dz = dz + 2.0**-20 * (z.abs() + softcap) + 2.0**-21
    z = z.masked_fill(~seen, -np.inf)
    lse = torch.logsumexp(z, -1)
    fin = torch.isfinite(lse)
    w = torch.exp(z - torch.where(fin, lse, 0.0)[:, None])
    o = w @ v
    d_lse = torch.where(seen, dz, 0.0).amax(1) if dz.shape[1] else torch.zeros_like(lse)
    d_lse = d_lse + 2.0**-22 * torch.where(fin, lse.abs(), 0.0)
    av = v.abs()
    big = w.amax(1) if w.shape[1] else torch.zeros_like(lse)
    d_o = 2.0**-8 * o.abs() + (w * (2 * dz + p_rel + 2.0**-12)) @ av + p_floor * big[:, None] * (seen.double() @ av)
    return o, lse, d_o, d_lse


def check_rows(o, lse, ref, where=""):
    """Kernel rows against attend()'s."""
    o64, lse64, d_o, d_lse = ref
    fin = torch.isfinite(lse64)
    assert not torch.isnan(o).any(), f"{where}: NaN in O"
    off = (o.double() - o64).abs()
    bad = off > d_o
    assert not bad.any(), (where, torch.nonzero(bad)[:4].tolist(), off.max().item(), (off / d_o.clamp_min(1e-30)).max().item())
    assert (o[~fin] == 0).all(), f"{where}: rows without a key"
    if lse is not None:
        assert torch.equal(torch.isneginf(lse), ~fin), f"{where}: LSE of rows without a key"
        worst = ((lse.double() - lse64).abs() - d_lse)[fin]
        assert (worst <= 0).all(), (where, worst.max().item())
