"""Cases of the operators around the paged e4m3 KV cache: rotary positions
written into the cache, attention with modified scores over it, the weight
each cached key has received, and the eviction of the light ones.

Inputs are random, made from a seed.  ``run`` computes a case in plain torch
operations, or (``own``) with the framework's calls.  d is 128 throughout.

Lengths are a function of the case alone, spread over [len_lo, len_hi]; a case
with ``skew`` has one sequence of len_hi keys and the rest near len_lo.
"""

import math

import numpy as np
import torch

own = False

D = 128
E4M3_MAX = 448.0
CUDA = "cuda"


# ---------------------------------------------------------------- the cases


def _rope(name, **kw):
    case = {"op": "rope", "name": name, "seqs": 64, "q_len": 1, "h_k": 8, "h_r": 4, "page": 16, "len_lo": 512,
            "len_hi": 8192, "skew": False, "rot": 128, "axes": 1, "mixed": False, "pairs": False, "packed": True}
    return {**case, **kw}


def _attn(name, **kw):
    case = {"op": "attn", "name": name, "seqs": 64, "q_len": 1, "h_k": 8, "h_r": 4, "page": 16, "len_lo": 512,
            "len_hi": 8192, "skew": False, "cap": 0.0, "alibi": False, "window": 0, "prefix": 0, "doc": 0,
            "causal": True, "q8": False}
    return {**case, **kw}


def _weights(name, **kw):
    case = {"op": "weights", "name": name, "seqs": 64, "q_len": 1, "h_k": 8, "h_r": 4, "page": 16, "len_lo": 512,
            "len_hi": 8192, "skew": False, "cap": 0.0, "alibi": False, "window": 0, "decay": 1.0, "q8": False}
    return {**case, **kw}


def _evict(name, **kw):
    case = {"op": "evict", "name": name, "seqs": 64, "h_k": 8, "page": 16, "len_lo": 512, "len_hi": 8192,
            "skew": False, "budget": 2048, "first": 4, "last": 256}
    return {**case, **kw}


def listed():
    return [
        # one new token of each sequence of a decode batch: positions, cache write, Q packed
        _rope("rope_decode"),
        # drafted tokens under verification, positions in time, height and width whose frequencies alternate
        _rope("rope_verify_axes", seqs=32, q_len=4, h_r=8, page=64, len_lo=2048, len_hi=32768, axes=3, mixed=True),
        # prompts with images written whole: axes in sections, half of each head rotated, neighbouring pairs
        _rope("rope_prompt", seqs=5, q_len=3001, h_r=4, page=128, len_lo=3001, len_hi=9000, axes=3, rot=64,
              pairs=True, packed=False),
        # the smallest decode call: two short sequences of one kv head, capped scores and a distance bias
        _attn("attn_tiny", seqs=2, h_k=1, h_r=8, len_lo=37, len_hi=100, cap=30.0, alibi=True),
        # decode of a layer that sees the last 1024 keys, scores capped
        _attn("attn_window_cap", cap=50.0, window=1024),
        # speculative verification under a distance bias: the largest
        _attn("attn_verify_alibi", seqs=32, q_len=4, h_r=8, page=64, len_lo=2048, len_hi=32768, alibi=True),
        # one very long sequence among short ones, e4m3 queries, capped scores
        _attn("attn_skewed_cap_e4m3", seqs=8, h_k=1, h_r=16, page=128, len_lo=1000, len_hi=131072, skew=True,
              cap=30.0, q8=True),
        # a chunk of a prompt of several documents behind a shared prefix that every token sees
        _attn("attn_chunk_docs", seqs=6, q_len=61, h_k=2, h_r=4, page=32, len_lo=700, len_hi=6000, prefix=300,
              doc=1500),
        # a decode step's attention weights added to each cached key's
        _weights("weights_decode"),
        # the same for drafted tokens, capped scores, older weight fading
        _weights("weights_verify_cap", seqs=32, q_len=4, h_r=8, page=64, len_lo=2048, len_hi=32768, cap=50.0,
                 decay=0.97),
        # a decode batch's caches cut to 2048 keys a head
        _evict("evict_decode"),
        # long caches of few heads cut to a quarter
        _evict("evict_long", seqs=4, h_k=2, page=128, len_lo=60001, len_hi=131072, budget=32768, first=16, last=2048),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "attn", "weights", "evict"))
    page = rng.choice((16, 32, 64, 128))
    h_k = rng.choice((1, 2, 3, 4, 8))
    h_r = rng.choice((1, 2, 4, 5, 8, 16))
    seqs = _log_int(rng, 1, 64)
    if op == "rope":
        q_len = _log_int(rng, 1, 4096)
        seqs = max(1, min(seqs, 15000 * 12 // (q_len * h_k * (h_r + 2))))
        rot = rng.choice((32, 64, 96, 128))
        axes = rng.choice((1, 2, 3))
        c = _rope("", seqs=seqs, q_len=q_len, h_k=h_k, h_r=h_r, page=page, len_lo=q_len, len_hi=q_len + _log_int(rng, 1, 8000),
                  rot=rot, axes=axes, mixed=axes > 1 and rng.random() < 0.5, pairs=rng.random() < 0.5,
                  packed=q_len * h_r <= 4096 and rng.random() < 0.7)
    elif op == "evict":
        hi = _log_int(rng, 64, 65536)
        seqs = max(1, min(seqs, 4_000_000 // (hi * h_k)))
        budget = _log_int(rng, 32, hi)
        last = rng.randrange(0, budget // 2 + 1)
        first = rng.randrange(0, min(16, budget - last) + 1)
        c = _evict("", seqs=seqs, h_k=h_k, page=page, len_lo=rng.randrange(1, hi + 1), len_hi=hi,
                   skew=rng.random() < 0.2, budget=budget, first=first, last=last)
    else:
        q_len = 1 if rng.random() < 0.4 else _log_int(rng, 1, 64)
        hi = q_len + _log_int(rng, 32, 65536)
        room = 3_500_000 // (h_k * max(1, -(-q_len * h_r // 32)))
        seqs = max(1, min(seqs, room // hi))
        common = dict(seqs=seqs, q_len=q_len, h_k=h_k, h_r=h_r, page=page, len_lo=rng.randrange(q_len, hi + 1),
                      len_hi=hi, skew=rng.random() < 0.2, cap=rng.choice((0.0, 20.0, 30.0, 50.0)),
                      alibi=rng.random() < 0.4, window=_log_int(rng, 64, hi + 64) if rng.random() < 0.4 else 0,
                      q8=rng.random() < 0.3)
        if op == "attn":
            c = _attn("", **common)
            c["causal"] = c["window"] > 0 or rng.random() < 0.8
            if rng.random() < 0.4:
                c["prefix"] = _log_int(rng, 1, 2000)
            if rng.random() < 0.4:
                c["doc"] = _log_int(rng, 20, 4000)
        else:
            c = _weights("", **common)
            c["decay"] = rng.choice((0.0, 0.9, 1.0))
    del c["name"]
    return c


def _lens(c):
    """The sequences' lengths, by the case alone."""
    n, lo, hi = c["seqs"], c["len_lo"], c["len_hi"]
    if c["skew"]:
        return [hi] + [min(hi, lo + (37 * i) % 130) for i in range(1, n)]
    if n == 1:
        return [hi]
    return [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n - 1)] + [hi]


# ------------------------------------------------------------------- inputs


def _random_codes(gen, shape):
    """e4m3 codes of normal values, in blocks (the float form is large)."""
    out = torch.empty(shape, dtype=torch.uint8, device=CUDA)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, generator=gen, device=CUDA)
        flat[i : i + n] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _cache(c, gen, both=True):
    """Pools of K and V pages in random order, and the table that lists each sequence's."""
    lens, ps = _lens(c), c["page"]
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=gen, device=CUDA).to(torch.int32)
    table = torch.full((c["seqs"], max(need)), -1, dtype=torch.int32)
    at = torch.tensor([0] + need).cumsum(0).tolist()
    perm = perm.cpu()
    for b, n in enumerate(need):
        table[b, :n] = perm[at[b] : at[b] + n]
    s = {"lens": lens, "pages": pages, "table": table.to(CUDA), "seq_lens": torch.tensor(lens, dtype=torch.int32, device=CUDA)}
    shape = (pages, ps, c["h_k"], D)
    s["k"] = _random_codes(gen, shape)
    s["v"] = _random_codes(gen, shape) if both else s["k"]
    s["kd"] = torch.rand(c["seqs"], c["h_k"], generator=gen, device=CUDA) * 0.75 + 0.25
    s["vd"] = torch.rand(c["seqs"], c["h_k"], generator=gen, device=CUDA) * 1.5 + 0.5
    return s


def _queries(c, gen):
    n_q = c["q_len"] * c["h_r"]
    q = 1.5 * torch.randn(c["seqs"], c["h_k"], n_q, D, generator=gen, device=CUDA)
    qd = torch.ones(c["seqs"], c["h_k"], device=CUDA)
    if c["q8"]:
        qd = torch.rand(c["seqs"], c["h_k"], generator=gen, device=CUDA) + 0.5
        return (q / qd[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), qd
    return q.to(torch.bfloat16), qd


def _mods(c, s, gen):
    """What changes the scores: slopes per query head, each query token's first key, each sequence's prefix."""
    s["slopes"] = s["first_key"] = s["prefix"] = None
    heads = c["h_k"] * c["h_r"]
    if c["alibi"]:
        s["slopes"] = 2.0 ** (-8.0 * (torch.arange(heads, device=CUDA) + 1) / heads) * (0.75 + 0.5 * torch.rand(heads, generator=gen, device=CUDA))
    if c.get("doc"):  # documents of about `doc` keys: a token sees its own document's keys
        lens = s["seq_lens"].long()[:, None]
        pos = (lens - c["q_len"] + torch.arange(c["q_len"], device=CUDA)).clamp_min(0)
        jitter = torch.randint(0, c["doc"], (c["seqs"], 1), generator=gen, device=CUDA)
        start = (pos + jitter) // c["doc"] * c["doc"] - jitter
        s["first_key"] = start.clamp_min(0).to(torch.int32).contiguous()
    if c.get("prefix"):
        r = torch.randint(0, c["prefix"] + 1, (c["seqs"],), generator=gen, device=CUDA)
        s["prefix"] = torch.minimum(r, s["seq_lens"].long()).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(CUDA).manual_seed(seed)
    return {"rope": _prepare_rope, "attn": _prepare_attn, "weights": _prepare_weights, "evict": _prepare_evict}[case["op"]](case, gen)


def _prepare_rope(c, gen):
    s = {"c": c, **_cache(c, gen)}
    tokens, h_q, half = c["seqs"] * c["q_len"], c["h_k"] * c["h_r"], c["rot"] // 2
    qkv = torch.randn(tokens, h_q + 2 * c["h_k"], D, generator=gen, device=CUDA).to(torch.bfloat16)  # one projection's output
    s["q"], s["kn"], s["vn"] = qkv[:, :h_q], qkv[:, h_q : h_q + c["h_k"]], qkv[:, h_q + c["h_k"] :]
    max_pos = c["len_hi"] + 64
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=CUDA) / half)
    angle = torch.arange(max_pos, dtype=torch.float64, device=CUDA)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    pos = (s["seq_lens"].long()[:, None] - c["q_len"] + torch.arange(c["q_len"], device=CUDA)).reshape(1, -1)
    shift = torch.randint(0, 64, (c["axes"] - 1, tokens), generator=gen, device=CUDA)
    s["pos"] = torch.cat([pos, torch.where(shift < 32, pos, pos // 2 + shift)], 0).to(torch.int32).contiguous()
    third = -(-half // c["axes"])
    s["axis"] = [i % c["axes"] if c["mixed"] else min(i // third, c["axes"] - 1) for i in range(half)]  # each frequency's axis
    shape = (c["seqs"], c["h_k"], c["q_len"] * c["h_r"], D) if c["packed"] else (tokens, h_q, D)
    s["q_out"] = torch.zeros(shape, dtype=torch.bfloat16, device=CUDA)
    if own:
        import paged_fp8_kv_gb300 as mj

        params = mj.make_rope_params(c["seqs"], c["q_len"], c["h_k"], c["h_r"], c["page"], int(s["table"].shape[1]), s["pages"],
                                     rot_dim=c["rot"], n_axes=c["axes"], interleaved=c["pairs"], max_pos=max_pos)
        s["call"] = mj.RopeAppend(params, q=s["q"], k=s["kn"], v=s["vn"], positions=s["pos"], cos_sin=s["cos_sin"],
                                  freq_axis=s["axis"], q_out=s["q_out"], k_cache=s["k"], v_cache=s["v"],
                                  block_table=s["table"], seq_lens=s["seq_lens"], k_descale=s["kd"], v_descale=s["vd"])
    return s


def _decode_params(mj, c, s):
    return mj.make_params(c["seqs"], c["q_len"], c["h_k"], c["h_r"], c["page"], int(s["table"].shape[1]), s["pages"],
                          causal=c.get("causal", True), q_dtype=mj.MJ_E4M3 if c["q8"] else mj.MJ_BF16,
                          max_splits=256 if c["seqs"] * c["h_k"] <= 64 else 64)  # few heads: as many as the library takes


def _prepare_attn(c, gen):
    s = {"c": c, **_cache(c, gen)}
    s["q"], s["qd"] = _queries(c, gen)
    _mods(c, s, gen)
    if own:
        import paged_fp8_kv_gb300 as mj

        params = _decode_params(mj, c, s)
        mod = mj.ScoreMod(softcap=c["cap"], window=c["window"], alibi_slopes=s["slopes"], key_begin=s["first_key"], prefix=s["prefix"])
        spans, plan_lens = mj.score_spans(params, mod, s["lens"])
        plan = mj.decode_plan(params, plan_lens)
        s["o"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=CUDA)
        s["lse"] = torch.empty(s["q"].shape[:3], device=CUDA)
        ws = mj.workspace_bytes(params)
        s["call"] = mj.DecodeAttnMod(
            params, mod, spans=torch.from_numpy(spans).to(CUDA), q=s["q"], k_cache=s["k"], v_cache=s["v"], block_table=s["table"],
            seq_lens=s["seq_lens"], work=torch.from_numpy(plan.work).to(CUDA), n_splits=torch.from_numpy(plan.n_splits).to(CUDA),
            q_descale=s["qd"], k_descale=s["kd"], v_descale=s["vd"], o=s["o"], lse=s["lse"],
            workspace=torch.empty(max(ws, 1), dtype=torch.uint8, device=CUDA), softmax_scale=D**-0.5,
            max_n_splits=plan.max_n_splits)
    return s


def _prepare_weights(c, gen):
    s = {"c": c, **_cache(c, gen, both=False)}
    s["q"], s["qd"] = _queries(c, gen)
    _mods(c, s, gen)
    room = -(-c["len_hi"] // 64) * 64 + 64
    s["acc"] = torch.rand(c["seqs"], c["h_k"], room, generator=gen, device=CUDA) ** 4
    s["lse"] = _exact_lse(c, s)
    if own:
        import paged_fp8_kv_gb300 as mj

        params = _decode_params(mj, c, s)
        mod = mj.ScoreMod(softcap=c["cap"], window=c["window"], alibi_slopes=s["slopes"])
        plan = mj.decode_plan(params, s["lens"])
        s["call"] = mj.KeyWeights(
            params, mod, q=s["q"], k_cache=s["k"], block_table=s["table"], seq_lens=s["seq_lens"],
            work=torch.from_numpy(plan.work).to(CUDA), q_descale=s["qd"], k_descale=s["kd"], lse=s["lse"], acc=s["acc"],
            softmax_scale=D**-0.5, decay=c["decay"], fresh=c["q_len"])
    return s


def _prepare_evict(c, gen):
    s = {"c": c, **_cache(c, gen)}
    room = -(-c["len_hi"] // 64) * 64 + 64
    acc = torch.exp(2.0 * torch.randn(c["seqs"], c["h_k"], room, generator=gen, device=CUDA))
    coarse = torch.rand(acc.shape, generator=gen, device=CUDA) < 0.25  # equal weights among them
    s["acc"] = torch.where(coarse, torch.round(4 * acc) / 4, acc)
    s["acc_out"] = torch.zeros_like(s["acc"])
    # positions of a cache that was cut before: the first keys older, in no order
    pos = torch.arange(room, device=CUDA, dtype=torch.int32) + 100
    s["pos"] = (pos - torch.randint(0, 90, acc.shape, generator=gen, device=CUDA, dtype=torch.int32)).contiguous()
    s["pos_out"] = torch.zeros_like(s["pos"])
    s["next_pos"] = s["seq_lens"] + 100
    s["new_lens"] = torch.zeros_like(s["seq_lens"])
    if own:
        import paged_fp8_kv_gb300 as mj

        params = mj.make_params(c["seqs"], 1, c["h_k"], 1, c["page"], int(s["table"].shape[1]), s["pages"])
        ws = torch.empty(mj.evict_workspace_bytes(params, c["budget"]), dtype=torch.uint8, device=CUDA)
        s["call"] = mj.Evict(params, k_cache=s["k"], v_cache=s["v"], block_table=s["table"], seq_lens=s["seq_lens"],
                             acc=s["acc"], acc_out=s["acc_out"], key_pos=s["pos"], key_pos_out=s["pos_out"], next_pos=s["next_pos"],
                             new_lens=s["new_lens"], budget=c["budget"], keep_first=c["first"], keep_last=c["last"], workspace=ws)
    return s


# -------------------------------------------------------------------- a pass


def run(state):
    return {"rope": _run_rope, "attn": _run_attn, "weights": _run_weights, "evict": _run_evict}[state["c"]["op"]](state)


def _codes(x, descale):
    return (x / descale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(pool):
    return pool.view(torch.float8_e4m3fn)


def _rotate(x, cos, sin, rot, pairs):
    x = x.float()
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _run_rope(s):
    c = s["c"]
    if own:
        s["call"]()
        return {"q": s["q_out"], "k": _values(s["k"]), "v": _values(s["v"])}
    half, dev = c["rot"] // 2, s["q"].device
    axis = torch.tensor(s["axis"], device=dev)
    at = s["pos"].long()[axis].t()  # (tokens, half): each frequency's position
    f = torch.arange(half, device=dev)
    cos, sin = s["cos_sin"][at, f][:, None], s["cos_sin"][at, half + f][:, None]
    q = _rotate(s["q"], cos, sin, c["rot"], c["pairs"]).to(torch.bfloat16)
    if c["packed"]:
        q = q.view(c["seqs"], c["q_len"], c["h_k"], c["h_r"], D).transpose(1, 2).reshape(c["seqs"], c["h_k"], -1, D)
    seq = torch.arange(c["seqs"], device=dev).repeat_interleave(c["q_len"])
    slot = (s["seq_lens"].long()[:, None] - c["q_len"] + torch.arange(c["q_len"], device=dev)).reshape(-1)
    row = s["table"][seq, slot // c["page"]].long() * c["page"] + slot % c["page"]
    k = _rotate(s["kn"], cos, sin, c["rot"], c["pairs"])
    s["k"].view(-1, c["h_k"], D)[row] = _codes(k, s["kd"][seq][..., None])
    s["v"].view(-1, c["h_k"], D)[row] = _codes(s["vn"].float(), s["vd"][seq][..., None])
    return {"q": q, "k": _values(s["k"]), "v": _values(s["v"])}


def _gather(s, pool):
    """(seqs, h_k, longest, d) in 32 bits: each sequence's rows through the table."""
    c = s["c"]
    j = torch.arange(max(s["lens"]), device=pool.device)
    page = s["table"][:, j // c["page"]].clamp_min(0).long()
    return _values(pool[page, j % c["page"]]).float().transpose(1, 2)


def _scores(s, k):
    """The modified scores and which of them count: (seqs, h_k, rows, longest)."""
    c, dev = s["c"], k.device
    q = _values(s["q"]).float() if c["q8"] else s["q"].float()
    z = torch.matmul(q, k.transpose(2, 3)) * (D**-0.5 * s["qd"] * s["kd"])[:, :, None, None]
    if c["cap"]:
        z = c["cap"] * torch.tanh(z / c["cap"])
    n_q = c["q_len"] * c["h_r"]
    lens = s["seq_lens"].long()[:, None, None]
    token = torch.arange(n_q, device=dev) // c["h_r"]
    pos = lens - c["q_len"] + token[:, None]  # (seqs, rows, 1)
    j = torch.arange(k.shape[2], device=dev)
    if s["slopes"] is not None:
        slope = s["slopes"].view(c["h_k"], 1, c["h_r"]).expand(-1, c["q_len"], -1).reshape(1, c["h_k"], n_q, 1)
        z = z - slope * (pos - j).abs().float()[:, None]
    seen = (j < lens) & ((j <= pos) if c.get("causal", True) else (j >= 0))
    if c["window"]:
        seen = seen & (j > pos - c["window"])
    if s["first_key"] is not None:
        seen = seen & (j >= s["first_key"].long()[:, token][:, :, None])
    if s["prefix"] is not None:
        seen = seen | (j < s["prefix"].long()[:, None, None])
    return z, seen[:, None]


def _run_attn(s):
    if own:
        s["call"]()
        return {"o": s["o"], "lse": s["lse"]}
    z, seen = _scores(s, _gather(s, s["k"]))
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _gather(s, s["v"])) * s["vd"][:, :, None, None]
    o = torch.where(total > 0, o / total, 0.0)
    return {"o": o.to(torch.bfloat16), "lse": (m + torch.log(total)).squeeze(-1)}


def _run_weights(s):
    if own:
        s["call"]()
        return {"acc": s["acc"]}
    c = s["c"]
    k = _gather(s, s["k"])
    z, seen = _scores(s, k)
    lse = s["lse"][..., None]
    w = torch.where(seen & (lse > -math.inf), torch.exp(z - lse), 0.0).sum(2)
    n, j = k.shape[2], torch.arange(k.shape[2], device=k.device)
    lens = s["seq_lens"].long()[:, None, None]
    acc = s["acc"][:, :, :n]
    old = torch.where(j < lens - c["q_len"], c["decay"] * acc, 0.0)
    acc.copy_(torch.where(j < lens, old + w, acc))
    return {"acc": s["acc"]}


def _run_evict(s):
    if own:
        s["call"]()
        return {"k": _values(s["k"]), "v": _values(s["v"]), "acc": s["acc_out"], "pos": s["pos_out"], "lens": s["new_lens"]}
    c, dev = s["c"], s["acc"].device
    n = max(s["lens"])
    lens = s["seq_lens"].long()[:, None, None]
    new = lens.clamp_max(c["budget"])
    j = torch.arange(n, device=dev)
    acc, pos = s["acc"][:, :, :n], s["pos"][:, :, :n]
    held = (pos < c["first"]) | (pos >= (s["next_pos"] - c["last"])[:, None, None])
    rank = torch.where(j < lens, torch.where(held, math.inf, acc), -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    keep = torch.zeros(rank.shape, dtype=torch.bool, device=dev).scatter_(-1, order, (j < new).expand(rank.shape))
    keep = keep & (j < lens)
    hole, mover = ~keep & (j < new), keep & (j >= new)  # the i-th hole takes the i-th row from behind
    dst, src = hole.nonzero(), mover.nonzero()
    b, g = dst[:, 0], dst[:, 1]
    row = lambda at: s["table"][at[:, 0], at[:, 2] // c["page"]].long() * c["page"] + at[:, 2] % c["page"]  # noqa: E731
    to, of = row(dst), row(src)
    for_all = torch.where(j < new, 1, 0).bool().expand(rank.shape)
    s["acc_out"][:, :, :n] = torch.where(for_all, acc, s["acc_out"][:, :, :n])
    s["pos_out"][:, :, :n] = torch.where(for_all, pos, s["pos_out"][:, :, :n])
    s["acc_out"][b, g, dst[:, 2]] = acc[b, g, src[:, 2]]
    s["pos_out"][b, g, dst[:, 2]] = pos[b, g, src[:, 2]]
    k, v = s["k"].view(-1, c["h_k"], D), s["v"].view(-1, c["h_k"], D)
    k[to, g] = k[of, g]
    v[to, g] = v[of, g]
    s["new_lens"].copy_(new.view(-1))
    return {"k": _values(s["k"]), "v": _values(s["v"]), "acc": s["acc_out"], "pos": s["pos_out"], "lens": s["new_lens"]}


# ------------------------------------------------------ the definition, in 64 bits


def _rows64(s, pool, b):
    """One sequence's rows, (h_k, L, d)."""
    c, n = s["c"], s["lens"][b]
    j = torch.arange(n, device=pool.device)
    at = s["table"][b].long()[j // c["page"]] * c["page"] + j % c["page"]
    return pool.view(-1, c["h_k"], D)[at].view(torch.float8_e4m3fn).double().permute(1, 0, 2)


def _logits64(s, b):
    """(h_k, rows, L) logits of sequence b, minus infinity where a row does not see a key."""
    c, n = s["c"], s["lens"][b]
    dev = s["k"].device
    q = s["q"][b].view(torch.float8_e4m3fn).double() if c["q8"] else s["q"][b].double()
    z = torch.einsum("gnd,gjd->gnj", q, _rows64(s, s["k"], b))
    z *= (s["qd"][b].double() * s["kd"][b].double() / math.sqrt(D))[:, None, None]
    if c["cap"]:
        z = torch.tanh(z / c["cap"]) * c["cap"]
    i = torch.arange(c["q_len"], device=dev).repeat_interleave(c["h_r"])[:, None]
    at, j = n - c["q_len"] + i, torch.arange(n, device=dev)[None]
    if s["slopes"] is not None:
        per_row = s["slopes"].double().view(c["h_k"], c["h_r"]).repeat(1, c["q_len"])
        z -= per_row[:, :, None] * (at - j).abs().double()
    lo = torch.zeros_like(at)
    if c["window"]:
        lo = torch.maximum(lo, at - c["window"] + 1)
    if s["first_key"] is not None:
        lo = torch.maximum(lo, s["first_key"][b].long()[i])
    hi = at if c.get("causal", True) else torch.full_like(at, n - 1)
    seen = (j >= lo) & (j <= hi)
    if s["prefix"] is not None:
        seen |= j < int(s["prefix"][b])
    return z.masked_fill(~seen, -math.inf)


def _exact_lse(c, s):
    return torch.stack([torch.logsumexp(_logits64(s, b), -1) for b in range(c["seqs"])]).float()


def _round_e4m3(x):
    """Nearest e4m3 value, ties to even, saturating."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0**-6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](case, s)


def _exact_rope(c, s):
    half, ps = c["rot"] // 2, c["page"]
    cs = s["cos_sin"].double().cpu().numpy()
    pos = s["pos"].cpu().numpy()
    f = np.arange(half)
    cos = torch.from_numpy(np.stack([cs[pos[a], i] for i, a in zip(f, s["axis"])], 1)).to(CUDA)
    sin = torch.from_numpy(np.stack([cs[pos[a], half + i] for i, a in zip(f, s["axis"])], 1)).to(CUDA)
    first = torch.arange(half, device=CUDA) * 2 if c["pairs"] else torch.arange(half, device=CUDA)
    second = first + (1 if c["pairs"] else half)

    def turn(x):
        x = x.double()
        y, a, b = x.clone(), x[:, :, first], x[:, :, second]
        y[:, :, first] = a * cos[:, None] - b * sin[:, None]
        y[:, :, second] = a * sin[:, None] + b * cos[:, None]
        return y

    q, kn, vn = turn(s["q"]), turn(s["kn"]), s["vn"].double()
    if c["packed"]:
        q = torch.stack([q[b * c["q_len"] : (b + 1) * c["q_len"]].view(c["q_len"], c["h_k"], c["h_r"], D).permute(1, 0, 2, 3).reshape(c["h_k"], -1, D)
                         for b in range(c["seqs"])])
    pools = []
    for pool, x, d in ((s["k"], kn, s["kd"]), (s["v"], vn, s["vd"])):
        out = _values(pool).float().view(-1, c["h_k"], D)
        for b, n in enumerate(s["lens"]):
            j = torch.arange(n - c["q_len"], n, device=CUDA)
            at = s["table"][b].long()[j // ps] * ps + j % ps
            out[at] = _round_e4m3(x[b * c["q_len"] : (b + 1) * c["q_len"]] / d[b].double()[:, None]).float()
        pools.append(out.view(pool.shape))
    return {"q": q, "k": pools[0], "v": pools[1]}


def _exact_attn(c, s):
    o, lse = [], []
    for b in range(c["seqs"]):
        z = _logits64(s, b)
        total = torch.logsumexp(z, -1)
        w = torch.exp(z - torch.where(total == -math.inf, 0.0, total)[..., None])
        o.append((w @ _rows64(s, s["v"], b)) * s["vd"][b].double()[:, None, None])
        lse.append(total)
    return {"o": torch.stack(o), "lse": torch.stack(lse)}


def _exact_weights(c, s):
    acc = s["acc"].double()
    for b, n in enumerate(s["lens"]):
        z, lse = _logits64(s, b), s["lse"][b].double()[..., None]
        w = torch.exp(z - lse).masked_fill(lse == -math.inf, 0.0).sum(1)
        acc[b, :, max(0, n - c["q_len"]) : n] = 0.0
        acc[b, :, : max(0, n - c["q_len"])] *= c["decay"]
        acc[b, :, :n] += w
    return {"acc": acc}


def _exact_evict(c, s):
    acc, pos = s["acc"].cpu().numpy(), s["pos"].cpu().numpy()
    acc_out, pos_out = s["acc_out"].cpu().numpy().astype(np.float64), s["pos_out"].cpu().numpy()
    table, ps = s["table"].cpu().numpy(), c["page"]
    k, v = s["k"].view(-1, c["h_k"], D), s["v"].view(-1, c["h_k"], D)
    ends, lens = s["next_pos"].tolist(), []
    for b, n in enumerate(s["lens"]):
        new = min(n, c["budget"])
        lens.append(new)
        for g in range(c["h_k"]):
            w = acc[b, g, :n].astype(np.float64)
            w[(pos[b, g, :n] < c["first"]) | (pos[b, g, :n] >= ends[b] - c["last"])] = np.inf
            kept = np.sort(np.lexsort((np.arange(n), -w))[:new])
            holes, movers = np.setdiff1d(np.arange(new), kept), kept[kept >= new]
            slots = np.arange(new)
            slots[holes] = movers
            acc_out[b, g, :new], pos_out[b, g, :new] = acc[b, g, slots], pos[b, g, slots]
            to, of = (torch.from_numpy(table[b, x // ps].astype(np.int64) * ps + x % ps).to(CUDA) for x in (holes, movers))
            k[to, g], v[to, g] = k[of, g], v[of, g]
    return {"k": _values(s["k"]).float(), "v": _values(s["v"]).float(), "acc": torch.from_numpy(acc_out).float(),
            "pos": torch.from_numpy(pos_out), "lens": torch.tensor(lens, dtype=torch.int32)}


# ------------------------------------------------------------- what a pass needs


def _seen_keys(c):
    """Keys that some query token of each sequence sees, summed (documents and prefixes by their mean)."""
    total = 0
    for n in _lens(c):
        see = n
        if c["window"]:
            see = min(see, c["window"] + c["q_len"] - 1)
        if c.get("doc"):
            see = min(see, c["doc"] // 2 + c["q_len"])
        if c.get("prefix"):
            see = min(n, see + c["prefix"] // 2)
        total += see
    return total


def work(case):
    c = case
    lens = _lens(c)
    if c["op"] == "rope":
        tokens = c["seqs"] * c["q_len"]
        elems = tokens * c["h_k"] * (c["h_r"] + 1) * c["rot"]
        bytes_ = tokens * c["h_k"] * D * (4 * c["h_r"] + 6) + tokens * c["axes"] * 4
        tables = min(tokens * c["axes"], c["len_hi"] + 64) * c["rot"] * 4
        return {"bytes": bytes_ + tables, "flops": 3 * elems}
    if c["op"] == "evict":
        moved = kept = 0.0
        for n in lens:
            new = min(n, c["budget"])
            kept += new
            if n > new:
                behind = min(c["last"], n - new)
                free = max(0.0, new - c["last"])
                moved += behind + free * max(0, n - new - c["last"]) / max(1, n - c["last"])
        return {"bytes": c["h_k"] * (8 * sum(lens) + 8 * kept + moved * 4 * D), "flops": c["h_k"] * sum(lens)}
    rows = c["q_len"] * c["h_r"]
    q = c["seqs"] * c["h_k"] * rows * D * (1 if c["q8"] else 2)
    if c["op"] == "attn":
        keys = _seen_keys(c) * c["h_k"]
        return {"bytes": keys * 2 * D + q + c["seqs"] * c["h_k"] * rows * (2 * D + 4), "flops": 4 * D * keys * rows}
    keys = sum(lens) * c["h_k"]
    seen = _seen_keys(c) * c["h_k"]
    return {"bytes": seen * D + keys * (8 if c["decay"] else 4) + q + c["seqs"] * c["h_k"] * rows * 4, "flops": 2 * D * seen * rows}
