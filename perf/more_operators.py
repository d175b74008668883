"""Cases of the operators a serving step needs around the paged e4m3 KV cache
beside the decode batch: pages handed out and taken back with the block tables
and slot maps that go with them, attention over whole prompts of different
lengths, attention of a drafted token tree, and the accepted branch's rows
moved to the front of the tree.

Inputs are random, made from a seed.  ``run`` computes a case in plain torch
operations, or (``own``) with the framework's calls.  d is 128 throughout.

Lengths are a function of the case alone.
"""

import math

import numpy as np
import torch

own = False

D = 128
CUDA = "cuda"


# ---------------------------------------------------------------- the cases


def _reserve(name, **kw):
    case = {"op": "reserve", "name": name, "seqs": 256, "new_lo": 1, "new_hi": 1, "len_lo": 512, "len_hi": 8192, "page": 16,
            "pad": 0}
    return {**case, **kw}


def _release(name, **kw):
    case = {"op": "release", "name": name, "seqs": 64, "len_lo": 512, "len_hi": 8192, "keep": 2048, "page": 16}
    return {**case, **kw}


def _prompt(name, **kw):
    case = {"op": "prompt", "name": name, "seqs": 5, "new_lo": 2001, "new_hi": 4001, "ctx_lo": 0, "ctx_hi": 0, "singles": 0,
            "h_k": 8, "h_r": 4, "page": 16, "causal": True, "window": 0, "cap": 0.0, "q8": False, "pad": 0}
    return {**case, **kw}


def _tree(name, **kw):
    case = {"op": "tree", "name": name, "seqs": 32, "q_len": 16, "h_k": 8, "h_r": 4, "page": 64, "len_lo": 2048,
            "len_hi": 32768, "ragged": False, "cap": 0.0, "window": 0, "q8": False}
    return {**case, **kw}


def _commit(name, **kw):
    case = {"op": "commit", "name": name, "seqs": 32, "q_len": 16, "accept": 5, "h_k": 8, "page": 64, "len_lo": 2048,
            "len_hi": 32768}
    return {**case, **kw}


def listed():
    return [
        # a decode batch's next step: a token more each, a new page where the last one is full
        _reserve("reserve_decode"),
        # prompts admitted together: their pages, tables and 65 thousand slots
        _reserve("reserve_prompts", seqs=33, new_lo=37, new_hi=4001, len_lo=0, len_hi=0, page=64, pad=61),
        # a decode batch's caches cut to 2048 keys: the pages behind go back
        _release("release_trim"),
        # the smallest prompt: one short sequence of one kv head
        _prompt("prompt_tiny", seqs=1, new_lo=37, new_hi=37, h_k=1, h_r=8),
        # five prompts of a batch, packed, written and attended whole
        _prompt("prompt_packed", pad=13),
        # a long prompt's chunk behind its cached beginning, in one batch with decode tokens of others
        _prompt("prompt_chunk_mixed", seqs=49, new_lo=2001, new_hi=2001, ctx_lo=512, ctx_hi=32768, singles=48, page=64),
        # e4m3 queries of a layer that sees the last 1024 keys, scores capped
        _prompt("prompt_window_cap_e4m3", seqs=3, new_lo=3001, new_hi=6001, window=1024, cap=50.0, q8=True, page=128),
        # one long prompt: the largest
        _prompt("prompt_long", seqs=1, new_lo=20001, new_hi=20001, page=128),
        # a small tree a sequence of a decode batch
        _tree("tree_small", seqs=64, q_len=4, page=16, len_lo=512, len_hi=8192),
        # speculative verification of trees of up to 61 tokens
        _tree("tree_verify", q_len=61, ragged=True),
        # the accepted branches of small trees
        _commit("commit_small"),
        # deep branches of wide trees, many sequences
        _commit("commit_deep", seqs=250, q_len=64, accept=13, page=16, len_lo=512, len_hi=8192),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("reserve", "release", "prompt", "prompt", "tree", "tree", "commit"))
    page = rng.choice((16, 32, 64, 128))
    h_k = rng.choice((1, 2, 3, 4, 8))
    h_r = rng.choice((1, 2, 4, 5, 8, 16))
    hi = _log_int(rng, 40, 65536)
    lo = rng.randrange(1, hi + 1)
    if op == "reserve":
        seqs = _log_int(rng, 1, 1000)
        room = max(1, 65000 // seqs)
        new_hi = 1 if rng.random() < 0.3 else _log_int(rng, 1, room)
        hi = max(1, min(hi, 4_000_000 // seqs))
        c = _reserve("", seqs=seqs, new_lo=rng.randrange(0, new_hi + 1), new_hi=new_hi, len_lo=rng.randrange(0, hi + 1),
                     len_hi=hi, page=page, pad=rng.choice((0, 0, 7, 100)))
    elif op == "release":
        seqs = _log_int(rng, 1, 1000)
        hi = max(1, min(hi, 4_000_000 // seqs))
        c = _release("", seqs=seqs, len_lo=rng.randrange(0, hi + 1), len_hi=hi, keep=rng.randrange(0, hi + 1), page=page)
    elif op == "commit":
        seqs = _log_int(rng, 1, 250)
        q_len = _log_int(rng, 2, 64)
        hi = max(q_len, min(hi, 2_000_000 // seqs))
        c = _commit("", seqs=seqs, q_len=q_len, accept=rng.randrange(1, max(1, q_len // 2) + 1), h_k=h_k, page=page,
                    len_lo=rng.randrange(q_len, hi + 1), len_hi=hi)
    elif op == "tree":
        q_len = _log_int(rng, 2, 64)
        hi = q_len + hi
        room = 3_500_000 // (h_k * max(1, -(-q_len * h_r // 32)))
        seqs = max(1, min(_log_int(rng, 1, 64), room // hi))
        c = _tree("", seqs=seqs, q_len=q_len, h_k=h_k, h_r=h_r, page=page, len_lo=rng.randrange(q_len, hi + 1), len_hi=hi,
                  ragged=rng.random() < 0.5, cap=rng.choice((0.0, 0.0, 20.0, 50.0)),
                  window=_log_int(rng, 128, hi + 64) if rng.random() < 0.3 else 0, q8=rng.random() < 0.3)
    else:
        new_hi = _log_int(rng, 1, 16000)
        ctx_hi = 0 if rng.random() < 0.4 else _log_int(rng, 1, 32768)
        most = 20001 * 20001 * 16 // (h_k * h_r)  # pairs of a token and a key, about the largest listed case's
        new_hi = max(1, min(new_hi, math.isqrt(most), most // (2 * ctx_hi + 1)))
        seqs = max(1, min(_log_int(rng, 1, 32), 60000 // new_hi, 200_000 // (ctx_hi + 1), most // (new_hi * (ctx_hi + new_hi))))
        causal = rng.random() < 0.8
        c = _prompt("", seqs=seqs, new_lo=rng.randrange(1, new_hi + 1), new_hi=new_hi, ctx_lo=rng.randrange(0, ctx_hi + 1),
                    ctx_hi=ctx_hi, singles=rng.randrange(0, seqs) if rng.random() < 0.3 else 0, h_k=h_k, h_r=h_r, page=page,
                    causal=causal, window=_log_int(rng, 64, 8000) if causal and rng.random() < 0.3 else 0,
                    cap=rng.choice((0.0, 0.0, 0.0, 30.0, 50.0)), q8=rng.random() < 0.3, pad=rng.choice((0, 0, 1, 61)))
    del c["name"]
    return c


def _spread(n, lo, hi):
    """n lengths over [lo, hi], the last one hi."""
    return [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n - 1)] + [hi]


def _lens(c):
    """Each sequence's keys (before a reservation or release, after the append of a prompt or a tree)."""
    if c["op"] != "prompt":
        return _spread(c["seqs"], c["len_lo"], c["len_hi"])
    return [x + n for x, n in zip(_spread(c["seqs"], c["ctx_lo"], c["ctx_hi"]), _news(c))]


def _news(c):
    """Each sequence's new tokens."""
    news = _spread(c["seqs"], c["new_lo"], c["new_hi"])
    return [1 if i < c.get("singles", 0) else n for i, n in enumerate(news)]


def _trees(c):
    """Each sequence's drafted tokens."""
    return [c["q_len"] if not c["ragged"] or i % 4 == 3 else 1 + (7 * i + 3) % c["q_len"] for i in range(c["seqs"])]


# ------------------------------------------------------------------- inputs


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=CUDA)


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


def _table(c, lens, seed, blocks, spare):
    """Sequences' pages in random order, and the pages no sequence holds."""
    need = [-(-n // c["page"]) for n in lens]
    pages = sum(need) + spare
    perm = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    table = np.full((c["seqs"], blocks), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at : at + n]
        at += n
    return torch.from_numpy(table).to(CUDA), torch.from_numpy(perm[at:]).to(CUDA), pages


def _pool(c, gen, lens, seed):
    s = {"c": c, "lens": lens, "seq_lens": _i32(lens)}
    s["table"], _, s["pages"] = _table(c, lens, seed, max(-(-n // c["page"]) for n in lens), 3)
    shape = (s["pages"], c["page"], c["h_k"], D)
    s["k"], s["v"] = _random_codes(gen, shape), _random_codes(gen, shape)
    s["kd"] = torch.rand(c["seqs"], c["h_k"], generator=gen, device=CUDA) * 0.75 + 0.25
    s["vd"] = torch.rand(c["seqs"], c["h_k"], generator=gen, device=CUDA) * 1.5 + 0.5
    return s


def prepare(case, seed):
    gen = torch.Generator(CUDA).manual_seed(seed)
    return {"reserve": _prepare_reserve, "release": _prepare_release, "prompt": _prepare_prompt, "tree": _prepare_tree,
            "commit": _prepare_commit}[case["op"]](case, gen, seed)


def _prepare_reserve(c, gen, seed):
    lens, news = _lens(c), _news(c)
    blocks = max(-(-(n + m) // c["page"]) for n, m in zip(lens, news)) + 1
    need = sum(-(-(n + m) // c["page"]) - -(-n // c["page"]) for n, m in zip(lens, news))
    s = {"c": c, "seq_lens": _i32(lens), "news": _i32(news)}
    s["table"], free, s["pages"] = _table(c, lens, seed, blocks, need + 5)
    s["free"] = torch.cat([free, torch.full((s["pages"] - free.numel(),), -1, dtype=torch.int32, device=CUDA)])
    s["num_free"] = _i32([free.numel()])
    tokens = sum(news) + c["pad"]
    s["num_free_out"], s["lens_out"] = torch.zeros_like(s["num_free"]), torch.zeros_like(s["seq_lens"])
    s["cu"] = torch.zeros(c["seqs"] + 1, dtype=torch.int32, device=CUDA)
    s["pos"] = torch.zeros(tokens, dtype=torch.int32, device=CUDA)
    s["slots"] = torch.zeros(tokens, dtype=torch.int64, device=CUDA)
    if own:
        import paged_fp8_kv_gb300 as mj

        s["call"] = mj.PagesReserve(
            mj.make_page_params(c["seqs"], c["page"], blocks, s["pages"]), seq_lens=s["seq_lens"], new_tokens=s["news"],
            free_pages=s["free"], num_free=s["num_free"], num_free_out=s["num_free_out"], block_table=s["table"],
            seq_lens_out=s["lens_out"], cu_tokens=s["cu"], positions=s["pos"], slots=s["slots"])
    return s


def _prepare_release(c, gen, seed):
    lens = _lens(c)
    blocks = max(1, max(-(-n // c["page"]) for n in lens))
    s = {"c": c, "seq_lens": _i32(lens), "keep": _i32([min(n, c["keep"]) for n in lens])}
    s["table"], free, s["pages"] = _table(c, lens, seed, blocks, 7)
    s["free"] = torch.cat([free, torch.full((s["pages"] - free.numel(),), -1, dtype=torch.int32, device=CUDA)])
    s["num_free"] = _i32([free.numel()])
    s["num_free_out"] = torch.zeros_like(s["num_free"])
    if own:
        import paged_fp8_kv_gb300 as mj

        s["call"] = mj.PagesRelease(
            mj.make_page_params(c["seqs"], c["page"], blocks, s["pages"]), seq_lens=s["seq_lens"], keep_lens=s["keep"],
            free_pages=s["free"], num_free=s["num_free"], num_free_out=s["num_free_out"], block_table=s["table"])
    return s


def _queries(c, gen, shape, per_row):
    """Queries and their descales; per_row broadcasts a (seqs, h_k) array over them."""
    q = 1.5 * torch.randn(shape, generator=gen, device=CUDA)
    qd = torch.ones(c["seqs"], c["h_k"], device=CUDA)
    if c["q8"]:
        qd = torch.rand(c["seqs"], c["h_k"], generator=gen, device=CUDA) + 0.5
        return (q / per_row(qd)).to(torch.float8_e4m3fn).view(torch.uint8), qd
    return q.to(torch.bfloat16), qd


def _prepare_prompt(c, gen, seed):
    news, h_q = _news(c), c["h_k"] * c["h_r"]
    s = _pool(c, gen, _lens(c), seed)
    total = sum(news)
    tokens = total + c["pad"]
    s["news"], s["starts"] = news, [sum(news[:b]) for b in range(c["seqs"])]
    s["cu"] = _i32(s["starts"] + [total])
    seq = torch.repeat_interleave(torch.arange(c["seqs"]), torch.tensor(news)).to(CUDA)
    seq = torch.cat([seq, seq.new_zeros(c["pad"])])
    q, s["qd"] = _queries(c, gen, (tokens, h_q, D), lambda d: d[seq].repeat_interleave(c["h_r"], 1)[..., None])
    s["q"] = q
    s["o"] = torch.zeros(tokens, h_q, D, dtype=torch.bfloat16, device=CUDA)
    s["lse"] = torch.zeros(tokens, h_q, device=CUDA)
    if own:
        import paged_fp8_kv_gb300 as mj

        params = mj.make_params(c["seqs"], 1, c["h_k"], c["h_r"], c["page"], int(s["table"].shape[1]), s["pages"],
                                causal=c["causal"], q_dtype=mj.MJ_E4M3 if c["q8"] else mj.MJ_BF16, max_splits=256)
        plan = torch.empty(mj.prompt_plan_bytes(params, tokens), dtype=torch.uint8, device=CUDA)
        mj.prompt_plan(params, cu_tokens=s["cu"], seq_lens=s["seq_lens"], num_tokens=tokens, window=c["window"], plan=plan)
        s["call"] = mj.PromptAttn(
            params, q=s["q"], k_cache=s["k"], v_cache=s["v"], block_table=s["table"], plan=plan, q_descale=s["qd"],
            k_descale=s["kd"], v_descale=s["vd"], o=s["o"], lse=s["lse"], softmax_scale=D**-0.5, softcap=c["cap"],
            window=c["window"],
            workspace=torch.empty(max(1, mj.prompt_workspace_bytes(params)), dtype=torch.uint8, device=CUDA))
    return s


def _parents(n, rng):
    """A tree of n tokens, level by level: node 0 is the root, a node's parent one of the last few levels' nodes."""
    return [-1] + [int(rng.integers(max(0, (i - 1) // 3 - 2), i)) for i in range(1, n)]


def _prepare_tree(c, gen, seed):
    s = _pool(c, gen, _lens(c), seed)
    rng = np.random.default_rng(seed)
    trees, n = _trees(c), c["q_len"]
    see = np.zeros((c["seqs"], n, n), dtype=bool)  # token i sees its ancestors and itself
    for b, t in enumerate(trees):
        for i, p in enumerate(_parents(t, rng)):
            if p >= 0:
                see[b, i] = see[b, p]
            see[b, i, i] = True
    words = -(-n // 32)
    bits = np.zeros((c["seqs"], n, words * 32), dtype=np.uint8)
    bits[:, :, :n] = see
    s["mask"] = torch.from_numpy(np.packbits(bits, axis=-1, bitorder="little").view(np.int32)).to(CUDA)
    s["trees"], s["tree_lens"] = trees, _i32(trees)
    s["first_key"] = None
    if c["window"]:  # the window ends at the token's own position, its depth behind the cached keys
        at = np.asarray(s["lens"])[:, None] - np.asarray(trees)[:, None] + see.sum(-1) - 1
        first = np.maximum(at - c["window"] + 1, 0)
        first = np.minimum(first, (np.asarray(s["lens"]) - np.asarray(trees))[:, None])
        s["first_key"] = torch.from_numpy(first.astype(np.int32)).to(CUDA)
    rows = n * c["h_r"]
    s["q"], s["qd"] = _queries(c, gen, (c["seqs"], c["h_k"], rows, D), lambda d: d[:, :, None, None])
    if own:
        import paged_fp8_kv_gb300 as mj

        params = mj.make_params(c["seqs"], n, c["h_k"], c["h_r"], c["page"], int(s["table"].shape[1]), s["pages"],
                                q_dtype=mj.MJ_E4M3 if c["q8"] else mj.MJ_BF16,
                                max_splits=256 if c["seqs"] * c["h_k"] <= 64 else 64)
        mod = mj.ScoreMod(softcap=c["cap"], key_begin=s["first_key"])
        spans, lens = None, s["lens"]
        if c["window"]:
            spans, lens = mj.score_spans(params, mod, s["lens"])
            spans = torch.from_numpy(spans).to(CUDA)
        plan = mj.decode_plan(params, lens)
        s["o"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=CUDA)
        s["lse"] = torch.empty(s["q"].shape[:3], device=CUDA)
        s["call"] = mj.DecodeAttnTree(
            params, mod, spans=spans, tree_mask=s["mask"], tree_lens=s["tree_lens"], q=s["q"], k_cache=s["k"], v_cache=s["v"],
            block_table=s["table"], seq_lens=s["seq_lens"], work=torch.from_numpy(plan.work).to(CUDA),
            n_splits=torch.from_numpy(plan.n_splits).to(CUDA), q_descale=s["qd"], k_descale=s["kd"], v_descale=s["vd"],
            o=s["o"], lse=s["lse"], softmax_scale=D**-0.5, max_n_splits=plan.max_n_splits,
            workspace=torch.empty(max(mj.workspace_bytes(params), 1), dtype=torch.uint8, device=CUDA))
    return s


def _prepare_commit(c, gen, seed):
    s = _pool(c, gen, _lens(c), seed)
    rng = np.random.default_rng(seed)
    # branches of trees laid out level by level whose first level is at least
    # as wide as a branch is long: the root, then nodes behind the first ones
    most = c["accept"]
    path = np.zeros((c["seqs"], most), dtype=np.int32)
    count = 1 + rng.integers(0, most, c["seqs"])
    count[-1] = most
    for b in range(c["seqs"]):
        path[b, 1:] = np.sort(rng.choice(np.arange(most, c["q_len"]), most - 1, replace=False))
    s["accepted"], s["num_accepted"] = torch.from_numpy(path).to(CUDA), _i32(count.tolist())
    s["tree_lens"] = _i32([c["q_len"]] * c["seqs"])
    s["new_lens"] = torch.zeros_like(s["seq_lens"])
    if own:
        import paged_fp8_kv_gb300 as mj

        params = mj.make_params(c["seqs"], c["q_len"], c["h_k"], 1, c["page"], int(s["table"].shape[1]), s["pages"])
        s["call"] = mj.TreeCommit(params, k_cache=s["k"], v_cache=s["v"], block_table=s["table"], seq_lens=s["seq_lens"],
                                  tree_lens=s["tree_lens"], accepted=s["accepted"], num_accepted=s["num_accepted"],
                                  new_lens=s["new_lens"])
    return s


# -------------------------------------------------------------------- a pass


def run(state):
    return {"reserve": _run_reserve, "release": _run_release, "prompt": _run_prompt, "tree": _run_tree,
            "commit": _run_commit}[state["c"]["op"]](state)


def _values(pool):
    return pool.view(torch.float8_e4m3fn)


def _run_reserve(s):
    out = {"table": s["table"], "lens": s["lens_out"], "num_free": s["num_free_out"], "cu": s["cu"], "pos": s["pos"],
           "slots": s["slots"]}
    if own:
        s["call"]()
        return out
    c, page = s["c"], s["c"]["page"]
    old, new = s["seq_lens"], s["seq_lens"] + s["news"]
    held, want = (old + page - 1) // page, (new + page - 1) // page
    end = torch.cumsum(want - held, 0)
    j = torch.arange(s["table"].shape[1], device=CUDA)
    grow = (j >= held[:, None]) & (j < want[:, None])
    at = s["num_free"] - 1 - ((end - (want - held))[:, None] + j - held[:, None])
    s["table"].copy_(torch.where(grow, s["free"][at.clamp(0, s["pages"] - 1)], s["table"]))
    s["lens_out"].copy_(new)
    s["num_free_out"].copy_(s["num_free"] - end[-1:])
    s["cu"][1:] = torch.cumsum(s["news"], 0)
    t = torch.arange(s["pos"].numel(), dtype=torch.int32, device=CUDA)
    b = torch.searchsorted(s["cu"][1:], t, right=True).clamp_max(c["seqs"] - 1)
    real = t < s["cu"][-1]
    pos = torch.where(real, old[b] + t - s["cu"][b], 0)
    s["pos"].copy_(pos)
    s["slots"].copy_(torch.where(real, s["table"][b, pos // page].long() * page + pos % page, -1))
    return out


def _run_release(s):
    out = {"free": s["free"], "num_free": s["num_free_out"]}
    if own:
        s["call"]()
        return out
    page = s["c"]["page"]
    held, keep = (s["seq_lens"] + page - 1) // page, (s["keep"] + page - 1) // page
    end = torch.cumsum(held - keep, 0)
    j = torch.arange(s["table"].shape[1], device=CUDA)
    gone = (j >= keep[:, None]) & (j < held[:, None])
    at = s["num_free"] + (end - (held - keep))[:, None] + j - keep[:, None]
    # entries that stay are written to one place behind the list
    room = torch.cat([s["free"], s["free"].new_zeros(1)])
    room.scatter_(0, torch.where(gone, at, s["pages"]).long().view(-1), s["table"].view(-1))
    s["free"].copy_(room[:-1])
    s["num_free_out"].copy_(s["num_free"] + end[-1:])
    return out


def _seq_rows(s, pool, b):
    """One sequence's rows, (h_k, L, d), 32 bits."""
    c, n = s["c"], s["lens"][b]
    at = s["table"][b, : -(-n // c["page"])].long()
    return _values(pool)[at].view(-1, c["h_k"], D)[:n].float().permute(1, 0, 2)


def _softmax_rows(z, seen, v):
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, torch.matmul(p, v) / total, 0.0)
    return o, (m + torch.log(total)).squeeze(-1)


def _cap(z, cap):
    return cap * torch.tanh(z / cap) if cap else z


def _run_prompt(s):
    out = {"o": s["o"], "lse": s["lse"]}
    if own:
        s["call"]()
        return out
    c, hr = s["c"], s["c"]["h_r"]
    q = _values(s["q"]) if c["q8"] else s["q"]
    for b, (n, t0, length) in enumerate(zip(s["news"], s["starts"], s["lens"])):
        k, v = _seq_rows(s, s["k"], b), _seq_rows(s, s["v"], b)
        step = max(1, (1 << 29) // (length * c["h_k"] * hr))  # tokens whose scores are held at once
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            first, last = length - n + i0, length - n + i1 - 1  # their positions
            a = max(0, first - c["window"] + 1) if c["window"] else 0
            e = last + 1 if c["causal"] else length
            x = q[t0 + i0 : t0 + i1].float().view(i1 - i0, c["h_k"], hr, D).permute(1, 0, 2, 3).reshape(c["h_k"], -1, D)
            z = torch.matmul(x, k[:, a:e].transpose(1, 2)) * (s["qd"][b] * s["kd"][b] / math.sqrt(D))[:, None, None]
            z = _cap(z, c["cap"])
            at = torch.arange(first, last + 1, device=CUDA).repeat_interleave(hr)[:, None]
            j = torch.arange(a, e, device=CUDA)
            seen = (j <= at if c["causal"] else j < length) & (j > at - (c["window"] or length + 1))
            o, lse = _softmax_rows(z, seen, v[:, a:e])
            o = (o * s["vd"][b][:, None, None]).view(c["h_k"], i1 - i0, hr, D).permute(1, 0, 2, 3)
            s["o"][t0 + i0 : t0 + i1] = o.reshape(i1 - i0, -1, D).to(torch.bfloat16)
            s["lse"][t0 + i0 : t0 + i1] = lse.view(c["h_k"], i1 - i0, hr).permute(1, 0, 2).reshape(i1 - i0, -1)
    return out


def _tree_seen(s, n):
    """(seqs, q_len, n) whether token i of each tree sees key j."""
    c = s["c"]
    j = torch.arange(n, device=CUDA)
    i = torch.arange(c["q_len"], device=CUDA)
    ctx = (s["seq_lens"] - s["tree_lens"])[:, None, None]
    node = (j - ctx).clamp(0, c["q_len"] - 1)
    word = s["mask"].gather(2, (node // 32).expand(-1, c["q_len"], -1).long())
    drafted = ((word >> (node % 32)) & 1).bool() & (j < s["seq_lens"][:, None, None])
    first = 0 if s["first_key"] is None else s["first_key"][:, :, None]
    return torch.where(j < ctx, j >= first, drafted) & (i[:, None] < s["tree_lens"][:, None, None])


def _run_tree(s):
    if own:
        s["call"]()
        return {"o": s["o"], "lse": s["lse"]}
    c = s["c"]
    n = max(s["lens"])
    blocks = -(-n // c["page"])
    at = s["table"][:, :blocks].clamp_min(0).long()
    rows = lambda pool: _values(pool)[at].view(c["seqs"], -1, c["h_k"], D)[:, :n].float().permute(0, 2, 1, 3)  # noqa: E731
    q = (_values(s["q"]) if c["q8"] else s["q"]).float()
    z = torch.matmul(q, rows(s["k"]).transpose(2, 3)) * (s["qd"] * s["kd"] / math.sqrt(D))[:, :, None, None]
    seen = _tree_seen(s, n).repeat_interleave(c["h_r"], 1)[:, None]
    v = torch.where((torch.arange(n, device=CUDA) < s["seq_lens"][:, None])[:, None, :, None], rows(s["v"]), 0.0)
    o, lse = _softmax_rows(_cap(z, c["cap"]), seen, v)
    return {"o": (o * s["vd"][:, :, None, None]).to(torch.bfloat16), "lse": lse}


def _run_commit(s):
    out = {"k": _values(s["k"]), "v": _values(s["v"]), "lens": s["new_lens"]}
    if own:
        s["call"]()
        return out
    c = s["c"]
    ctx = (s["seq_lens"] - s["tree_lens"])[:, None]
    i = torch.arange(c["accept"], dtype=torch.int32, device=CUDA)
    kept = i < s["num_accepted"][:, None]
    row = lambda slot: s["table"].gather(1, (slot // c["page"]).long()).long() * c["page"] + slot % c["page"]  # noqa: E731
    of = row(ctx + torch.where(kept, s["accepted"], i))  # what is not accepted stays where it is
    to = row(ctx + i)
    of = torch.where(kept, of, to)
    for pool in (s["k"], s["v"]):
        p = pool.view(-1, c["h_k"] * D)
        p[to.view(-1)] = p[of.view(-1)]
    s["new_lens"].copy_(ctx[:, 0] + s["num_accepted"])
    return out


# ------------------------------------------------------ the definition, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"reserve": _exact_reserve, "release": _exact_release, "prompt": _exact_prompt, "tree": _exact_tree,
            "commit": _exact_commit}[case["op"]](case, s)


def _exact_reserve(c, s):
    lens, news, page = s["seq_lens"].tolist(), s["news"].tolist(), c["page"]
    table, stack = s["table"].tolist(), s["free"][: int(s["num_free"])].tolist()
    cu, pos, slots, out = [0], [], [], []
    for b, (n, m) in enumerate(zip(lens, news)):
        held = -(-n // page)
        for t in range(n, n + m):
            if t // page >= held:
                table[b][held] = stack.pop()
                held += 1
            pos.append(t)
            slots.append(table[b][t // page] * page + t % page)
        cu.append(len(pos))
        out.append(n + m)
    i32 = dict(dtype=torch.int32)
    return {"table": torch.tensor(table, **i32), "lens": torch.tensor(out, **i32), "num_free": torch.tensor([len(stack)], **i32),
            "cu": torch.tensor(cu, **i32), "pos": torch.tensor(pos + [0] * c["pad"], **i32),
            "slots": torch.tensor(slots + [-1] * c["pad"], dtype=torch.int64)}


def _exact_release(c, s):
    lens, keep, page = s["seq_lens"].tolist(), s["keep"].tolist(), c["page"]
    table, count = s["table"].tolist(), int(s["num_free"])
    stack = s["free"].tolist()
    for b, (n, m) in enumerate(zip(lens, keep)):
        for j in range(-(-m // page), -(-n // page)):
            stack[count] = table[b][j]
            count += 1
    return {"free": torch.tensor(stack, dtype=torch.int32), "num_free": torch.tensor([count], dtype=torch.int32)}


def _rows64(s, pool, b):
    """One sequence's rows, (h_k, L, d)."""
    c, n = s["c"], s["lens"][b]
    j = torch.arange(n, device=pool.device)
    at = s["table"][b].long()[j // c["page"]] * c["page"] + j % c["page"]
    return pool.view(-1, c["h_k"], D)[at].view(torch.float8_e4m3fn).double().permute(1, 0, 2)


def _attend64(q, k, v, scale, cap, seen):
    """One head's rows: (rows, d) and their log sums."""
    z = (q @ k.T) * scale
    if cap:
        z = torch.tanh(z / cap) * cap
    z = z.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(z, -1)
    w = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return w @ v, lse


def _exact_prompt(c, s):
    o, lse = s["o"].double(), s["lse"].double()
    q = s["q"].view(torch.float8_e4m3fn) if c["q8"] else s["q"]
    for b, (n, t0, length) in enumerate(zip(s["news"], s["starts"], s["lens"])):
        k, v = _rows64(s, s["k"], b), _rows64(s, s["v"], b)
        for i0 in range(0, n, 2048):
            i1 = min(n, i0 + 2048)
            pos = torch.arange(length - n + i0, length - n + i1, device=CUDA)[:, None]
            end = int(pos[-1]) + 1 if c["causal"] else length
            j = torch.arange(end, device=CUDA)[None]
            seen = (j <= pos) if c["causal"] else torch.ones(i1 - i0, end, dtype=torch.bool, device=CUDA)
            if c["window"]:
                seen = seen & (pos - j < c["window"])
            for h in range(c["h_k"] * c["h_r"]):
                g = h // c["h_r"]
                scale = float(s["qd"][b, g].double() * s["kd"][b, g].double()) / math.sqrt(D)
                rows, sums = _attend64(q[t0 + i0 : t0 + i1, h].double(), k[g, :end], v[g, :end], scale, c["cap"], seen)
                o[t0 + i0 : t0 + i1, h] = rows * s["vd"][b, g].double()
                lse[t0 + i0 : t0 + i1, h] = sums
    return {"o": o, "lse": lse}


def _exact_tree(c, s):
    rows = c["q_len"] * c["h_r"]
    o = torch.zeros(c["seqs"], c["h_k"], rows, D, dtype=torch.float64, device=CUDA)
    lse = torch.full((c["seqs"], c["h_k"], rows), -math.inf, dtype=torch.float64, device=CUDA)
    mask = s["mask"].cpu().numpy().view(np.uint32)
    q = s["q"].view(torch.float8_e4m3fn) if c["q8"] else s["q"]
    for b, (t, n) in enumerate(zip(s["trees"], s["lens"])):
        see = np.ones((c["q_len"], n), dtype=bool)
        if s["first_key"] is not None:
            see &= np.arange(n)[None] >= s["first_key"][b].cpu().numpy()[:, None]
        for i in range(c["q_len"]):
            see[i, n - t :] = [(int(mask[b, i, m // 32]) >> (m % 32)) & 1 for m in range(t)]
        see[t:] = False
        seen = torch.from_numpy(np.repeat(see, c["h_r"], axis=0)).to(CUDA)
        k, v = _rows64(s, s["k"], b), _rows64(s, s["v"], b)
        for g in range(c["h_k"]):
            scale = float(s["qd"][b, g].double() * s["kd"][b, g].double()) / math.sqrt(D)
            x, sums = _attend64(q[b, g].double(), k[g], v[g], scale, c["cap"], seen)
            o[b, g], lse[b, g] = x * s["vd"][b, g].double(), sums
    return {"o": o, "lse": lse}


def _exact_commit(c, s):
    path, count, table = s["accepted"].tolist(), s["num_accepted"].tolist(), s["table"].tolist()
    page, to, of, lens = c["page"], [], [], []
    for b, n in enumerate(s["lens"]):
        ctx = n - c["q_len"]
        for i in range(count[b]):
            a, e = ctx + path[b][i], ctx + i
            of.append(table[b][a // page] * page + a % page)
            to.append(table[b][e // page] * page + e % page)
        lens.append(ctx + count[b])
    pools = []
    for pool in (s["k"], s["v"]):
        x = _values(pool).float().view(-1, c["h_k"], D)
        x[torch.tensor(to, device=CUDA)] = x[torch.tensor(of, device=CUDA)]
        pools.append(x.view(pool.shape))
    return {"k": pools[0], "v": pools[1], "lens": torch.tensor(lens, dtype=torch.int32)}


# ------------------------------------------------------------- what a pass needs


def work(case):
    c, lens, page = case, _lens(case), case["page"]
    if c["op"] == "reserve":
        news = _news(c)
        grown = sum(-(-(n + m) // page) - -(-n // page) for n, m in zip(lens, news))
        return {"bytes": 16 * c["seqs"] + 8 * grown + 12 * (sum(news) + c["pad"]), "flops": sum(news)}
    if c["op"] == "release":
        gone = sum(-(-n // page) - -(-min(n, c["keep"]) // page) for n in lens)
        return {"bytes": 8 * c["seqs"] + 8 * gone, "flops": c["seqs"]}
    if c["op"] == "commit":
        moved = (c["accept"] - 1) / 2 * (c["seqs"] - 1) + c["accept"] - 1  # branches are of 1 to `accept` tokens; the root stays
        return {"bytes": moved * c["h_k"] * 4 * D + c["seqs"] * 12, "flops": 0}
    q_bytes = 1 if c["q8"] else 2
    h_q = c["h_k"] * c["h_r"]
    if c["op"] == "tree":
        rows = sum(_trees(c)) * h_q
        keys = [min(n, c["window"] + c["q_len"]) if c["window"] else n for n in lens]
        pairs = sum(t * n for t, n in zip(_trees(c), keys)) * h_q
        read = sum(keys) * c["h_k"] * 2 * D
    else:
        rows = sum(_news(c)) * h_q
        pairs = read = 0
        for n, m in zip(lens, _news(c)):
            w = min(c["window"], n) if c["window"] else n
            below = max(0, min(m, w - (n - m)))  # tokens whose view is not cut by the window
            seen = n * m if not c["causal"] else below * (n - m) + below * (below + 1) // 2 + (m - below) * w
            pairs += seen * h_q
            read += min(n, w + m) * c["h_k"] * 2 * D
    return {"bytes": read + rows * (D * (q_bytes + 2) + 4), "flops": 4 * D * pairs}
