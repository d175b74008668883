"""GPU parity of the rotary append (mj_rope_append) against the float64
reference: pair layouts, partial rotation, axes, ragged and padded batches,
strided inputs, pool layouts, the token and packed outputs, bad pages and
positions, key positions.

Bounds: q is fp32 arithmetic (two products and a sum, 3 * 2^-24 of |a| + |b|)
rounded to bf16 (2^-8 relative).  A code is the rounding of a value that is
within 4 * 2^-24 (|a| + |b|) / descale of the exact one: it equals the exact
code unless the exact value lies that near a border."""

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from oracle import cache_ref
from paged_fp8_kv_gb300 import synthetic as syn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Case:
    def __init__(self, news, olds, h_k=2, h_r=3, page_size=16, rot=128, axes=1, mixed=False, pairs=False, packed=False, pad=0,
                 ragged=None, layout="nhd", slices=True, seed=0, max_pos=300):
        rng = np.random.default_rng(seed)
        self.__dict__.update(locals())
        b = len(news)
        self.b = b
        q_len = news[0]
        ragged = len(set(news)) > 1 or pad > 0 if ragged is None else ragged
        self.lens = np.asarray([o + n for o, n in zip(olds, news)], dtype=np.int32)
        self.cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        n = self.n = int(self.cu[-1]) + pad
        h_q = h_k * h_r
        width = h_q + 2 * h_k if slices else 0
        x = syn.bf16_encode(rng.standard_normal((n, h_q + 2 * h_k, 128)).astype(np.float32) * 2)
        self.x = syn.bf16_bits_to_float(x).astype(np.float64)
        t = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
        parts = [t[:, :h_q], t[:, h_q : h_q + h_k], t[:, h_q + h_k :]]
        if not width:
            parts = [p.contiguous() for p in parts]
        self.q, self.k, self.v = parts
        self.pos = rng.integers(0, max_pos, (axes, n)).astype(np.int32)
        half = rot // 2
        self.axis = np.asarray([i % axes if mixed else min(i * axes // half, axes - 1) for i in range(half)])
        ang = rng.uniform(-20, 20, (max_pos, half))
        self.table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.kd = rng.uniform(0.01, 0.6, (b, h_k)).astype(np.float32)  # some codes saturate
        self.vd = rng.uniform(0.005, 2, (b, h_k)).astype(np.float32)
        need = [max(1, -(-int(L) // page_size)) for L in self.lens]
        self.max_blocks = max(need) + 1
        pages = self.pages = sum(need) + 3
        perm = rng.permutation(pages)
        self.bt = np.full((b, self.max_blocks), -1, dtype=np.int32)
        at = 0
        for i, m in enumerate(need):
            self.bt[i, :m] = perm[at : at + m]
            at += m
        codes = rng.integers(0, 256, (2, pages, page_size, h_k, 128)).astype(np.uint8)
        kv = torch.from_numpy(codes).cuda()
        if layout == "hnd":
            buf = kv.permute(1, 0, 3, 2, 4).contiguous()  # (pages, 2, h_k, ps, d)
            self.kc, self.vc = buf[:, 0].transpose(1, 2), buf[:, 1].transpose(1, 2)
        elif layout == "interleaved":
            buf = torch.cat([kv[0], kv[1]], -1).transpose(1, 2).contiguous().transpose(1, 2)
            self.kc, self.vc = buf[..., :128], buf[..., 128:]
        else:
            self.kc, self.vc = kv[0], kv[1]
        self.before = codes
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        shape = (b, h_k, q_len * h_r, 128) if packed else (n, h_q, 128)
        self.q_out = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        self.key_pos = torch.full((b, h_k, self.max_blocks * page_size), -9, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.params = mj.make_rope_params(b, q_len, h_k, h_r, page_size, self.max_blocks, pages, rot_dim=rot, n_axes=axes,
                                          interleaved=pairs, max_pos=max_pos)
        self.dev = dict(positions=dev(self.pos), cos_sin=dev(self.table), block_table=dev(self.bt), seq_lens=dev(self.lens),
                        k_descale=dev(self.kd), v_descale=dev(self.vd), cu_tokens=dev(self.cu) if ragged else None)

    def call(self, **kw):
        args = dict(q=self.q, k=self.k, v=self.v, q_out=self.q_out, k_cache=self.kc, v_cache=self.vc, freq_axis=self.axis,
                    key_pos=self.key_pos, status=self.status, **self.dev)
        args.update(kw)
        return mj.RopeAppend(self.params, **args)

    def check(self, skip_tokens=(), skip_rows=(), status=0):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        h_q, h_k, h_r = self.h_k * self.h_r, self.h_k, self.h_r
        y = cache_ref.rotate(self.x[:, : h_q + h_k], self.pos, self.table, self.axis, self.rot, self.pairs)
        # |a| + |b| of each element's pair
        mag = np.zeros_like(y)
        half = self.rot // 2
        for i in range(half):
            a, c = (2 * i, 2 * i + 1) if self.pairs else (i, i + half)
            mag[:, :, a] = mag[:, :, c] = np.abs(self.x[:, : h_q + h_k, a]) + np.abs(self.x[:, : h_q + h_k, c])
        got = self.q_out.float().cpu().numpy().astype(np.float64)
        used = int(self.cu[-1])
        if self.packed:
            q_len = self.news[0]
            got = got.reshape(self.b, h_k, q_len, h_r, 128).transpose(0, 2, 1, 3, 4).reshape(self.n, h_q, 128)
        live = [t for t in range(used) if t not in skip_tokens]
        err = np.abs(got[live] - y[live, :h_q])
        assert (err <= 2.0**-8 * np.abs(y[live, :h_q]) + 2.0**-21 * mag[live, :h_q]).all(), err.max()
        rest = [t for t in range(self.n) if t not in live]
        assert (got[rest] == 7.0).all()
        # the pools: every row a token owns, and nothing else
        kc, vc = self.kc.cpu().numpy(), self.vc.cpu().numpy()
        untouched = np.ones(kc.shape[:2], dtype=bool)
        key_pos = np.full(self.key_pos.shape, -9)
        vals = cache_ref.values_of
        for t, b, i, slot, page, r in cache_ref.append_slots(self.lens, self.cu, used, self.bt, self.page_size):
            if t in skip_tokens or (b, slot) in skip_rows:
                continue
            untouched[page, r] = False
            key_pos[b, :, slot] = self.pos[0, t]
            for g in range(h_k):
                for got_c, x, m, d in ((kc, y[t, h_q + g], mag[t, h_q + g], self.kd[b, g]),
                                       (vc, self.x[t, h_q + h_k + g], 0.0, self.vd[b, g])):
                    exact, slack = x / float(d), 2.0**-22 * (m + np.abs(x)) / float(d)
                    lo, hi = cache_ref.round_e4m3(exact - slack), cache_ref.round_e4m3(exact + slack)
                    v = vals(got_c[page, r, g])
                    assert ((v >= lo) & (v <= hi)).all(), (t, g)
        assert np.array_equal(kc[untouched], self.before[0][untouched])
        assert np.array_equal(vc[untouched], self.before[1][untouched])
        assert np.array_equal(self.key_pos.cpu().numpy(), key_pos)


@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("rot", [16, 32, 64, 96, 128])
@pytest.mark.parametrize("axes,mixed", [(1, False), (3, False), (3, True), (4, True)])
def test_rotation_forms(pairs, rot, axes, mixed):
    c = Case([3, 3], [20, 0], rot=rot, axes=axes, mixed=mixed, pairs=pairs, packed=True, seed=rot + axes)
    c.call()()
    c.check()


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "interleaved"])
def test_pages_and_layouts(page_size, layout):
    c = Case([40, 40, 40], [0, 5, 130], page_size=page_size, layout=layout, seed=page_size)
    c.call()()
    c.check()


@pytest.mark.parametrize("h_k,h_r", [(1, 1), (1, 16), (8, 4), (8, 8), (3, 5), (8, 17)])
def test_heads_and_single_tokens(h_k, h_r):
    c = Case([1] * 9, [0, 1, 15, 16, 17, 31, 100, 127, 128], h_k=h_k, h_r=h_r, packed=True, axes=3, slices=h_r != 4)
    c.call()()
    c.check()


def test_ragged_padded_and_empty_sequences():
    c = Case([5, 0, 1, 17, 0], [3, 9, 0, 31, 0], pad=6, axes=2, mixed=True)
    c.pos[:, -6:] = -123  # a padding token's position is nobody's
    c.dev["positions"].copy_(torch.from_numpy(c.pos))
    c.call()()
    c.pos[:, -6:] = 0
    c.check()


def test_long_ragged_prompts():
    """Several tokens a CTA, sequences ending inside one."""
    for h_r in (2, 6):  # 12 and 6 tokens a CTA would have room for
        c = Case([9001, 1, 12003], [0, 5, 77], h_k=1, h_r=h_r, axes=3, page_size=64, pad=5, max_pos=2000)
        c.call()()
        c.check()


def test_more_new_tokens_than_the_length_counts():
    """Rows whose slot would be negative: Q is written, no cache row is."""
    c = Case([4, 4], [0, 7], packed=True)
    c.lens[0] = 2
    c.dev["seq_lens"].copy_(torch.from_numpy(c.lens))
    c.call()()
    c.check()


def test_in_place_in_the_projection():
    c = Case([3, 5], [8, 0], h_k=2, h_r=3)
    q = c.q
    x = c.x[:, :6].copy()
    c.call(q_out=q)()
    torch.cuda.synchronize()
    want = cache_ref.rotate(x, c.pos, c.table, c.axis, 128, False)
    got = q.float().cpu().numpy()
    assert (np.abs(got - want) <= 2.0**-8 * np.abs(want) + 2.0**-18).all()
    # k and v of the same projection are as they were
    assert np.array_equal(c.k.float().cpu().numpy(), c.x[:, 6:8]) and np.array_equal(c.v.float().cpu().numpy(), c.x[:, 8:])


def test_bad_positions_and_pages_are_left_out():
    c = Case([3, 3], [20, 40], packed=False)
    c.pos[0, 1] = 300  # past the table
    c.pos[0, 4] = -1
    c.dev["positions"].copy_(torch.from_numpy(c.pos))
    c.call()()
    c.pos[0, 1] = c.pos[0, 4] = 0
    c.check(skip_tokens=(1, 4), status=mj.MJ_ERR_INVALID_ARG)
    for entry in (-1, 2**31 - 1):
        c = Case([3, 3], [30, 40], packed=False)
        bt = c.bt.copy()
        bt[0, 2] = entry  # slot 32 of sequence 0
        c.dev["block_table"].copy_(torch.from_numpy(bt))
        c.call()()
        c.check(skip_rows=((0, 32),), status=mj.MJ_ERR_INVALID_ARG)
    c = Case([2], [14])
    c.lens[0] = 5000  # past the table's blocks
    c.dev["seq_lens"].copy_(torch.from_numpy(c.lens))
    c.call()()
    torch.cuda.synchronize()
    assert int(c.status.item()) == mj.MJ_ERR_INVALID_ARG
    assert np.array_equal(c.kc.cpu().numpy(), c.before[0])


def test_nonfinite_values():
    c = Case([2], [3], h_k=1, h_r=1)
    t = c.v
    t[0, 0, 0], t[0, 0, 1], t[0, 0, 2] = float("nan"), float("inf"), -float("inf")
    c.call()()
    torch.cuda.synchronize()
    row = c.vc.cpu().numpy()[c.bt[0, 0], 3, 0]
    assert row[0] & 0x7F == 0x7F and row[1] == 0x7E and row[2] == 0xFE


def test_codes_are_those_of_the_division():
    """K (turned by nothing) and V codes equal torch's division and rounding,
    bit for bit, for descales over the whole range."""
    n = 4096
    rng = np.random.default_rng(5)
    c = Case([n], [0], h_k=4, h_r=1, seed=9, max_pos=1, page_size=128)
    c.pos[:] = 0
    c.dev["positions"].zero_()
    c.dev["cos_sin"][:, :64], c.dev["cos_sin"][:, 64:] = 1.0, 0.0
    for exps in ((-3, 3), (-70, 70), (-126, 127)):
        d = torch.from_numpy((2.0 ** rng.uniform(*exps, (1, 4))).astype(np.float32)).cuda()
        scale = torch.from_numpy(2.0 ** rng.uniform(-12, 12, (n, 4, 1))).cuda()
        x = (torch.from_numpy(rng.standard_normal((n, 4, 128))).cuda() * scale * d[..., None].double()).to(torch.bfloat16)
        c.call(k=x, v=x, k_descale=d, v_descale=d)()
        torch.cuda.synchronize()
        want = (x.float() / d[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        page = c.dev["block_table"][0, torch.arange(n, device="cuda") // 128].long()
        row = torch.arange(n, device="cuda") % 128
        for got in (c.kc, c.vc):
            g = got[page, row]
            nan = torch.isnan(x.float() / d[..., None])
            assert torch.equal(torch.where(nan, 0x7F, g), torch.where(nan, 0x7F, want)), exps


@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "neighbours"])
def test_results_are_the_formulas_in_fp32(pairs):
    """Q and K equal the formula evaluated operation by operation, bit for bit."""
    n, h_k, h_r, rot = 6000, 4, 2, 96
    c = Case([n], [0], h_k=h_k, h_r=h_r, page_size=128, rot=rot, axes=3, mixed=True, pairs=pairs)
    c.call()()
    torch.cuda.synchronize()
    at = c.dev["positions"].long()[torch.from_numpy(c.axis).cuda()].t()
    f = torch.arange(rot // 2, device="cuda")
    cos, sin = c.dev["cos_sin"][at, f][:, None], c.dev["cos_sin"][at, rot // 2 + f][:, None]

    def turn(x):
        x = x.float()
        y = x.clone()
        ia, ib = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
        y[..., ia] = x[..., ia] * cos - x[..., ib] * sin
        y[..., ib] = x[..., ib] * cos + x[..., ia] * sin
        return y

    assert torch.equal(c.q_out, turn(c.q).to(torch.bfloat16))
    slot = torch.arange(n, device="cuda")
    got = c.kc[c.dev["block_table"][0, slot // 128].long(), slot % 128]
    want = (turn(c.k) / c.dev["k_descale"][0][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(got, want)


def test_signed_zeros_keep_their_sign():
    c = Case([3, 3], [5, 40], h_k=2, h_r=1, packed=False)
    v = c.v.clone()
    v[:, :, 0::4], v[:, :, 1::4] = 0.0, -0.0
    c.call(v=v)()
    torch.cuda.synchronize()
    for b in range(2):
        for i in range(3):
            slot = int(c.lens[b]) - 3 + i
            row = c.vc.cpu().numpy()[c.bt[b, slot // 16], slot % 16]
            assert (row[:, 0::4] == 0x00).all() and (row[:, 1::4] == 0x80).all()


def test_no_tokens():
    c = Case([3, 3], [5, 40], packed=False)
    before = c.kc.clone(), c.vc.clone()
    empty = {n: c.dev[n][..., :0] if n == "positions" else getattr(c, n)[:0] for n in ("q", "k", "v", "positions", "q_out")}
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    c.call(**empty, cu_tokens=cu)()
    torch.cuda.synchronize()
    assert torch.equal(c.kc, before[0]) and torch.equal(c.vc, before[1]) and int(c.status.item()) == 0


def test_a_call_keeps_its_shape():
    """Parameters changed after the call was made do not change it."""
    c = Case([4, 4], [100, 3])
    call = c.call()
    c.params.interleaved, c.params.rot_dim = 1, 64
    call()
    c.check()


def test_graph_and_stream():
    c = Case([4, 4], [100, 3], packed=True, axes=3)
    call = c.call()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call(side)
    graph.replay()
    c.check()


def test_binding_refuses():
    c = Case([4, 4], [10, 3], packed=True, axes=2)
    with pytest.raises(ValueError):
        c.call(q=c.q.float())
    with pytest.raises(ValueError):
        c.call(k=c.k[:3])
    with pytest.raises(ValueError):
        c.call(positions=c.dev["positions"][:1])
    with pytest.raises(ValueError):
        c.call(cos_sin=c.dev["cos_sin"][:, :64])
    with pytest.raises(ValueError):
        c.call(freq_axis=[0] * 10)
    with pytest.raises(ValueError):
        c.call(q_out=c.q_out[:, :1])
    with pytest.raises(ValueError):
        c.call(key_pos=c.key_pos[:, :, :16])
    with pytest.raises(mj.MjError):
        c.call(freq_axis=[2] * 64)()
