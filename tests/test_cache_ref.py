"""The cache operators' oracle against what their definitions fix, and the
host span rule against brute force (CPU only)."""

import numpy as np
import pytest

import oracle
import paged_fp8_kv_gb300 as mj
from oracle import cache_ref


def test_round_e4m3_hits_every_code_and_border():
    vals = cache_ref.values_of(np.arange(256))
    fin = np.unique(vals[np.isfinite(vals)])
    assert np.array_equal(cache_ref.round_e4m3(fin), fin)
    mid = (fin[1:] + fin[:-1]) / 2
    r = cache_ref.round_e4m3(mid)
    # a tie goes to the neighbour with the even code
    codes = {float(v): c for c, v in enumerate(vals[:128]) if np.isfinite(v)}
    for m, x in zip(mid, r):
        if m != 0:
            assert codes[abs(float(x))] % 2 == 0
    assert cache_ref.round_e4m3(1e9) == 448.0 and cache_ref.round_e4m3(-460.0) == -448.0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_angles(interleaved):
    rng = np.random.default_rng(3)
    rot, half = 64, 32
    ang = rng.uniform(0, 6, (50, half))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x = rng.standard_normal((7, 3, 128))
    pos = rng.integers(0, 50, (2, 7))
    axis = rng.integers(0, 2, half)
    y = cache_ref.rotate(x, pos, cs, axis, rot, interleaved)
    assert np.allclose((y**2).sum(-1), (x**2).sum(-1), rtol=1e-12)
    assert np.array_equal(y[:, :, rot:], x[:, :, rot:])
    i = 5
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    turn = np.angle((y[:, 0, a] + 1j * y[:, 0, b]) / (x[:, 0, a] + 1j * x[:, 0, b]))
    assert np.allclose(np.exp(1j * turn), np.exp(1j * ang[pos[axis[i]], i]))


def test_evict_slots_small_cases():
    src = cache_ref.evict_slots([5, 1, 4, 1, 9], np.arange(5), 5, 3, 5, 0, 0)
    assert src.tolist() == [0, 4, 2]  # slots 1 and 3 leave, 4 fills the hole
    src = cache_ref.evict_slots([1, 1, 1, 1], np.arange(4), 4, 2, 4, 0, 0)
    assert src.tolist() == [0, 1]  # ties: lowest slots
    src = cache_ref.evict_slots([np.nan, 0.0, -0.0, 3], np.arange(4), 4, 2, 4, 0, 0)
    assert src.tolist() == [3, 1]  # NaN last, -0 ties with 0
    src = cache_ref.evict_slots([9, 9, 0, 0], np.arange(4), 4, 2, 4, 0, 2)
    assert src.tolist() == [2, 3]  # the newest two are protected


def _params(b, q_len, causal, max_blocks=64, h_k=1, h_r=2):
    return mj.make_params(b, q_len, h_k, h_r, 16, max_blocks, 100, causal, kernel=mj.MJ_KERNEL_TENSOR_CORE_QROWS)


@pytest.mark.parametrize("seed", range(40))
def test_host_spans_cover_exactly_what_is_seen(seed):
    rng = np.random.default_rng(seed)
    b, q_len = 5, int(rng.integers(1, 6))
    causal = bool(rng.random() < 0.7)
    lens = rng.integers(0, 700, b)
    lens[0] = 0
    lens[1] = int(rng.integers(0, q_len + 1))  # fewer keys than query tokens
    window = int(rng.integers(1, 400)) if causal and rng.random() < 0.5 else 0
    kb = rng.integers(-5, 720, (b, q_len)).astype(np.int32) if rng.random() < 0.5 else None
    ke = rng.integers(-5, 720, (b, q_len)).astype(np.int32) if rng.random() < 0.4 else None
    px = rng.integers(-3, 300, b).astype(np.int32) if rng.random() < 0.5 else None
    p = _params(b, q_len, causal)
    mod = mj.ScoreMod(window=window, key_begin=kb, key_end=ke, prefix=px)
    spans, plan_lens = mj.score_spans(p, mod, lens)
    for i in range(b):
        L = int(lens[i])
        see = cache_ref.visible(L, q_len, causal, window, None if kb is None else kb[i], None if ke is None else ke[i],
                                0 if px is None else int(px[i]))
        any_row = see.any(0)
        n_prefix, first, end, zero = spans[i]
        assert zero == 0 and 0 <= n_prefix <= first <= end <= L
        inside = np.zeros(L, dtype=bool)
        inside[:n_prefix] = True
        inside[first:end] = True
        assert not (any_row & ~inside).any()
        # the planned tiles, listed as the kernel lists them, hold every seen key
        tiles = -(-int(plan_lens[i]) // 128)
        pt = -(-int(n_prefix) // 128)
        jump = max(0, int(first) // 128 - pt)
        listed = [v if v < pt else v + jump for v in range(tiles)]
        assert sorted(set(listed)) == listed
        held = np.zeros(L + 256, dtype=bool)
        for t in listed:
            held[t * 128 : t * 128 + 128] = True
        assert not (any_row & ~held[:L]).any()
        assert 0 <= plan_lens[i] <= L


def test_spans_refuse():
    p = _params(2, 1, True)
    with pytest.raises(mj.MjError):
        mj.score_spans(p, mj.ScoreMod(softcap=-1.0), [3, 4])
    with pytest.raises(mj.MjError):
        mj.score_spans(p, mj.ScoreMod(softcap=float("nan")), [3, 4])
    with pytest.raises(mj.MjError):
        mj.score_spans(p, mj.ScoreMod(), [3, 16 * 64 + 1])
    with pytest.raises(mj.MjError):
        mj.score_spans(_params(2, 1, False), mj.ScoreMod(window=8), [3, 4])
    with pytest.raises(ValueError):
        mj.score_spans(p, mj.ScoreMod(key_begin=np.zeros((2, 3), np.int32)), [3, 4])
    assert oracle is not None
