"""Which kernel attends trees: the one that was asked for is the one that runs
and the one that is named; each within the bounds of its own roundings."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_fp8_kv_gb300 as mj
from tests.serving_helpers import HALF_P, SPLIT_P, attend, check_rows, value_of
from tests.test_gpu_tree import D, Tree

pytestmark = pytest.mark.gpu
QROWS = mj.MJ_KERNEL_TENSOR_CORE_QROWS


def check(t, bounds, by_row):
    """Tree.check with the given bounds of P, and rows of Q scaled by themselves or all of a head's together."""
    c = t.c
    for b, (L, n) in enumerate(zip(c.lens, t.nodes)):
        ctx, j = L - n, np.arange(L)
        see = np.zeros((t.q_len, L), dtype=bool)
        for i in range(n):
            see[i, :ctx] = j[:ctx] >= (0 if t.begin is None else t.begin[b, i])
            if t.prefix is not None:
                see[i, :ctx] |= j[:ctx] < t.prefix[b]
            see[i, ctx:] = t.see[b][i]
        seen = torch.from_numpy(np.repeat(see, t.h_r, axis=0)).cuda()
        k, v = c.rows(c.k, b), c.rows(c.v, b)
        for g in range(c.h_k):
            q = value_of(t.q[b, g])
            scale = float(t.qd[b, g].double() * c.kd[b, g].double()) * D**-0.5
            ref = attend(q, k[g], v[g] * c.vd[b, g].double() * 0.75, scale, seen, t.softcap, bounds, None if by_row else q.abs().max())
            check_rows(t.o[b, g], t.lse[b, g], ref, f"sequence {b}, head {g}")


SHAPES = [(31, 5), (61, 4), (70, 5), (256, 1), (300, 2)]  # above 128 rows


@pytest.mark.parametrize("q_len,h_r", SHAPES)
@pytest.mark.parametrize("kw", [{}, dict(e4m3=True), dict(softcap=20.0), dict(prefix=True, begin=True), dict(force_splits=3)])
def test_above_128_rows(q_len, h_r, kw):
    """Eleven bits of P and rows of Q scaled one by one; some rows of Q are far smaller than others."""
    nodes = [q_len, q_len // 2, 1, 0]
    t = Tree([1200, 128 + q_len, 129, 40], nodes, q_len, 2, h_r, 16, **kw)
    if t.q.dtype == torch.bfloat16:
        t.q[:, :, ::3] *= 2.0**-9
        t.q[:, :, 1::7] *= 2.0**6
    t.run()
    check(t, HALF_P, True)


@pytest.mark.parametrize("q_len,h_r", SHAPES)
@pytest.mark.parametrize("kw", [{}, dict(e4m3=True), dict(softcap=20.0), dict(prefix=True, begin=True, force_splits=3)])
def test_query_rows_kernel_when_asked_for(q_len, h_r, kw):
    nodes = [q_len, q_len // 2, 1, 0]
    lens = [1200, 128 + q_len, 129, 40]
    t = Tree(lens, nodes, q_len, 2, h_r, 16, kernel=QROWS, **kw).run()
    check(t, SPLIT_P, False)
    other = Tree(lens, nodes, q_len, 2, h_r, 16, **kw).run()
    assert not torch.equal(t.o, other.o)  # another kernel's roundings


SCRIPT = """
import sys
from tests.test_gpu_tree import Tree
q_len, h_r, kernel, e4m3 = map(int, sys.argv[1:])
Tree([300], [q_len], q_len, 1, h_r, 16, kernel=kernel, e4m3=bool(e4m3)).run()
"""


@pytest.mark.parametrize("q_len,h_r,kernel,e4m3,name", [(61, 4, mj.MJ_KERNEL_AUTO, 0, "prompt_bf16"), (61, 4, mj.MJ_KERNEL_AUTO, 1, "prompt_e4m3"),
                                                        (61, 4, QROWS, 0, "qm_pair_bf16"), (16, 4, mj.MJ_KERNEL_AUTO, 0, "qm_r64_bf16"),
                                                        (4, 4, mj.MJ_KERNEL_AUTO, 1, "tc_r16_e4m3")])
def test_the_named_kernel_is_the_one_that_runs(q_len, h_r, kernel, e4m3, name):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", SCRIPT, *map(str, (q_len, h_r, kernel, e4m3))], cwd=root, capture_output=True, text=True,
                         env=dict(os.environ, MJ_VERBOSE="1", PYTHONPATH=root), timeout=300, check=True)
    assert f"mj_decode_attn_tree: kernel={name} " in out.stderr, out.stderr
