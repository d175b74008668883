"""Prompts and trees whose scores are far below one: scales that leave fp32's
normal range must not turn masked keys into NaN."""

import pytest
import torch

from tests.serving_helpers import HALF_P
from tests.test_gpu_prompt import Prompt
from tests.test_gpu_tree import Tree
from tests.test_gpu_tree_kernels import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kd,softcap,window", [(2.0**-24, 0.0, 0), (2.0**-60, 0.0, 70), (2.0**-60, 5.0, 0), (2.0**-126, 0.0, 0)])
def test_prompts_of_tiny_scores(kd, softcap, window, e4m3):
    """Rows of bf16 Q at its smallest values, e4m3 Q under descales whose product no fp32 holds."""
    p = Prompt([200, 900, 129], [40, 300, 1], 2, 4, 16, softcap=softcap, window=window, e4m3=e4m3)
    p.c.kd.fill_(kd)
    if e4m3:
        p.qd.fill_(2.0**-100)
    else:
        sign = torch.where(p.q < 0, -1.0, 1.0)
        for first, size in ((0, 2.0**-125), (1, 2.0**-133), (2, 2.0**-110), (3, 0.0)):
            p.q[first::5] = (sign * size).to(torch.bfloat16)[first::5]
    p.run().check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_trees_of_tiny_scores(e4m3):
    t = Tree([900, 300, 129], [61, 20, 1], 61, 2, 4, 16, e4m3=e4m3, begin=True)
    t.c.kd.fill_(2.0**-60)
    if e4m3:
        t.qd.fill_(2.0**-100)
    else:
        t.q.copy_((torch.where(t.q < 0, -1.0, 1.0) * 2.0**-125).to(torch.bfloat16))
    t.run()
    check(t, HALF_P, True)
