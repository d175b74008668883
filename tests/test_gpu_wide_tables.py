"""GPU: eviction under a block table far wider than the sequences are long, as
a server's is (the model's whole context): the kept set, the rows and the
planes byte for byte, as in the tests with tables of the sequences' width."""

import numpy as np
import pytest
import torch

from tests.test_gpu_evict import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("longest", [20000, 60000])
def test_many_groups(longest):
    """One sequence that makes the table wide, and more groups than the GPU
    holds: a run is then as wide as the table, whose keys do not fit shared
    memory beside another CTA's, or at all."""
    rng = np.random.default_rng(longest)
    c = Case([longest] + rng.integers(0, 1200, 39).tolist(), 300, h_k=8, page_size=64, first=2, last=20, pos=True)
    c.call()()
    c.check()


def test_few_groups():
    c = Case([450001, 0, 65, 3000, 3001], 3000, h_k=2, page_size=128, first=4, last=100, weights="mixed")
    c.call()()
    c.check()
