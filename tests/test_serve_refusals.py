"""More refusals of the serving operators' entry points, on the host (CPU only;
the pointers are aligned and never dereferenced)."""

import ctypes

import pytest

import paged_fp8_kv_gb300 as mj

BAD = mj.MJ_ERR_INVALID_ARG


@pytest.mark.parametrize("out", ["positions", "block_table", "num_free_out", "cu_tokens"])
@pytest.mark.parametrize("over", ["seq_lens", "num_free", "new_tokens"])
def test_only_lengths_and_the_lists_size_are_in_place(out, over):
    """An output as long as the lengths (one new token a sequence, a table of one page) is not their place."""
    p, a = mj.make_page_params(1, 16, 1, 40), mj.ReserveArgs()
    at = iter(range(1 << 20, 1 << 60, 1 << 32))
    for f in ("seq_lens", "new_tokens", "free_pages", "num_free", "num_free_out", "block_table", "seq_lens_out", "positions"):
        setattr(a, f, next(at))
    a.num_tokens = 1
    if (out, over) != ("num_free_out", "num_free"):
        setattr(a, out, getattr(a, over))
        assert mj.lib().mj_pages_reserve(ctypes.byref(p), ctypes.byref(a), None) == BAD
