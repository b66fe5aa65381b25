"""Refusals of the attention entry points at the ends of their ranges (no GPU needed)."""
import ctypes

import pytest

from test_attend_abi import DIMS, L, cache, cache_dims  # noqa: F401


@pytest.mark.parametrize("batch", [(1 << 17) + 1, 1 << 24])
def test_cache_batches_whose_walk_could_outlast_a_wait(L, batch):  # noqa: F811
    """Empty sequences are passed over one by one while other warps wait."""
    d = cache_dims(batch=batch, num_heads=1, table_rows=batch)
    assert cache(L, d) == DIMS
    n = ctypes.c_size_t(0)
    assert L.mla_prolog_attend_cache_workspace(ctypes.byref(d), ctypes.byref(n)) == DIMS
