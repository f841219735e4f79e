"""The page table of a PagedCache: written in place or replaced by another
tensor, the calls take the one that the cache holds (no GPU needed)."""
import pytest

import __graft_entry__
from hierarchical_quantized_kv_gb300 import qs

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def cache():
    __graft_entry__.build()
    return qs.PagedCache(2, 3, 4, 5, device="cpu")


def test_the_calls_take_the_assigned_table(cache):
    assert cache.pages_struct.table == cache.table.data_ptr()
    assert (cache.table == -1).all()
    old = cache.table
    cache.table = torch.arange(8, dtype=torch.int32).reshape(2, 4)
    assert cache.pages_struct.table == cache.table.data_ptr() != old.data_ptr()
    assert cache._pages_ref._obj is cache.pages_struct
    cache.table += 1  # in place, through the attribute
    assert cache.table[1, 3] == 8 and cache.pages_struct.table == cache.table.data_ptr()
    assert cache.nbytes() - qs.Cache.nbytes(cache) == 2 * 4 * 4


@pytest.mark.parametrize("bad", [
    lambda: torch.zeros((2, 4), dtype=torch.int64), lambda: torch.zeros((2, 4)),
    lambda: torch.zeros((2, 5), dtype=torch.int32), lambda: torch.zeros(8, dtype=torch.int32),
    lambda: torch.zeros((4, 2), dtype=torch.int32).t(),
    lambda: torch.zeros((2, 4), dtype=torch.int32, device="meta")])
def test_other_tensors_are_refused(cache, bad):
    held = cache.table
    with pytest.raises(ValueError):
        cache.table = bad()
    assert cache.table is held and cache.pages_struct.table == held.data_ptr()
