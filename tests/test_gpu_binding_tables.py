"""A page table that is replaced between two calls: the second call reads the
new one's pages, after the first table's memory has been given back."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_listed_attn import run
from tests.test_gpu_qs import DRAFT, _oracle_state, assert_close, h16

pytestmark = pytest.mark.gpu


def test_replaced_table():
    torch = pytest.importorskip("torch")
    import __graft_entry__
    __graft_entry__.build()
    rng = np.random.default_rng(1)
    oc = _oracle_state(rng, 1, 2, [6], [40], cap=6)
    cache = paging.paged_copy(torch, oc, rng)
    q = h16(rng, (1, 2, 1, 128))
    ref, rl = paging.attention(oc, q, True)
    assert_close(*(x for p in zip(run(torch, cache, DRAFT, q), (ref, rl)) for x in p))
    # the groups in other pages, named by a table of its own
    perm = torch.randperm(cache.n_pages, device="cuda")
    for name in paging.GROUP_ARRAYS:
        t = getattr(cache, name)
        t[perm] = t.clone()
    cache.table = perm[cache.table.long()].to(torch.int32)
    torch.full((64, 6), -9, dtype=torch.int32, device="cuda")  # where the first table was
    got, gl = run(torch, cache, DRAFT, q)
    assert_close(got, ref, gl, rl)
    assert np.all(qs.qs_get_errors(cache) == 0)
