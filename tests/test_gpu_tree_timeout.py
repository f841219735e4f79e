"""The bounded waits of the tree attention, on both sides of the 24 rows: with no
copy issued and a 1 ms limit the waits run out, the sequences are flagged, the
call returns, and the next ordinary call on the same cache is right."""
import ctypes
import time

import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import trees
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, h16, to_dev
from tests.test_gpu_tree_attn import check, run

pytestmark = pytest.mark.gpu

WAIT_NS = 1_000_000


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def entry():
    f = qs.lib().qs_test_attn_tree_timeout
    p, i = ctypes.c_void_p, ctypes.c_int32
    f.argtypes = [ctypes.POINTER(qs.QsCacheStruct), ctypes.POINTER(qs.QsPagesStruct), ctypes.c_int, p, i, p, i,
                  i, ctypes.c_float, p, p, p, ctypes.c_size_t, ctypes.c_uint64, p]
    f.restype = ctypes.c_int
    return f


@pytest.mark.parametrize("n,group", [(9, 1), (40, 1), (64, 4)])
@pytest.mark.parametrize("ng", [4, 200])
def test_waits_run_out(torch, n, group, ng):
    rng = np.random.default_rng([n, group, ng])
    B, H = 1, 2
    oc = _oracle_state(rng, B, H, [ng], [90], cap=ng)
    cache = load(torch, oc, rng)
    parent = trees.random_parents(rng, B, n)
    for mode in (DRAFT, VERIFY):
        q = h16(rng, (B, H * group, n, 128))
        qd, pd = to_dev(torch, q), to_dev(torch, parent)
        out = torch.full_like(qd, float("nan"))
        ws = torch.zeros(qs.qs_attn_tree_workspace_size(cache, n, group), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        assert entry()(cache._ref, cache._pages_ref, mode, pd.data_ptr(), n, qd.data_ptr(), n, group, 0.1,
                       out.data_ptr(), None, ws.data_ptr(), ws.numel(), WAIT_NS,
                       torch.cuda.current_stream().cuda_stream) == qs.QS_OK
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 5.0
        assert list(qs.qs_get_errors(cache)) == [qs.DEV_TIMEOUT]
        assert int(cache.arrive.abs().sum()) == 0
        got, gl = run(torch, cache, mode, q, parent, group)
        ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group)
        check(got, gl, ref, rl)
        assert np.all(qs.qs_get_errors(cache) == 0)


def test_wait_limit_outside_its_range_is_rejected(torch):
    cache = qs.PagedCache(1, 2, 3, 4)
    p = 0x10000
    for limit in (0, 999, 100_000_001):
        assert entry()(cache._ref, cache._pages_ref, 0, p, 40, p, 40, 1, 0.1, p, None, p, 1 << 20, limit,
                       None) == qs.QS_ERR_ARG
