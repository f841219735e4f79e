"""The bounded waits of the listed attention kernels (split, one cluster a
segment, several): with no copy issued and a 1 ms limit every wait runs out,
the sequences are flagged, nothing is written, the counters are at zero and
the next ordinary call on the same cache is right."""
import ctypes
import time

import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_listed_attn import load, run
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, assert_close, h16, to_dev

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
    f = qs.lib().qs_test_attn_paged_timeout
    f.argtypes = [ctypes.POINTER(qs.QsCacheStruct), ctypes.POINTER(qs.QsPagesStruct), ctypes.c_int,
                  ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p,
                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64, ctypes.c_void_p]
    f.restype = ctypes.c_int
    return f


@pytest.mark.parametrize("B,H,ng", [(2, 3, 9), (1, 2, 3), (1, 20, 6), (1, 8, 130)])
def test_waits_run_out(torch, B, H, ng):
    rng = np.random.default_rng([B, H, ng])
    oc = _oracle_state(rng, B, H, [ng] * B, [70] * B, cap=ng)
    cache = load(torch, oc, rng)
    for mode, n_q in ((DRAFT, 1), (VERIFY, 5)):
        q = h16(rng, (B, H, n_q, 128))
        qd = to_dev(torch, q)
        out = torch.full_like(qd, float("nan"))
        lse = torch.full(q.shape[:3], float("nan"), dtype=torch.float32, device="cuda")
        ws = torch.empty(qs.qs_attn_workspace_size(cache, n_q), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        assert entry()(cache._ref, cache._pages_ref, mode, qd.data_ptr(), n_q, 1, 0.1, out.data_ptr(),
                       lse.data_ptr(), ws.data_ptr(), ws.numel(), WAIT_NS,
                       torch.cuda.current_stream().cuda_stream) == qs.QS_OK
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 5.0
        assert list(qs.qs_get_errors(cache)) == [qs.DEV_TIMEOUT] * B
        assert int(cache.arrive.abs().sum()) == 0
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
        got, gl = run(torch, cache, mode, q)
        ref, rl = paging.attention(oc, q, mode == DRAFT)
        assert_close(got, ref, gl, rl)
        assert np.all(qs.qs_get_errors(cache) == 0)


def test_wait_limit_outside_its_range_is_rejected(torch):
    cache = qs.PagedCache(1, 2, 3, 4)
    p = 0x10000
    for limit in (0, 999, 100_000_001):
        assert entry()(cache._ref, cache._pages_ref, 0, p, 1, 1, 0.1, p, None, p, 1 << 20, limit,
                       None) == qs.QS_ERR_ARG
