"""The quantizer at every CTA width its sizes lead to (prefill: sixteen, eight
and four warps, one to eight quarters a CTA; flush: sixteen and four warps),
both plane layouts, contiguous and paged: bit for bit against the oracle, on
degenerate groups and on values at exact ties."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import layout, paging
from tests.test_gpu_qs import _degenerate_tokens, assert_state_equal, h16, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def prompt(rng, H, T):
    """Degenerate groups (moderate, then the fp16 extremes), values at exact
    ties of their group's scale, and plain ones."""
    parts = [_degenerate_tokens(rng, H, False), _degenerate_tokens(rng, H, True)]
    ties = (rng.integers(0, 255, (1, H, 128, 128)) + 0.5) * 2.0 ** -6
    ties[:, :, 0], ties[:, :, 1] = 0.0, 255 * 2.0 ** -6
    ties[..., 0], ties[..., 1] = 0.0, 255 * 2.0 ** -6
    parts.append((ties.astype(np.float16), ties.astype(np.float16)))
    n = T - 384
    parts.append((h16(rng, (1, H, n, 128), 2.0), h16(rng, (1, H, n, 128))))
    return tuple(np.concatenate([p[i] for p in parts], 2) for i in range(2))


@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("H,T", [(3, 700), (40, 640), (40, 1000), (80, 900), (80, 2300), (150, 4200)])
def test_prefill(torch, H, T, ub):
    rng = np.random.default_rng([H, T, ub])
    k, v = prompt(rng, H, T)
    lens = np.array([T], np.int32)
    n = -(-(T - 256) // 128)
    oc = oracle.OracleCache(1, H, 128, 128, n)
    oc.prefill(k, v, lens)
    kd, vd, ld = (to_dev(torch, x) for x in (k, v, lens))
    cache = qs.Cache(1, H, n, upper_bits=ub)
    qs.qs_prefill(cache, kd, vd, ld)
    f = oc.counters(0)["fill"]
    oc.bk[:, :, f:] = oc.bv[:, :, f:] = 0
    assert_state_equal(cache, oc)
    pages = qs.PagedCache(1, H, n, n + 4, upper_bits=ub)
    pages.table.copy_(torch.from_numpy(paging.random_table(rng, [n], n, n + 4)))
    qs.qs_prefill_paged(pages, kd, vd, ld)
    paging.assert_groups_equal(pages, oc)
    assert np.all(qs.qs_get_errors(cache) == 0) and np.all(qs.qs_get_errors(pages) == 0)


@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("H", [5, 76, 77, 130])
def test_flush(torch, H, ub):
    rng = np.random.default_rng([H, ub])
    k, v = prompt(rng, H, 385)
    cache = qs.Cache(1, H, 4, upper_bits=ub)
    oc = oracle.OracleCache(1, H, 128, 128, 4)
    zero = to_dev(torch, np.zeros(1, np.int32))
    for i in range(3):  # (each flush takes the oldest of two halves)
        part = [np.ascontiguousarray(x[:, :, 128 * i:128 * i + 128]) for x in (k, v)]
        qs.qs_buffer_append(cache, *(to_dev(torch, x) for x in part))
        qs.qs_buffer_rollback(cache, zero)
        qs.qs_quantize_flush(cache)
        oc.append(*part)
        oc.rollback([0])
        oc.flush()
    torch.cuda.synchronize()
    assert oc.counters(0)["n_groups"] == 3
    got, want = layout.read_device(cache), layout.device_arrays(oc, ub)
    for name in paging.GROUP_ARRAYS + ("state",):
        assert np.array_equal(got[name].reshape(want[name].shape), want[name]), name
