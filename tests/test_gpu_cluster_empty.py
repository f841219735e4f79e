"""Clusters with nothing to do: sequences with fewer buffered tokens than
queries, and selections that take every group.  Outputs and error bits as
documented, counters back at zero, the calls after them right."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_listed_attn import load, random_sel, run
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, assert_close, h16, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


@pytest.mark.parametrize("mode", [DRAFT, VERIFY])
@pytest.mark.parametrize("H,n", [(1, 200), (8, 130), (32, 40), (3, 2)])  # several clusters a segment, one
def test_fewer_tokens_than_queries(torch, H, n, mode):
    rng = np.random.default_rng([H, n, mode])
    oc = _oracle_state(rng, 1, H, [n], [3], cap=n)
    cache = load(torch, oc, rng)
    for n_q in (5, 3, 8, 1):
        q = h16(rng, (1, H, n_q, 128))
        got, gl = run(torch, cache, mode, q)
        if n_q > 3:
            assert not got.any() and np.all(gl == -np.inf)
        else:
            ref, rl = paging.attention(oc, q, mode == DRAFT)
            assert_close(got, ref, gl, rl)
        assert list(qs.qs_get_errors(cache)) == [qs.DEV_NQ_GT_FILL if n_q > 3 else 0]


@pytest.mark.parametrize("mode", [DRAFT, VERIFY])
def test_append_that_overflows_into_too_few_tokens(torch, mode):
    """The append fails and the queries outnumber the buffer: both flagged, the
    counters unchanged, the ticket back at zero."""
    rng = np.random.default_rng(5 + mode)
    B, H = 2, 4
    oc = _oracle_state(rng, B, H, [6, 6], [2, 100], cap=6)
    cache = load(torch, oc, rng)
    sel = random_sel(rng, B, H, 3, [6, 6])
    k = h16(rng, (B, H, 200, 128))
    q = h16(rng, (B, H, 8, 128))
    oc.append(k, k)
    state = cache.state.clone()
    got, gl = run(torch, cache, mode, q, sel=sel, k=k, v=k)
    # sequence 0 takes the tokens, sequence 1 cannot (100 + 200 > 256)
    ref, rl = paging.attention(oc, q, mode == DRAFT, sel=sel)
    assert_close(got, ref, gl, rl)
    assert list(qs.qs_get_errors(cache)) == [0, qs.DEV_OVERFLOW]
    assert cache.state[0, 1] == 202 and cache.state[1, 1] == 100 and not cache.state[:, 5].any()
    cache.state.copy_(state)
    cache.state[:, 1] = torch.tensor([60, 4])
    cache.state[:, 2] = 0
    got, gl = run(torch, cache, mode, q, sel=sel, k=k, v=k)  # 60 + 200 and 4 + 200
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_OVERFLOW, 0]
    assert list(cache.state[:, 1].cpu().numpy()) == [60, 204] and not cache.state[:, 5].any()
    cache.state[:, 1] = torch.tensor([250, 7])
    got, gl = run(torch, cache, mode, q, sel=sel, k=k[:, :, :7].copy(), v=k[:, :, :7].copy())
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_OVERFLOW, 0]
    cache.state[:, 1] = torch.tensor([255, 3])
    got, gl = run(torch, cache, mode, q, sel=sel, k=k[:, :, :2].copy(), v=k[:, :, :2].copy())
    assert not got[1].any() and np.all(gl[1] == -np.inf) and got[0].any()
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_OVERFLOW, qs.DEV_NQ_GT_FILL]
    assert list(cache.state[:, 1].cpu().numpy()) == [255, 5] and not cache.state[:, 5].any()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,H,n", [(1, 2, 100), (1, 2, 200), (2, 4, 400), (3, 2, 1100), (9, 32, 300)])
def test_selection_of_every_group(torch, B, H, n, paged):
    rng = np.random.default_rng([B, H, n])
    ng = [int(x) for x in rng.integers(0, 5, B)]
    oc = _oracle_state(rng, B, H, ng, [4] * B, cap=n)
    cache = load(torch, oc, rng, paged=paged)
    q = h16(rng, (B, H, 1, 128))
    qd = to_dev(torch, q)
    for k in (7, 1, 4, 2):  # every group, some of them, in turn
        sel = torch.full((B, H, k), -9, dtype=torch.int32, device="cuda")
        qs.qs_select_groups(cache, qd, sel)
        assert np.array_equal(sel.cpu().numpy(), paging.select(oc, q, k))
    assert np.all(qs.qs_get_errors(cache) == 0)
