"""The quantizing writes of a paged cache (flush, due flush, prefill) against
the oracle: the pages the table names bit for bit, every other page untouched."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import layout, paging
from tests.test_gpu_qs import _oracle_state, assert_state_equal, h16, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def pool(cache):
    got = layout.read_device(cache)
    return {n: got[n].copy() for n in paging.GROUP_ARRAYS}


@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("T,lens", [(1, [1, 0]), (256, [256, 255]), (257, [257, 129]),
                                    (700, [700, 300]), (1000, [385, 1000])])
def test_prefill_bit_exact(torch, ub, T, lens):
    rng = np.random.default_rng(T + ub)
    B, H, cap = 2, 3, 7
    k, v = h16(rng, (B, H, T, 128), 2.0), h16(rng, (B, H, T, 128))
    oc = oracle.OracleCache(B, H, 128, 128, cap)
    oc.prefill(k, v, lens)
    n = [oc.counters(b)["n_groups"] for b in range(B)]
    cache = qs.PagedCache(B, H, cap, 20, upper_bits=ub)
    cache.table.copy_(torch.from_numpy(paging.random_table(rng, n, cap, 20)))
    cache.k_upper.fill_(0x5A)
    qs.qs_prefill_paged(cache, to_dev(torch, k), to_dev(torch, v), to_dev(torch, np.array(lens, np.int32)))
    assert np.all(qs.qs_get_errors(cache) == 0)
    # buffer slots past each prompt's fill are not written: compare the rest
    for b in range(B):
        f = oc.counters(b)["fill"]
        oc.bk[b, :, f:] = 0
        oc.bv[b, :, f:] = 0
    paging.assert_groups_equal(cache, oc, "prefill")
    owned = np.concatenate([cache.table.cpu().numpy()[b, :n[b]] for b in range(B)])
    rest = np.setdiff1d(np.arange(20), owned)
    assert np.all(cache.k_upper.cpu().numpy()[rest] == 0x5A)


@pytest.mark.parametrize("ub", [4, 2])
def test_flush_rounds_bit_exact(torch, ub):
    """Appends, rollbacks and flushes (all three forms) of a batch at unequal
    fill levels, pages handed out as the groups come."""
    rng = np.random.default_rng(3 + ub)
    B, H, cap, n_pages = 3, 4, 4, 14
    cache = qs.PagedCache(B, H, cap, n_pages, upper_bits=ub)
    free = list(rng.permutation(n_pages))
    table = np.full((B, cap), -1, np.int32)
    oc = oracle.OracleCache(B, H, 128, 128, cap)
    qs.qs_state_reset(cache)
    mask_d = torch.zeros(B, dtype=torch.uint8, device="cuda")
    for step in range(24):
        for b in range(B):  # the page of the next group, before the call that may write it
            n = oc.counters(b)["n_groups"]
            if n < cap and table[b, n] < 0 and free:
                table[b, n] = free.pop()
        cache.table.copy_(torch.from_numpy(table))
        n = int(rng.integers(20, 60))
        if step % 2:
            qs.qs_quantize_flush_due_paged(cache, n)
        else:
            qs.qs_need_flush(cache, n, mask_d)
            qs.qs_quantize_flush_paged(cache, mask_d)
        oc.flush(oc.need_flush(n))
        k, v = h16(rng, (B, H, n, 128), 3.0), h16(rng, (B, H, n, 128))
        qs.qs_buffer_append(cache, to_dev(torch, k), to_dev(torch, v))
        oc.append(k, v)
        drop = rng.integers(0, n, B).astype(np.int32)
        qs.qs_buffer_rollback(cache, to_dev(torch, drop))
        oc.rollback(drop)
        assert np.array_equal(qs.qs_get_errors(cache), oc.state[:, oracle.ERR]), step
        oc.state[:, oracle.ERR] = 0
    assert oc.state[:, oracle.N_GROUPS].sum() >= 4
    paging.assert_groups_equal(cache, oc, "rounds")


@pytest.mark.parametrize("bad", [-1, 9, 1 << 30, -(1 << 31)])
def test_bad_page_is_flagged_and_a_no_op(torch, bad):
    """A page out of range for one sequence of the batch: that sequence keeps
    its state, the other one is written."""
    rng = np.random.default_rng(5)
    B, H, cap, n_pages = 2, 2, 4, 9
    k, v = h16(rng, (B, H, 640, 128)), h16(rng, (B, H, 640, 128))
    lens = np.array([640, 500], np.int32)
    cache = qs.PagedCache(B, H, cap, n_pages)
    cache.table.copy_(torch.from_numpy(np.array([[0, 1, bad, 3], [4, 5, 6, bad]], np.int32)))
    qs.qs_prefill_paged(cache, to_dev(torch, k), to_dev(torch, v), to_dev(torch, lens))
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_PAGE, 0]
    assert cache.state[:, :4].tolist() == [[0, 0, 0, 0], [2, 244, 0, 0]]
    # a prompt that stays in the buffer needs no page
    short = np.array([200, 0], np.int32)
    cache.table[0].fill_(bad)
    cache.state.zero_()
    qs.qs_prefill_paged(cache, to_dev(torch, k), to_dev(torch, v), to_dev(torch, short))
    assert list(qs.qs_get_errors(cache)) == [0, 0]
    # flush into it: nothing changes
    before, state = pool(cache), cache.state.clone()
    mask = to_dev(torch, np.array([1, 0], np.uint8))
    qs.qs_quantize_flush_paged(cache, mask)
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_PAGE, 0]
    qs.qs_quantize_flush_due_paged(cache, 100)
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_PAGE, 0]
    after = pool(cache)
    assert all(np.array_equal(before[n], after[n]) for n in before)
    assert torch.equal(cache.state, state)
    # a good page: the same flush goes through
    cache.table[0, 0] = 7
    qs.qs_quantize_flush_due_paged(cache, 100)
    assert list(qs.qs_get_errors(cache)) == [0, 0]
    assert cache.state[0, :4].tolist() == [1, 72, 0, 1]


def test_contiguous_cache_unchanged_by_the_new_calls(torch):
    """The binding's paged calls refuse a contiguous cache and the others a
    paged one (an exception, nothing launched)."""
    dense, paged = qs.Cache(1, 1, 2), qs.PagedCache(1, 1, 2, 3)
    for call, c in ((qs.qs_quantize_flush_paged, dense), (qs.qs_quantize_flush, paged)):
        with pytest.raises(qs.QsError) as e:
            call(c)
        assert e.value.status == qs.QS_ERR_ARG
    oc = _oracle_state(np.random.default_rng(0), 1, 1, [1], [30], cap=2)
    layout.load_into(dense, oc)
    assert_state_equal(dense, oc)
