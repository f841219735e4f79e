"""The bounds-checked build over the selection, the read back and the clustered
attention: no failed check, results as in the ordinary build."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_checked import checked  # noqa: F401  (fixture)
from tests.test_gpu_listed_attn import load, random_sel, run
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, assert_close, h16, to_dev
from tests.test_gpu_read import expected, read

pytestmark = pytest.mark.gpu


def test_every_file_with_checks_reports(checked):  # noqa: F811
    for name in ("quantize", "listed", "select", "read"):
        assert hasattr(qs.lib(), "qs_checked_failures_" + name)


def select(torch, cache, q, k, group):
    sel = torch.full((cache.B, cache.H, k), -9, dtype=torch.int32, device="cuda")
    qs.qs_select_groups(cache, to_dev(torch, q), sel, group=group)
    torch.cuda.synchronize()
    return sel.cpu().numpy()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n,k", [(5, 2), (17, 16), (150, 9), (600, 64)])  # one to eight CTAs a cluster
@pytest.mark.parametrize("n_q,group", [(1, 1), (5, 3), (1, 24)])
def test_selection(checked, n, k, n_q, group, paged):  # noqa: F811
    torch, failures = checked
    rng = np.random.default_rng([n, k, n_q, group])
    B, H = 2, 2
    ng = [n, max(0, n - 3)]
    oc = _oracle_state(rng, B, H, ng, [9, 20], cap=n + 2)
    cache = load(torch, oc, rng, paged=paged)
    q = h16(rng, (B, H * group, n_q, 128))
    got = select(torch, cache, q, k, group)
    assert failures() == (0, 0)
    assert np.array_equal(got, paging.select(oc, q, k, group))


def test_selection_among_equal_scores(checked):  # noqa: F811
    """700 copies of one group: all of them in the list of close groups."""
    torch, failures = checked
    rng = np.random.default_rng(3)
    oc = _oracle_state(rng, 1, 1, [1], [4], cap=1)
    cache = paging.paged_copy(torch, oc, rng)
    wide = qs.PagedCache(1, 1, 700, cache.n_pages)
    for name in paging.GROUP_ARRAYS + ("state",):
        getattr(wide, name).copy_(getattr(cache, name))
    wide.table.fill_(int(cache.table[0, 0]))
    wide.state[0, 0] = 700
    got = select(torch, wide, h16(rng, (1, 1, 1, 128)), 300, 1)
    assert np.array_equal(got[0, 0], np.arange(300))  # the lowest of equal ones
    assert failures() == (0, 0)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("tok0,T", [(0, 1), (127, 2), (130, 900), (500, 257), (1000, 5), (0, 128 * 9)])
def test_read_back(checked, tok0, T, ub, paged):  # noqa: F811
    torch, failures = checked
    rng = np.random.default_rng([tok0, T, ub])
    oc = _oracle_state(rng, 2, 3, [6, 1], [200, 255], cap=6)
    oc.state[1, oracle.HALF_BASE] = 1
    cache = load(torch, oc, rng, ub, paged)
    for mode in (DRAFT, VERIFY):
        for got, want in zip(read(torch, cache, mode, tok0, T), expected(oc, mode, ub, tok0, T)):
            assert np.array_equal(got, want)
    assert failures() == (0, 0)


@pytest.mark.parametrize("mode,n_q,group", [(DRAFT, 1, 1), (DRAFT, 1, 7), (VERIFY, 5, 1), (VERIFY, 5, 4)])
@pytest.mark.parametrize("H,n", [(8, 130), (1, 200), (3, 30)])
def test_several_clusters_a_segment(checked, H, n, mode, n_q, group):  # noqa: F811
    torch, failures = checked
    rng = np.random.default_rng([H, n, n_q, group])
    oc = _oracle_state(rng, 1, H, [n], [201], cap=n)
    cache = load(torch, oc, rng, n_pages=n + 2)
    q = h16(rng, (1, H * group, n_q, 128))
    got, gl = run(torch, cache, mode, q, group)
    ref, rl = paging.attention(oc, q, mode == DRAFT, group)
    assert_close(got, ref, gl, rl)
    assert failures() == (0, 0)


@pytest.mark.parametrize("mode,n_q", [(DRAFT, 1), (VERIFY, 4)])
@pytest.mark.parametrize("H", [1, 8, 33])
def test_clusters_over_selections(checked, H, mode, n_q):  # noqa: F811
    torch, failures = checked
    rng = np.random.default_rng([H, n_q])
    ng = [20, 3]
    oc = _oracle_state(rng, 2, H, ng, [30, 250], cap=20)
    cache = load(torch, oc, rng)
    sel = random_sel(rng, 2, H, 12, ng)
    q = h16(rng, (2, H, n_q, 128))
    got, gl = run(torch, cache, mode, q, sel=sel)
    ref, rl = paging.attention(oc, q, mode == DRAFT, sel=sel)
    assert_close(got, ref, gl, rl)
    assert failures() == (0, 0)
