"""Decode attention over listed groups (paged caches, selected groups) against
textbook softmax attention in 64 bits over the oracle's dequantized tokens.

Tolerances are those of the contiguous kernel, whose arithmetic this is:
max-abs 1e-2, relative RMS 2e-3, log-sum-exp 5e-3 (tests/test_gpu_qs.py)."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import layout, paging
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, assert_close, h16, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def load(torch, oc, rng, ub=4, paged=True, **kw):
    if paged:
        return paging.paged_copy(torch, oc, rng, ub, **kw)
    cache = qs.Cache(oc.B, oc.H, oc.cap, upper_bits=ub)
    layout.load_into(cache, oc)
    return cache


def run(torch, cache, mode, q, group=1, sel=None, k=None, v=None, stream=None):
    qd = to_dev(torch, q)
    out = torch.full_like(qd, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), dtype=torch.float32, device="cuda")
    ws = torch.empty(qs.qs_attn_workspace_size_gqa(cache, q.shape[2], group), dtype=torch.uint8,
                     device="cuda")
    kw = dict(lse=lse, workspace=ws, group=group, stream=stream)
    if k is not None:
        kw.update(k_new=to_dev(torch, k), v_new=to_dev(torch, v))
    if sel is None:
        qs.qs_attn_decode_paged(cache, mode, qd, 1.0 / np.sqrt(128), out, **kw)
    else:
        sd = to_dev(torch, sel.astype(np.int32))
        qs.qs_attn_decode_sparse(cache, mode, sd, qd, 1.0 / np.sqrt(128), out, **kw)
    torch.cuda.synchronize()
    assert int(cache.arrive.abs().sum().item()) == 0, "segment counters not back at zero"
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def random_sel(rng, B, H, k, n_groups):
    """Rows of distinct groups in random order, -1 strewn in."""
    sel = np.full((B, H, k), -1, np.int64)
    for b in range(B):
        for h in range(H):
            n = min(k, n_groups[b])
            row = rng.permutation(n_groups[b])[:n]
            sel[b, h, :n] = np.where(rng.random(n) < 0.2, -1, row)
    return sel


SHAPES = [([0, 0], [1, 8]), ([1, 3], [33, 64]), ([5, 2], [256, 200]), ([7, 0], [129, 31])]


@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("n_q,group", [(1, 1), (1, 4), (5, 1), (8, 1), (5, 4), (8, 3), (1, 24)])
@pytest.mark.parametrize("n_groups,fill", SHAPES)
def test_paged(torch, n_groups, fill, n_q, group, ub):
    rng = np.random.default_rng([n_q, group, ub] + n_groups + fill)
    B, H = 2, 3
    oc = _oracle_state(rng, B, H, n_groups, fill, cap=8)
    oc.state[1, oracle.HALF_BASE] = 1
    cache = load(torch, oc, rng, ub)
    q = h16(rng, (B, H * group, n_q, 128))
    short = [n_q > f for f in fill]
    for mode in (DRAFT, VERIFY):
        got, gl = run(torch, cache, mode, q, group)
        ref, rl = paging.attention(oc, q, mode == DRAFT, group, ub)
        assert_close(got, ref, gl, rl, "mode %d" % mode)
        assert list(qs.qs_get_errors(cache)) == [qs.DEV_NQ_GT_FILL if s else 0 for s in short]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n_q,group,ub", [(1, 1, 4), (1, 4, 2), (5, 1, 4), (5, 4, 4), (3, 2, 2)])
@pytest.mark.parametrize("k", [1, 3, 8, 20])
def test_sparse(torch, k, n_q, group, ub, paged):
    rng = np.random.default_rng([k, n_q, group, ub])
    ng, fill = [12, 0, 5, 1], [70, 9, 256, 31]
    B, H = 4, 3
    oc = _oracle_state(rng, B, H, ng, fill, cap=12)
    oc.state[2, oracle.HALF_BASE] = 1
    cache = load(torch, oc, rng, ub, paged)
    sel = random_sel(rng, B, H, k, ng)
    sel[2, 1] = -1                       # a row with no group at all
    q = h16(rng, (B, H * group, n_q, 128))
    for mode in (DRAFT, VERIFY):
        got, gl = run(torch, cache, mode, q, group, sel)
        ref, rl = paging.attention(oc, q, mode == DRAFT, group, ub, sel)
        assert_close(got, ref, gl, rl, "mode %d" % mode)
    assert np.all(qs.qs_get_errors(cache) == 0)


@pytest.mark.parametrize("mode,n_q,group", [(DRAFT, 1, 1), (DRAFT, 1, 8), (VERIFY, 5, 1), (VERIFY, 5, 4),
                                            (VERIFY, 8, 3)])
@pytest.mark.parametrize("B,H", [(1, 1), (1, 8), (1, 32), (2, 20), (3, 24), (5, 31)])
def test_cluster_sizes(torch, B, H, mode, n_q, group):
    """Eight, four and two CTAs a segment, and the split kernel; sequences
    with fewer groups than the list, and one with too few buffered tokens."""
    rng = np.random.default_rng([B, H, n_q, group])
    ng = [int(x) for x in rng.integers(0, 14, B)]
    fill = [int(x) for x in rng.integers(1, 257, B)]
    ng[0], fill[0] = 13, 250
    oc = _oracle_state(rng, B, H, ng, fill, cap=13)
    cache = load(torch, oc, rng, paged=False)
    sel = random_sel(rng, B, H, 9, ng)
    q = h16(rng, (B, H * group, n_q, 128))
    got, gl = run(torch, cache, mode, q, group, sel)
    ref, rl = paging.attention(oc, q, mode == DRAFT, group, sel=sel)
    assert_close(got, ref, gl, rl)
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_NQ_GT_FILL if n_q > f else 0 for f in fill]


@pytest.mark.parametrize("mode,n_q,group", [(DRAFT, 1, 1), (DRAFT, 1, 4), (DRAFT, 1, 7), (VERIFY, 5, 1),
                                            (VERIFY, 1, 3), (VERIFY, 5, 4)])
@pytest.mark.parametrize("H,n", [(8, 130), (1, 200), (3, 100)])
def test_several_clusters_a_segment(torch, H, n, mode, n_q, group):
    """Few heads with a long context: two to nineteen clusters a segment,
    joined through the workspace, twice (the counters are back at zero)."""
    rng = np.random.default_rng([H, n, n_q, group])
    oc = _oracle_state(rng, 1, H, [n], [201], cap=n)
    cache = load(torch, oc, rng, n_pages=n + 2)
    for _ in range(2):
        q = h16(rng, (1, H * group, n_q, 128))
        got, gl = run(torch, cache, mode, q, group)
        ref, rl = paging.attention(oc, q, mode == DRAFT, group)
        assert_close(got, ref, gl, rl)
    assert np.all(qs.qs_get_errors(cache) == 0)


@pytest.mark.parametrize("paged", [False, True])
def test_every_group_selected_equals_dense(torch, paged):
    """All groups in order give the contiguous kernel's result (within the
    tolerance: which warp takes which half-unit varies from run to run)."""
    rng = np.random.default_rng(6)
    B, H, n = 2, 4, 40
    oc = _oracle_state(rng, B, H, [n, n], [100, 256], cap=n)
    dense, cache = load(torch, oc, rng, paged=False), load(torch, oc, rng, paged=paged)
    sel = np.broadcast_to(np.arange(n), (B, H, n))
    for mode, n_q in ((DRAFT, 1), (VERIFY, 5)):
        q = h16(rng, (B, H, n_q, 128))
        qd = to_dev(torch, q)
        out = torch.empty_like(qd)
        lse = torch.empty((B, H, n_q), dtype=torch.float32, device="cuda")
        ws = torch.empty(qs.qs_attn_workspace_size(dense, n_q), dtype=torch.uint8, device="cuda")
        qs.qs_attn_decode(dense, mode, qd, 1.0 / np.sqrt(128), out, lse, ws)
        got = [run(torch, cache, mode, q, sel=sel)]
        if paged:
            got.append(run(torch, cache, mode, q))
        ref = out.double().cpu().numpy()
        for o, l in got:
            assert_close(o, ref, l, lse.double().cpu().numpy(), "mode %d" % mode)


def test_bad_entries_are_left_out(torch):
    """Indices outside the sequence's groups, pages outside the pool, a group
    named twice: left out and flagged, or counted twice; the neighbours in
    the batch see nothing of it."""
    rng = np.random.default_rng(12)
    B, H, ng = 3, 2, [6, 6, 6]
    oc = _oracle_state(rng, B, H, ng, [50, 60, 70], cap=9)
    cache = load(torch, oc, rng)
    sel = np.tile(np.array([4, 1, 1, 5, -1, 0]), (B, H, 1))
    sel[0, 0, 2], sel[0, 1, 0], sel[1, 1, 3] = 6, -2, 1 << 30
    for mode, n_q in ((DRAFT, 1), (VERIFY, 4)):
        q = h16(rng, (B, H, n_q, 128))
        got, gl = run(torch, cache, mode, q, sel=sel)
        ref, rl = paging.attention(oc, q, mode == DRAFT, sel=sel)
        assert_close(got, ref, gl, rl, "mode %d" % mode)
        assert list(qs.qs_get_errors(cache)) == [qs.DEV_SELECT, qs.DEV_SELECT, 0]
    cache.table[1, 1] = -1
    cache.table[2, 5] = cache.n_pages
    c = [paging.counts(oc, b, sel) for b in range(B)]
    c[1][:, 1] = 0
    c[2][:, 5] = 0
    q = h16(rng, (B, H, 1, 128))
    got, gl = run(torch, cache, DRAFT, q, sel=sel)
    ref, rl = paging.attention(oc, q, True, times=c)
    assert_close(got, ref, gl, rl, "bad pages")
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_SELECT, qs.DEV_SELECT | qs.DEV_PAGE, qs.DEV_PAGE]
    c = [np.ones((H, 6)) for _ in range(B)]
    c[1][:, 1] = 0
    c[2][:, 5] = 0
    got, gl = run(torch, cache, VERIFY, q)
    ref, rl = paging.attention(oc, q, False, times=c)
    assert_close(got, ref, gl, rl, "bad pages, all groups")
    assert list(qs.qs_get_errors(cache)) == [0, qs.DEV_PAGE, qs.DEV_PAGE]


@pytest.mark.parametrize("mode", [DRAFT, VERIFY])
def test_more_units_than_the_kernel_lists(torch, mode):
    """A sequence of 10,400 groups in 32 heads: over 2,048 units a CTA, the
    last of them looked up when they are issued.  All groups lie in 40 pages,
    each named 260 times by the table: the reference counts each page so often."""
    rng = np.random.default_rng(21)
    H, n_pages, times = 32, 40, 260
    oc = _oracle_state(rng, 1, H, [n_pages], [90], cap=n_pages)
    cache = qs.PagedCache(1, H, n_pages * times, n_pages)
    arrs = layout.device_arrays(oc)
    for name in paging.GROUP_ARRAYS:
        paging.put(torch, getattr(cache, name), np.ascontiguousarray(arrs[name][0].swapaxes(0, 1)))
    for name in ("buf_k", "buf_v"):
        paging.put(torch, getattr(cache, name), arrs[name])
    table = rng.permutation(np.repeat(np.arange(n_pages), times)).astype(np.int32)
    cache.table.copy_(torch.from_numpy(table[None]))
    cache.state[0, 0], cache.state[0, 1] = n_pages * times, 90
    assert H * n_pages * times > 2048 * 152
    q = h16(rng, (1, H, 1, 128))
    got, gl = run(torch, cache, mode, q)
    ref, rl = paging.attention(oc, q, mode == DRAFT, times=[np.full((H, n_pages), float(times))])
    assert_close(got, ref, gl, rl)
    assert np.all(qs.qs_get_errors(cache) == 0)


@pytest.mark.parametrize("paged", [False, True])
def test_fused_append(torch, paged):
    """Append and attend in one launch: the buffer and counters as after a
    separate append, an overflowing sequence flagged (beside a bad selection
    in the same call) and left as it was."""
    rng = np.random.default_rng(31)
    B, H, ng = 3, 2, [4, 2, 3]
    oc = _oracle_state(rng, B, H, ng, [100, 255, 7], cap=4)
    cache = load(torch, oc, rng, paged=paged)
    sel = random_sel(rng, B, H, 3, ng)
    for mode, n in ((DRAFT, 1), (VERIFY, 5)):
        k, v = h16(rng, (B, H, n, 128), 2.0), h16(rng, (B, H, n, 128))
        q = h16(rng, (B, H, n, 128))
        oc.append(k, v)
        bad = sel.copy()
        bad[1, 0, 0] = 99
        got, gl = run(torch, cache, mode, q, sel=bad, k=k, v=v)
        ref, rl = paging.attention(oc, q, mode == DRAFT, sel=bad)
        assert_close(got, ref, gl, rl, "mode %d" % mode)
        over = qs.DEV_OVERFLOW if oc.state[1, oracle.ERR] else 0
        assert list(qs.qs_get_errors(cache)) == [0, over | qs.DEV_SELECT, 0]
        oc.state[:, oracle.ERR] = 0
        if paged:
            paging.assert_groups_equal(cache, oc, "append")
            got, gl = run(torch, cache, mode, q, k=k[:, :, :1], v=v[:, :, :1])
            oc.append(k[:, :, :1], v[:, :, :1])
            ref, rl = paging.attention(oc, q, mode == DRAFT)
            assert_close(got, ref, gl, rl, "paged append, mode %d" % mode)
            qs.qs_get_errors(cache)
            oc.state[:, oracle.ERR] = 0
    assert np.array_equal(cache.state[:, :4].cpu().numpy(), oc.state[:, :4])


def test_host_errors(torch):
    cache = qs.PagedCache(1, 2, 3, 4)
    q = torch.zeros((1, 2, 1, 128), dtype=torch.float16, device="cuda")
    sel = torch.zeros((1, 2, 1), dtype=torch.int32, device="cuda")
    for call in (lambda: qs.qs_attn_decode_paged(cache, DRAFT, q, 0.1, torch.empty_like(q)),
                 lambda: qs.qs_attn_decode_sparse(cache, DRAFT, sel, q, 0.1, torch.empty_like(q))):
        with pytest.raises(qs.QsError) as e:
            call()
        assert e.value.status == qs.QS_ERR_WORKSPACE
    with pytest.raises(qs.QsError) as e:
        qs.qs_attn_decode_paged(qs.Cache(1, 2, 3), DRAFT, q, 0.1, torch.empty_like(q))
    assert e.value.status == qs.QS_ERR_ARG


def test_captured_round_replays(torch):
    """Append + sparse draft, append + paged verify and the rollbacks captured
    into one graph: each replay advances the cache as the eager calls do."""
    rng = np.random.default_rng(44)
    B, H, ng = 2, 4, [9, 5]
    oc = _oracle_state(rng, B, H, ng, [40, 90], cap=9)
    cache = load(torch, oc, rng)
    sel = random_sel(rng, B, H, 4, ng)
    k, v, q = (h16(rng, (B, H, 3, 128)) for _ in range(3))
    drop = np.array([1, 2], np.int32)
    dev = [to_dev(torch, x) for x in (k[:, :, :1], v[:, :, :1], q[:, :, :1], k, v, q)]
    d1, dr, sd = to_dev(torch, np.ones(B, np.int32)), to_dev(torch, drop), to_dev(torch, sel.astype(np.int32))
    out = [torch.empty_like(dev[2]), torch.empty_like(dev[5])]
    ws = torch.empty(qs.qs_attn_workspace_size(cache, 3), dtype=torch.uint8, device="cuda")

    def step():
        qs.qs_attn_decode_sparse(cache, DRAFT, sd, dev[2], 1 / np.sqrt(128), out[0], None, ws,
                                 k_new=dev[0], v_new=dev[1])
        qs.qs_buffer_rollback(cache, d1)
        qs.qs_attn_decode_paged(cache, VERIFY, dev[5], 1 / np.sqrt(128), out[1], None, ws,
                                k_new=dev[3], v_new=dev[4])
        qs.qs_buffer_rollback(cache, dr)

    def want():
        oc.append(k[:, :, :1], v[:, :, :1])
        a = paging.attention(oc, q[:, :, :1], True, sel=sel)[0]
        oc.rollback([1, 1])
        oc.append(k, v)
        b = paging.attention(oc, q, False)[0]
        oc.rollback(drop)
        return a, b

    step()
    torch.cuda.synchronize()
    want()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(out, want()):
            assert_close(got.double().cpu().numpy(), ref)
    assert np.array_equal(cache.state[:, :4].cpu().numpy(), oc.state[:, :4])
    assert np.all(qs.qs_get_errors(cache) == 0)
