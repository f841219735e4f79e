"""qs_select_groups against the definition in 64 bits: the indices have to be
equal (close scores are summed exactly, ties go to the lower index)."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import DRAFT, VERIFY, assert_close, h16, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def metadata_cache(rng, B, H, n_groups, cap, spread=1.0):
    """An oracle cache with random key boxes (codes and values stay zero: the
    selection reads neither)."""
    oc = oracle.OracleCache(B, H, 128, 128, cap)
    lo = rng.standard_normal(oc.kz.shape) * spread - 2.5
    oc.kz[:] = lo.astype(np.float16).view(np.uint16)
    oc.ks[:] = (rng.random(oc.ks.shape) * 0.02 + 0.01).astype(np.float16).view(np.uint16)
    oc.state[:, oracle.N_GROUPS] = n_groups
    oc.state[:, oracle.FILL] = 10
    return oc


def run(torch, cache, q, k, group=1, stream=None):
    sel = torch.full((cache.B, cache.H, k), -99, dtype=torch.int32, device="cuda")
    qs.qs_select_groups(cache, to_dev(torch, q), sel, group=group, stream=stream)
    torch.cuda.synchronize()
    return sel.cpu().numpy()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n_q,group", [(1, 1), (1, 4), (5, 1), (8, 1), (3, 3), (4, 4), (5, 4), (8, 3)])
@pytest.mark.parametrize("k", [1, 7, 32, 100])
def test_select(torch, k, n_q, group, paged):
    rng = np.random.default_rng([k, n_q, group])
    B, H, ng, cap = 5, 3, [33, 0, 200, 7, 129], 200
    oc = metadata_cache(rng, B, H, ng, cap)
    cache = load(torch, oc, rng, paged=paged)
    q = h16(rng, (B, H * group, n_q, 128))
    assert np.array_equal(run(torch, cache, q, k, group), paging.select(oc, q, k, group))
    assert np.all(qs.qs_get_errors(cache) == 0)


@pytest.mark.parametrize("B,H,n,k", [(1, 2, 1022, 64), (1, 1, 5000, 300), (2, 3, 1300, 1299),
                                     (1, 2, 300, 299), (40, 32, 20, 3), (1, 32, 254, 32),
                                     (1, 1, 12800, 500)])
def test_sizes(torch, B, H, n, k):
    """Clusters of one to eight CTAs, several passes a warp."""
    rng = np.random.default_rng(n + k)
    oc = metadata_cache(rng, B, H, rng.integers(n // 2, n + 1, B), n)
    cache = load(torch, oc, rng, paged=False)
    q = h16(rng, (B, H, 1, 128))
    for _ in range(2):
        assert np.array_equal(run(torch, cache, q, k), paging.select(oc, q, k))


@pytest.mark.parametrize("n", [40, 600])
def test_close_scores(torch, n):
    """Boxes that differ by one fp16 step in one small channel, under large
    terms that cancel: fp32 sums cannot order them."""
    rng = np.random.default_rng(n)
    oc = metadata_cache(rng, 1, 2, [n], n)
    oc.kz[:] = oc.kz[:, :, :1]
    oc.ks[:] = oc.ks[:, :, :1]
    z = oc.kz.view(np.float16)
    z[..., 0], z[..., 1] = 3000.0, 3000.0
    z[..., 5] = (2.0 ** -9 * (1 + rng.integers(0, 64, z.shape[:3]) / 1024)).astype(np.float16)
    q = h16(rng, (1, 2, 1, 128))
    q[..., 0], q[..., 1], q[..., 5] = 50.0, -50.0, 0.5
    cache = load(torch, oc, rng, paged=False)
    for k in (1, 5, n // 2, n - 1):
        assert np.array_equal(run(torch, cache, q, k), paging.select(oc, q, k)), k


@pytest.mark.parametrize("scale", [1e-4, 2e-6])
def test_subnormal_boxes(torch, scale):
    """Zeros and scales below the smallest normal fp16 number."""
    rng = np.random.default_rng(11)
    oc = metadata_cache(rng, 1, 3, [400], 400)
    for x in (oc.kz, oc.ks):
        x[:] = (x.view(np.float16).astype(np.float64) * scale).astype(np.float16).view(np.uint16)
    cache = load(torch, oc, rng, paged=False)
    for q in (h16(rng, (1, 3, 1, 128)), h16(rng, (1, 3, 1, 128), 1e-4), h16(rng, (1, 3, 1, 128), 1e3)):
        for k in (1, 50, 200):
            assert np.array_equal(run(torch, cache, q, k), paging.select(oc, q, k))


def test_ties_go_to_the_lower_index(torch):
    rng = np.random.default_rng(3)
    oc = metadata_cache(rng, 2, 2, [500, 90], 500)
    cache = load(torch, oc, rng, paged=False)
    zero = np.zeros((2, 2, 1, 128), np.float16)
    zero[1] = -0.0
    got = run(torch, cache, zero, 37)  # queries of zeros: every score is zero
    assert np.array_equal(got, np.broadcast_to(np.arange(37), got.shape))
    # every group three times over
    oc.kz[:] = oc.kz[:, :, np.arange(500) % 167]
    oc.ks[:] = oc.ks[:, :, np.arange(500) % 167]
    cache = load(torch, oc, rng, paged=False)
    q = h16(rng, (2, 2, 1, 128))
    for k in (1, 2, 50, 89):
        assert np.array_equal(run(torch, cache, q, k), paging.select(oc, q, k)), k


def test_empty_and_small_sequences(torch):
    rng = np.random.default_rng(4)
    oc = metadata_cache(rng, 3, 2, [0, 1, 4], 4)
    cache = load(torch, oc, rng)
    for k in (1, 4, 9):
        q = h16(rng, (3, 2, 1, 128))
        assert np.array_equal(run(torch, cache, q, k), paging.select(oc, q, k))


def test_bad_pages_come_last(torch):
    rng = np.random.default_rng(5)
    oc = metadata_cache(rng, 2, 2, [60, 20], 60)
    cache = load(torch, oc, rng)
    bad = [(0, 3), (0, 40), (0, 59)]
    for b, g in bad:
        cache.table[b, g] = -1 if g == 3 else cache.n_pages
    q = h16(rng, (2, 2, 1, 128))
    for k in (1, 30, 57):
        assert np.array_equal(run(torch, cache, q, k), paging.select(oc, q, k, left_out=bad))
        errs = qs.qs_get_errors(cache)
        assert list(errs) == [qs.DEV_PAGE, 0]
    got = run(torch, cache, q, 58)  # one more than there are good pages: the lowest bad one
    assert np.array_equal(got, paging.select(oc, q, 58, left_out=bad))
    assert got[0, 0].tolist().count(3) == 1


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_queries_that_are_not_finite(torch, bad):
    """Some valid selection: distinct ascending indices, no error, and the
    other heads' selections untouched by it."""
    rng = np.random.default_rng(6)
    oc = metadata_cache(rng, 1, 3, [300], 300)
    cache = load(torch, oc, rng, paged=False)
    q = h16(rng, (1, 3, 2, 128))
    want = paging.select(oc, q, 40)
    q[0, 1, 1, 17] = bad
    got = run(torch, cache, q, 40)
    assert np.array_equal(got[0, [0, 2]], want[0, [0, 2]])
    row = got[0, 1]
    assert np.all(np.diff(row) > 0) and row[0] >= 0 and row[-1] < 300


def test_select_then_attend_round(torch):
    """The operators as a server uses them, on one stream and without a host
    wait: prompts written to pages, a selection, draft steps over the selected
    groups (append fused), rollback, verify over everything, rollback, flush
    into a new page, and the cache read back."""
    rng = np.random.default_rng(7)
    B, H, group, cap, k, gamma = 2, 2, 4, 12, 4, 3
    lens = np.array([1500, 700], np.int32)
    oc = oracle.OracleCache(B, H, 128, 128, cap)
    k0, v0 = h16(rng, (B, H, 1500, 128), 2.0), h16(rng, (B, H, 1500, 128))
    oc.prefill(k0, v0, lens)
    cache = qs.PagedCache(B, H, cap, 30)
    cache.table.copy_(torch.from_numpy(paging.random_table(rng, [cap, cap], cap, 30)))
    hq, scale = H * group, 1 / np.sqrt(128)
    dk, dv = h16(rng, (gamma, B, H, 1, 128), 2.0), h16(rng, (gamma, B, H, 1, 128))
    dq = h16(rng, (gamma, B, hq, 1, 128))
    vk, vv = h16(rng, (B, H, gamma + 1, 128), 2.0), h16(rng, (B, H, gamma + 1, 128))
    vq = h16(rng, (B, hq, gamma + 1, 128))
    drop = np.array([2, 0], np.int32)
    d = [to_dev(torch, x) for x in (k0, v0, lens, dk, dv, dq, vk, vv, vq, np.full(B, gamma, np.int32), drop)]
    ws = torch.empty(qs.qs_attn_workspace_size_gqa(cache, gamma + 1, group), dtype=torch.uint8, device="cuda")
    sel = torch.empty((B, H, k), dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(x) for x in d[5]] + [torch.empty_like(d[8])]
    rd = [torch.zeros((B, H, 1510, 128), dtype=torch.float16, device="cuda") for _ in "kv"]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    qs.qs_prefill_paged(cache, *d[:3], stream=s)
    qs.qs_select_groups(cache, d[5][0], sel, group=group, stream=s)
    for i in range(gamma):
        qs.qs_attn_decode_sparse(cache, DRAFT, sel, d[5][i], scale, outs[i], None, ws, group=group,
                                 k_new=d[3][i], v_new=d[4][i], stream=s)
    qs.qs_buffer_rollback(cache, d[9], stream=s)
    qs.qs_attn_decode_paged(cache, VERIFY, d[8], scale, outs[-1], None, ws, group=group, k_new=d[6],
                            v_new=d[7], stream=s)
    qs.qs_buffer_rollback(cache, d[10], stream=s)
    qs.qs_quantize_flush_due_paged(cache, 128, stream=s)
    qs.qs_cache_read(cache, VERIFY, *rd, stream=s)
    s.synchronize()
    want = paging.select(oc, dq[0], k, group)
    assert np.array_equal(sel.cpu().numpy(), want)
    for i in range(gamma):
        oc.append(dk[i], dv[i])
        assert_close(outs[i].double().cpu().numpy(), paging.attention(oc, dq[i], True, group, sel=want)[0])
    oc.rollback([gamma, gamma])
    oc.append(vk, vv)
    assert_close(outs[-1].double().cpu().numpy(), paging.attention(oc, vq, False, group)[0])
    oc.rollback(drop)
    oc.flush(oc.need_flush(128))
    paging.assert_groups_equal(cache, oc, "round")
    for b in range(B):
        for got, x in zip(rd, paging.dequantized(oc, b, False)):
            got = got[b].cpu().numpy()
            assert np.array_equal(got[:, :x.shape[1]], x.astype(np.float16))
            assert not got[:, x.shape[1]:].any()
    assert np.all(qs.qs_get_errors(cache) == 0)


def test_no_token_left_out_scores_above_the_selected_boxes(torch):
    """What the score promises: it bounds every key of its group, so no token
    of a group that is left out scores above the lowest box score among the
    selected groups (queries aligned to one token of the context each)."""
    rng = np.random.default_rng(8)
    B, H, T = 1, 4, 6000
    k, v = h16(rng, (B, H, T, 128)), h16(rng, (B, H, T, 128))
    cache = qs.Cache(B, H, 60)
    qs.qs_prefill(cache, to_dev(torch, k), to_dev(torch, v), to_dev(torch, np.array([T], np.int32)))
    oc = oracle.OracleCache(B, H, 128, 128, 60)
    oc.prefill(k, v, [T])
    at = [7, 1000, 2500, 5000]
    q = np.stack([k[0, h, at[h]] for h in range(H)])[None, :, None]
    got = run(torch, cache, q, 4)
    assert np.array_equal(got, paging.select(oc, q, 4))
    n = oc.counters(0)["n_groups"]
    keys = paging.dequantized(oc, 0, False)[0][:, :n * 128].reshape(H, n, 128, 128)
    for h in range(H):
        qh = q[0, h, 0].astype(np.float64)
        best = (keys[h] @ qh).max(-1)
        lo, s = (x[0, h, :n].view(np.float16).astype(np.float64) for x in (oc.kz, oc.ks))
        box = np.maximum(qh * lo, qh * (lo + 255 * s)).sum(-1)
        assert np.all(best <= box)
        rest = np.setdiff1d(np.arange(n), got[0, h])
        assert best[rest].max() <= box[got[0, h]].min()
