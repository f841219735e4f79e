"""The paged and sparse calls beside one another: two caches on two streams,
the largest batch, selections and reads captured into graphs, and what one
call leaves for the next."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_listed_attn import load, random_sel, run
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, assert_close, h16, to_dev
from tests.test_gpu_read import expected

pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(128)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def test_two_caches_on_two_streams(torch):
    """Each stream selects and attends on its own cache, forty calls deep and
    never waited for in between."""
    rng = np.random.default_rng(1)
    B, H, k = 1, 8, 5
    side = []
    for _ in range(2):
        oc = _oracle_state(rng, B, H, [30], [120], cap=30)
        q = h16(rng, (20, B, H, 1, 128))
        side.append(dict(oc=oc, q=q, cache=load(torch, oc, rng), qd=to_dev(torch, q),
                         sel=torch.empty((20, B, H, k), dtype=torch.int32, device="cuda"),
                         out=torch.empty((20, B, H, 1, 128), dtype=torch.float16, device="cuda"),
                         s=torch.cuda.Stream()))
        side[-1]["ws"] = torch.empty(qs.qs_attn_workspace_size(side[-1]["cache"], 1), dtype=torch.uint8,
                                     device="cuda")
    torch.cuda.synchronize()
    for i in range(20):
        for x in side:
            qs.qs_select_groups(x["cache"], x["qd"][i], x["sel"][i], stream=x["s"])
            qs.qs_attn_decode_sparse(x["cache"], DRAFT, x["sel"][i], x["qd"][i], SCALE, x["out"][i], None,
                                     x["ws"], stream=x["s"])
    torch.cuda.synchronize()
    for x in side:
        for i in range(20):
            want = paging.select(x["oc"], x["q"][i], k)
            assert np.array_equal(x["sel"][i].cpu().numpy(), want)
            assert_close(x["out"][i].double().cpu().numpy(),
                         paging.attention(x["oc"], x["q"][i], True, sel=want)[0])


def test_largest_batch(torch):
    rng = np.random.default_rng(2)
    B, H = 256, 2
    ng = [int(x) for x in rng.integers(0, 5, B)]
    fill = [int(x) for x in rng.integers(1, 257, B)]
    oc = _oracle_state(rng, B, H, ng, fill, cap=4)
    cache = load(torch, oc, rng)
    sel = random_sel(rng, B, H, 2, ng)
    q = h16(rng, (B, H, 1, 128))
    for mode in (DRAFT, VERIFY):
        for s in (None, sel):
            got, gl = run(torch, cache, mode, q, sel=s)
            ref, rl = paging.attention(oc, q, mode == DRAFT, sel=s)
            assert_close(got, ref, gl, rl)
    got = torch.empty((B, H, 2), dtype=torch.int32, device="cuda")
    qs.qs_select_groups(cache, to_dev(torch, q), got)
    assert np.array_equal(got.cpu().numpy(), paging.select(oc, q, 2))
    qs.qs_quantize_flush_due_paged(cache, 0)  # nobody is due
    assert np.all(qs.qs_get_errors(cache) == 0)


def test_captured_selection_and_read(torch):
    """Select, attend, flush and read in a graph: a replay follows the cache as
    it is then, not as it was when captured."""
    rng = np.random.default_rng(3)
    B, H, k, cap = 2, 4, 3, 8
    oc = _oracle_state(rng, B, H, [5, 2], [256, 140], cap=cap)
    cache = paging.paged_copy(torch, oc, rng, spare=12)
    table = cache.table.cpu().numpy()
    free = iter(np.setdiff1d(np.arange(cache.n_pages), np.concatenate([table[0, :5], table[1, :2]])))
    for b, n in ((0, 5), (1, 2)):
        for g in range(n, n + 3):
            table[b, g] = next(free)
    cache.table.copy_(torch.from_numpy(table))
    q = h16(rng, (B, H, 1, 128))
    kn, vn = h16(rng, (B, H, 60, 128), 2.0), h16(rng, (B, H, 60, 128))
    qd, kd, vd = (to_dev(torch, x) for x in (q, kn, vn))
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    sel = torch.empty((B, H, k), dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(qd), torch.empty(qs.qs_attn_workspace_size(cache, 1), dtype=torch.uint8, device="cuda")
    rd = [torch.zeros((B, H, 1200, 128), dtype=torch.float16, device="cuda") for _ in "kv"]

    def step():
        qs.qs_quantize_flush_due_paged(cache, 60)
        qs.qs_buffer_append(cache, kd, vd)
        qs.qs_buffer_rollback(cache, zero)
        qs.qs_select_groups(cache, qd, sel)
        qs.qs_attn_decode_sparse(cache, VERIFY, sel, qd, SCALE, out, None, ws)
        qs.qs_cache_read(cache, VERIFY, *rd)

    def advance():
        oc.flush(oc.need_flush(60))
        oc.append(kn, vn)
        oc.rollback([0, 0])

    step()
    advance()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        g.replay()
        advance()
        torch.cuda.synchronize()
        want = paging.select(oc, q, k)
        assert np.array_equal(sel.cpu().numpy(), want)
        assert_close(out.double().cpu().numpy(), paging.attention(oc, q, False, sel=want)[0])
        for got, x in zip(rd, expected(oc, VERIFY, 4, 0, 1200)):
            for b in range(B):
                n = oc.counters(b)["n_groups"] * 128 + oc.counters(b)["fill"]
                assert np.array_equal(got[b, :, :n].cpu().numpy().view(np.uint16), x[b, :, :n])
    assert oc.state[0, oracle.N_GROUPS] >= 7
    assert np.all(qs.qs_get_errors(cache) == 0)


def test_reset_empties_a_paged_cache(torch):
    rng = np.random.default_rng(4)
    cache = qs.PagedCache(3, 5, 4, 9)
    cache.state.random_(0, 100)
    cache.arrive.fill_(3)
    qs.qs_state_reset(cache)
    assert not cache.state.any() and not cache.arrive.any()
    wide = qs.Cache(200, 7, 1)
    wide.state.fill_(5)
    wide.arrive.fill_(5)
    qs.qs_state_reset(wide)
    assert not wide.state.any() and not wide.arrive.any()
    del rng
