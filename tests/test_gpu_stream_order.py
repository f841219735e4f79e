"""What one call writes and the next one reads, many calls deep on one stream
without a host wait, the same buffers reused with changing contents: flush
masks, drop counts, rows read back that are appended, prefilled or used as
queries.  The results are those of the calls one after the other."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import (DRAFT, VERIFY, _oracle_state, assert_close, assert_state_equal, h16,
                               to_dev)
from tests.test_gpu_read import expected
from tests.test_gpu_spec import draw, softmax_rows

pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(128)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


@pytest.mark.parametrize("paged", [False, True])
def test_masks_of_need_flush(torch, paged):
    """One mask array for every round: other sequences are due each time."""
    rng = np.random.default_rng(1)
    B, H, cap, rounds = 9, 2, 12, 150
    n = rng.integers(1, 10, rounds)
    k, v = (h16(rng, (rounds, B, H, 9, 128)) for _ in "kv")
    oc = oracle.OracleCache(B, H, 128, 128, cap)
    first = h16(rng, (B, H, 256, 128))
    lens = rng.integers(0, 257, B).astype(np.int32)
    oc.prefill(first, first, lens)
    if paged:
        cache = qs.PagedCache(B, H, cap, B * cap)
        cache.table.copy_(torch.from_numpy(rng.permutation(B * cap).astype(np.int32).reshape(B, cap)))
        qs.qs_prefill_paged(cache, to_dev(torch, first), to_dev(torch, first), to_dev(torch, lens))
        flush = qs.qs_quantize_flush_paged
    else:
        cache = qs.Cache(B, H, cap)
        qs.qs_prefill(cache, to_dev(torch, first), to_dev(torch, first), to_dev(torch, lens))
        flush = qs.qs_quantize_flush
    new = [[to_dev(torch, x[i, :, :, :n[i]]) for i in range(rounds)] for x in (k, v)]
    mask = torch.zeros(B, dtype=torch.uint8, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for i in range(rounds):
        qs.qs_need_flush(cache, n[i], mask)
        flush(cache, mask)
        qs.qs_buffer_append(cache, new[0][i], new[1][i])
        qs.qs_buffer_rollback(cache, zero)
    due = 0
    for i in range(rounds):
        m = oc.need_flush(n[i])
        due += 0 < m.sum() < B
        oc.flush(m)
        oc.append(k[i, :, :, :n[i]], v[i, :, :, :n[i]])
        oc.rollback([0] * B)
    assert due > 20  # the masks do differ from round to round
    if paged:
        paging.assert_groups_equal(cache, oc)
    else:
        torch.cuda.synchronize()
        assert_state_equal(cache, oc)
    assert np.all(qs.qs_get_errors(cache) == 0)


def test_drop_counts_of_spec_accept(torch):
    """Append, accept, roll back, with one n_drop array."""
    rng = np.random.default_rng(2)
    B, H, g, V, rounds = 6, 2, 4, 90, 120
    p = softmax_rows(rng, (rounds, B, g + 1, V), 1.0)
    q = (0.7 * p[:, :, :g] + 0.3 * softmax_rows(rng, (rounds, B, g, V), 1.0)).astype(np.float32)
    draft = np.stack([draw(rng, x) for x in q])
    u, e = rng.random((rounds, B, g)).astype(np.float32), rng.exponential(size=(rounds, B, V)).astype(np.float32)
    k, v = (h16(rng, (rounds, B, H, g, 128)) for _ in "kv")
    dev = [to_dev(torch, x) for x in (p, q, draft, u, e, k, v)]
    n_accept, token, n_drop = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    tokens = torch.zeros((rounds, B), dtype=torch.int32, device="cuda")
    cache, oc = qs.Cache(B, H, 6), oracle.OracleCache(B, H, 128, 128, 6)
    torch.cuda.synchronize()
    for i in range(rounds):
        qs.qs_quantize_flush_due(cache, g)
        qs.qs_buffer_append(cache, dev[5][i], dev[6][i])
        qs.qs_spec_accept(*(x[i] for x in dev[:5]), n_accept, tokens[i], n_drop)
        qs.qs_buffer_rollback(cache, n_drop)
    want, drops = [], set()
    for i in range(rounds):
        oc.flush(oc.need_flush(g))
        oc.append(k[i], v[i])
        _, t, d = oracle.spec_accept(p[i], q[i], draft[i], u[i], e[i])
        oc.rollback(d)
        want.append(t)
        drops.add(tuple(d))
    assert len(drops) > 20
    torch.cuda.synchronize()
    assert np.array_equal(tokens.cpu().numpy(), np.stack(want))
    assert_state_equal(cache, oc)
    assert np.all(qs.qs_get_errors(cache) == 0)


def test_rows_read_back(torch):
    """Rows of one cache, read into the same arrays round after round, are
    appended to another and are the queries of attention over a third."""
    rng = np.random.default_rng(3)
    B, H, T, rounds = 2, 3, 5, 100
    src = _oracle_state(rng, B, H, [3, 3], [120, 116], cap=3)
    third = _oracle_state(rng, B, H, [4, 6], [90, 33], cap=6, k_scale=0.5)
    a, c = load(torch, src, rng), load(torch, third, rng)
    dst, od = qs.Cache(B, H, 4), oracle.OracleCache(B, H, 128, 128, 4)
    k, v = (torch.zeros((B, H, T, 128), dtype=torch.float16, device="cuda") for _ in "kv")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.zeros((rounds, B, H, T, 128), dtype=torch.float16, device="cuda")
    ws = torch.empty(qs.qs_attn_workspace_size(c, T), dtype=torch.uint8, device="cuda")
    starts = [int(x) for x in rng.integers(0, 490, rounds)]
    torch.cuda.synchronize()
    for i, t in enumerate(starts):
        qs.qs_cache_read(a, VERIFY, k, v, tok0=t)
        qs.qs_quantize_flush_due(dst, T)
        qs.qs_buffer_append(dst, k, v)
        qs.qs_buffer_rollback(dst, zero)
        qs.qs_attn_decode_paged(c, (DRAFT, VERIFY)[i & 1], v, SCALE, out[i], None, ws)
    torch.cuda.synchronize()
    rows = [x.view(np.float16) for x in expected(src, VERIFY, 4, 0, 500)]
    got = out.double().cpu().numpy()
    for i, t in enumerate(starts):
        kr, vr = (x[:, :, t:t + T] for x in rows)
        od.flush(od.need_flush(T))
        od.append(kr, vr)
        od.rollback([0, 0])
        assert_close(got[i], paging.attention(third, vr, i & 1 == 0)[0], what="round %d" % i)
    assert_state_equal(dst, od)
    for x in (a, dst, c):
        assert np.all(qs.qs_get_errors(x) == 0)


def test_prompts_read_back(torch):
    """A prompt read from one cache, of another length each time, fills the
    next one."""
    rng = np.random.default_rng(4)
    B, H, T = 2, 2, 700
    src = _oracle_state(rng, B, H, [4, 4], [200, 200], cap=4)
    a = load(torch, src, rng)
    k, v = (torch.zeros((B, H, T, 128), dtype=torch.float16, device="cuda") for _ in "kv")
    lens = rng.integers(0, T + 1, (12, B)).astype(np.int32)
    starts = [int(x) for x in rng.integers(0, 12, len(lens))]
    dl = to_dev(torch, lens)
    caches = [qs.Cache(B, H, 6) for _ in lens]
    torch.cuda.synchronize()
    for i, cache in enumerate(caches):
        qs.qs_cache_read(a, VERIFY, k, v, tok0=starts[i])
        qs.qs_prefill(cache, k, v, dl[i])
    torch.cuda.synchronize()
    rows = [x.view(np.float16) for x in expected(src, VERIFY, 4, 0, 712)]
    for i, cache in enumerate(caches):
        oc = oracle.OracleCache(B, H, 128, 128, 6)
        oc.prefill(*(np.ascontiguousarray(x[:, :, starts[i]:starts[i] + T]) for x in rows), lens[i])
        assert_state_equal(cache, oc, "prompt %d" % i)
