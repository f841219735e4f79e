"""qs_cache_read against the oracle's codes, scales and zeros in 64 bits: the
row of a quantized token is s * code + z rounded once to fp16, so it is
compared bit for bit; buffered rows are the appended bytes; rows past the end
stay as they were."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import layout, paging
from tests.test_gpu_qs import DRAFT, VERIFY, _degenerate_tokens, _oracle_state, h16, to_dev

pytestmark = pytest.mark.gpu

MARK = np.float16(-77.0)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def read(torch, cache, mode, tok0, T, which="kv"):
    shape = (cache.B, cache.H, T, 128)
    k, v = (torch.full(shape, float(MARK), dtype=torch.float16, device="cuda") if n in which else None
            for n in "kv")
    qs.qs_cache_read(cache, mode, k, v, tok0=tok0)
    torch.cuda.synchronize()
    return tuple(None if x is None else x.cpu().numpy().view(np.uint16) for x in (k, v))


def to_fp16(x):
    with np.errstate(over="ignore"):
        return np.clip(x, -65504.0, 65504.0).astype(np.float16)


def expected(oc, mode, ub, tok0, T):
    out = [np.full((oc.B, oc.H, T, 128), MARK, np.float16) for _ in "kv"]
    for b in range(oc.B):
        for x, d in zip(out, paging.dequantized(oc, b, mode == DRAFT, ub)):
            rows = to_fp16(d[:, tok0:tok0 + T])
            x[b, :, :rows.shape[1]] = rows
    return tuple(x.view(np.uint16) for x in out)


def load(torch, oc, rng, ub, paged):
    if paged:
        return paging.paged_copy(torch, oc, rng, ub)
    cache = qs.Cache(oc.B, oc.H, oc.cap, upper_bits=ub)
    layout.load_into(cache, oc)
    return cache


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("mode", [DRAFT, VERIFY])
def test_windows(torch, mode, ub, paged):
    rng = np.random.default_rng(17)
    ng, fill = [3, 0, 1], [200, 1, 256]
    oc = _oracle_state(rng, 3, 2, ng, fill, cap=4)
    oc.state[2, oracle.HALF_BASE] = 1
    oc.state[0, oracle.PENDING] = 5
    cache = load(torch, oc, rng, ub, paged)
    for tok0, T in ((0, 584), (0, 1), (0, 128), (1, 127), (127, 2), (129, 300), (383, 1), (384, 256),
                    (500, 400), (583, 1), (584, 10), (1 << 30, 3)):
        got, want = read(torch, cache, mode, tok0, T), expected(oc, mode, ub, tok0, T)
        for n, g, w in zip("kv", got, want):
            assert np.array_equal(g, w), (tok0, T, n)
    for which in "kv":  # one of the two alone
        got, want = read(torch, cache, mode, 100, 350, which), expected(oc, mode, ub, 100, 350)
        i = "kv".index(which)
        assert got[1 - i] is None and np.array_equal(got[i], want[i])
    assert np.all(qs.qs_get_errors(cache) == 0)


@pytest.mark.parametrize("extreme", [False, True])
def test_degenerate_groups(torch, extreme):
    """Constant groups, subnormal scales, the fp16 extremes (a value past the
    largest fp16 is held there), each reading still one rounding away from
    s * code + z."""
    rng = np.random.default_rng(41 + extreme)
    k, v = _degenerate_tokens(rng, 2, extreme)
    pad = [h16(rng, (1, 2, 256, 128)) for _ in "kv"]
    k, v = np.concatenate([k, pad[0]], 2), np.concatenate([v, pad[1]], 2)
    oc = oracle.OracleCache(1, 2, 128, 128, 2)
    oc.prefill(k, v, [384])
    for ub in (4, 2):
        cache = load(torch, oc, rng, ub, False)
        for mode in (DRAFT, VERIFY):
            got, want = read(torch, cache, mode, 0, 384), expected(oc, mode, ub, 0, 384)
            for g, w in zip(got, want):
                g, w = g.view(np.float16), w.view(np.float16)
                assert np.array_equal(g, w)  # (by value: -0 equals +0)
                assert np.all(np.isfinite(g))


def test_bad_page_leaves_its_rows(torch):
    rng = np.random.default_rng(8)
    oc = _oracle_state(rng, 2, 2, [3, 2], [40, 40], cap=3)
    cache = paging.paged_copy(torch, oc, rng)
    want = expected(oc, VERIFY, 4, 0, 424)
    cache.table[0, 1] = cache.n_pages
    got = read(torch, cache, VERIFY, 0, 424)
    for g, w in zip(got, want):
        w[0, :, 128:256] = MARK.view(np.uint16)
        assert np.array_equal(g, w)
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_PAGE, 0]
    read(torch, cache, VERIFY, 256, 10)  # a window that does not need it
    assert list(qs.qs_get_errors(cache)) == [0, 0]


def test_after_writes_on_one_stream(torch):
    """Prefill, append, flush and reads in one stream order, no host wait
    between them, on a stream of its own; the read sees each write."""
    rng = np.random.default_rng(9)
    B, H, cap = 2, 3, 6
    lens = np.array([600, 257], np.int32)
    k, v = h16(rng, (B, H, 600, 128), 2.0), h16(rng, (B, H, 600, 128))
    kn, vn = h16(rng, (B, H, 50, 128), 2.0), h16(rng, (B, H, 50, 128))
    oc = oracle.OracleCache(B, H, 128, 128, cap)
    oc.prefill(k, v, lens)
    want1 = expected(oc, VERIFY, 4, 0, 700)
    oc.flush(oc.need_flush(50))
    oc.append(kn, vn)
    want2 = expected(oc, DRAFT, 4, 0, 700)
    cache = qs.PagedCache(B, H, cap, 12)
    cache.table.copy_(torch.from_numpy(paging.random_table(rng, [cap, cap], cap, 12)))
    args = [to_dev(torch, x) for x in (k, v, lens, kn, vn)]
    out = [torch.full((B, H, 700, 128), float(MARK), dtype=torch.float16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    qs.qs_prefill_paged(cache, *args[:3], stream=s)
    qs.qs_cache_read(cache, VERIFY, out[0], out[1], stream=s)
    qs.qs_quantize_flush_due_paged(cache, 50, stream=s)
    qs.qs_buffer_append(cache, *args[3:], stream=s)
    qs.qs_cache_read(cache, DRAFT, out[2], out[3], stream=s)
    s.synchronize()
    for g, w in zip(out, want1 + want2):
        assert np.array_equal(g.cpu().numpy().view(np.uint16), w)
    assert np.all(qs.qs_get_errors(cache) == 0)
