"""Paged caches and the read back: what the host refuses before any CUDA
call, and the sizes of a paged cache's arrays (no GPU needed)."""
import ctypes

import pytest

import __graft_entry__
from hierarchical_quantized_kv_gb300 import qs

P = ctypes.c_void_p(0x20000)


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return qs.lib()


def cache(paged, **kw):
    c = qs.QsCacheStruct(1, 2, 128, 128, 4, 4 | (qs.QS_PAGED if paged else 0), *([0x10000] * 9))
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def pages(table=0x30000, n_pages=5):
    return ctypes.byref(qs.QsPagesStruct(table, n_pages))


#: calls that take (cache, pages, ...): for a paged cache alone, or for either kind
PAGED_ONLY = {
    "qs_quantize_flush_paged": lambda f, c, pg: f(c, pg, None, None),
    "qs_quantize_flush_due_paged": lambda f, c, pg: f(c, pg, 1, None),
    "qs_prefill_paged": lambda f, c, pg: f(c, pg, P, P, 10, P, None),
    "qs_attn_decode_paged": lambda f, c, pg: f(c, pg, 0, None, None, 0, P, 1, 1, ctypes.c_float(0.1), P,
                                               None, P, 1 << 30, None),
}
F = ctypes.c_float
EITHER = {
    "qs_select_groups": lambda f, c, pg: f(c, pg, P, 1, 1, 3, P, None),
    "qs_attn_decode_sparse": lambda f, c, pg: f(c, pg, 0, P, 3, None, None, 0, P, 1, 1, F(0.1), P, None,
                                                P, 1 << 30, None),
    "qs_cache_read": lambda f, c, pg: f(c, pg, 1, 0, 5, P, P, None),
}
#: calls for contiguous groups
CONTIGUOUS = {
    "qs_quantize_flush": lambda f, c: f(c, None, None),
    "qs_quantize_flush_due": lambda f, c: f(c, 1, None),
    "qs_prefill": lambda f, c: f(c, P, P, 10, P, None),
    "qs_attn_decode": lambda f, c: f(c, 0, P, 1, ctypes.c_float(0.1), P, None, P, 1 << 30, None),
    "qs_attn_decode_gqa": lambda f, c: f(c, 0, P, 1, 1, ctypes.c_float(0.1), P, None, P, 1 << 30, None),
    "qs_attn_decode_append": lambda f, c: f(c, 0, P, P, 1, P, 1, 1, ctypes.c_float(0.1), P, None, P,
                                            1 << 30, None),
    "qs_attn_decode_static_ws": lambda f, c: f(c, 0, P, 1, ctypes.c_float(0.1), P, None, None),
}


@pytest.mark.parametrize("name", sorted(PAGED_ONLY) + sorted(EITHER))
def test_pages_are_checked(L, name):
    call = {**PAGED_ONLY, **EITHER}[name]
    f = getattr(L, name)
    assert call(f, cache(True), None) == qs.QS_ERR_ARG          # a paged cache without its pages
    assert call(f, cache(False), pages()) == qs.QS_ERR_ARG      # pages for a contiguous cache
    if name in PAGED_ONLY:
        assert call(f, cache(False), None) == qs.QS_ERR_ARG
    assert call(f, cache(True), pages(table=None)) == qs.QS_ERR_ARG
    assert call(f, cache(True), pages(n_pages=0)) == qs.QS_ERR_SHAPE
    assert call(f, cache(True), pages(table=0x30002)) == qs.QS_ERR_ALIGN
    assert call(f, cache(True, upper_bits=qs.QS_PAGED | 3), pages()) == qs.QS_ERR_ARG
    assert call(f, cache(True, D=64), pages()) == qs.QS_ERR_UNSUPPORTED
    assert call(f, cache(True, meta=0x10002), pages()) == qs.QS_ERR_ALIGN
    assert call(f, None, pages()) == qs.QS_ERR_ARG


@pytest.mark.parametrize("name", sorted(CONTIGUOUS))
def test_contiguous_calls_refuse_a_paged_cache(L, name):
    assert CONTIGUOUS[name](getattr(L, name), cache(True)) == qs.QS_ERR_ARG


def test_paged_cache_bytes(L):
    b = qs.qs_paged_cache_bytes(2, 3, 7)
    assert b["k_upper"] == b["v_lower"] == 7 * 3 * 128 * 64
    assert b["meta"] == 7 * 3 * 4 * 128 * 2
    assert b["buf_k"] == 2 * 3 * 256 * 128 * 2 and b["state"] == 2 * 8 * 4 and b["arrive"] == 2 * 3 * 4
    out = qs.QsCacheBytes()
    assert L.qs_paged_cache_bytes(1, 1, 128, 128, 0, ctypes.byref(out)) == qs.QS_ERR_ARG
    assert L.qs_paged_cache_bytes(1, 1, 64, 128, 1, ctypes.byref(out)) == qs.QS_ERR_UNSUPPORTED
    assert L.qs_paged_cache_bytes(1, 1, 128, 128, 1, None) == qs.QS_ERR_ARG


def test_prefill_and_flush_arguments(L):
    c, pg = cache(True), pages()
    for bad in (-1, 257):
        assert L.qs_quantize_flush_due_paged(c, pg, bad, None) == qs.QS_ERR_ARG
    assert L.qs_prefill_paged(c, pg, None, P, 10, P, None) == qs.QS_ERR_ARG
    assert L.qs_prefill_paged(c, pg, P, P, -1, P, None) == qs.QS_ERR_ARG
    assert L.qs_prefill_paged(c, pg, ctypes.c_void_p(0x20008), P, 1, P, None) == qs.QS_ERR_ALIGN


@pytest.mark.parametrize("paged", [False, True])
def test_read_arguments(L, paged):
    c, pg = cache(paged), pages() if paged else None
    f, odd = L.qs_cache_read, ctypes.c_void_p(0x20008)
    assert f(c, pg, 2, 0, 5, P, P, None) == qs.QS_ERR_ARG
    assert f(c, pg, 1, 0, 5, None, None, None) == qs.QS_ERR_ARG
    assert f(c, pg, 1, -1, 5, P, P, None) == qs.QS_ERR_ARG
    assert f(c, pg, 1, (1 << 30) + 1, 5, P, P, None) == qs.QS_ERR_ARG
    for T in (0, -3, (1 << 26) + 1):
        assert f(c, pg, 1, 0, T, P, P, None) == qs.QS_ERR_ARG
    assert f(c, pg, 1, 0, 5, odd, P, None) == qs.QS_ERR_ALIGN
    assert f(c, pg, 1, 0, 5, None, odd, None) == qs.QS_ERR_ALIGN


def test_listed_attention_arguments(L):
    c, pg, odd = cache(True), pages(), ctypes.c_void_p(0x20002)

    def paged(mode=0, k=None, v=None, n=0, q=P, n_q=1, group=1, scale=0.1, out=P, lse=None):
        return L.qs_attn_decode_paged(c, pg, mode, k, v, n, q, n_q, group, F(scale), out, lse, P,
                                      1 << 30, None)

    def sparse(sel=P, k_sel=3, **kw):
        a = dict(dict(mode=0, k=None, v=None, n=0, q=P, n_q=1, group=1, scale=0.1, out=P, lse=None), **kw)
        return L.qs_attn_decode_sparse(c, pg, a["mode"], sel, k_sel, a["k"], a["v"], a["n"], a["q"],
                                       a["n_q"], a["group"], F(a["scale"]), a["out"], a["lse"], P,
                                       1 << 30, None)

    for f in (paged, sparse):
        for kw in (dict(mode=2), dict(q=None), dict(out=None), dict(n_q=0), dict(n_q=9), dict(group=0),
                   dict(n_q=5, group=5), dict(n_q=8, group=1 << 29), dict(scale=0.0),
                   dict(scale=float("nan")), dict(k=P), dict(v=P, n=1), dict(n=1), dict(k=P, v=P),
                   dict(k=P, v=P, n=257), dict(k=P, v=P, n=-1)):
            assert f(**kw) == qs.QS_ERR_ARG, kw
        for kw in (dict(q=odd), dict(out=odd), dict(lse=odd), dict(k=odd, v=P, n=1), dict(k=P, v=odd, n=1)):
            assert f(**kw) == qs.QS_ERR_ALIGN, kw
    assert sparse(sel=None) == qs.QS_ERR_ARG
    assert sparse(k_sel=0) == qs.QS_ERR_ARG
    assert sparse(sel=odd) == qs.QS_ERR_ALIGN


@pytest.mark.parametrize("paged", [False, True])
def test_select_arguments(L, paged):
    c, pg = cache(paged), pages() if paged else None

    def f(c=c, q=P, n_q=1, group=1, k=3, sel=P):
        return L.qs_select_groups(c, pg, q, n_q, group, k, sel, None)

    for kw in (dict(q=None), dict(sel=None), dict(n_q=0), dict(n_q=9), dict(group=0), dict(group=25),
               dict(n_q=5, group=5), dict(n_q=8, group=1 << 29), dict(k=0), dict(k=-1)):
        assert f(**kw) == qs.QS_ERR_ARG, kw
    assert f(q=ctypes.c_void_p(0x20008)) == qs.QS_ERR_ALIGN
    assert f(sel=ctypes.c_void_p(0x20002)) == qs.QS_ERR_ALIGN
    assert f(c=cache(paged, cap_groups=12801)) == qs.QS_ERR_UNSUPPORTED


def test_binding_checks_shapes_and_types(L):
    """The binding turns tensors that do not fit the cache away (no GPU: CPU
    tensors stand in, nothing is called)."""
    torch = pytest.importorskip("torch")
    c = qs.PagedCache(2, 3, 4, 5, device="cpu")
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16)
    q, sel = f16(2, 6, 1, 128), torch.zeros((2, 3, 2), dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    bad = [
        lambda: qs.qs_attn_decode_paged(c, 0, q, 0.1, f16(2, 6, 1, 128), group=1),
        lambda: qs.qs_attn_decode_paged(c, 0, q, 0.1, f16(2, 6, 2, 128), group=2),
        lambda: qs.qs_attn_decode_paged(c, 0, q.float(), 0.1, q, group=2),
        lambda: qs.qs_attn_decode_paged(c, 0, f16(2, 6, 128, 2).transpose(2, 3), 0.1, f16(2, 6, 2, 128),
                                        group=2),
        lambda: qs.qs_attn_decode_paged(c, 0, q, 0.1, f16(2, 6, 1, 128), torch.zeros(5), group=2),
        lambda: qs.qs_attn_decode_paged(c, 0, q, 0.1, f16(2, 6, 1, 128), group=2, k_new=f16(2, 6, 1, 128),
                                        v_new=f16(2, 6, 1, 128)),
        lambda: qs.qs_attn_decode_sparse(c, 0, sel.long(), q, 0.1, f16(2, 6, 1, 128), group=2),
        lambda: qs.qs_attn_decode_sparse(c, 0, sel[:1], q, 0.1, f16(2, 6, 1, 128), group=2),
        lambda: qs.qs_select_groups(c, q, sel.float(), group=2),
        lambda: qs.qs_select_groups(c, q, sel),
        lambda: qs.qs_cache_read(c, 1, f16(2, 3, 5, 64), None),
        lambda: qs.qs_cache_read(c, 1, torch.zeros((2, 3, 5, 128)), None),
        lambda: qs.qs_prefill_paged(c, f16(2, 6, 5, 128), f16(2, 6, 5, 128), lens),
        lambda: qs.qs_prefill_paged(c, f16(2, 3, 5, 128), f16(2, 3, 5, 128), lens[:1]),
        lambda: qs.qs_quantize_flush_paged(c, torch.zeros(3, dtype=torch.uint8)),
    ]
    for call in bad:
        with pytest.raises(AssertionError):
            call()
