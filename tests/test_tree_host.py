"""The calls of a round over a tree: what they turn away before anything is
launched, in the library and in the binding (no GPU needed)."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import __graft_entry__
from hierarchical_quantized_kv_gb300 import qs
from tests import trees
from tests.test_abi import _fake_cache
from tests.test_binding_arguments import half, zeros

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x20002)


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return qs.lib()


def rows(data=0x20000, b=0, h=128, t=256):
    return qs.QsRowsStruct(data, b, h, t)


def test_append_rotary(L):
    def call(c=None, k=rows(), v=rows(), q=rows(), q_out=P, group=2, n=4, offset=P, freq=P, rot=64, inter=0):
        c = c or _fake_cache()
        ref = lambda r: None if r is None else ctypes.byref(r)
        return L.qs_buffer_append_rotary(ctypes.byref(c), ref(k), ref(v), ref(q), q_out, group, n, offset,
                                         freq, rot, inter, None)
    for bad in (dict(k=None), dict(v=None), dict(freq=None), dict(q=None), dict(q_out=None), dict(n=0),
                dict(n=257), dict(group=0), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144),
                dict(k=rows(data=None)), dict(q=rows(data=None))):
        assert call(**bad) == qs.QS_ERR_ARG, bad
    for bad in (dict(k=rows(b=4)), dict(v=rows(h=1)), dict(q=rows(t=129))):
        assert call(**bad) == qs.QS_ERR_SHAPE, bad
    for bad in (dict(k=rows(data=0x20008)), dict(q_out=ctypes.c_void_p(0x20008)), dict(freq=ODD),
                dict(offset=ODD)):
        assert call(**bad) == qs.QS_ERR_ALIGN, bad
    assert call(c=_fake_cache(D=64)) == qs.QS_ERR_UNSUPPORTED


def test_attention(L):
    n = ctypes.c_size_t()
    c = _fake_cache()
    for n_q, g in ((0, 1), (65, 1), (64, 9), (1, 513), (1, 0), (8, -1)):
        assert L.qs_attn_tree_workspace_size(ctypes.byref(c), n_q, g, ctypes.byref(n)) == qs.QS_ERR_ARG
    assert L.qs_attn_tree_workspace_size(ctypes.byref(c), 4, 1, None) == qs.QS_ERR_ARG

    def call(c=None, pg=None, mode=0, parent=P, n_tree=8, q=P, n_q=8, group=4, scale=0.1, out=P, lse=None,
             ws=P, size=1 << 30):
        c = c or _fake_cache()
        return L.qs_attn_decode_tree(ctypes.byref(c), pg, mode, parent, n_tree, q, n_q, group,
                                     ctypes.c_float(scale), out, lse, ws, size, None)
    pages = qs.QsPagesStruct(0x10000, 4)
    for group in (1, 4):  # both sides of the 24 rows
        for bad in (dict(parent=None), dict(n_tree=7), dict(n_tree=65), dict(n_q=0), dict(n_tree=64, n_q=65),
                    dict(group=0), dict(n_tree=64, n_q=64, group=9), dict(mode=2), dict(q=None),
                    dict(out=None), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
                    dict(pg=ctypes.byref(pages)), dict(c=_fake_cache(upper_bits=4 | qs.QS_PAGED))):
            assert call(**{**dict(group=group), **bad}) == qs.QS_ERR_ARG, (group, bad)
        for bad in (dict(parent=ODD), dict(q=ctypes.c_void_p(0x20008)), dict(out=ctypes.c_void_p(0x20008)),
                    dict(lse=ctypes.c_void_p(0x20004))):
            assert call(**{**dict(group=group), **bad}) == qs.QS_ERR_ALIGN, (group, bad)


def test_accept(L):
    def call(**kw):
        a = dict(parent=P, draft=P, target=P, n=8, n_keep=P, path=P, emitted=P)
        a.update(kw)
        c = _fake_cache()
        return L.qs_tree_accept(ctypes.byref(c), a["parent"], a["draft"], a["target"], a["n"], a["n_keep"],
                                a["path"], a["emitted"], None)
    for name in ("parent", "draft", "target", "n_keep", "path", "emitted"):
        assert call(**{name: None}) == qs.QS_ERR_ARG, name
        assert call(**{name: ODD}) == qs.QS_ERR_ALIGN, name
    assert call(n=0) == call(n=65) == qs.QS_ERR_ARG


def test_sample(L):
    def call(**kw):
        a = dict(x=P, dtype=qs.QS_FP16, rows=3, V=100, stride=100, t=P, k=P, p=P, m=P, u=P, token=P, probs=P)
        a.update(kw)
        return L.qs_sample(a["x"], a["dtype"], a["rows"], a["V"], a["stride"], a["t"], a["k"], a["p"],
                           a["m"], a["u"], a["token"], a["probs"], None)
    for bad in (dict(x=None), dict(u=None), dict(token=None), dict(rows=0), dict(V=0), dict(stride=99),
                dict(dtype=3), dict(dtype=-1)):
        assert call(**bad) == qs.QS_ERR_ARG, bad
    assert call(V=qs.QS_MAX_VOCAB + 1, stride=1 << 20) == qs.QS_ERR_UNSUPPORTED
    for bad in (dict(x=ctypes.c_void_p(0x20001)), dict(x=ODD, dtype=qs.QS_FP32), dict(t=ODD), dict(k=ODD),
                dict(p=ODD), dict(m=ODD), dict(u=ODD), dict(token=ODD), dict(probs=ODD)):
        assert call(**bad) == qs.QS_ERR_ALIGN, bad


# ------------------------------------------------------------------ binding

I32, BF = torch.int32, torch.bfloat16
i32 = lambda *s, away=False: zeros(*s, dtype=I32, away=away)  # noqa: E731
B, H, N = 2, 3, 5


def append(c, kw):
    a = dict(k=half(B, H, N, 128), v=half(B, H, N, 128), inv_freq=torch.zeros(32), q=half(B, 2 * H, N, 128),
             q_out=half(B, 2 * H, N, 128), offset=i32(B, N))
    a.update(kw)
    qs.qs_buffer_append_rotary(c, **a)


def attend(c, kw):
    a = dict(parent=i32(B, N), q=half(B, 2 * H, N, 128), softmax_scale=0.1, out=half(B, 2 * H, N, 128),
             lse=torch.zeros((B, 2 * H, N)), workspace=torch.zeros(8, dtype=torch.uint8), group=2)
    a.update(kw)
    qs.qs_attn_decode_tree(c, 0, **a)


def accept(c, kw):
    a = dict(parent=i32(B, N), draft=i32(B, N), target=i32(B, N), n_keep=i32(B), path=i32(B, N),
             emitted=i32(B, N))
    a.update(kw)
    qs.qs_tree_accept(c, **a)


def draw(c, kw):
    """(a tensor that says it lies on a device stands for one there)"""
    f = lambda *s, **k: zeros(*s, away=True, **k)  # noqa: E731
    a = dict(logits=f(B, 7), u=f(B), token=f(B, dtype=I32), probs=f(B, 7), temperature=f(B),
             top_k=f(B, dtype=I32), top_p=f(B), min_p=f(B))
    a.update(kw)
    held, qs._current_device = qs._current_device, lambda: kw.pop("current", 3)
    try:
        qs.qs_sample(**{k: v for k, v in a.items() if k != "current"})
    finally:
        qs._current_device = held


BAD = [
    (append, dict(k=half(B, H, N, 128, dtype=BF))), (append, dict(k=half(B, H, N, 64))),
    (append, dict(k=half(B, H, 128))), (append, dict(v=half(B, H, N + 1, 128))),
    (append, dict(v=half(B, H, N, 128, away=True))), (append, dict(k=half(B, H, N, 256)[..., ::2])),
    (append, dict(q=None)), (append, dict(q_out=None)), (append, dict(q=half(B, 2 * H + 1, N, 128))),
    (append, dict(q=half(B, 2, N, 128), q_out=half(B, 2, N, 128))),
    (append, dict(q_out=half(B, 2 * H, 128, N).transpose(2, 3))), (append, dict(q_out=half(B, H, N, 128))),
    (append, dict(inv_freq=torch.zeros(32, dtype=torch.float64))), (append, dict(inv_freq=torch.zeros(8, 4))),
    (append, dict(inv_freq=torch.zeros(64)[::2])), (append, dict(inv_freq=zeros(32, away=True))),
    (append, dict(offset=i32(B, N + 1))), (append, dict(offset=torch.zeros((B, N), dtype=torch.int64))),
    (append, dict(offset=i32(N, B).t())), (append, dict(offset=i32(B, N, away=True))),
    (attend, dict(parent=i32(B + 1, N))), (attend, dict(parent=i32(B * N))),
    (attend, dict(parent=torch.zeros((B, N)))), (attend, dict(parent=i32(N, B).t())),
    (attend, dict(parent=i32(B, N, away=True))), (attend, dict(q=half(B, 2 * H, N, 128, dtype=BF))),
    (attend, dict(q=half(B, H, N, 128))), (attend, dict(out=half(B, 2 * H, N, 128, away=True))),
    (attend, dict(lse=torch.zeros((B, 2 * H, N + 1)))), (attend, dict(workspace=zeros(8, away=True))),
    (accept, dict(draft=i32(B, N + 1))), (accept, dict(target=torch.zeros((B, N)))),
    (accept, dict(parent=i32(B, N, away=True))), (accept, dict(path=i32(N, B).t())),
    (accept, dict(emitted=i32(B, 1))), (accept, dict(n_keep=i32(B, 1))),
    (accept, dict(n_keep=torch.zeros(B, dtype=torch.int64))),
    (draw, dict(logits=zeros(B, 7))), (draw, dict(logits=zeros(B, 7, dtype=torch.float64, away=True))),
    (draw, dict(logits=zeros(B, 7, 1, away=True))), (draw, dict(logits=zeros(B, 14, away=True)[:, ::2])),
    (draw, dict(current=0)), (draw, dict(u=zeros(B + 1, away=True))), (draw, dict(u=zeros(B))),
    (draw, dict(token=zeros(B, away=True))), (draw, dict(token=zeros(2 * B, dtype=I32, away=True)[::2])),
    (draw, dict(probs=zeros(7, B, away=True).t())), (draw, dict(probs=zeros(B, 8, away=True))),
    (draw, dict(temperature=zeros(1, away=True))), (draw, dict(top_k=zeros(B, away=True))),
    (draw, dict(top_p=zeros(B, dtype=torch.float16, away=True))), (draw, dict(min_p=zeros(B))),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_the_binding_refuses(L, i):
    call, kw = BAD[i]
    with pytest.raises(qs.QsArgumentError):
        call(qs.PagedCache(B, H, 4, 5, device="cpu"), dict(kw))


def test_refusals_hold_without_assertions(L):
    code = ("import sys; sys.path.insert(0, %r)\n"
            "from tests import test_tree_host as t\n"
            "from hierarchical_quantized_kv_gb300 import qs\n"
            "c = qs.PagedCache(t.B, t.H, 4, 5, device='cpu')\n"
            "n = 0\n"
            "for call, kw in t.BAD:\n"
            "    try:\n"
            "        call(c, dict(kw))\n"
            "    except qs.QsArgumentError:\n"
            "        n += 1\n"
            "print(n, __debug__)\n" % ROOT)
    r = subprocess.run([sys.executable, "-O", "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.stdout.split() == [str(len(BAD)), "False"], r.stdout + r.stderr


def test_rows_of_any_strides_reach_the_library():
    """Slices of a projection's output, broadcast heads and a single token give
    the strides that the library is told."""
    c = qs.PagedCache(B, H, 4, 5, device="cpu")
    x = half(B, N, 4 * H, 128).transpose(1, 2)
    assert qs._rows(c, x[:, H:2 * H], "k", H, N) == (x.data_ptr() + H * 256, N * 4 * H * 128, 128, 4 * H * 128)
    assert qs._rows(c, half(B, 1, N, 128).expand(B, H, N, 128), "k", H, N)[2:] == (0, 128)
    assert qs._rows(c, half(B, H, 1, 128), "k", H, 1)[1:] == (H * 128, 128, 0)


# -------------------------------------------------- the model these tests use

def test_the_model_of_a_tree():
    parent = np.array([-1, 0, 0, 1, 1, 2, 5, -1])
    sees = trees.ancestors(parent)
    assert [np.flatnonzero(r).tolist() for r in sees] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 4], [0, 2, 5],
                                                          [0, 2, 5, 6], [7]]
    assert trees.depths(parent[None]).tolist() == [[0, 1, 1, 2, 2, 2, 3, 0]]
    assert trees.accept(parent, [9, 4, 5, 6, 6, 5, 8, 4], [5, 0, 5, 0, 0, 7, 0, 0]) == [0, 2, 5]
    token, probs = trees.sample([1.0, 3.0, 3.0, 2.0], 0.6, top_k=2)
    assert token == 2 and probs.tolist() == [0, 0.5, 0.5, 0]
    assert trees.sample([1.0, 3.0, 3.0, 2.0], 0.6, temperature=0)[0] == 1
