"""Outputs of a tree round's calls that lie on what other CTAs may still read are
turned away before anything is launched (no GPU needed)."""
import ctypes

import pytest

import __graft_entry__
from hierarchical_quantized_kv_gb300 import qs
from tests.test_abi import _fake_cache

B, N = 2, 8
BYTES = 4 * B * N


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return qs.lib()


INT_ARRAYS = ("parent", "draft", "target", "n_keep", "path", "emitted")


def accept(L, **kw):
    """Six arrays of one size, side by side."""
    a = {name: 0x20000 + i * BYTES for i, name in enumerate(INT_ARRAYS)}
    a.update(kw)
    c = _fake_cache(B=B)
    p = {name: ctypes.c_void_p(v) for name, v in a.items()}
    return L.qs_tree_accept(ctypes.byref(c), p["parent"], p["draft"], p["target"], N, p["n_keep"], p["path"],
                            p["emitted"], None)


@pytest.mark.parametrize("out,other", [(o, x) for o in INT_ARRAYS[3:] for x in INT_ARRAYS if x != o])
def test_accept(L, out, other):
    """Each output on each other array: at its start, on its last element, and with
    its own last on the first."""
    i = INT_ARRAYS.index(other)
    at = 0x20000 + i * BYTES
    size = 4 * B if other == "n_keep" else BYTES
    mine = 4 * B if out == "n_keep" else BYTES
    for start in (at, at + size - 4, at - mine + 4):
        assert accept(L, **{other: at, out: start}) == qs.QS_ERR_ARG, hex(start)


H, GROUP, T = 3, 2, 5  # KV heads, query heads on each, new tokens
ROW = 256              # bytes


def append(L, q_out, **rows):
    """k, v and q heads of a token side by side from 0x100000 on, as one projection
    leaves them (rows: (data, stride_b, stride_h, stride_t), strides in rows)."""
    heads = (2 + GROUP) * H
    a = {n: (0x100000 + at * ROW, T * heads, 1, heads) for n, at in (("q", 0), ("k", GROUP * H), ("v", GROUP * H + H))}
    a.update(rows)
    r = {n: qs.QsRowsStruct(x[0], *(128 * s for s in x[1:])) for n, x in a.items()}
    c = _fake_cache(B=B, H=H)
    return L.qs_buffer_append_rotary(ctypes.byref(c), ctypes.byref(r["k"]), ctypes.byref(r["v"]),
                                     ctypes.byref(r["q"]), ctypes.c_void_p(q_out), GROUP, T, None,
                                     ctypes.c_void_p(0x20000), 64, 0, None)


def test_append(L):
    end = 0x100000 + B * T * (2 + GROUP) * H * ROW
    size = B * T * GROUP * H * ROW
    for q_out in (0x100000, 0x100000 + 16, end - 16, 0x100000 - size + 16):
        assert append(L, q_out) == qs.QS_ERR_ARG, hex(q_out)
    own = (0x400000, T * GROUP * H, T, 1)  # q_out's layout
    for q_out in (0x400000 + ROW, 0x400000 - ROW, 0x400000 + size - 16):
        assert append(L, q_out, q=own) == qs.QS_ERR_ARG
    for q in ((own[0], own[1], 1, GROUP * H), (own[0], 0, T, 1), (own[0], own[1], 0, 1)):
        assert append(L, 0x400000, q=q) == qs.QS_ERR_ARG, q
    # strides below zero: the rows lie in front of the first
    last = (0x900000, -T * H, -T, -1)
    for name in ("k", "v"):
        assert append(L, 0x900000 - ROW, **{name: last}) == qs.QS_ERR_ARG
        assert append(L, 0x900000 - (B * T * H - 1) * ROW - size + 16, **{name: last}) == qs.QS_ERR_ARG


def sample(L, probs, dtype=qs.QS_FP32, rows=4, vocab=100, stride=100):
    at = ctypes.c_void_p
    return L.qs_sample(at(0x100000), dtype, rows, vocab, stride, None, None, None, None, at(0x20000), at(0x30000),
                       at(probs), None)


def test_sample(L):
    """Probabilities in the logits' memory, but not in their place: of another type, with
    another stride, or shifted."""
    x, row = 0x100000, 400
    for kw in (dict(dtype=qs.QS_FP16), dict(dtype=qs.QS_BF16), dict(stride=104), dict(dtype=qs.QS_FP16, rows=1)):
        assert sample(L, x, **kw) == qs.QS_ERR_ARG, kw
    for probs in (x + 4, x - 4, x + row, x - row, x + 4 * row - 4, x - 4 * row + 4):
        assert sample(L, probs) == qs.QS_ERR_ARG, hex(probs)
    # in front of the second, or behind the first, of rows far apart
    for probs in (x + 4000 - 1600 + 4, x + row - 4, x + 3 * 4000 + row - 4):
        assert sample(L, probs, stride=1000) == qs.QS_ERR_ARG, hex(probs)
