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
