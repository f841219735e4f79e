"""What the binding of the paged, sparse, selecting and reading calls turns
away before the library is called: types that only have the right size,
tensors elsewhere than the cache, half an append.  Also under python -O (no
GPU needed: CPU tensors stand in, some of which say they are elsewhere)."""
import os
import subprocess
import sys

import pytest

import __graft_entry__
from hierarchical_quantized_kv_gb300 import qs

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on another device."""

    def get_device(self):
        return 3


def zeros(*s, dtype=torch.float32, away=False):
    t = torch.zeros(s, dtype=dtype)
    return t.as_subclass(Elsewhere) if away else t


def half(*s, dtype=torch.float16, away=False):
    return zeros(*s, dtype=dtype, away=away)


Q, KV = (2, 6, 1, 128), (2, 3, 2, 128)


class Args(dict):
    """Arguments that fit, with some replaced."""

    def __init__(self, **kw):
        super().__init__(q=half(*Q), out=half(*Q), lse=torch.zeros(Q[:3]), k_new=half(*KV), v_new=half(*KV),
                         sel=torch.zeros((2, 3, 2), dtype=torch.int32), ws=torch.zeros(8, dtype=torch.uint8))
        self.update(kw)
        self.__dict__ = self


def paged(c, a):
    qs.qs_attn_decode_paged(c, 0, a.q, 0.1, a.out, a.lse, a.ws, group=2, k_new=a.k_new, v_new=a.v_new,
                            stream=a.get("stream"))


def sparse(c, a):
    qs.qs_attn_decode_sparse(c, 0, a.sel, a.q, 0.1, a.out, a.lse, a.ws, group=2, k_new=a.k_new,
                             v_new=a.v_new, stream=a.get("stream"))


def select(c, a):
    qs.qs_select_groups(c, a.q, a.sel, group=2)


def read(c, a):
    qs.qs_cache_read(c, 1, a.k_new, a.v_new)


def prefill(c, a):
    qs.qs_prefill_paged(c, a.k_new, a.v_new, a.get("lens", torch.zeros(2, dtype=torch.int32)))


def flush(c, a):
    qs.qs_quantize_flush_paged(c, a.mask)


BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
BAD = [
    (paged, dict(q=half(*Q, dtype=BF))), (paged, dict(out=half(*Q, dtype=BF))),
    (paged, dict(q=half(*Q, away=True))), (paged, dict(out=half(*Q, away=True))),
    (paged, dict(q=half(2, 6, 128))), (paged, dict(lse=torch.zeros(Q[:3], dtype=torch.int32))),
    (paged, dict(lse=zeros(*Q[:3], away=True))), (paged, dict(k_new=None)), (paged, dict(v_new=None)),
    (paged, dict(k_new=half(*KV, dtype=BF))), (paged, dict(v_new=half(*KV, dtype=torch.int16))),
    (paged, dict(k_new=half(*KV, away=True))), (paged, dict(v_new=half(*KV, away=True))),
    (paged, dict(k_new=half(3, 2, 128))), (paged, dict(ws=zeros(8, away=True))),
    (paged, dict(ws=torch.zeros((8, 8), dtype=torch.uint8).t()[::2])),
    (sparse, dict(q=half(*Q, dtype=BF))), (sparse, dict(v_new=None)),
    (sparse, dict(sel=zeros(2, 3, 2, dtype=I32, away=True))),
    (sparse, dict(sel=torch.zeros((2, 3), dtype=torch.int32))),
    (sparse, dict(ws=zeros(8, away=True))),
    (select, dict(q=half(*Q, dtype=BF))), (select, dict(q=half(*Q, away=True))),
    (select, dict(sel=zeros(2, 3, 2, dtype=I32, away=True))),
    (read, dict(k_new=half(*KV, dtype=BF))), (read, dict(v_new=half(*KV, away=True))),
    (read, dict(k_new=half(2, 3))), (read, dict(k_new=None, v_new=half(2, 3, 128))),
    (prefill, dict(v_new=None)), (prefill, dict(k_new=half(2, 3, 128), v_new=half(2, 3, 128))),
    (prefill, dict(k_new=half(*KV, dtype=BF), v_new=half(*KV, dtype=BF))),
    (prefill, dict(v_new=half(*KV, away=True))), (prefill, dict(lens=torch.zeros(2))),
    (prefill, dict(lens=zeros(2, dtype=I32, away=True))),
    (flush, dict(mask=zeros(2, dtype=U8, away=True))),
    (flush, dict(mask=torch.zeros(4, dtype=torch.uint8)[::2])),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refused(i):
    call, kw = BAD[i]
    __graft_entry__.build()
    c = qs.PagedCache(2, 3, 4, 5, device="cpu")
    with pytest.raises(qs.QsArgumentError):
        call(c, Args(**kw))


def test_refusals_hold_without_assertions():
    """python -O drops assert statements, not these checks."""
    code = ("import sys; sys.path.insert(0, %r)\n"
            "from tests import test_binding_arguments as t\n"
            "from hierarchical_quantized_kv_gb300 import qs\n"
            "c = qs.PagedCache(2, 3, 4, 5, device='cpu')\n"
            "n = 0\n"
            "for call, kw in t.BAD:\n"
            "    try:\n"
            "        call(c, t.Args(**kw))\n"
            "    except qs.QsArgumentError:\n"
            "        n += 1\n"
            "print(n, __debug__)\n" % ROOT)
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-O", "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.stdout.split() == [str(len(BAD)), "False"], r.stdout + r.stderr


def test_fitting_arguments_reach_the_library():
    """The same arguments unspoilt pass the checks: the library itself answers
    (there is no device to ask; no kernel is launched)."""
    if torch.cuda.is_available():
        pytest.skip("CPU tensors must not reach a device")
    __graft_entry__.build()
    c = qs.PagedCache(2, 3, 4, 5, device="cpu")
    for call in (paged, sparse):
        with pytest.raises(qs.QsError) as e:
            call(c, Args(stream=0))
        assert e.value.status == qs.QS_ERR_CUDA
