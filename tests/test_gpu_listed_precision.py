"""What the listed drafts gain over the contiguous kernel's rounding, against 64
bits: codes further up in their fp16 operands, q s_K carried fourfold.

Outputs: relative RMS below sqrt(2) 2^-11 / sqrt(3) = 4.0e-4.  An output is
rounded to fp16 (off by up to 2^-11 of itself, evenly spread: RMS at most
2^-11 / sqrt(3)), and so is each probability times value scale before the
product, which the sum carries into the output at no more than that rate (codes
are taken from 128, so the terms are of the values' size).  The contiguous
two-bit draft is 5 to 8e-4 off.

Log-sum-exp: one case made to show the residual of q s_K.  Every odd channel
holds q s = hi + r with r = 2^-21 - 2^-25 past the nearest fp16 number, every
token the largest code, so all 64 residuals add up.  The odd channels' operand is
q s / 16 onefold, where r / 16 < 2^-25 is less than half an fp16 step and lost
whole: 64 * 240 r / sqrt(128) = 6.1e-4 (two bits: 64 * 192, 4.9e-4) would be
missing.  Fourfold, r / 4 is rounded by 2^-27: 4.1e-5.  A sum of 17 addends is cut
no coarser than 2^-23 of the largest (2^-18.9 of a score of 43: 8.8e-5), and the
score's own fp32 steps are below 2e-5: 1.5e-4 together."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_listed_attn import load, run
from tests.test_gpu_qs import DRAFT, _oracle_state, assert_close, h16

pytestmark = pytest.mark.gpu

RMS = np.sqrt(2 / 3) * 2.0 ** -11


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


@pytest.mark.parametrize("sharp", [1.0, 3.0])
@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("B,group", [(1, 4), (1, 8), (3, 2), (3, 16)])  # packed rows and not, clusters and not
def test_outputs(torch, B, group, ub, sharp):
    rng = np.random.default_rng([B, group, ub, int(sharp)])
    H, n = 8, 24
    oc = _oracle_state(rng, B, H, [n] * B, [100] * B, cap=n)
    cache = load(torch, oc, rng, ub)
    sel = np.stack([[rng.permutation(n)[:16] for _ in range(H)] for _ in range(B)])
    err = np.zeros((2, 2))
    for _ in range(3):
        q = h16(rng, (B, H * group, 1, 128), sharp)
        for i, s in enumerate((None, sel)):
            got, _ = run(torch, cache, DRAFT, q, group, s)
            ref, _ = paging.attention(oc, q, True, group, ub, s)
            err[i] += ((got - ref) ** 2).sum(), (ref ** 2).sum()
    rel = np.sqrt(err[:, 0] / err[:, 1])
    print("relative RMS: pages %.3g, selected %.3g" % tuple(rel))
    assert np.all(rel < RMS)


Q, S = 1 + 2.0 ** -10, 0.031707763671875  # fp16 numbers


@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("B,group", [(1, 1), (1, 8), (2, 4), (2, 24)])
def test_residuals_of_the_scores(torch, B, group, ub):
    p = Q * S
    assert p - float(np.float16(p)) == 2.0 ** -21 - 2.0 ** -25 and p < 2.0 ** -4
    assert float(np.float16(Q)) == Q and float(np.float16(S)) == S
    rng = np.random.default_rng([B, group, ub])
    H, n = 2, 5
    oc = oracle.OracleCache(B, H, 128, 128, n)
    k = np.zeros((B, H, 128 * n + 256, 128), np.float16)
    oc.prefill(k, h16(rng, k.shape), np.full(B, k.shape[2], np.int32))
    oc.kq[:] = 255
    oc.ks.view(np.float16)[:] = S
    oc.kz[:] = 0
    q = np.zeros((B, H * group, 1, 128), np.float16)
    q[..., 1::2] = Q
    cache = load(torch, oc, rng, ub)
    sel = np.broadcast_to(np.arange(n), (B, H, n))
    ref, rl = paging.attention(oc, q, True, group, ub)
    assert 40 < rl.min() and rl.max() - np.log(128 * n) < 55
    for s in (None, sel):
        got, gl = run(torch, cache, DRAFT, q, group, s)
        print("log-sum-exp off by up to %.3g" % np.abs(gl - rl).max())
        assert_close(got, ref, gl, rl)
        assert np.abs(gl - rl).max() < 1.5e-4
