"""Drafts over listed groups whose q s_K (query times key scale) goes to the
end of fp16's range: finite, and the attention of the definition in 64 bits.

Tolerances of tests/test_gpu_qs.py, the log-sum-exp within 1e-4: the softmax
scale keeps scores below 6 (plus the ordinary channels' 1e-3), a score's error is
some 20 fp32 steps of that (products of an fp16 pair that is exact to 2^-22, eight
sums of tensor core results), about 1e-5."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import DRAFT, assert_close, h16, to_dev

pytestmark = pytest.mark.gpu

WIDE = (4, 7, 97)  # channels of both operand registers


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def wide_state(rng, B, H, n, A):
    """n groups and 256 buffered tokens; the wide channels of the keys fill [-A, A]."""
    oc = oracle.OracleCache(B, H, 128, 128, n + 1)
    T = 128 * n + 256
    k, v = rng.standard_normal((B, H, T, 128)), rng.standard_normal((B, H, T, 128))
    for c in WIDE:
        k[..., c] = rng.uniform(-A, A, (B, H, T))
        k[:, :, 0::128, c], k[:, :, 1::128, c] = -A, A
    oc.prefill(k.astype(np.float16), v.astype(np.float16), np.full(B, T, np.int32))
    return oc


def call(torch, cache, q, scale, group, sel=None, dense=False):
    qd = to_dev(torch, q)
    out = torch.full_like(qd, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), dtype=torch.float32, device="cuda")
    ws = torch.empty(qs.qs_attn_workspace_size_gqa(cache, q.shape[2], group), dtype=torch.uint8, device="cuda")
    if dense:
        qs.qs_attn_decode_gqa(cache, DRAFT, qd, group, scale, out, lse, ws)
    elif sel is None:
        qs.qs_attn_decode_paged(cache, DRAFT, qd, scale, out, lse, ws, group=group)
    else:
        qs.qs_attn_decode_sparse(cache, DRAFT, to_dev(torch, sel), qd, scale, out, lse, ws, group=group)
    assert np.all(qs.qs_get_errors(cache) == 0)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


# |q| and half the key range: q s_K = 20,000, 17,500, 16,500, 60,000, and the two
# sides of the largest query that is carried fourfold, at the largest scale
CASES = [(200, 12750), (70, 31875), (330, 6375), (1200, 6375), (31.75, 65504), (31.765625, 65504)]


@pytest.mark.parametrize("n_q,group", [(1, 1), (1, 4), (5, 1), (1, 8), (1, 24)])
@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("Q,A", CASES)
def test_wide_scores(torch, Q, A, ub, n_q, group):
    rng = np.random.default_rng([int(Q * 64), ub, n_q, group])
    for B, H in ((1, 3), (2, 2)):  # clusters; the split kernel
        n = 9
        oc = wide_state(rng, B, H, n, A)
        q = h16(rng, (B, H * group, n_q, 128))
        q[..., WIDE] = np.float16(Q) * rng.choice([-1, 1], (B, H * group, n_q, len(WIDE)))
        if group == 4:
            q[:, 1::4] = h16(rng, (B, H, n_q, 128))  # an ordinary row beside wide ones
        scale = 2.0 / (Q * A)
        ks = oc.ks[:, :, :n][..., WIDE].view(np.float16).astype(np.float64)
        assert 4 * Q * ks.max() > 64e3 and Q * ks.max() < 65504
        paged, dense = load(torch, oc, rng, ub), load(torch, oc, rng, ub, False)
        got, gl = call(torch, paged, q, scale, group)
        ref, rl = paging.attention(oc, q, True, group, ub, scale=scale)
        assert_close(got, ref, gl, rl, "paged")
        assert np.abs(gl - rl).max() < 1e-4
        cont, cl = call(torch, dense, q, scale, group, dense=True)
        assert_close(got, cont, gl, cl, "against the contiguous call")
        sel = np.stack([[rng.permutation(n)[:6] for _ in range(H)] for _ in range(B)]).astype(np.int32)
        for cache in (paged, dense):
            got, gl = call(torch, cache, q, scale, group, sel)
            ref, rl = paging.attention(oc, q, True, group, ub, sel, scale=scale)
            assert_close(got, ref, gl, rl, "sparse")
            assert np.abs(gl - rl).max() < 1e-4
