"""How the attention of many rows weighs what its CTAs have found, against softmax
attention in 64 bits."""
import numpy as np
import oracle
import pytest

from tests import trees
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import DRAFT, VERIFY, h16
from tests.test_gpu_tree_attn import run, torch  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def filled(k, v, ng, fill):
    """An oracle cache of one sequence with tokens k, v [H, ng * 128 + fill, 128]."""
    oc = oracle.OracleCache(1, k.shape[0], 128, 128, ng)
    oracle.prefill(oc, lambda b, t0, m: (k[:, t0:t0 + m], v[:, t0:t0 + m]), [ng], [fill])
    return oc


@pytest.mark.parametrize("size", [1, 200, 8000])
@pytest.mark.parametrize("ng", [6, 330])
@pytest.mark.parametrize("n,group", [(40, 1), (35, 2), (50, 3)])
def test_equal_scores_of_any_size_weigh_the_same(torch, n, group, ng, size):  # noqa: F811
    """All keys alike, so that every token weighs the same, whatever the score (up to
    10^9, where a step of fp32 is 64) and whatever its group's values: their sizes
    differ by 2^12 from group to group.  Rounded, in rms of 2^-11 / sqrt(3): the
    weights, times the values' scales, and the output; 4e-4 in squares."""
    rng = np.random.default_rng([n, group, ng, size])
    H, fill = 2, 200
    T = ng * 128 + fill
    k = np.broadcast_to(np.float16(size) * rng.choice([-1, 1], 128).astype(np.float16), (H, T, 128)).copy()
    sizes = 2.0 ** (rng.permutation(np.arange(T // 128 + 1)) % 13 - 6)
    v = (rng.standard_normal((H, T, 128)) + 1) * sizes[np.arange(T) // 128][:, None]
    oc = filled(k, v.astype(np.float16), ng, fill)
    parent = trees.random_parents(rng, 1, n)
    # (a query's channels are the keys' times 1/2, 1/4 .. of it: sums without rounding)
    q = (k[:1, :1, :] * (2.0 ** -rng.integers(0, 3, (1, H * group, n, 1)))).astype(np.float16)
    cache = load(torch, oc, rng)
    for mode in (DRAFT, VERIFY):
        got, gl = run(torch, cache, mode, q, parent, group)
        ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group)
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= 1e-3, (mode, rel)
        assert np.all(np.abs(gl - rl) <= 2.0 ** -21 * np.abs(rl) + 1e-5), mode
