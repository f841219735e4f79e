"""How near the attention of many rows per KV head comes to softmax attention in 64
bits: near enough to tell that its keys are not rounded to fp16.

What is rounded, in rms of at most a rounding's 2^-11 / sqrt(3) = 2.8e-4 each: a weight
times its value's scale (one token may carry a sum), and the output; 4.0e-4 in squares.
Of the keys only a second part, 1 / 14 of their size (a scale is off by 1 / 8 at most,
evenly, from its three bits): 2.0e-5 of a key, the mean over a step, and so with unit
queries, three channels of 16 and 125 of 2, 2.0e-5 * 35.5 / sqrt(128) = 6e-5 of a
score and of its weight: 4.1e-4 together.  Keys rounded once move the output by 5.8e-4
and more (shown below, on the CPU)."""
import numpy as np
import oracle
import pytest

from tests import paging, trees
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, h16
from tests.test_gpu_tree_attn import run, torch  # noqa: F401  (fixture)

CLOSE = 4.1e-4


def case(n, group, B=1, ub=4):
    rng = np.random.default_rng([n, group, B])
    ng = [12, 5, 9][:B]
    oc = _oracle_state(rng, B, 3, ng, [200, 256, 97][:B], cap=12)  # (three channels eightfold)
    parent = trees.random_parents(rng, B, n)
    return rng, oc, parent, h16(rng, (B, 3 * group, n, 128))


@pytest.mark.gpu
@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("n,group", [(26, 1), (33, 1), (64, 1), (32, 2), (13, 5), (43, 3), (60, 4), (64, 5), (64, 8)])
def test_many_rows(torch, n, group, B, ub):  # noqa: F811
    rng, oc, parent, q = case(n, group, B)
    cache = load(torch, oc, rng, ub)
    for mode in (DRAFT, VERIFY):
        got, gl = run(torch, cache, mode, q, parent, group)
        ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group, ub)
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= CLOSE, (mode, rel)


@pytest.mark.gpu
@pytest.mark.parametrize("n,group", [(17, 1), (9, 2), (5, 4), (24, 1)])
def test_verifications_next_to_the_border(torch, n, group):  # noqa: F811
    rng, oc, parent, q = case(n, group, 3)
    got, gl = run(torch, load(torch, oc, rng), VERIFY, q, parent, group)
    ref, rl = trees.attention(oc, q, parent, False, group)
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rel <= CLOSE, rel


@pytest.mark.parametrize("n,group", [(26, 1), (60, 4), (17, 1)])
def test_keys_rounded_once_would_not_pass(n, group, monkeypatch):
    _, oc, parent, q = case(n, group)
    for upper in (True, False):
        ref, _ = trees.attention(oc, q, parent, upper, group)
        plain = paging.dequantized
        with monkeypatch.context() as m:
            m.setattr(paging, "dequantized", lambda *a: [x.astype(np.float16).astype(np.float64) if i == 0 else x
                                                         for i, x in enumerate(plain(*a))])
            once, _ = trees.attention(oc, q, parent, upper, group)
        assert np.linalg.norm(once - ref) / np.linalg.norm(ref) > 1.4 * CLOSE


def large(rng, k_size, T, H=2):
    k = np.clip(rng.standard_normal((H, T, 128)) * k_size, -65504, 65504).astype(np.float16)
    return k, rng.standard_normal((H, T, 128)).astype(np.float16)


def ahead(oc, q, parent, upper, group):
    """bool [B, Hq, n]: rows whose largest score leads by more than scores of this size may
    be off (1.1e-4 of the log-sum-exp each, tests/test_gpu_tree_attn.py) and 40: what comes
    second then weighs 2^-57 at most."""
    B, Hq, n, _ = q.shape
    lead = np.zeros(q.shape[:3], bool)
    sees = trees.ancestors(parent[0])
    k, _ = paging.dequantized(oc, 0, upper, 4)
    for i in range(Hq):
        s = float(np.float32(1 / np.sqrt(128))) * (q[0, i].astype(np.float64) @ k[i // group].T)
        s[:, s.shape[1] - n:][~sees] = -np.inf
        top = np.sort(s, 1)[:, -2:]
        lead[0, i] = top[:, 1] - top[:, 0] > 2 * 1.1e-4 * np.abs(top[:, 1]) + 40
    return lead


@pytest.mark.gpu
@pytest.mark.parametrize("q_size,k_size", [(1, 3000), (100, 100), (3000, 3000), (8000, 8000)])
@pytest.mark.parametrize("n,group", [(40, 1), (30, 5)])
def test_large_scores_pick_their_token(torch, n, group, q_size, k_size):  # noqa: F811
    """A row whose best token leads is that token's values: its weight is a power of two,
    so codes, scale and zero meet without a rounding but those of fp32 sums, and the
    output is rounded once (2^-11 of it; 2^-20 of the largest value for the sums)."""
    rng = np.random.default_rng([n, group, q_size, k_size])
    ng, fill = 4, 200
    k, v = large(rng, k_size, ng * 128 + fill)
    oc = oracle.OracleCache(1, 2, 128, 128, ng)
    oracle.prefill(oc, lambda b, t0, m: (k[:, t0:t0 + m], v[:, t0:t0 + m]), [ng], [fill])
    parent = trees.random_parents(rng, 1, n)
    q = np.clip(rng.standard_normal((1, 2 * group, n, 128)) * q_size, -65504, 65504).astype(np.float16)
    cache = load(torch, oc, rng)
    for mode in (DRAFT, VERIFY):
        got, gl = run(torch, cache, mode, q, parent, group)
        ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group)
        lead = ahead(oc, q, parent, mode == DRAFT, group)
        assert lead.mean() > 0.5
        err = np.abs(got - ref)[lead]
        assert np.all(err <= 2.0 ** -11 * np.abs(ref[lead]) + 2.0 ** -20 * np.abs(v).max()), err.max()
