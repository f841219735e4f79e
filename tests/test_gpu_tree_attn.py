"""qs_attn_decode_tree against softmax attention in 64 bits under the mask of the
nodes' ancestors.

Tolerances: those of the other attention calls (max-abs 1e-2, log-sum-exp 5e-3),
and 1e-3 of the output in norm.  What is rounded, in rms of a rounding's 2^-11 /
sqrt(3) = 2.8e-4: the output (once); the weights and values of a sum (which average
out over its tokens, but a single token may carry it: twice more); the keys, which
move a score by up to 4e-4 with the eightfold channels of these inputs.  In squares
7e-4."""
import numpy as np
import oracle
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import trees
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, assert_close, h16, to_dev

pytestmark = pytest.mark.gpu

RRMS = 1e-3


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def run(torch, cache, mode, q, parent, group=1, stream=None, lse=True):
    qd = to_dev(torch, q)
    out = torch.full_like(qd, float("nan"))
    ld = torch.full(q.shape[:3], float("nan"), dtype=torch.float32, device="cuda") if lse else None
    ws = torch.empty(qs.qs_attn_tree_workspace_size(cache, q.shape[2], group), dtype=torch.uint8, device="cuda")
    qs.qs_attn_decode_tree(cache, mode, to_dev(torch, parent), qd, 1.0 / np.sqrt(128), out, ld, ws, group=group,
                           stream=stream)
    torch.cuda.synchronize()
    assert int(cache.arrive.abs().sum().item()) == 0
    return out.double().cpu().numpy(), ld.double().cpu().numpy() if lse else None


def check(got, gl, ref, rl, what=""):
    assert_close(got, ref, gl, rl, what)
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
    assert rel <= RRMS, "%s: %.3g" % (what, rel)


SHAPES = [(1, 1, 1), (2, 2, 1), (7, 7, 1), (21, 8, 1), (24, 24, 1), (12, 2, 12), (25, 25, 1), (26, 26, 1),
          (64, 64, 1), (33, 17, 3), (64, 1, 32), (43, 43, 3), (64, 64, 2), (61, 26, 5), (64, 64, 4),
          (60, 60, 5), (64, 64, 8)]


@pytest.mark.parametrize("n_groups,fill", [(0, 64), (1, 127), (2, 129), (4, 256)])
@pytest.mark.parametrize("n_tree,n_q,group", SHAPES)
def test_sizes(torch, n_groups, fill, n_tree, n_q, group):
    rng = np.random.default_rng([n_groups, fill, n_tree, n_q, group])
    B, H = 2, 3
    oc = _oracle_state(rng, B, H, [n_groups, max(n_groups - 1, 0)], [fill, max(fill // 2, n_tree)],
                       cap=n_groups + 1)
    parent = trees.random_parents(rng, B, n_tree, roots=0.1)
    q = h16(rng, (B, H * group, n_q, 128))
    for paged in (False, True):
        cache = load(torch, oc, rng, paged=paged)
        for mode in (DRAFT, VERIFY):
            got, gl = run(torch, cache, mode, q, parent, group)
            ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group)
            check(got, gl, ref, rl, "mode %d paged %d" % (mode, paged))
        assert np.all(qs.qs_get_errors(cache) == 0)


@pytest.mark.parametrize("n_tree,n_q,group", [(7, 7, 1), (20, 5, 4), (30, 30, 1), (64, 64, 3)])
@pytest.mark.parametrize("paged", [False, True])
def test_two_bit_layout(torch, n_tree, n_q, group, paged):
    rng = np.random.default_rng([n_tree, n_q, group, paged])
    B, H = 2, 2
    oc = _oracle_state(rng, B, H, [6, 3], [200, 99], cap=6)
    parent = trees.random_parents(rng, B, n_tree)
    q = h16(rng, (B, H * group, n_q, 128))
    cache = load(torch, oc, rng, 2, paged)
    for mode in (DRAFT, VERIFY):
        got, gl = run(torch, cache, mode, q, parent, group)
        ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group, 2)
        check(got, gl, ref, rl, "mode %d" % mode)


@pytest.mark.parametrize("B,H,ng,n_q,group", [(1, 2, 300, 64, 4), (1, 1, 70, 40, 1), (3, 8, 40, 26, 1),
                                              (1, 40, 9, 64, 1), (5, 7, 33, 30, 7), (1, 3, 150, 5, 4)])
def test_many_units(torch, B, H, ng, n_q, group):
    """Segments over many CTAs, CTAs over many segments, ragged."""
    rng = np.random.default_rng([B, H, ng, n_q, group])
    n = [max(0, ng - 11 * b) for b in range(B)]
    oc = _oracle_state(rng, B, H, n, [int(x) for x in rng.integers(n_q, 257, B)], cap=ng)
    parent = trees.random_parents(rng, B, n_q)
    q = h16(rng, (B, H * group, n_q, 128))
    cache = load(torch, oc, rng)
    for mode in (DRAFT, VERIFY):
        got, gl = run(torch, cache, mode, q, parent, group)
        ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group)
        check(got, gl, ref, rl, "mode %d" % mode)


@pytest.mark.parametrize("n,group", [(5, 1), (24, 1), (40, 1), (64, 8)])
def test_a_chain_is_the_causal_attention(torch, n, group):
    """Each node the child of the one before: what the calls for chains see."""
    rng = np.random.default_rng([n, group])
    B, H = 2, 2
    oc = _oracle_state(rng, B, H, [3, 1], [140, 70], cap=3)
    parent = np.tile(np.arange(-1, n - 1, dtype=np.int32), (B, 1))
    q = h16(rng, (B, H * group, n, 128))
    cache = load(torch, oc, rng)
    got, gl = run(torch, cache, VERIFY, q, parent, group)
    for j0 in range(0, n, 8 if group == 1 else 1):  # the queries the chain calls take, from the last on
        j1 = min(n, j0 + (8 if group == 1 else 1))
        drop = n - j1
        cache.state[:, 1] -= drop
        out = torch.empty((B, H * group, j1 - j0, 128), dtype=torch.float16, device="cuda")
        ws = torch.empty(qs.qs_attn_workspace_size_gqa(cache, j1 - j0, group), dtype=torch.uint8, device="cuda")
        qs.qs_attn_decode_paged(cache, VERIFY, to_dev(torch, q[:, :, j0:j1]), 1 / np.sqrt(128), out, None, ws,
                                group=group)
        torch.cuda.synchronize()
        cache.state[:, 1] += drop
        check(got[:, :, j0:j1], None, out.double().cpu().numpy(), None, "nodes %d.." % j0)


@pytest.mark.parametrize("n,n_q,group", [(9, 9, 1), (40, 33, 1), (64, 64, 4)])
def test_preconditions_on_the_device(torch, n, n_q, group):
    """Too few tokens, parents that are none, pages out of range: flagged, and the
    other sequences are as they should be."""
    rng = np.random.default_rng([n, n_q])
    B, H = 4, 2
    oc = _oracle_state(rng, B, H, [3, 2, 4, 1], [n, n - 1, 200, n + 3], cap=4)
    parent = trees.random_parents(rng, B, n)
    parent[2, 3], parent[2, 5], parent[2, 0] = 3, -2, 7
    q = h16(rng, (B, H * group, n_q, 128))
    cache = load(torch, oc, rng)
    cache.table[3, 0] = 10 ** 6
    cache.table[0, 2] = -1
    for mode in (DRAFT, VERIFY):
        got, gl = run(torch, cache, mode, q, parent, group)
        ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group, left_out=[(3, 0), (0, 2)])
        check(got, gl, ref, rl, "mode %d" % mode)
        assert np.all(got[1] == 0) and np.all(gl[1] == -np.inf)
        assert list(qs.qs_get_errors(cache)) == [qs.DEV_PAGE, qs.DEV_NQ_GT_FILL, qs.DEV_TREE, qs.DEV_PAGE]


@pytest.mark.parametrize("n,group", [(8, 1), (8, 3), (40, 1), (64, 2), (64, 5)])
@pytest.mark.parametrize("fill", [64, 128, 191, 256])
def test_what_a_node_does_not_see_may_hold_anything(torch, n, group, fill):
    """Infinities and NaN in the keys and values of nodes reach the rows that see
    them and no others, nor does what lies in the ring behind the last token."""
    rng = np.random.default_rng([n, group, fill])
    B, H = 1, 2
    oc = _oracle_state(rng, B, H, [2], [fill], cap=2)
    parent = trees.random_parents(rng, B, n, reach=4, roots=0.3)
    sick_v, sick_k = n // 2, n // 3
    parent[0, sick_k] = parent[0, sick_v] = 0
    sees = trees.ancestors(parent[0])
    q = h16(rng, (B, H * group, n, 128))
    cache = load(torch, oc, rng)
    ref, rl = trees.attention(oc, q, parent, False, group)
    slot = lambda j: (int(cache.state[0, 3]) * 128 + fill - n + j) % 256  # noqa: E731
    for j in range(n, n + 256 - fill):
        cache.buf_k[:, :, slot(j)] = float("nan")
        cache.buf_v[:, :, slot(j)] = float("inf")
    cache.buf_v[:, 0, slot(sick_v), 77] = float("inf")
    cache.buf_v[:, 1, slot(sick_v), 12] = float("nan")
    cache.buf_v[:, 1, slot(sick_v), 13] = -float("inf")
    cache.buf_k[:, :, slot(sick_k), 5] = float("nan")
    got, gl = run(torch, cache, VERIFY, q, parent, group)
    well = ~(sees[:, sick_v] | sees[:, sick_k])
    assert 0 < well.sum() < n
    check(got[:, :, well], gl[:, :, well], ref[:, :, well], rl[:, :, well])
    assert np.isnan(got[:, :, ~well]).all()


def test_streams_graphs_and_no_lse(torch):
    """Two caches on two streams, calls not waited for; then a captured call that
    follows its queries, its tree and its cache through replays."""
    rng = np.random.default_rng(8)
    B, H, n, group = 1, 4, 40, 2
    side = []
    for i in range(2):
        oc = _oracle_state(rng, B, H, [20 + i], [200], cap=22)
        parent = trees.random_parents(rng, B, n)
        q = h16(rng, (6, B, H * group, n, 128))
        cache = load(torch, oc, rng)
        ws = torch.empty(qs.qs_attn_tree_workspace_size(cache, n, group), dtype=torch.uint8, device="cuda")
        side.append(dict(oc=oc, parent=parent, q=q, cache=cache, ws=ws, qd=to_dev(torch, q),
                         pd=to_dev(torch, parent), s=torch.cuda.Stream(),
                         out=torch.empty((6, B, H * group, n, 128), dtype=torch.float16, device="cuda")))
    torch.cuda.synchronize()

    def call(x, i, stream=None):
        qs.qs_attn_decode_tree(x["cache"], VERIFY, x["pd"], x["qd"][i], 1 / np.sqrt(128), x["out"][i], None,
                               x["ws"], group=group, stream=stream)
    for i in range(6):
        for x in side:
            call(x, i, x["s"])
    torch.cuda.synchronize()
    refs = [[trees.attention(x["oc"], x["q"][i], x["parent"], False, group)[0] for i in range(6)] for x in side]
    for x, ref in zip(side, refs):
        for i in range(6):
            check(x["out"][i].double().cpu().numpy(), None, ref[i], None)
    x = side[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, 0)
        call(x, 1)
    x["out"].zero_()
    g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        check(x["out"][i].double().cpu().numpy(), None, refs[0][i], None)
    x["qd"][1] = x["qd"][4]
    parent = trees.random_parents(rng, B, n, reach=2)
    x["pd"].copy_(torch.from_numpy(parent))
    x["cache"].state[:, 1] -= 3
    g.replay()
    torch.cuda.synchronize()
    x["oc"].state[:, 1] -= 3  # (its fill)
    want = trees.attention(x["oc"], x["q"][4], parent, False, group)[0]
    check(x["out"][1].double().cpu().numpy(), None, want, None)


@pytest.mark.parametrize("size", [-10, 0, 12])
@pytest.mark.parametrize("n,group", [(8, 1), (40, 1), (50, 2), (64, 4)])
def test_keys_with_offsets_and_values_of_any_size(torch, n, group, size):
    """Values of 2^size, three channels of the keys far from zero, and one that reaches
    both ends of fp16 (against small queries).  The offset channels stand at 15 +- 2
    or more: what lies outside a tile's range there, up to 16, is rounded by 2^-8 /
    sqrt(3) in rms, three of them move a score by 3.4e-4, so 8e-4 with the rest."""
    rng = np.random.default_rng([n, group, size + 20])
    B, H, ng, fill = 1, 2, 4, 200
    k = rng.standard_normal((B, H, ng * 128 + fill, 128)) * 2
    k[..., :3] += 15
    k[..., 9] = np.where(rng.random(k.shape[:3]) < 0.1, 65504 * np.sign(k[..., 8]), 100 * k[..., 9])
    v = rng.standard_normal(k.shape) * 2.0 ** size + 2.0 ** size
    k, v = k.astype(np.float16), v.astype(np.float16)
    oc = oracle.OracleCache(B, H, 128, 128, ng)
    oracle.prefill(oc, lambda b, t0, m: (k[b, :, t0:t0 + m], v[b, :, t0:t0 + m]), [ng], [fill])
    parent = trees.random_parents(rng, B, n)
    q = h16(rng, (B, H * group, n, 128))
    q[..., 9] *= np.float16(2.0 ** -13)
    for ub in (4, 2):
        cache = load(torch, oc, rng, ub)
        for mode in (DRAFT, VERIFY):
            got, gl = run(torch, cache, mode, q, parent, group)
            ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group, ub)
            rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
            assert rel <= RRMS and np.abs(gl - rl).max() <= 5e-3, (mode, ub, rel, np.abs(gl - rl).max())


@pytest.mark.parametrize("q_size,k_size", [(1, 3000), (100, 100), (3000, 3000), (8000, 8000)])
@pytest.mark.parametrize("n,group", [(40, 1), (30, 5)])
def test_scores_of_any_size(torch, n, group, q_size, k_size):
    """Above 24 rows finite queries and keys give finite results, however large their
    products.  A score is then off by the rounding of the keys' second part, a
    fifteenth of their range, so 2^-12 / sqrt(3) of 2 / 15 of the largest key (4 of its
    sizes) in each of 128 channels, against a log-sum-exp of some 3.5 of a
    score's sizes: 2.1e-5 of it in rms, and five of those are allowed."""
    rng = np.random.default_rng([n, group, q_size, k_size])
    B, H, ng, fill = 1, 2, 4, 200
    k = np.clip(rng.standard_normal((B, H, ng * 128 + fill, 128)) * k_size, -65504, 65504).astype(np.float16)
    v = rng.standard_normal(k.shape).astype(np.float16)
    oc = oracle.OracleCache(B, H, 128, 128, ng)
    oracle.prefill(oc, lambda b, t0, m: (k[b, :, t0:t0 + m], v[b, :, t0:t0 + m]), [ng], [fill])
    parent = trees.random_parents(rng, B, n)
    q = np.clip(rng.standard_normal((B, H * group, n, 128)) * q_size, -65504, 65504).astype(np.float16)
    cache = load(torch, oc, rng)
    for mode in (DRAFT, VERIFY):
        got, gl = run(torch, cache, mode, q, parent, group)
        _, rl = trees.attention(oc, q, parent, mode == DRAFT, group)
        assert np.isfinite(got).all() and np.abs(got).max() <= np.abs(v).max() * 1.01
        assert np.all(np.abs(gl - rl) <= 1.1e-4 * np.abs(rl))


@pytest.mark.parametrize("B,H,n,group", [(256, 1, 30, 1), (256, 2, 3, 2), (1, 1, 1, 512), (2, 1, 2, 256)])
def test_many_sequences_and_many_heads(torch, B, H, n, group):
    """As many sequences as a cache holds, some without room for the tree (all of them
    in the last call); a KV head with as many query heads as a call takes."""
    rng = np.random.default_rng([B, H, n, group])
    ng = [int(x) for x in rng.integers(0, 2, B)]
    fill = [int(x) for x in rng.integers(max(1, n - 2), n + 40, B)]
    oc = _oracle_state(rng, B, H, ng, fill, cap=1)
    parent = trees.random_parents(rng, B, n)
    q = h16(rng, (B, H * group, n, 128))
    cache = load(torch, oc, rng)
    got, gl = run(torch, cache, VERIFY, q, parent, group)
    ref, rl = trees.attention(oc, q, parent, False, group)
    fits = np.array(fill) >= n
    check(got, gl, ref, rl)
    assert np.all(got[~fits] == 0) and np.all(gl[~fits] == -np.inf)
    assert list(qs.qs_get_errors(cache)) == [0 if f else qs.DEV_NQ_GT_FILL for f in fits]
    cache.state[:, 1] = 0
    got, gl = run(torch, cache, VERIFY, q, parent, group)
    assert np.all(got == 0) and np.all(gl == -np.inf)
    assert list(qs.qs_get_errors(cache)) == [qs.DEV_NQ_GT_FILL] * B
