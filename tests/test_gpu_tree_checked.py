"""The bounds-checked build over the attention of a tree's nodes, by both of its
ways: no failed check, results as in the ordinary build."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import trees
from tests.test_gpu_checked import checked  # noqa: F401  (fixture)
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, h16
from tests.test_gpu_tree_attn import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("n_tree,n_q,group", [(1, 1, 1), (12, 6, 4), (25, 25, 1), (64, 33, 2), (50, 50, 2), (64, 64, 5)])
def test_tree_attention(checked, n_tree, n_q, group, ub):  # noqa: F811
    torch, failures = checked
    rng = np.random.default_rng([n_tree, n_q, group, ub])
    B, H = 3, 3
    oc = _oracle_state(rng, B, H, [9, 0, 4], [255, n_tree, 150], cap=9)
    parent = trees.random_parents(rng, B, n_tree)
    q = h16(rng, (B, H * group, n_q, 128))
    for paged in (True, False):
        cache = load(torch, oc, rng, ub, paged)
        if paged:
            cache.table[2, 1] = -5
        for mode in (DRAFT, VERIFY):
            got, gl = run(torch, cache, mode, q, parent, group)
            ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group, ub, left_out=[(2, 1)] if paged else ())
            check(got, gl, ref, rl, "mode %d paged %d" % (mode, paged))
        assert list(qs.qs_get_errors(cache)) == [0, 0, qs.DEV_PAGE if paged else 0]
    assert failures() == (0, 0)
