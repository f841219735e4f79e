"""Row counts on both sides of the borders between the two ways of a tree's attention:
16 rows of a verification, 24 of a draft (both layouts, contiguous and in pages; the
workspace of exactly the size that is asked for).  Tolerances: those of
tests/test_gpu_tree_attn.py."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import trees
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, h16
from tests.test_gpu_tree_attn import check, run, torch  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("n_q,group", [(15, 1), (5, 3), (16, 1), (4, 4), (1, 16), (17, 1), (1, 17), (9, 2), (23, 1),
                                       (24, 1), (6, 4), (25, 1), (5, 5)])
@pytest.mark.parametrize("B", [1, 3])
def test_rows(torch, B, n_q, group, ub):  # noqa: F811
    rng = np.random.default_rng([B, n_q, group, ub])
    H, n = 2, n_q + 2
    oc = _oracle_state(rng, B, H, [11, 0, 3][:B], [201, n, 140][:B], cap=11)
    parent = trees.random_parents(rng, B, n, roots=0.1)
    q = h16(rng, (B, H * group, n_q, 128))
    for paged in (False, True):
        cache = load(torch, oc, rng, ub, paged)
        for mode in (DRAFT, VERIFY):
            got, gl = run(torch, cache, mode, q, parent, group)
            ref, rl = trees.attention(oc, q, parent, mode == DRAFT, group, ub)
            check(got, gl, ref, rl, "mode %d paged %d" % (mode, paged))
        assert np.all(qs.qs_get_errors(cache) == 0)
