"""One workspace, of the size that the whole tree's verification asks for, serves the
narrower calls of the round too."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import trees
from tests.test_gpu_listed_attn import load
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, h16, to_dev
from tests.test_gpu_tree_attn import check, torch  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,ub", [(1, 32, 4), (8, 8, 4), (3, 5, 2)])
def test_the_size_grows_with_the_rows(torch, B, H, ub):  # noqa: F811
    cache = qs.Cache(B, H, 4, upper_bits=ub)
    of_rows = {}
    for group in (1, 2, 3, 4, 8, 12, 24, 64, 512):
        for n_q in range(1, min(64, 512 // group) + 1):
            size = qs.qs_attn_tree_workspace_size(cache, n_q, group)
            assert of_rows.setdefault(group * n_q, size) == size
    sizes = [of_rows[r] for r in sorted(of_rows)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("n,group", [(60, 1), (30, 4), (9, 8), (20, 1)])
def test_levels_in_the_trees_workspace(torch, n, group):  # noqa: F811
    rng = np.random.default_rng([n, group])
    B, H = 1, 6
    oc = _oracle_state(rng, B, H, [40], [150], cap=40)
    cache = load(torch, oc, rng)
    parent = trees.random_parents(rng, B, n)
    ws = torch.empty(qs.qs_attn_tree_workspace_size(cache, n, group), dtype=torch.uint8, device="cuda")
    for mode in (DRAFT, VERIFY):
        for n_q in sorted({1, 2, 4, 5, 8, 9, 16, 17, 24, 25, n} & set(range(1, n + 1))):
            q = h16(rng, (B, H * group, n_q, 128))
            out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
            qs.qs_attn_decode_tree(cache, mode, to_dev(torch, parent), to_dev(torch, q), 1 / np.sqrt(128), out, None,
                                   ws, group=group)
            torch.cuda.synchronize()
            ref, _ = trees.attention(oc, q, parent, mode == DRAFT, group)
            check(out.double().cpu().numpy(), None, ref, None, "mode %d, %d queries" % (mode, n_q))
