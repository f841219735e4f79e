"""The bounds-checked build over the listed attention, the paged writes and
their edge cases: no failed check, results as in the ordinary build."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import paging
from tests.test_gpu_checked import checked  # noqa: F401  (fixture)
from tests.test_gpu_listed_attn import load, random_sel, run
from tests.test_gpu_qs import DRAFT, VERIFY, _oracle_state, assert_close, h16, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("n_q,group", [(1, 1), (5, 1), (5, 4)])
def test_listed_attention(checked, n_q, group, ub):  # noqa: F811
    torch, failures = checked
    rng = np.random.default_rng(n_q + group + ub)
    ng, fill = [9, 0, 3], [255, 30, 64]
    B, H = 3, 2
    oc = _oracle_state(rng, B, H, ng, fill, cap=9)
    sel = random_sel(rng, B, H, 5, ng)
    sel[0, 0, 1] = 50
    for paged in (True, False):
        cache = load(torch, oc, rng, ub, paged)
        if paged:
            cache.table[2, 1] = -5
        q = h16(rng, (B, H * group, n_q, 128))
        times = [paging.counts(oc, b, sel) for b in range(B)]
        if paged:
            times[2][:, 1] = 0
        for mode in (DRAFT, VERIFY):
            got, gl = run(torch, cache, mode, q, group, sel)
            ref, rl = paging.attention(oc, q, mode == DRAFT, group, ub, times=times)
            assert_close(got, ref, gl, rl, "mode %d" % mode)
    assert failures() == (0, 0)


def test_paged_writes(checked):  # noqa: F811
    torch, failures = checked
    rng = np.random.default_rng(2)
    B, H = 2, 3
    k, v = h16(rng, (B, H, 800, 128)), h16(rng, (B, H, 800, 128))
    cache = qs.PagedCache(B, H, 6, 13)
    cache.table.copy_(torch.from_numpy(paging.random_table(rng, [6, 5], 6, 13)))
    qs.qs_prefill_paged(cache, to_dev(torch, k), to_dev(torch, v), to_dev(torch, np.array([800, 500], np.int32)))
    qs.qs_quantize_flush_due_paged(cache, 200)
    assert np.all(qs.qs_get_errors(cache) == 0)
    assert failures() == (0, 0)
