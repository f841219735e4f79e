"""Queries rotated where they lie inside a projection's output, next to the keys and
values of the same call."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import trees
from tests.test_gpu_qs import h16, to_dev
from tests.test_gpu_tree_buffer import close, make, torch  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("group", [1, 4])
def test_queries_in_a_projections_output(torch, n, group):  # noqa: F811
    rng = np.random.default_rng([n, group])
    H, heads = 3, (2 + group) * 3
    c, st = make(torch, rng, 1, H, [20], [2])
    # (one token's heads side by side, or each head's tokens)
    x = h16(rng, (1, heads, n, 128))
    xd = to_dev(torch, x)
    q, k, v = xd[:, :group * H], xd[:, group * H:group * H + H], xd[:, group * H + H:]
    freq = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    qs.qs_buffer_append_rotary(c, k, v, to_dev(torch, freq), q=q, q_out=q)
    got, pos = xd.cpu().numpy(), 276 + np.arange(n)
    close(got[:, :group * H], trees.rotate(x[:, :group * H], pos[None, None], freq, False), x[:, :group * H])
    assert np.array_equal(got[:, group * H:], x[:, group * H:])
    at = (st[0, 3] * 128 + 20 + np.arange(n)) % 256
    kx = x[:, group * H:group * H + H]
    close(c.buf_k.cpu().numpy()[:, :, at], trees.rotate(kx, pos[None, None], freq, False), kx)
    assert np.array_equal(c.buf_v.cpu().numpy()[:, :, at], x[:, group * H + H:])
