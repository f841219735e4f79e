"""The bounds-checked build over the rest of a tree's round: sampling, the append with
rotation and the acceptance.  No failed check, results as in the ordinary build."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import test_gpu_sample as sample
from tests import trees
from tests.test_gpu_checked import checked  # noqa: F401  (fixture)
from tests.test_gpu_qs import h16, to_dev
from tests.test_gpu_tree_buffer import close, make, tokens_for

pytestmark = pytest.mark.gpu


def test_every_file_with_checks_reports(checked):  # noqa: F811
    for name in ("buffer_tree", "sample", "tree"):
        assert hasattr(qs.lib(), "qs_checked_failures_" + name)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("V", [1, 31, 1001, 8193, 33793, 67585, 100003, 368640])
def test_sampling(checked, dtype, V):  # noqa: F811
    """Odd vocabularies, remainders of a slice, and the most a slice holds."""
    torch, failures = checked
    rng = np.random.default_rng([len(dtype), V])
    rows = 12 if V < 100000 else 4
    x = sample.logits(torch, rng, rows, V, dtype)
    x[0] = 1.0  # one value: full bins and lists
    sample.check(torch, x, rng.random(rows), **sample.settings(rng, rows))
    for k, t in ((700, 0.25), (40, 1), (0, 1)):
        s = sample.settings(rng, rows, top_k=k, temperature=t)
        sample.check(torch, x, rng.random(rows), **s)
    assert failures() == (0, 0)


def test_sampling_strided_rows(checked):  # noqa: F811
    torch, failures = checked
    rng = np.random.default_rng(2)
    for dtype in ("float16", "float32"):
        big = sample.logits(torch, rng, 9, 7777, dtype)
        for x in (big[:, 3:7003], big[::2, 1:20], big[2:3, 5:]):
            sample.check(torch, x, rng.random(len(x)), **sample.settings(rng, len(x)))
    assert failures() == (0, 0)


@pytest.mark.parametrize("n", [1, 5, 63, 256])
@pytest.mark.parametrize("rot,interleaved", [(16, False), (96, False), (128, False), (48, True), (128, True)])
def test_append(checked, n, rot, interleaved):  # noqa: F811
    """Into rings that end inside the tokens, and one without room."""
    torch, failures = checked
    rng = np.random.default_rng([n, rot])
    B, H, group = 3, 2, 3
    fill = np.array([0, 256 - n, min(255, 257 - n + 9)])
    c, st = make(torch, rng, B, H, fill, [3, 1, 2])
    room = fill + n <= 256
    k, v, q = h16(rng, (B, H, n, 128)), h16(rng, (B, H, n, 128)), h16(rng, (B, H * group, n, 128))
    freq = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    q_out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    x = to_dev(torch, np.concatenate([q, k, v], 1).transpose(0, 2, 1, 3)).transpose(1, 2)  # heads side by side
    qs.qs_buffer_append_rotary(c, x[:, H * group:H * group + H], x[:, H * group + H:], to_dev(torch, freq),
                               q=x[:, :H * group], q_out=q_out, interleaved=interleaved)
    pos = st[:, :1] * 128 + fill[:, None] + np.arange(n)
    close(q_out.cpu().numpy(), trees.rotate(q, pos[:, None], freq, interleaved), q)
    want = trees.rotate(k, pos[:, None], freq, interleaved)
    for b in np.flatnonzero(room):
        at = (st[b, 3] * 128 + fill[b] + np.arange(n)) % 256
        close(c.buf_k[b].cpu().numpy()[:, at], want[b], k[b])
        assert np.array_equal(c.buf_v[b].cpu().numpy()[:, at], v[b])
    assert failures() == (0, 0)


@pytest.mark.parametrize("n", [1, 33, 64])
def test_accept(checked, n):  # noqa: F811
    torch, failures = checked
    rng = np.random.default_rng(n)
    B, H = 6, 3
    fill = rng.integers(n, 257, B)
    c, st = make(torch, rng, B, H, fill, [1] * B, pending=n)
    parent = trees.random_parents(rng, B, n, reach=3)
    parent[1] = np.arange(-1, n - 1)
    if n > 1:
        parent[2, n - 1] = n  # no tree
    dt = [tokens_for(rng, parent[b], n, 0.9) for b in range(B)]
    draft, target = np.stack([d for d, _ in dt]), np.stack([t for _, t in dt])
    draft[1], target[1] = np.arange(n), np.arange(1, n + 1)
    bk = c.buf_k.cpu().numpy()
    out = [torch.full((B, n) if i else (B,), -77, dtype=torch.int32, device="cuda") for i in range(3)]
    qs.qs_tree_accept(c, to_dev(torch, parent), to_dev(torch, draft), to_dev(torch, target), *out)
    gk = c.buf_k.cpu().numpy()
    for b in range(B):
        want = [] if n > 1 and b == 2 else trees.accept(parent[b], draft[b], target[b])
        assert out[0][b] == len(want) and out[1][b].tolist() == want + [-1] * (n - len(want))
        src = np.arange(256)
        first = st[b, 3] * 128 + fill[b] - n
        src[(first + np.arange(len(want))) % 256] = (first + np.array(want, int)) % 256
        assert np.array_equal(gk[b], bk[b][:, src])
    assert failures() == (0, 0)
