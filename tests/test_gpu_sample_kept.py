"""Which tokens qs_sample keeps, told by its probabilities, where the filters reach
far down: a top-k that takes in more logits than weigh anything in the draw (fewer
than k of them above 2^-46 of the largest)."""
import numpy as np
import pytest

from tests import trees
from tests.test_gpu_sample import logits, run, torch  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def check_kept(torch, x, u, least, **s):  # noqa: F811
    """As the definition says: the token, no probability outside the kept tokens, and
    inside, from a weight of 2^least of the largest on, the quotient to 2^-22 (half a
    step, 2^-24, each for the weight, the total, their quotient's scale and the product)."""
    token, pr = run(torch, x, u, **s)
    xs = x.double().cpu().numpy()
    for r in range(len(xs)):
        one = {k: v[r] for k, v in s.items()}
        want, wp = trees.sample(xs[r], u[r], **one)
        assert token[r] == want, (r, one)
        assert not pr[r][wp == 0].any(), (r, one, int((pr[r][wp == 0] > 0).sum()))
        near = wp >= 2.0 ** least * wp.max()
        assert np.all(np.abs(pr[r] - wp)[near] <= 2.0 ** -22 * wp[near]), (r, one)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("V,k,T", [(32000, 1000, 0.25), (1000, 200, 0.3), (8192, 3000, 0.5), (600, 599, 0.1),
                                   (131073, 5000, 0.2)])
def test_a_top_k_beyond_what_weighs(torch, dtype, V, k, T):  # noqa: F811
    rng = np.random.default_rng([V, k, len(dtype)])
    rows = 6
    x = logits(torch, rng, rows, V, dtype)
    x[2] = (x[2] * 2).round() / 2  # (many equal ones: the border lies among them)
    x[3, 5:] = -float("inf")       # fewer logits than k
    x[4, ::3] = float("nan")
    full = lambda v, t: np.full(rows, v, t)  # noqa: E731
    s = dict(temperature=full(T, np.float32), top_k=full(k, np.int32))
    check_kept(torch, x, rng.random(rows), -60, **s)
    s["min_p"] = np.array([0, 1e-20, 0, 1e-30, 0, 0.5], np.float32)
    check_kept(torch, x, rng.random(rows), -60, **s)
    s["top_p"] = np.array([1, 1, 0.999, 1, 0.5, 1], np.float32)
    check_kept(torch, x, rng.random(rows), -60, **s)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("V,T", [(1000, 0.2), (32000, 0.25), (131073, 0.3), (368640, 0.25)])
def test_kept_tokens_of_small_weights(torch, dtype, V, T):  # noqa: F811
    """Whatever is kept has its share, down to 2^-107 of the largest weight: with up to
    2^18.5 tokens the quotient is a normal number of fp32 there."""
    rng = np.random.default_rng([V, len(dtype)])
    rows = 4
    x = logits(torch, rng, rows, V, dtype)
    full = lambda v, t: np.full(rows, v, t)  # noqa: E731
    s = dict(temperature=full(T, np.float32))
    check_kept(torch, x, rng.random(rows), -106.9, **s)
    s["top_k"] = np.array([0, 700, V - 1, 0], np.int32)
    s["min_p"] = np.array([1e-25, 0, 0, 1e-31], np.float32)
    check_kept(torch, x, rng.random(rows), -106.9, **s)
