"""qs_sample against its definition in 64 bits: the same tokens, the same tokens
kept, and probabilities to fp32: weights of 2^-36, and half a step, 2^-24, each for the
weight, the total, their quotient's scale and the product, 2^-22 together; what
weighs less than 2^-45 of the largest may be 0)."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def settings(rng, rows, **kw):
    pick = lambda xs, dt: np.array([xs[i] for i in rng.integers(0, len(xs), rows)], dt)  # noqa: E731
    s = dict(temperature=pick([0, 0.5, 0.8, 1, 1.7, 30], np.float32), top_k=pick([0, 1, 2, 7, 50, 900, 3000, 10 ** 6], np.int32),
             top_p=pick([1, 0.999, 0.95, 0.9, 0.5, 0.1, 0.0], np.float32), min_p=pick([0, 0.02, 0.2, 1], np.float32))
    for k, v in kw.items():
        s[k] = np.full(rows, v, s[k].dtype)
    return s


def run(torch, x, u, probs=True, stream=None, **s):
    rows, V = x.shape
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    token = torch.full((rows,), -77, dtype=torch.int32, device="cuda")
    pr = torch.full((rows, V), float("nan"), device="cuda") if probs else None
    qs.qs_sample(x, dev(u.astype(np.float32)), token, probs=pr, stream=stream, **{k: dev(v) for k, v in s.items()})
    torch.cuda.synchronize()
    return token.cpu().numpy(), pr.double().cpu().numpy() if probs else None


def check(torch, x, u, probs=True, **s):
    """x: a device tensor of logits."""
    token, pr = run(torch, x, u, probs, **s)
    xs = x.double().cpu().numpy()
    for r in range(len(xs)):
        one = {k: v[r] for k, v in s.items()}
        want, wp = trees.sample(xs[r], u[r], **one)
        assert token[r] == want, (r, one, u[r])
        if probs:
            tiny = wp < 2.0 ** -44 * wp.max()
            assert np.array_equal((pr[r] > 0)[~tiny], (wp > 0)[~tiny]), (r, one)
            assert np.all(np.abs(pr[r] - wp)[~tiny] <= 2.0 ** -22 * wp[~tiny]), (r, one)
            assert np.all(pr[r][tiny] <= wp[tiny] * 1.01), (r, one)


def logits(torch, rng, rows, V, dtype, std=2.5):
    x = rng.standard_normal((rows, V)) * std
    x[np.arange(rows)[:, None], rng.integers(0, V, (rows, 20))] += rng.uniform(4, 12, (rows, 20))
    return torch.from_numpy(x.astype(np.float32)).cuda().to(getattr(torch, dtype))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 8192, 8193, 32000, 65537, 131073, 262144])
def test_settings(torch, dtype, V):
    rng = np.random.default_rng([len(dtype), V])
    rows = 24 if V < 100000 else 8
    x = logits(torch, rng, rows, V, dtype)
    check(torch, x, rng.random(rows), **settings(rng, rows))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("one", [dict(top_p=0.9), dict(top_k=40), dict(top_k=5000), dict(min_p=0.03),
                                 dict(top_k=200, top_p=0.9, min_p=0.001), dict(temperature=0), dict()])
def test_each_filter_on_flat_and_peaked_rows(torch, dtype, one):
    rng = np.random.default_rng(len(dtype) + len(one))
    rows, V = 6, 50001
    off = dict(temperature=1, top_k=0, top_p=1, min_p=0)
    for std in (0.01, 1.0, 6.0):
        x = logits(torch, rng, rows, V, dtype, std)
        check(torch, x, rng.random(rows), **settings(rng, rows, **{**off, **one}))


def test_without_settings(torch):
    rng = np.random.default_rng(1)
    x = logits(torch, rng, 5, 12345, "float32")
    u = rng.random(5)
    token, pr = run(torch, x, u)
    for r in range(5):
        want, wp = trees.sample(x[r].double().cpu().numpy(), u[r])
        assert token[r] == want
        assert np.all(np.abs(pr[r] - wp) <= 2.0 ** -22 * wp + 2.0 ** -60)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("V", [9, 3001, 40000])
def test_equal_logits(torch, dtype, V):
    """Whole rows of one value, and of few: the lower index first, exact borders."""
    rng = np.random.default_rng(V)
    rows = 40
    x = np.full((rows, V), 1.5, np.float32)
    x[10:20] = rng.integers(-1, 2, (10, V))
    x[20:30] = np.where(rng.random((10, V)) < 0.5, -0.0, 0.0)
    x[30:] = rng.integers(0, 2, (10, V)) * 1e-3
    s = settings(rng, rows)
    s["top_p"][:5] = 0.5
    s["top_k"][:5] = 0
    s["min_p"][:5] = 0
    s["temperature"][:5] = 1
    check(torch, torch.from_numpy(x).cuda().to(getattr(torch, dtype)), rng.random(rows), **s)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_masked_and_odd_values(torch, dtype):
    """-inf, NaN, the type's lowest and largest values, +inf, subnormal steps; rows
    with one token left and with none."""
    rng = np.random.default_rng(3)
    rows, V = 16, 20011
    dt = getattr(torch, dtype)
    x = torch.from_numpy((rng.standard_normal((rows, V)) * 2).astype(np.float32)).cuda().to(dt)
    low, high = torch.finfo(dt).min, torch.finfo(dt).max
    hide = torch.from_numpy(rng.random((rows, V)) < 0.7).cuda()
    x[0][hide[0]] = -float("inf")
    x[1][hide[1]] = float("nan")
    x[2][hide[2]] = low
    x[3] = low
    x[4] = -float("inf")
    x[5] = float("nan")
    x[6] = -float("inf")
    x[6, 17] = -3.0
    x[7, 5], x[7, 9000], x[7, 3] = float("inf"), float("inf"), high
    x[8, 100] = high
    x[9] = low
    x[9, 77], x[9, 78] = high, high
    x[10] = -float("inf")
    x[10, V - 1] = low
    x[11] = x[11] * 1e-3 + (10000 if dtype == "float16" else 1e6)
    tiny = torch.finfo(dt).tiny
    x[12] = torch.from_numpy(rng.integers(0, 4, V).astype(np.float32)).cuda().to(dt) * (tiny / 4)
    x[13, ::2] = low
    x[13, 1::2] = x[13, 1::2] * 0 + high
    x[14][hide[14]] = -float("inf")
    x[14, 0] = float("nan")
    x[15, :-1] = -float("inf")
    for seed in range(4):
        r = np.random.default_rng(seed)
        s = settings(r, rows)
        check(torch, x, r.random(rows), **s)
    token, pr = run(torch, x, rng.random(rows), **settings(rng, rows))
    assert token[4] == -1 and token[5] == -1 and not pr[4].any() and not pr[5].any()


def test_uniform_numbers_at_their_ends(torch):
    rng = np.random.default_rng(4)
    x = logits(torch, rng, 1, 5000, "float32").expand(12, 5000).contiguous()
    u = np.array([0, 1e-45, 1e-30, 2.0 ** -24, 0.5, 1 - 2.0 ** -24, 1, 1.5, np.inf, -1, np.nan, -np.inf], np.float32)
    s = settings(rng, 12, temperature=1, top_k=0, top_p=1, min_p=0)
    check(torch, x, u, **s)
    s["top_k"][:] = 3
    check(torch, x, u, **s)


def test_odd_settings(torch):
    """NaN and out of range: off, or the end of the range."""
    rng = np.random.default_rng(5)
    x = logits(torch, rng, 12, 3000, "float32")
    s = settings(rng, 12, temperature=1, top_k=0, top_p=1, min_p=0)
    s["temperature"][:4] = [np.nan, -1, 1e-20, np.inf]
    s["top_k"][4:6] = [-5, 2 ** 31 - 1]
    s["top_p"][6:9] = [np.nan, -1, 2]
    s["min_p"][9:12] = [np.nan, -1, 5]
    check(torch, x, rng.random(12), **s)


def test_strides_and_offsets(torch):
    """Rows of a larger array, one that starts at an odd element, one row given to
    all."""
    rng = np.random.default_rng(6)
    for dtype in ("float16", "bfloat16", "float32"):
        big = logits(torch, rng, 9, 7777, dtype)
        for x in (big[:, 3:7003], big[::2, 1:20], big.reshape(-1)[5:5 + 3 * 9001].as_strided((3, 9001), (9001, 1))):
            check(torch, x, rng.random(len(x)), **settings(rng, len(x)))


def test_many_rows_largest_vocabulary_and_no_probs(torch):
    rng = np.random.default_rng(7)
    x = logits(torch, rng, 700, 400, "float16")
    check(torch, x, rng.random(700), False, **settings(rng, 700))
    for dtype in ("bfloat16", "float32"):
        x = logits(torch, rng, 2, qs.QS_MAX_VOCAB, dtype)
        check(torch, x, rng.random(2), **settings(rng, 2, top_k=0, temperature=1))


def test_frequencies(torch):
    """20,000 draws from a small row: each token as often as its probability says,
    within five standard deviations."""
    rng = np.random.default_rng(8)
    n = 20000
    x = logits(torch, rng, 1, 40, "float32", 1.0).expand(n, 40)
    token, _ = run(torch, x.contiguous(), rng.random(n), False, temperature=np.full(n, 2.0, np.float32))
    _, p = trees.sample(x[0].double().cpu().numpy(), 0.5, temperature=2.0)
    count = np.bincount(token, minlength=40)
    assert np.all(np.abs(count - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1)


def test_streams_and_graphs(torch):
    rng = np.random.default_rng(9)
    sides = [dict(x=logits(torch, rng, 3, 20000, "float16"), u=torch.from_numpy(rng.random(3).astype(np.float32)).cuda(),
                  token=torch.empty((10, 3), dtype=torch.int32, device="cuda"), s=torch.cuda.Stream())
             for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(10):
        for d in sides:
            qs.qs_sample(d["x"], d["u"], d["token"][i], stream=d["s"])
    torch.cuda.synchronize()
    for d in sides:
        want = [trees.sample(d["x"][r].double().cpu().numpy(), float(d["u"][r]))[0] for r in range(3)]
        assert (d["token"].cpu().numpy() == want).all()
    d = sides[0]
    g = torch.cuda.CUDAGraph()
    k = torch.full((3,), 20, dtype=torch.int32, device="cuda")
    with torch.cuda.graph(g):
        qs.qs_sample(d["x"], d["u"], d["token"][0], top_k=k)
    d["x"].copy_(logits(torch, rng, 3, 20000, "float16"))
    k[1] = 1
    g.replay()
    torch.cuda.synchronize()
    want = [trees.sample(d["x"][r].double().cpu().numpy(), float(d["u"][r]), top_k=int(k[r]))[0] for r in range(3)]
    assert d["token"][0].tolist() == want


@pytest.mark.parametrize("V", [1000, 32000, 65537])
def test_probabilities_in_the_place_of_the_logits(torch, V):
    rng = np.random.default_rng(V)
    rows = 5
    x, u = logits(torch, rng, rows, V, "float32"), rng.random(rows)
    s = settings(rng, rows, top_p=0.9)
    token, pr = run(torch, x, u, **s)
    dev = {k: torch.from_numpy(v).cuda() for k, v in s.items()}
    t2 = torch.full((rows,), -77, dtype=torch.int32, device="cuda")
    qs.qs_sample(x, torch.from_numpy(u.astype(np.float32)).cuda(), t2, probs=x, **dev)
    torch.cuda.synchronize()
    assert np.array_equal(t2.cpu().numpy(), token) and np.array_equal(x.double().cpu().numpy(), pr)
