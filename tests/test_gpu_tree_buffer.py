"""qs_buffer_append_rotary and qs_tree_accept against their definitions in 64 bits.

A rotated element is rounded to fp16 once (half a step, 2^-11 of it) from an fp32
value whose error is that of three roundings and of the sine and cosine: a few
2^-23 of the pair's length (2^-20 is allowed); below the normal numbers half a
step is 2^-25."""
import numpy as np
import pytest

from hierarchical_quantized_kv_gb300 import qs
from tests import trees
from tests.test_gpu_qs import h16, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def make(torch, rng, B, H, fill, groups, pending=None, half=None):
    c = qs.Cache(B, H, 4)
    st = np.zeros((B, 8), np.int32)
    st[:, 0], st[:, 1], st[:, 2] = groups, fill, 0 if pending is None else pending
    st[:, 3] = np.arange(B) % 2 if half is None else half
    c.state.copy_(torch.from_numpy(st))
    for t in (c.buf_k, c.buf_v):
        t.copy_(torch.from_numpy(h16(rng, t.shape)))
    return c, st


def close(got, want, x, what=""):
    """got: fp16 results, want: fp64, x: the rows before."""
    pair = np.abs(x.astype(np.float64)).max(-1, keepdims=True) * 2
    err = np.abs(got.astype(np.float64) - want)
    assert np.all(err <= 2.0 ** -11 * np.abs(want) + 2.0 ** -20 * pair + 2.0 ** -25), (what, err.max())


def strided(torch, a, kind):
    """The rows a [B, h, n, D] on the device, laid out as a user may hold them."""
    B, h, n, D = a.shape
    if kind == "plain":
        return to_dev(torch, a)
    if kind == "tokens":  # heads of a token side by side, among others
        t = torch.full((B, n, h + 3, D), float("nan"), dtype=torch.float16, device="cuda")
        v = t[:, :, 2:2 + h].transpose(1, 2)
    elif kind == "padded":  # rows of 136 elements
        v = torch.full((B, h, n, D + 8), float("nan"), dtype=torch.float16, device="cuda")[..., :D]
    else:  # tokens of all sequences one after the other, the heads outermost
        v = torch.full((h, n, B, D), float("nan"), dtype=torch.float16, device="cuda").permute(2, 0, 1, 3)
    v.copy_(torch.from_numpy(a))
    return v


@pytest.mark.parametrize("rot", [16, 48, 64, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,kind", [(1, "tokens"), (3, "padded"), (5, "outer"), (64, "tokens"), (97, "plain")])
def test_append(torch, rot, interleaved, n, kind):
    rng = np.random.default_rng([rot, interleaved, n])
    B, H, group = 3, 2, 3
    fill = np.array([0, 256 - n, 100])
    c, st = make(torch, rng, B, H, fill, [0, 17, 1000])
    bk, bv = c.buf_k.cpu().numpy(), c.buf_v.cpu().numpy()
    k, v, q = h16(rng, (B, H, n, 128), 3), h16(rng, (B, H, n, 128)), h16(rng, (B, H * group, n, 128))
    freq = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    tree = n == 64
    off = trees.depths(trees.random_parents(rng, B, n)) if tree else np.tile(np.arange(n), (B, 1))
    q_out = torch.full((B, H * group, n, 128), float("nan"), dtype=torch.float16, device="cuda")
    kw = dict(offset=to_dev(torch, off.astype(np.int32))) if tree else {}
    qs.qs_buffer_append_rotary(c, strided(torch, k, kind), strided(torch, v, kind), to_dev(torch, freq),
                               q=strided(torch, q, kind), q_out=q_out, interleaved=interleaved, **kw)
    pos = st[:, :1] * 128 + fill[:, None] + off
    close(q_out.cpu().numpy(), trees.rotate(q, pos[:, None], freq, interleaved), q, "q")
    want = trees.rotate(k, pos[:, None], freq, interleaved)
    gk, gv = c.buf_k.cpu().numpy(), c.buf_v.cpu().numpy()
    for b in range(B):
        at = (st[b, 3] * 128 + fill[b] + np.arange(n)) % 256
        close(gk[b][:, at], want[b], k[b], "k")
        assert np.array_equal(gv[b][:, at], v[b])
        rest = np.setdiff1d(np.arange(256), at)
        assert np.array_equal(gk[b][:, rest], bk[b][:, rest]) and np.array_equal(gv[b][:, rest], bv[b][:, rest])
    st[:, 1:3] += n
    assert np.array_equal(c.state.cpu().numpy(), st)


def test_far_positions_and_frequencies(torch):
    """Positions up to 2^31, offsets below 0, frequencies of more than a turn, and
    zero: whole turns go without a trace."""
    rng = np.random.default_rng(5)
    groups = np.array([0, 1000, 100_000, 16_700_000])
    c, st = make(torch, rng, 4, 1, [5, 6, 7, 8], groups, pending=[0, 6, 3, 0])
    k = h16(rng, (4, 1, 2, 128))
    freq = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    freq[:4] = [7.5, 100.25, -0.3, 0.0]
    off = np.array([[-3, 0], [0, -128000], [2, 5], [70000, 77775]], np.int32)
    qs.qs_buffer_append_rotary(c, to_dev(torch, k), to_dev(torch, k), to_dev(torch, freq), offset=to_dev(torch, off))
    pos = (groups * 128 + st[:, 1] - st[:, 2])[:, None] + off
    assert pos.max() < 2 ** 31
    want = trees.rotate(k, pos[:, None], freq, False)
    for b in range(4):
        at = (st[b, 3] * 128 + st[b, 1] + np.arange(2)) % 256
        close(c.buf_k[b].cpu().numpy()[:, at], want[b], k[b], "sequence %d" % b)


def test_append_without_room_and_in_place(torch):
    rng = np.random.default_rng(6)
    c, st = make(torch, rng, 2, 3, [250, 249], [3, 3])
    bk = c.buf_k.clone()
    k, q = h16(rng, (2, 3, 7, 128)), h16(rng, (2, 6, 7, 128))
    freq = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    qd = to_dev(torch, q)
    qs.qs_buffer_append_rotary(c, to_dev(torch, k), to_dev(torch, k), to_dev(torch, freq), q=qd, q_out=qd)
    assert list(qs.qs_get_errors(c)) == [qs.DEV_OVERFLOW, 0]
    assert torch.equal(c.buf_k[0], bk[0])
    got = c.state.cpu().numpy()
    assert list(got[:, 1]) == [250, 256] and list(got[:, 2]) == [0, 7] and not got[:, 5].any()
    pos = 3 * 128 + np.array([[250], [249]]) + np.arange(7)
    close(qd.cpu().numpy(), trees.rotate(q, pos[:, None], freq, False), q)


def test_keys_alone_and_one_head_for_all(torch):
    """Without queries; and one row given to all heads (stride 0)."""
    rng = np.random.default_rng(7)
    c, st = make(torch, rng, 1, 4, [10], [1])
    k = h16(rng, (1, 1, 5, 128))
    freq = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    kd = to_dev(torch, k).expand(1, 4, 5, 128)
    qs.qs_buffer_append_rotary(c, kd, kd, to_dev(torch, freq), interleaved=True)
    want = trees.rotate(k, (138 + np.arange(5))[None, None], freq, True)
    at = (st[0, 3] * 128 + 10 + np.arange(5)) % 256
    for h in range(4):
        close(c.buf_k[0, h].cpu().numpy()[at], want[0, 0], k[0, 0])


def test_it_is_the_plain_append_at_angle_zero(torch):
    """With frequencies of zero the same bits as qs_buffer_append, subnormals,
    infinities and signed zeros of the values among them."""
    rng = np.random.default_rng(8)
    a, _ = make(torch, rng, 2, 2, [100, 200], [1, 2])
    b = qs.Cache(2, 2, 4)
    for x in ("buf_k", "buf_v", "state"):
        getattr(b, x).copy_(getattr(a, x))
    k, v = h16(rng, (2, 2, 40, 128)), h16(rng, (2, 2, 40, 128))
    v[0, 0, 0, :6] = [np.inf, -np.inf, np.nan, -0.0, 6e-8, -6e-8]
    kd, vd = to_dev(torch, k), to_dev(torch, v)
    qs.qs_buffer_append_rotary(a, kd, vd, torch.zeros(64, device="cuda"))
    qs.qs_buffer_append(b, kd, vd)
    for x in ("buf_k", "buf_v", "state"):
        g, w = getattr(a, x), getattr(b, x)
        assert torch.equal(g.view(torch.int16) if g.dtype == torch.float16 else g,
                           w.view(torch.int16) if w.dtype == torch.float16 else w)


# ---------------------------------------------------------------- acceptance

def tokens_for(rng, parent, n, p_hit):
    """Draft and target tokens of which many agree, siblings with the same token
    and negative drafts among them."""
    draft = rng.integers(0, 6, n).astype(np.int32)
    draft[rng.random(n) < 0.1] = -1
    target = rng.integers(0, 6, n).astype(np.int32)
    for j in range(n):
        kids = np.flatnonzero(parent == j)
        if len(kids) and rng.random() < p_hit:
            target[j] = draft[rng.choice(kids)]
    return draft, target


@pytest.mark.parametrize("n", [1, 2, 7, 31, 32, 33, 64])
@pytest.mark.parametrize("extra", [0, 9])
def test_accept(torch, n, extra):
    rng = np.random.default_rng([n, extra])
    B, H = 12, 3
    fill = rng.integers(n + extra, 257, B)
    c, st = make(torch, rng, B, H, fill, rng.integers(0, 4, B), pending=n + extra)
    bk, bv = c.buf_k.cpu().numpy(), c.buf_v.cpu().numpy()
    parent = trees.random_parents(rng, B, n, reach=[1, 3, 20][n % 3], roots=0.05)
    parent[1] = np.arange(-1, n - 1)  # a chain, all of it accepted
    dt = [tokens_for(rng, parent[b], n, 0.9) for b in range(B)]
    draft, target = np.stack([d for d, _ in dt]), np.stack([t for _, t in dt])
    draft[1] = np.arange(n)
    target[1] = np.arange(1, n + 1)
    out = [torch.full((B, n) if i else (B,), -77, dtype=torch.int32, device="cuda") for i in range(3)]
    qs.qs_tree_accept(c, to_dev(torch, parent), to_dev(torch, draft), to_dev(torch, target), out[0], out[1], out[2])
    keep, path, emitted = (x.cpu().numpy() for x in out)
    gk, gv, gs = c.buf_k.cpu().numpy(), c.buf_v.cpu().numpy(), c.state.cpu().numpy()
    assert not gs[:, 4:].any()
    for b in range(B):
        want = trees.accept(parent[b], draft[b], target[b])
        m = len(want)
        assert keep[b] == m and list(path[b]) == want + [-1] * (n - m)
        assert list(emitted[b]) == [target[b, j] for j in want] + [-1] * (n - m)
        src = np.arange(256)
        first = st[b, 3] * 128 + fill[b] - n
        src[(first + np.arange(m)) % 256] = (first + np.array(want)) % 256
        assert np.array_equal(gk[b], bk[b][:, src]) and np.array_equal(gv[b], bv[b][:, src])
        assert list(gs[b, :4]) == [st[b, 0], fill[b] - n + m, 0, st[b, 3]]
    assert keep[1] == n


def test_accept_refuses_what_is_no_tree(torch):
    """Fewer pending tokens than nodes, a parent out of range, a first node that
    has one: flagged, and nothing of the sequence changes."""
    rng = np.random.default_rng(2)
    B, n = 5, 6
    c, st = make(torch, rng, B, 2, [50] * B, [0] * B, pending=[6, 5, 6, 6, 6])
    bk = c.buf_k.clone()
    parent = np.tile(np.arange(-1, n - 1, dtype=np.int32), (B, 1))
    parent[2, 4], parent[3, 2], parent[4, 0] = 4, -2, 1
    same = to_dev(torch, np.ones((B, n), np.int32))
    out = [torch.full((B, n) if i else (B,), -77, dtype=torch.int32, device="cuda") for i in range(3)]
    qs.qs_tree_accept(c, to_dev(torch, parent), same, same, *out)
    assert list(qs.qs_get_errors(c)) == [0] + [qs.DEV_TREE] * 4
    assert out[0].tolist() == [6, 0, 0, 0, 0]
    assert (out[1][1:] == -1).all() and (out[2][1:] == -1).all()
    got = c.state.cpu().numpy()
    assert np.array_equal(got[1:], st[1:]) and list(got[0, 1:3]) == [50, 0]
    assert torch.equal(c.buf_k[1:], bk[1:])


def test_captured_round_of_append_and_accept(torch):
    """Captured, a round works on the counters it finds: three replays in a row."""
    rng = np.random.default_rng(3)
    B, H, n = 2, 2, 9
    c, st = make(torch, rng, B, H, [30, 100], [1, 1])
    parent = trees.random_parents(rng, B, n)
    dt = [tokens_for(rng, parent[b], n, 1.0) for b in range(B)]
    draft, target = np.stack([d for d, _ in dt]), np.stack([t for _, t in dt])
    k = to_dev(torch, h16(rng, (B, H, n, 128)))
    freq, off = torch.full((64,), 0.01, device="cuda"), to_dev(torch, trees.depths(parent))
    a = [to_dev(torch, x) for x in (parent, draft, target)]
    out = [torch.zeros((B, n) if i else (B,), dtype=torch.int32, device="cuda") for i in range(3)]

    def round_():
        qs.qs_buffer_append_rotary(c, k, k, freq, offset=off)
        qs.qs_tree_accept(c, *a, *out)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        round_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        round_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    m = np.array([len(trees.accept(parent[b], draft[b], target[b])) for b in range(B)])
    assert np.array_equal(c.state.cpu().numpy()[:, 1], [30, 100] + 4 * m)
    assert not c.state[:, 2].any() and not c.state[:, 4:].any()
