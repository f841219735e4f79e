"""Test-side model of a paged cache: an oracle cache's groups scattered over a
pool of pages, and gathered back, in the layout include/qs.h gives."""
import numpy as np

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import layout

GROUP_ARRAYS = ("k_upper", "k_lower", "v_upper", "v_lower", "meta")


def random_table(rng, n_groups, cap, n_pages):
    """int32 [B, cap]: distinct pages for each sequence's first n_groups[b]
    groups in random order, the unused entries out of range on both sides."""
    B = len(n_groups)
    table = np.where(rng.random((B, cap)) < 0.5, -7, n_pages + 1000).astype(np.int32)
    pages = rng.permutation(n_pages)
    at = 0
    for b, n in enumerate(n_groups):
        table[b, :n] = pages[at:at + n]
        at += n
    return table


def paged_copy(torch, oc, rng, upper_bits=4, spare=3, n_pages=None):
    """A qs.PagedCache with the oracle cache's content in randomly chosen
    pages; the rest of the pool holds 0xA5 bytes."""
    n = [oc.counters(b)["n_groups"] for b in range(oc.B)]
    n_pages = n_pages or max(1, sum(n) + spare)
    cache = qs.PagedCache(oc.B, oc.H, oc.cap, n_pages, upper_bits=upper_bits)
    table = random_table(rng, n, oc.cap, n_pages)
    cache.table.copy_(torch.from_numpy(table))
    arrs = layout.device_arrays(oc, upper_bits)
    for name in GROUP_ARRAYS:
        a = arrs[name]
        pool = np.full((n_pages,) + a.shape[1:2] + a.shape[3:], 0xA5, a.dtype)
        if a.dtype == np.uint16:
            pool[:] = 0x7E00  # NaN scales and zeros in pages nobody owns
        for b in range(oc.B):
            for g in range(n[b]):
                pool[table[b, g]] = a[b, :, g]
        put(torch, getattr(cache, name), pool)
    for name in ("buf_k", "buf_v", "state"):
        put(torch, getattr(cache, name), arrs[name])
    return cache


def put(torch, t, a):
    src = torch.from_numpy(np.ascontiguousarray(a.view(np.int16) if a.dtype == np.uint16 else a))
    if t.dtype == torch.float16:
        src = src.view(torch.float16)
    t.copy_(src.reshape(t.shape))


def assert_groups_equal(cache, oc, what=""):
    """The pages the table names hold the oracle's groups bit for bit, the
    buffers and counters (but the error words) are the oracle's."""
    got = layout.read_device(cache)
    want = layout.device_arrays(oc, cache.upper_bits)
    table = cache.table.cpu().numpy()
    for b in range(oc.B):
        n = oc.counters(b)["n_groups"]
        for name in GROUP_ARRAYS:
            assert np.array_equal(got[name][table[b, :n]].swapaxes(0, 1), want[name][b, :, :n]), \
                "%s: %s of sequence %d differs" % (what, name, b)
    for name in ("buf_k", "buf_v"):
        assert np.array_equal(got[name].reshape(want[name].shape), want[name]), (what, name)
    g, w = got["state"].copy(), want["state"].copy()
    g[:, oracle.ERR] = w[:, oracle.ERR] = 0
    assert np.array_equal(g, w), what


def dequantized(oc, b, upper_only, upper_bits=4):
    """fp64 keys and values [H, n_groups * G + fill, D] of sequence b as one
    pass sees them, from the oracle's codes, scales and zeros."""
    n = oc.counters(b)["n_groups"]
    f = lambda x: x.view(np.float16).astype(np.float64)
    step = 1 << (8 - upper_bits)

    def value(code):
        code = code.astype(np.float64)
        return np.floor(code / step) * step + step / 2 if upper_only else code

    k = value(oc.kq[b, :, :n]) * f(oc.ks[b, :, :n])[:, :, None, :] + f(oc.kz[b, :, :n])[:, :, None, :]
    v = value(oc.vq[b, :, :n]) * f(oc.vs[b, :, :n])[:, :, :, None] + f(oc.vz[b, :, :n])[:, :, :, None]
    flat = lambda x: x.reshape(oc.H, n * oc.G, oc.D)
    buf = [oc.buffer_tokens(b, h) for h in range(oc.H)]
    return (np.concatenate([flat(k), f(np.stack([x[0] for x in buf]))], 1),
            np.concatenate([flat(v), f(np.stack([x[1] for x in buf]))], 1))


def counts(oc, b, sel=None):
    """How often each group of sequence b takes part, [H, n_groups]: once, or
    as often as the first min(k, n_groups) entries of the head's row name it."""
    n = oc.counters(b)["n_groups"]
    if sel is None:
        return np.ones((oc.H, n))
    c = np.zeros((oc.H, n))
    for h in range(oc.H):
        for g in sel[b, h, :min(sel.shape[2], n)]:
            if 0 <= g < n:
                c[h, g] += 1
    return c


def attention(oc, q, upper_only, group=1, upper_bits=4, sel=None, times=None, scale=None):
    """Textbook softmax attention in fp64 over the dequantized tokens, each
    weighted by how often its group takes part (counts, or times [B][H, n]),
    and the causal part of the buffer: (out, lse), zeros and -inf where
    n_q > fill."""
    B, Hq, n_q, D = q.shape
    scale = float(np.float32(1.0 / np.sqrt(D) if scale is None else scale))
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    for b in range(B):
        n, fill = oc.counters(b)["n_groups"], oc.counters(b)["fill"]
        if n_q > fill:
            continue
        k, v = dequantized(oc, b, upper_only, upper_bits)
        c = counts(oc, b, sel) if times is None else times[b]
        for i in range(Hq):
            h = i // group
            w = np.concatenate([np.repeat(c[h], oc.G), np.ones(fill)])
            with np.errstate(divide="ignore"):
                logw = np.log(w)
            for j in range(n_q):
                s = scale * (k[h] @ q[b, i, j].astype(np.float64)) + logw
                s[n * oc.G + fill - n_q + j + 1:] = -np.inf
                m = s.max()
                p = np.exp(s - m)
                out[b, i, j] = (p @ v[h]) / p.sum()
                lse[b, i, j] = m + np.log(p.sum())
    return out, lse


def select(oc, q, k, group=1, left_out=()):
    """The k groups of each KV head with the largest box scores, by definition:
    every channel's larger product, summed in fp64 (the sums of these fp16
    products are exact or nearly so), the largest over the head's query rows;
    ties to the lower index, ascending, -1 behind.  left_out: (b, g) pairs
    that score below all others."""
    f = lambda x: x.view(np.float16).astype(np.float64)
    n_q = q.shape[2]
    sel = np.full((oc.B, oc.H, k), -1, np.int32)
    for b in range(oc.B):
        n = oc.counters(b)["n_groups"]
        for h in range(oc.H):
            lo = f(oc.kz[b, h, :n])
            hi = lo + 255 * f(oc.ks[b, h, :n])
            rows = q[b, h * group:(h + 1) * group].reshape(group * n_q, -1).astype(np.float64)
            score = np.full(n, -np.inf)
            for row in rows:
                score = np.maximum(score, np.maximum(row * lo, row * hi).sum(-1))
            if n > k:
                score[[g for bb, g in left_out if bb == b]] = -np.inf
            best = np.sort(np.lexsort((np.arange(n), -score))[:k])
            sel[b, h, :len(best)] = best
    return sel
