"""Test-side model of a round over a tree of drafted tokens, in 64 bits."""
import numpy as np

from tests import paging


def random_parents(rng, B, n, reach=9, roots=0.0):
    """int32 [B, n]: node 0 the root, the others below one of the `reach` nodes
    before them, or (with probability `roots`) nobody's child."""
    parent = np.full((B, n), -1, np.int32)
    for b in range(B):
        for j in range(1, n):
            if rng.random() >= roots:
                parent[b, j] = rng.integers(max(0, j - reach), j)
    return parent


def ancestors(parent):
    """bool [n, n] of one tree: node i sees node j.  A parent that is not an
    earlier node counts as -1."""
    n = len(parent)
    sees = np.zeros((n, n), bool)
    for j, up in enumerate(parent):
        if 0 <= up < j:
            sees[j] = sees[up]
        sees[j, j] = True
    return sees


def depths(parent):
    return np.stack([ancestors(p).sum(1) - 1 for p in parent]).astype(np.int32)


def attention(oc, q, parent, upper_only, group=1, upper_bits=4, left_out=()):
    """Softmax attention of the last n_q nodes: (out, lse), zeros and -inf where
    n_tree > fill.  left_out: (b, g) groups that take no part."""
    B, Hq, n_q, D = q.shape
    n = parent.shape[1]
    scale = float(np.float32(1.0 / np.sqrt(D)))
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    for b in range(B):
        ng, fill = oc.counters(b)["n_groups"], oc.counters(b)["fill"]
        if n > fill:
            continue
        k, v = paging.dequantized(oc, b, upper_only, upper_bits)
        seen = np.ones((n_q, ng * oc.G + fill), bool)
        seen[:, ng * oc.G + fill - n:] = ancestors(parent[b])[n - n_q:]
        for bb, g in left_out:
            if bb == b:
                seen[:, g * oc.G:(g + 1) * oc.G] = False
        for i in range(Hq):
            kk, vv = k[i // group], v[i // group]
            with np.errstate(invalid="ignore"):
                s = np.where(seen, scale * (q[b, i].astype(np.float64) @ kk.T), -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            for j in range(n_q):  # (tokens that are not seen may hold anything)
                out[b, i, j] = p[j][seen[j]] @ vv[seen[j]] / p[j].sum()
            lse[b, i] = m[:, 0] + np.log(p.sum(1))
    return out, lse


def rotate(x, pos, freq, interleaved):
    """fp64 rows x [..., D] at positions pos (broadcast against x[..., 0])."""
    y = x.astype(np.float64).copy()
    m = len(freq)
    i = np.arange(m)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + m)
    # (the product of an int32 and a float32 has 55 bits)
    ang = np.asarray(pos, np.longdouble)[..., None] * np.asarray(freq, np.longdouble)
    c, s = np.cos(ang).astype(np.float64), np.sin(ang).astype(np.float64)
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


def accept(parent, draft, target):
    """The path of one tree."""
    path = [0]
    while True:
        nxt = [j for j in range(path[-1] + 1, len(parent))
               if parent[j] == path[-1] and draft[j] >= 0 and draft[j] == target[path[-1]]]
        if not nxt:
            return path
        path.append(nxt[0])


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, fp64 probabilities) of one row of logits."""
    x = np.asarray(x, np.float64) + 0.0
    V = len(x)
    probs = np.zeros(V)
    ok = np.flatnonzero(x > -np.inf)
    if not len(ok):
        return -1, probs
    m = x[ok].max()
    if m == np.inf:
        ok = ok[x[ok] == m]
    by = ok[np.argsort(-x[ok], kind="stable")]
    T = float(np.float32(temperature))
    if not T >= 2.0 ** -60:
        by, w = by[:1], np.ones(1)
    else:
        w = np.ones(len(by)) if m == np.inf else np.exp((x[by] - m) / T)
        if 0 < top_k < V:
            by, w = by[:top_k], w[:top_k]
        p = float(np.float32(top_p))
        if p < 1:
            mass = np.cumsum(w)
            n = 1 + int(np.searchsorted(mass, max(p, 0.0) * mass[-1], side="left"))
            by, w = by[:n], w[:n]
        mp = min(float(np.float32(min_p)), 1.0)
        if mp > 0 and m < np.inf:
            # w >= min_p, asked of the logits: exp(-2^-130) is less than 1, but a
            # double of 53 bits rounds it to 1
            kept = x[by] - m >= T * np.log(mp)
            by, w = by[kept], w[kept]
    at = np.argsort(by)
    by, w = by[at], w[at]
    probs[by] = w / w.sum()
    cum = np.cumsum(w)
    u = float(np.float32(u))
    if u >= 1:
        i = np.flatnonzero(w > 0)[-1]
    else:
        i = int(np.searchsorted(cum, (u if u > 0 else 0.0) * cum[-1], side="right"))
    return int(by[min(i, len(by) - 1)]), probs
