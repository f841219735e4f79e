"""Cases that measure the operators of a speculative round over a tree of drafted
tokens: the append with position rotation, the attention of the tree's nodes
over the hierarchical quantized cache, the sampling of a token for each row of
logits, and the acceptance of a path of the tree.

``own`` false computes each operator in elementary torch operations from the
bytes the cache stores (the layout of include/qs.h); ``own`` true calls the
library.  Sizes: head_dim 128 and groups of 128 tokens throughout (the only
ones the cache has), trees of up to 64 nodes, contexts from 1k to 128k tokens,
2 to 32 KV heads, up to eight query heads per KV head, vocabularies from 1k to
256k tokens.
"""
import math

import numpy as np
import torch

own = False

D = G = 128
RING = 2 * G
DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a single grouped-query sequence, heads sliced out of the fused
        # projection: latency counts
        dict(name="append_token", op="append", B=1, H=8, group=4, n=1, rot=128, pairs="halves",
             tree=False, fused=True),
        # a tree of 64 nodes for each of eight sequences
        dict(name="append_tree", op="append", B=8, H=8, group=4, n=64, rot=128, pairs="halves",
             tree=True, fused=True),
        # a whole buffer of tokens for sixteen sequences, half of the channels rotated, in
        # neighbouring pairs
        dict(name="append_long", op="append", B=16, H=32, group=1, n=256, rot=64, pairs="neighbours",
             tree=False, fused=False),
        # the smallest tree: seven nodes, two heads, 1k tokens
        dict(name="tree_small", op="tree", B=1, H=2, group=1, n_tree=7, n_q=7, groups=6, fill=256,
             ragged=False, paged=False, bits=4, mode="verify"),
        # drafting the last level of a 21-node tree over a 32k context
        dict(name="tree_draft_level", op="tree", B=1, H=32, group=1, n_tree=21, n_q=8, groups=254,
             fill=200, ragged=False, paged=False, bits=4, mode="draft"),
        # verifying a 60-node tree of a grouped-query 32k sequence: 240 rows a KV head
        dict(name="tree_verify_gqa_32k", op="tree", B=1, H=8, group=4, n_tree=60, n_q=60, groups=254,
             fill=256, ragged=False, paged=False, bits=4, mode="verify"),
        # verifying 26-node trees of eight ragged sequences up to 64k tokens, in pages
        dict(name="tree_verify_ragged", op="tree", B=8, H=32, group=1, n_tree=26, n_q=26, groups=510,
             fill=133, ragged=True, paged=True, bits=4, mode="verify"),
        # the next token of one sequence under the usual mixture of filters: latency counts
        dict(name="sample_row", op="sample", rows=1, V=32000, dtype="fp16", temperature=0.8, top_k=50,
             top_p=0.95, min_p=0.02, mixed=False, probs=False),
        # a token and the filtered probabilities for every node of a tree
        dict(name="sample_nodes", op="sample", rows=60, V=128000, dtype="bf16", temperature=1.0, top_k=0,
             top_p=0.9, min_p=0.0, mixed=False, probs=True),
        # a serving batch whose requests bring settings of their own, an odd vocabulary
        dict(name="sample_batch", op="sample", rows=257, V=65537, dtype="fp32", temperature=0.9, top_k=100,
             top_p=0.9, min_p=0.05, mixed=True, probs=False),
        # a 16-node tree of one sequence: latency counts
        dict(name="accept_one", op="accept", B=1, H=8, n=16, depth=5),
        # 64-node trees of sixteen sequences, long paths
        dict(name="accept_batch", op="accept", B=16, H=32, n=64, depth=20),
    ]


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = (max(most.get(c["op"], (0, 0))[0], w["bytes"]),
                         max(most.get(c["op"], (0, 0))[1], w["flops"]))

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["append", "tree", "tree", "sample", "sample", "accept"])
        c = dict(op=op)
        if op != "sample":
            c.update(B=log_int(1, 16), H=rng.choice([2, 4, 5, 8, 16, 32]))
        if op in ("append", "tree"):
            c["group"] = rng.choice([1, 2, 3, 4, 8])
        if op == "append":
            c.update(n=log_int(1, 256), rot=rng.choice([128, 128, 96, 64, 32]),
                     pairs=rng.choice(["halves", "neighbours"]), fused=rng.random() < 0.5)
            c["tree"] = c["n"] <= 64 and rng.random() < 0.5
        if op == "tree":
            c.update(n_tree=log_int(2, 64), groups=log_int(4, 1022), ragged=rng.random() < 0.5,
                     paged=rng.random() < 0.5, bits=rng.choice([4, 4, 2]),
                     mode=rng.choice(["draft", "verify"]))
            c["n_q"] = c["n_tree"] if c["mode"] == "verify" else rng.randint(1, c["n_tree"])
            c["fill"] = rng.randint(c["n_tree"], RING)
        if op == "sample":
            c.update(rows=log_int(1, 257), V=log_int(1000, 256000), dtype=rng.choice(list(DTYPES)),
                     temperature=rng.choice([0.0, 0.7, 1.0, 1.3]), top_k=rng.choice([0, 1, 20, 64, 1000]),
                     top_p=rng.choice([1.0, 0.95, 0.9, 0.5]), min_p=rng.choice([0.0, 0.05]),
                     mixed=rng.random() < 0.3, probs=rng.random() < 0.5)
        if op == "accept":
            c.update(n=log_int(2, 64))
            c["depth"] = rng.randint(1, c["n"])
        w = work(c)
        if 2e4 < w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def lengths(n, B, ragged):
    """Per-sequence values up to n, fixed by the case alone: spread from about
    n / 8 to n where ragged."""
    if not ragged:
        return [n] * B
    return [max(1, n - (n * 7 * ((5 * b) % B)) // (8 * max(1, B - 1)) if B > 1 else n) for b in range(B)]


def group_bytes(mode, bits):
    """Plane and scale bytes of a group and head that an attention in this mode
    needs."""
    if mode == "verify":
        return 4 * 8192 + 1024
    return (8192 if bits == 2 else 16384) + 1024


def work(case):
    c = case
    if c["op"] == "append":
        rows = c["B"] * c["n"] * c["H"]
        return {"bytes": rows * (2 + c["group"]) * 512, "flops": rows * (1 + c["group"]) * 3 * c["rot"]}
    if c["op"] == "accept":
        rows = c["B"] * c["H"]
        return {"bytes": rows * (c["n"] + c["depth"]) * 2 * 512, "flops": 0}
    if c["op"] == "sample":
        n = c["rows"] * c["V"]
        return {"bytes": n * ((4 if c["dtype"] == "fp32" else 2) + (4 if c["probs"] else 0)), "flops": 2 * n}
    ng = lengths(c["groups"], c["B"], c["ragged"])
    R, H = c["group"] * c["n_q"], c["H"]
    tok = sum(ng) * G + c["B"] * c["fill"]
    return {"bytes": H * (sum(ng) * group_bytes(c["mode"], c["bits"]) + c["B"] * c["fill"] * 512)
            + c["B"] * H * R * (512 + 4), "flops": 4 * 128 * R * H * tok}


# --------------------------------------------------------- stored layout

def v_token_of(p):
    """Token of a 32-token quarter in nibble position p of a value row."""
    return 16 * ((p >> 1) & 1) + 8 * (p & 1) + 2 * (p >> 3) + ((p >> 2) & 1)


def k_channel_of(p):
    """Channel in position p of a key scale / zero row."""
    return 32 * ((p >> 3) & 3) + 8 * (p >> 5) + 2 * ((p >> 2) & 1) + ((p >> 1) & 1) + 4 * (p & 1)


def v_row_token_of(p):
    """Token in position p of a value scale / zero row."""
    return 32 * (p >> 5) + ((p >> 2) & 7) + 16 * ((p >> 1) & 1) + 8 * (p & 1)


V_TOKEN = v_token_of(torch.arange(32, device=DEV))
K_CHANNEL = k_channel_of(torch.arange(128, device=DEV))
V_ROW_TOKEN = v_row_token_of(torch.arange(128, device=DEV))
V_TOKEN_AT, K_CHANNEL_AT, V_ROW_TOKEN_AT = V_TOKEN.argsort(), K_CHANNEL.argsort(), V_ROW_TOKEN.argsort()


def quantize(x, dim):
    """Asymmetric 8-bit groups along dim: codes, fp16 scale, fp16 zero."""
    x = x.float()
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s = (((hi - lo) / 255.0).half().view(torch.int16) + 1).view(torch.float16)  # the next larger fp16
    q = ((x - lo) / s.float()).round().clamp(0, 255)
    return q.to(torch.uint8), s, lo.half()


def pack_pairs(n):
    return n[..., 0::2] | (n[..., 1::2] << 4)


def two_bit(plane):
    """A nibble plane's groups in the two-bit draft layout."""
    w = plane.reshape(-1, 1024, 2, 4)
    a, b = w[:, :, 0], w[:, :, 1]
    u = ((a >> 2) & 0x33) | (b & 0xCC)
    m = (a & 0x33) | ((b & 0x33) << 2)
    return torch.cat([u.reshape(-1, 4096), m.reshape(-1, 4096)], 1).reshape(plane.shape)


def stored(k, v, bits):
    """Planes and scale rows of groups k, v: fp16 [..., G tokens, D]."""
    kq, ks, kz = quantize(k, -2)
    vq, vs, vz = quantize(v, -1)
    tok = V_TOKEN + 32 * torch.arange(4, device=DEV)[:, None]
    vq = vq[..., tok, :].transpose(-1, -2)
    kp, vp = K_CHANNEL, V_ROW_TOKEN
    st = dict(k_upper=pack_pairs(kq >> 4), k_lower=pack_pairs(kq & 15), v_upper=pack_pairs(vq >> 4),
              v_lower=pack_pairs(vq & 15),
              meta=torch.stack([ks[..., 0, :][..., kp], kz[..., 0, :][..., kp], vs[..., 0][..., vp],
                                vz[..., 0][..., vp]], -2))
    if bits == 2:
        st["k_upper"], st["v_upper"] = two_bit(st["k_upper"]), two_bit(st["v_upper"])
    return {n: t.contiguous() for n, t in st.items()}


# ------------------------------------------------------------------ inputs

PLANES = ("k_upper", "k_lower", "v_upper", "v_lower", "meta")


def tokens(gen, shape):
    """Keys and values as a model leaves them: unit variance, a few key
    channels of each head eight times as large."""
    k = torch.randn(shape, generator=gen, device=DEV)
    v = torch.randn(shape, generator=gen, device=DEV)
    big = torch.rand((1, shape[1]) + (1,) * (len(shape) - 3) + (D,), generator=gen, device=DEV) < 0.025
    return torch.where(big, 8 * k, k).half(), v.half()


def random_trees(gen, B, n):
    """int32 [B, n] parents: node 0 the root, the others below a recent node."""
    j = torch.arange(n, device=DEV)
    back = (torch.rand((B, n), generator=gen, device=DEV) * torch.clamp(j, max=9)).long()
    return torch.where(j > 0, j - 1 - back, -1).to(torch.int32)


def depths(parent):
    """int32 [B, n]: the number of ancestors of each node."""
    d = torch.zeros_like(parent)
    for j in range(1, parent.shape[1]):
        d[:, j] = d.gather(1, parent[:, j:j + 1].long())[:, 0] + 1
    return d


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=c)
    if c["op"] == "sample":
        rows, V = c["rows"], c["V"]
        x = 2.5 * torch.randn((rows, V), generator=gen, device=DEV)
        at = torch.randint(V, (rows, 20), generator=gen, device=DEV)
        x.scatter_add_(1, at, 4 + 8 * torch.rand((rows, 20), generator=gen, device=DEV))
        st["logits"] = x.to(DTYPES[c["dtype"]])
        st["u"] = torch.rand(rows, generator=gen, device=DEV)

        def setting(name, dtype, off):
            t = torch.full((rows,), c[name], dtype=dtype, device=DEV)
            if c["mixed"]:  # some requests do without
                t[torch.rand(rows, generator=gen, device=DEV) < 0.4] = off
            return t

        st["temperature"] = setting("temperature", torch.float32, 0)
        st["top_k"] = setting("top_k", torch.int32, 0)
        st["top_p"] = setting("top_p", torch.float32, 1)
        st["min_p"] = setting("min_p", torch.float32, 0)
        st["token"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        st["probs"] = torch.empty((rows, V), device=DEV) if c["probs"] else None
        return st
    B, H = c["B"], c["H"]
    cap, ng, fill, bits = c.get("groups", 16), None, c.get("fill", 0), c.get("bits", 4)
    state = torch.zeros((B, 8), dtype=torch.int32, device=DEV)
    if c["op"] == "tree":
        ng = torch.tensor(lengths(cap, B, c["ragged"]), dtype=torch.int32, device=DEV)
        if c["paged"]:
            pages = int(ng.sum()) + 5
            perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
            at = torch.arange(cap, device=DEV)
            first = torch.cumsum(ng, 0) - ng
            live = at < ng[:, None]
            st["table"] = torch.where(live, perm[torch.where(live, first[:, None] + at, 0)], -1).to(torch.int32)
            k, v = tokens(gen, (pages, H, G, D))
        else:
            k, v = tokens(gen, (B, H, cap, G, D))
        st.update(stored(k, v, bits))
        del k, v
        state[:, 0], state[:, 2] = ng, c["n_tree"]
        st["parent"] = random_trees(gen, B, c["n_tree"])
        st["q"] = torch.randn((B, H * c["group"], c["n_q"], D), generator=gen, device=DEV).half()
    else:
        state[:, 0] = torch.randint(cap, (B,), generator=gen, device=DEV)
        fill = torch.randint(RING - c["n"] + 1, (B,), generator=gen, device=DEV)
    state[:, 1] = fill
    state[:, 3] = torch.arange(B, device=DEV) % 2
    st["buf_k"], st["buf_v"] = tokens(gen, (B, H, RING, D))
    st["state"] = state
    if c["op"] == "append":
        hq, n = H * c["group"], c["n"]
        if c["fused"]:  # query, key and value heads of a token side by side, as one projection leaves them
            x = torch.randn((B, n, hq + 2 * H, D), generator=gen, device=DEV).half().transpose(1, 2)
            st["q"], st["k"], st["v"] = x[:, :hq], x[:, hq:hq + H], x[:, hq + H:]
        else:
            st["q"] = torch.randn((B, hq, n, D), generator=gen, device=DEV).half()
            st["k"], st["v"] = tokens(gen, (B, H, n, D))
        half = c["rot"] // 2
        st["inv_freq"] = (500000.0 ** (-torch.arange(half, device=DEV).double() / half)).float()
        st["offset"] = depths(random_trees(gen, B, n)) if c["tree"] else None
        st["q_out"] = torch.empty((B, hq, n, D), dtype=torch.float16, device=DEV)
    if c["op"] == "accept":
        n = c["n"]
        st["k"], st["v"] = tokens(gen, (B, H, n, D))
        st["parent"] = parent = random_trees(gen, B, n)
        # tokens of a path of `depth` nodes (or to the first leaf) are the target's, the others not
        st["draft"] = torch.randint(32000, (B, n), generator=gen, device=DEV).to(torch.int32)
        st["target"] = 32000 + torch.arange(n, device=DEV, dtype=torch.int32).expand(B, n).contiguous()
        at = torch.zeros((B,), dtype=torch.int64, device=DEV)
        row = torch.arange(B, device=DEV)
        for _ in range(c["depth"] - 1):
            child = (parent == at[:, None]) & (torch.arange(n, device=DEV) > 0)
            pick = (child * torch.rand((B, n), generator=gen, device=DEV)).argmax(1)
            ok = child.any(1)
            st["target"][row[ok], at[ok]] = st["draft"][row[ok], pick[ok]]
            at = torch.where(ok, pick, at)
        for name in ("path", "emitted"):
            st[name] = torch.empty((B, n), dtype=torch.int32, device=DEV)
        st["n_keep"] = torch.empty((B,), dtype=torch.int32, device=DEV)
    if c["op"] == "tree":
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(st["q"].shape[:3], dtype=torch.float32, device=DEV)
    if own:  # the handles a serving program keeps: the cache and its workspace
        from hierarchical_quantized_kv_gb300 import qs
        if "table" in st:
            cache = qs.PagedCache(B, H, cap, pages, upper_bits=bits)
            cache.table.copy_(st["table"])
        else:
            cache = qs.Cache(B, H, cap, upper_bits=bits)
        for n in PLANES + ("buf_k", "buf_v", "state"):
            if n in st:
                getattr(cache, n).copy_(st[n])
        st["cache"] = cache
        if c["op"] == "tree":
            size = qs.qs_attn_tree_workspace_size(cache, c["n_q"], c["group"])
            st["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------- plain forms

def unpack_pairs(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def one_nibble_plane(plane):
    """The nibble plane of groups stored in the two-bit draft layout."""
    w = plane.reshape(-1, 2, 1024, 4)
    u, m = w[:, 0], w[:, 1]
    a = ((u & 0x33) << 2) | (m & 0x33)
    b = (u & 0xCC) | ((m >> 2) & 0x33)
    return torch.stack([a, b], 2).reshape(plane.shape)


def code_values(upper, lower, mode, bits):
    """What a code stands for, in units of its scale (fp32)."""
    if mode == "verify":
        return (upper * 16 + lower).float()
    return (upper * 16 + 8).float() if bits == 4 else ((upper >> 2) * 64 + 32).float()


def dequantized(st, mode, bits):
    """fp32 keys and values of the groups, [B, H, n, G, D]."""
    B, H = st["buf_k"].shape[:2]
    g = {n: st[n] for n in PLANES}
    if "table" in st:
        page = st["table"].clamp(min=0).long()[:, None].expand(B, H, -1)
        g = {n: t[page, torch.arange(H, device=DEV)[:, None]] for n, t in g.items()}
    ku, vu = g["k_upper"], g["v_upper"]
    if bits == 2:
        ku, vu = one_nibble_plane(ku), one_nibble_plane(vu)
    kp, vp = K_CHANNEL_AT, V_ROW_TOKEN_AT
    meta = g["meta"].float()
    k = code_values(unpack_pairs(ku), unpack_pairs(g["k_lower"]), mode, bits)
    k = k * meta[..., 0, :][..., None, kp] + meta[..., 1, :][..., None, kp]
    v = code_values(unpack_pairs(vu), unpack_pairs(g["v_lower"]), mode, bits)
    v = v[..., V_TOKEN_AT].transpose(-1, -2).flatten(-3, -2)
    v = v * meta[..., 2, :][..., vp, None] + meta[..., 3, :][..., vp, None]
    return k, v


def ring_slots(st):
    """int64 [B, 2G]: the slot of each buffer token."""
    return (st["state"][:, 3:4].long() * G + torch.arange(RING, device=DEV)) % RING


def plain_tree(st):
    """Softmax attention of the tree's last n_q nodes over the groups, the
    buffer in front of the tree and each node's ancestors."""
    c = st["case"]
    B, H, n_q, n = c["B"], c["H"], c["n_q"], c["n_tree"]
    R = c["group"] * n_q
    sees = torch.zeros((B, n, n), dtype=torch.bool, device=DEV)
    for j in range(n):
        up = st["parent"][:, j].long()
        above = sees.gather(1, up.clamp(min=0)[:, None, None].expand(B, 1, n))[:, 0]
        sees[:, j] = torch.where((up >= 0)[:, None], above, False)
        sees[:, j, j] = True
    k, v = dequantized(st, c["mode"], c["bits"])
    ng = k.shape[2]
    at = ring_slots(st)[:, None, :, None].expand(B, H, RING, D)
    bk, bv = st["buf_k"].gather(2, at).float(), st["buf_v"].gather(2, at).float()
    q = st["q"].float().reshape(B, H, R, D)
    s1 = q @ k.reshape(B, H, ng * G, D).transpose(-1, -2)
    s2 = q @ bk.transpose(-1, -2)
    seen1 = torch.arange(ng * G, device=DEV) < (st["state"][:, 0].long() * G)[:, None, None, None]
    first = st["state"][:, 1].long()[:, None] - n
    i = torch.arange(RING, device=DEV)
    node = (i - first).clamp(0, n - 1)[:, None, :].expand(B, n, RING)
    seen2 = (i < first)[:, None] | ((i < first + n)[:, None] & (i >= first)[:, None] & sees.gather(2, node))
    seen2 = seen2[:, n - n_q:].repeat(1, c["group"], 1)[:, None]
    s1 = torch.where(seen1, s1 / math.sqrt(D), -math.inf)
    s2 = torch.where(seen2, s2 / math.sqrt(D), -math.inf)
    top = torch.maximum(s1.amax(-1, keepdim=True), s2.amax(-1, keepdim=True))
    p1, p2 = torch.exp(s1 - top), torch.exp(s2 - top)
    total = p1.sum(-1, keepdim=True) + p2.sum(-1, keepdim=True)
    o = (p1 @ v.reshape(B, H, ng * G, D) + p2 @ bv) / total
    shape = st["q"].shape
    return dict(out=o.half().reshape(shape), lse=(top + torch.log(total)).reshape(shape[:3]))


def rotated(x, cos, sin, rot, pairs):
    """fp16 rows x [B, h, n, D], their first rot channels turned by the angles
    [B, 1, n, rot / 2]."""
    x = x.float()
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if pairs == "halves" else (x[..., :rot:2], x[..., 1:rot:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([a, b], -1) if pairs == "halves" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).half()


def appended(st, k, v):
    """The buffers and counters with rows k, v [B, H, n, D] behind the last token."""
    B, H, n = k.shape[:3]
    at = (st["state"][:, 3:4].long() * G + st["state"][:, 1:2].long() + torch.arange(n, device=DEV)) % RING
    at = at[:, None, :, None].expand(B, H, n, D)
    state = st["state"][:, :4].clone()
    state[:, 1:3] += n
    return st["buf_k"].scatter(2, at, k), st["buf_v"].scatter(2, at, v), state


def plain_append(st):
    c = st["case"]
    pos = st["state"][:, 0].long() * G + st["state"][:, 1].long()
    step = torch.arange(c["n"], device=DEV) if st["offset"] is None else st["offset"].long()
    pos = pos[:, None] + step
    angle = pos.double()[:, None, :, None] * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    bk, bv, state = appended(st, rotated(st["k"], cos, sin, c["rot"], c["pairs"]), st["v"])
    return dict(q=rotated(st["q"], cos, sin, c["rot"], c["pairs"]), buf_k=bk, buf_v=bv, state=state)


def plain_accept(st):
    c = st["case"]
    B, H, n = c["B"], c["H"], c["n"]
    parent, draft, target = st["parent"].long(), st["draft"], st["target"]
    j = torch.arange(n, device=DEV)
    at = torch.zeros((B, 1), dtype=torch.int64, device=DEV)
    going = torch.ones((B, 1), dtype=torch.bool, device=DEV)
    path, emitted = [], []
    for _ in range(n):
        path.append(torch.where(going, at, -1))
        emitted.append(torch.where(going, target.gather(1, at), -1))
        hit = going & (parent == at) & (j > 0) & (draft >= 0) & (draft == target.gather(1, at))
        going = hit.any(1, keepdim=True)
        at = torch.where(going, torch.where(hit, j, n).amin(1, keepdim=True), at)
    path, emitted = torch.cat(path, 1), torch.cat(emitted, 1)
    n_keep = (path >= 0).sum(1)
    bk, bv, state = appended(st, st["k"], st["v"])
    first = st["state"][:, 3:4].long() * G + st["state"][:, 1:2].long()
    keep = torch.arange(n, device=DEV)
    into = ((first + keep) % RING)[:, None, :, None].expand(B, H, n, D)
    source = ((first + torch.where(path >= 0, path, keep)) % RING)[:, None, :, None].expand(B, H, n, D)
    bk, bv = bk.scatter(2, into, bk.gather(2, source)), bv.scatter(2, into, bv.gather(2, source))
    state[:, 1] = st["state"][:, 1] + n_keep
    state[:, 2] = 0
    return dict(buf_k=bk, buf_v=bv, state=state, n_keep=n_keep.to(torch.int32), path=path.to(torch.int32),
                emitted=emitted.to(torch.int32))


def plain_sample(st):
    """In fp64: which token a filter or the draw takes hangs on sums next to a
    border."""
    c = st["case"]
    V = c["V"]
    T = st["temperature"].double()[:, None]
    x, order = torch.sort(st["logits"].double(), dim=-1, descending=True, stable=True)
    greedy = T == 0
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, 1.0, T))
    rank = torch.arange(V, device=DEV)
    k = torch.where(st["top_k"] > 0, st["top_k"], V).long()[:, None]
    w = torch.where(rank < torch.where(greedy, 1, k), w, 0.0)
    before = torch.cumsum(w, -1) - w
    p = st["top_p"].double()[:, None]
    keep = (before < p * w.sum(-1, keepdim=True)) | (p >= 1) | (rank == 0)
    keep &= w >= st["min_p"].double()[:, None]
    w = torch.zeros_like(w).scatter(1, order, torch.where(keep, w, 0.0))
    total = w.sum(-1, keepdim=True)
    token = (torch.cumsum(w, -1) > st["u"].double()[:, None] * total).to(torch.uint8).argmax(-1)
    res = dict(token=token.to(torch.int32))
    if c["probs"]:
        res["probs"] = (w / total).float()
    return res


def run(state):
    st, c = state, state["case"]
    if not own:
        return dict(append=plain_append, tree=plain_tree, sample=plain_sample,
                    accept=plain_accept)[c["op"]](st)
    from hierarchical_quantized_kv_gb300 import qs
    if c["op"] == "sample":
        qs.qs_sample(st["logits"], st["u"], st["token"], probs=st["probs"], temperature=st["temperature"],
                     top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"])
        res = dict(token=st["token"])
        if c["probs"]:
            res["probs"] = st["probs"]
        return res
    cache = st["cache"]
    if c["op"] == "tree":
        mode = qs.QS_DRAFT_UPPER4 if c["mode"] == "draft" else qs.QS_VERIFY_INT8
        qs.qs_attn_decode_tree(cache, mode, st["parent"], st["q"], 1.0 / math.sqrt(D), st["out"], st["lse"],
                               st["ws"], group=c["group"])
        return dict(out=st["out"], lse=st["lse"])
    cache.state.copy_(st["state"])  # the counters as they were before the round
    if c["op"] == "append":
        qs.qs_buffer_append_rotary(cache, st["k"], st["v"], st["inv_freq"], q=st["q"], q_out=st["q_out"],
                                   offset=st["offset"], interleaved=c["pairs"] == "neighbours")
        return dict(q=st["q_out"], buf_k=cache.buf_k, buf_v=cache.buf_v, state=cache.state[:, :4])
    qs.qs_buffer_append(cache, st["k"], st["v"])
    qs.qs_tree_accept(cache, st["parent"], st["draft"], st["target"], st["n_keep"], st["path"], st["emitted"])
    return dict(buf_k=cache.buf_k, buf_v=cache.buf_v, state=cache.state[:, :4], n_keep=st["n_keep"],
                path=st["path"], emitted=st["emitted"])


# ------------------------------------------------- the definition, 64 bits

def nibbles_at(plane, byte, odd):
    """fp64 nibbles of a [..., bytes] plane at byte positions, odd ones high."""
    b = plane.flatten(1)[:, byte.reshape(-1)].to(torch.int64)
    return ((b >> (4 * odd.reshape(-1))) & 15).reshape(-1, *byte.shape)


def exact_groups(st, b, h, n, mode, bits):
    """fp64 keys and values [n * G, D] of the first n groups of sequence b,
    head h, each code looked up by its address in the stored layout."""
    g = {x: (st[x][st["table"][b, :n].long(), h] if "table" in st else st[x][b, h, :n]) for x in PLANES}
    t, d = torch.arange(G, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    v_pos = torch.empty(32, dtype=torch.int64, device=DEV)
    v_pos[V_TOKEN] = torch.arange(32, device=DEV)
    addr = {"k": 2 * (64 * t + d // 2) + d % 2, "v": 2 * 16 * (128 * (t // 32) + d) + v_pos[t % 32]}
    res = []
    for x, row, at_pos in (("k", 0, K_CHANNEL), ("v", 2, V_ROW_TOKEN)):
        nib = addr[x].expand(G, D)
        if bits == 4:
            up = nibbles_at(g[x + "_upper"], nib // 2, nib % 2)
        else:
            # nibble j of 32-bit word w: field w % 2 of nibble j of word w / 2
            w, j = nib // 8, nib % 8
            src, sh = 8 * (w // 2) + j, 2 * (w % 2)
            two = nibbles_at(g[x + "_upper"], src // 2, src % 2)
            mid = nibbles_at(g[x + "_upper"], 4096 + src // 2, src % 2)
            up = 4 * ((two >> sh) & 3) + ((mid >> sh) & 3)
        lo = nibbles_at(g[x + "_lower"], nib // 2, nib % 2)
        if mode == "verify":
            code = 16 * up + lo
        else:
            code = 16 * up + 8 if bits == 4 else 64 * (up // 4) + 32
        sz = torch.empty((n, 2, 128), dtype=torch.float64, device=DEV)
        sz[..., at_pos] = g["meta"][:, row:row + 2].double()
        sz = sz[:, :, None, :] if x == "k" else sz[:, :, :, None]
        res.append((sz[:, 0] * code + sz[:, 1]).reshape(-1, D))
    return res


def exact_rotation(x, pos, freq, pairs):
    """Rows x [h, D] at one position, as complex products."""
    y = x.double().cpu().numpy().copy()
    m = len(freq)
    i = np.arange(m)
    a, b = (i, i + m) if pairs == "halves" else (2 * i, 2 * i + 1)
    z = (y[:, a] + 1j * y[:, b]) * np.exp(1j * (pos * freq))
    y[:, a], y[:, b] = z.real, z.imag
    return torch.from_numpy(y)


def exact_append(st):
    c = st["case"]
    state = st["state"][:, :4].cpu().clone()
    freq = st["inv_freq"].cpu().double().numpy()
    q = torch.zeros(st["q"].shape, dtype=torch.float64)
    bk, bv = st["buf_k"].double().cpu(), st["buf_v"].double().cpu()
    k, v, qin = st["k"].cpu(), st["v"].cpu(), st["q"].cpu()
    for b in range(c["B"]):
        groups, fill, _, half = (int(x) for x in state[b])
        for j in range(c["n"]):
            pos = groups * G + fill + (j if st["offset"] is None else int(st["offset"][b, j]))
            slot = (half * G + fill + j) % RING
            q[b, :, j] = exact_rotation(qin[b, :, j], pos, freq, c["pairs"])
            bk[b, :, slot] = exact_rotation(k[b, :, j], pos, freq, c["pairs"])
            bv[b, :, slot] = v[b, :, j].double()
        state[b, 1] += c["n"]
        state[b, 2] += c["n"]
    return dict(q=q, buf_k=bk, buf_v=bv, state=state)


def exact_accept(st):
    c = st["case"]
    n = c["n"]
    state = st["state"][:, :4].cpu().clone()
    bk, bv = st["buf_k"].double().cpu(), st["buf_v"].double().cpu()
    k, v = st["k"].double().cpu(), st["v"].double().cpu()
    n_keep = torch.zeros(c["B"], dtype=torch.int32)
    path = torch.full((c["B"], n), -1, dtype=torch.int32)
    emitted = path.clone()
    for b in range(c["B"]):
        parent, draft, target = (st[x][b].tolist() for x in ("parent", "draft", "target"))
        nodes = [0]
        while True:
            nxt = [j for j in range(1, n) if parent[j] == nodes[-1] and draft[j] == target[nodes[-1]]]
            if not nxt:
                break
            nodes.append(nxt[0])
        fill, half = int(state[b, 1]), int(state[b, 3])
        for i in range(n):
            src = nodes[i] if i < len(nodes) else i
            slot = (half * G + fill + i) % RING
            bk[b, :, slot], bv[b, :, slot] = k[b, :, src], v[b, :, src]
        for i, node in enumerate(nodes):
            path[b, i], emitted[b, i] = node, target[node]
        n_keep[b] = len(nodes)
        state[b, 1], state[b, 2] = fill + len(nodes), 0
    return dict(buf_k=bk, buf_v=bv, state=state, n_keep=n_keep, path=path, emitted=emitted)


def exact_sample(st):
    c = st["case"]
    V = c["V"]
    rows = st["logits"].double().cpu().numpy()
    T, k, p, m, u = (st[n].double().cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p", "u"))
    token, probs = np.zeros(c["rows"], np.int32), np.zeros((c["rows"], V) if c["probs"] else (1, V))
    for r, x in enumerate(rows):
        by = np.argsort(-x, kind="stable")
        by = by[:1] if T[r] == 0 else by[:int(k[r])] if k[r] > 0 else by
        w = np.exp((x[by] - x[by[0]]) / T[r]) if T[r] > 0 else np.ones(1)
        if p[r] < 1:
            mass = np.cumsum(w)
            n = 1 + int(np.searchsorted(mass, p[r] * mass[-1], side="left"))  # the first to reach it, too
            by, w = by[:n], w[:n]
        by, w = by[w >= m[r]], w[w >= m[r]]
        at = np.argsort(by)
        by, w = by[at], w[at] / w.sum()
        token[r] = by[min(np.searchsorted(np.cumsum(w), u[r], side="right"), len(by) - 1)]
        if c["probs"]:
            probs[r, by] = w
    res = dict(token=torch.from_numpy(token))
    if c["probs"]:
        res["probs"] = torch.from_numpy(probs)
    return res


def exact_tree(st):
    c = st["case"]
    if work(c)["flops"] > 6e11:
        return None
    B, H, n_q, n, group = c["B"], c["H"], c["n_q"], c["n_tree"], c["group"]
    state = st["state"].cpu()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["q"].shape[:3], dtype=torch.float64, device=DEV)
    for b in range(B):
        ng, fill, half = int(state[b, 0]), int(state[b, 1]), int(state[b, 3])
        slots = (half * G + torch.arange(fill, device=DEV)) % RING
        hidden = np.ones((n_q, fill), bool)
        up = st["parent"][b].tolist()
        hidden[:, :fill - n] = False
        for j in range(n_q):
            node = n - n_q + j
            while node >= 0:
                hidden[j, fill - n + node] = False
                node = up[node]
        hidden = torch.from_numpy(np.concatenate([np.zeros((n_q, ng * G), bool), hidden], 1)).to(DEV)
        for h in range(H):
            k, v = exact_groups(st, b, h, ng, c["mode"], c["bits"])
            k = torch.cat([k, st["buf_k"][b, h, slots].double()])
            v = torch.cat([v, st["buf_v"][b, h, slots].double()])
            for i in range(h * group, (h + 1) * group):
                s = (st["q"][b, i].double() @ k.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lse[b, i] = torch.logsumexp(s, -1)
                out[b, i] = torch.exp(s - lse[b, i][:, None]) @ v
    return dict(out=out, lse=lse)


def exact(case, seed):
    st = prepare(case, seed)
    return dict(append=exact_append, tree=exact_tree, sample=exact_sample, accept=exact_accept)[case["op"]](st)
