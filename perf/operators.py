"""Cases that measure the paged and sparse operators of the hierarchical
quantized KV cache: group selection, sparse and paged decode attention, the
quantizing write of a paged cache with its read back, and the read back alone.

``own`` false computes each operator in elementary torch operations from the
bytes the cache stores (the layout of include/qs.h); ``own`` true calls the
library.  Sizes: head_dim 128 and groups of 128 tokens throughout (the only
ones the cache has), contexts from 1k to 128k tokens, 2 to 32 KV heads, one
query head per KV head or groups of up to eight.
"""
import math

import numpy as np
import torch

own = False

D = G = 128
RING = 2 * G
DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one draft step of a single 32k sequence picks its groups: latency counts
        dict(name="select_32k", op="select", B=1, H=32, group=1, n_q=1, groups=254, ragged=False,
             paged=False, k=32),
        # grouped-query heads, four 128k sequences in pages
        dict(name="select_gqa_128k", op="select", B=4, H=8, group=4, n_q=1, groups=1022, ragged=True,
             paged=True, k=64),
        # the draft's attention over the picked groups of a 32k context and the full buffer
        dict(name="sparse_draft_32k", op="sparse", B=1, H=32, group=1, n_q=1, groups=254,
             ragged=False, paged=False, k=32, fill=256, bits=4, mode="draft"),
        # the two-bit draft of four 128k grouped-query sequences in pages
        dict(name="sparse_gqa_2bit_128k", op="sparse", B=4, H=8, group=4, n_q=1, groups=1022,
             ragged=True, paged=True, k=64, fill=201, bits=2, mode="draft"),
        # a verify pass limited to the picked half of ragged contexts up to 64k
        dict(name="sparse_verify_ragged", op="sparse", B=16, H=32, group=1, n_q=5, groups=510,
             ragged=True, paged=False, k=128, fill=133, bits=4, mode="verify"),
        # the smallest call: two heads, 1k tokens
        dict(name="paged_draft_1k", op="paged", B=1, H=2, group=1, n_q=1, groups=6, ragged=False,
             fill=256, bits=4, mode="draft"),
        # one new token of a grouped-query 32k sequence
        dict(name="paged_gqa_draft_32k", op="paged", B=1, H=8, group=4, n_q=1, groups=254,
             ragged=False, fill=256, bits=4, mode="draft"),
        # verify of five tokens for eight ragged sequences up to 64k
        dict(name="paged_verify_ragged", op="paged", B=8, H=32, group=1, n_q=5, groups=510,
             ragged=True, fill=77, bits=4, mode="verify"),
        # a batch of short prompts written and read back
        dict(name="write_read_short", op="write", B=4, H=8, T=1000, ragged=True, bits=4),
        # a 32k prompt of 32 heads written and read back
        dict(name="write_read_32k", op="write", B=1, H=32, T=32768, ragged=False, bits=4),
        # an odd window of the draft's view
        dict(name="read_draft_window", op="read", B=2, H=8, groups=30, ragged=True, paged=True,
             fill=99, bits=4, mode="draft", tok0=1037, T=2001),
        # the whole of a 32k cache for a dense pass over it
        dict(name="read_verify_32k", op="read", B=1, H=32, groups=254, ragged=False, paged=False,
             fill=256, bits=4, mode="verify", tok0=0, T=32768),
    ]


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["select", "sparse", "paged", "write", "read"])
        mode = rng.choice(["draft", "verify"])
        c = dict(op=op, B=log_int(1, 16), H=rng.choice([2, 4, 5, 8, 16, 32]), ragged=rng.random() < 0.5)
        if op in ("select", "sparse", "paged"):
            c["n_q"] = rng.choice([1, 1, 1, 4, 5]) if mode == "verify" or op == "select" else 1
            c["group"] = rng.choice([g for g in (1, 2, 3, 4, 8) if g * c["n_q"] <= 24])
        if op != "write":
            c["groups"] = log_int(4, 1022)
        if op == "select":
            c["groups"] = max(16, c["groups"])
            c["k"] = min(log_int(1, 256), 3 * c["groups"] // 4)
        if op == "sparse":
            c["k"] = min(log_int(1, 256), c["groups"])
        if op in ("select", "sparse", "read"):
            c["paged"] = rng.random() < 0.5
        if op in ("sparse", "paged", "read"):
            c["fill"] = rng.randint(8, RING)
            c["mode"] = mode
        if op != "select":
            c["bits"] = rng.choice([4, 4, 2])
        if op == "write":
            c["T"] = log_int(200, 32768)
        if op == "read":
            n = c["groups"] * G + c["fill"]
            c["tok0"] = rng.choice([0, rng.randint(0, n - 1)])
            c["T"] = rng.randint(1, n - c["tok0"])
        w = work(c)["bytes"]
        if 2e5 < w <= most:
            return c


def lengths(n, B, ragged):
    """Per-sequence values up to n, fixed by the case alone: spread from about
    n / 8 to n where ragged."""
    if not ragged:
        return [n] * B
    return [max(1, n - (n * 7 * ((5 * b) % B)) // (8 * max(1, B - 1)) if B > 1 else n) for b in range(B)]


def group_bytes(mode, bits):
    """Plane and scale bytes of a group and head that an attention or a read
    in this mode needs."""
    if mode == "verify":
        return 4 * 8192 + 1024
    return (8192 if bits == 2 else 16384) + 1024


def prompt_split(L):
    """Quantized groups and buffered tokens of an L-token prompt."""
    ng = -(-(L - RING) // G) if L > RING else 0
    return ng, L - ng * G


def work(case):
    c = case
    B, H = c["B"], c["H"]
    if c["op"] == "write":
        byts = 0
        for L in lengths(c["T"], B, c["ragged"]):
            ng, fill = prompt_split(L)
            byts += H * (2 * L * 512 + ng * group_bytes("verify", 4) + fill * 512)
        return {"bytes": byts, "flops": 0}
    ng = lengths(c["groups"], B, c["ragged"])
    if c["op"] == "read":
        byts = 0
        for n in ng:
            lo, hi = c["tok0"], min(c["tok0"] + c["T"], n * G + c["fill"])
            q = max(0, min(hi, n * G) - lo)
            byts += H * (q * group_bytes(c["mode"], c["bits"]) / G + max(0, hi - max(lo, n * G)) * 512
                         + max(0, hi - lo) * 512)
        return {"bytes": byts, "flops": 0}
    R = c["group"] * c["n_q"]
    if c["op"] == "select":
        return {"bytes": sum(ng) * H * 512 + B * H * (R * 256 + 4 * c["k"]),
                "flops": 2 * 256 * R * H * sum(ng)}
    if c["op"] == "sparse":
        ng = [min(n, c["k"]) for n in ng]
    tok = sum(ng) * G + B * c["fill"]
    return {"bytes": H * (sum(ng) * group_bytes(c["mode"], c["bits"]) + B * c["fill"] * 512)
            + B * H * R * (512 + 4),
            "flops": 4 * 128 * R * H * tok}


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


def round_up_fp16(x):
    """The smallest fp16 value >= x (x >= 0, fp32)."""
    h = x.half()
    return torch.where(h.float() < x, (h.view(torch.int16) + 1).view(torch.float16), h)


def quantize(x, dim):
    """Asymmetric 8-bit groups along dim: codes, fp16 scale, fp16 zero."""
    x = x.float()
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s = round_up_fp16((hi - lo) / 255.0)
    sf = s.float()
    u = (x - lo) / torch.where(sf == 0, torch.ones_like(sf), sf)
    q = torch.where(sf == 0, torch.zeros_like(u), u.round().clamp(0, 255))
    return q.to(torch.uint8), s, (lo + 0.0).half()


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


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, H = c["B"], c["H"]
    st = dict(case=c)
    bits = c.get("bits", 4)
    if c["op"] == "write":
        T = c["T"]
        st["k"], st["v"] = tokens(gen, (B, H, T, D))
        st["lens"] = torch.tensor(lengths(T, B, c["ragged"]), dtype=torch.int32, device=DEV)
        cap = max(1, prompt_split(T)[0])
        pages = B * cap + 3
        st["table"] = torch.randperm(pages, generator=gen, device=DEV)[:B * cap].to(torch.int32).reshape(B, cap)
        st["k_out"], st["v_out"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
    else:
        cap = c["groups"]
        ng = torch.tensor(lengths(cap, B, c["ragged"]), dtype=torch.int32, device=DEV)
        paged = c["op"] == "paged" or c.get("paged", False)
        if paged:
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
        bk, bv = tokens(gen, (B, H, RING, D))
        fill = c.get("fill", 64)
        state = torch.zeros((B, 8), dtype=torch.int32, device=DEV)
        state[:, 0] = ng
        state[:, 1] = fill
        state[:, 3] = torch.arange(B, device=DEV) % 2
        st.update(buf_k=bk, buf_v=bv, state=state)
        if c["op"] == "read":
            for n in ("k_out", "v_out"):
                st[n] = torch.zeros((B, H, c["T"], D), dtype=torch.float16, device=DEV)
        else:
            hq = H * c["group"]
            st["q"] = torch.randn((B, hq, c["n_q"], D), generator=gen, device=DEV).half()
        if c["op"] == "sparse":
            kk = c["k"]
            r = torch.rand((B, H, cap), generator=gen, device=DEV)
            r = torch.where(torch.arange(cap, device=DEV) < ng[:, None, None], r, 2.0)
            pick = r.argsort(-1)[..., :kk].to(torch.int32)
            pick = torch.where(torch.arange(kk, device=DEV) < ng[:, None, None], pick, 1 << 30)
            pick = pick.sort(-1).values
            st["sel"] = torch.where(pick == 1 << 30, -1, pick).contiguous()
        if c["op"] == "select":
            st["sel"] = torch.zeros((B, H, c["k"]), dtype=torch.int32, device=DEV)
        if c["op"] in ("sparse", "paged"):
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
        if c["op"] in ("sparse", "paged"):
            size = qs.qs_attn_workspace_size_gqa(cache, c["n_q"], c["group"])
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


def groups_of(st, pick=None, names=PLANES):
    """The named arrays of each sequence's groups, [B, H, n, ...]: all of them, or
    the picked ones (pick [B, H, n], clamped to valid indices)."""
    B, H = st["buf_k"].shape[:2]
    heads = torch.arange(H, device=DEV)[:, None]
    got = {}
    for n in names:
        t = st[n]
        if "table" in st:
            page = st["table"].clamp(min=0).long()[:, None].expand(B, H, -1)
            if pick is not None:
                page = page.gather(-1, pick)
            got[n] = t[page, heads]
        elif pick is None:
            got[n] = t
        else:
            got[n] = t[torch.arange(B, device=DEV)[:, None, None], heads, pick]
    return got


def dequantized(st, mode, bits, pick=None):
    """fp32 keys and values of the groups, [B, H, n, G, D]."""
    g = groups_of(st, pick)
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


def ring_order(st):
    """The buffers in logical order, fp32 [B, H, 2G, D]."""
    slot = (st["state"][:, 3:4].long() * G + torch.arange(RING, device=DEV)) % RING
    at = slot[:, None, :, None].expand(-1, st["buf_k"].shape[1], -1, D)
    return st["buf_k"].gather(2, at).float(), st["buf_v"].gather(2, at).float()


def plain_attention(st, pick, count):
    """Softmax attention of the queries over count [B] of the groups and the
    causal part of the buffer."""
    c = st["case"]
    B, H, R = c["B"], c["H"], c["group"] * c["n_q"]
    k, v = dequantized(st, c["mode"], c["bits"], pick)
    n = k.shape[2]
    bk, bv = ring_order(st)
    q = st["q"].float().reshape(B, H, R, D)
    s1 = q @ k.reshape(B, H, n * G, D).transpose(-1, -2)
    s2 = q @ bk.transpose(-1, -2)
    seen1 = torch.arange(n * G, device=DEV) < (count.long() * G)[:, None, None, None]
    last = st["state"][:, 1].long()[:, None, None, None] - c["n_q"] + \
        (torch.arange(R, device=DEV) % c["n_q"])[:, None]
    seen2 = torch.arange(RING, device=DEV) <= last
    s1 = torch.where(seen1, s1 / math.sqrt(D), -math.inf)
    s2 = torch.where(seen2, s2 / math.sqrt(D), -math.inf)
    top = torch.maximum(s1.amax(-1, keepdim=True), s2.amax(-1, keepdim=True))
    p1, p2 = torch.exp(s1 - top), torch.exp(s2 - top)
    total = p1.sum(-1, keepdim=True) + p2.sum(-1, keepdim=True)
    o = (p1 @ v.reshape(B, H, n * G, D) + p2 @ bv) / total
    shape = st["q"].shape
    return dict(out=o.half().reshape(shape), lse=(top + torch.log(total)).reshape(shape[:3]))


def plain_select(st):
    """The k groups of each KV head whose keys' box allows the largest score
    for any of the head's query rows, in fp64 (which of two close groups is
    in hangs on it); ties to the lower index, listed in ascending order."""
    c = st["case"]
    B, H, R, kk = c["B"], c["H"], c["group"] * c["n_q"], c["k"]
    meta = groups_of(st, names=("meta",))["meta"][..., :2, :][..., K_CHANNEL_AT].double()
    q = st["q"].double().reshape(B, H, R, D)
    bound = q @ meta[..., 1, :].transpose(-1, -2) + 255 * (q.clamp(min=0) @ meta[..., 0, :].transpose(-1, -2))
    bound = bound.amax(2)
    ng = st["state"][:, 0].long()[:, None, None]
    at = torch.arange(bound.shape[-1], device=DEV)
    bound = torch.where(at < ng, bound, -math.inf)
    pick = torch.sort(bound, dim=-1, descending=True, stable=True).indices[..., :kk]
    pick = torch.where(pick < ng, pick, 1 << 30).sort(-1).values
    return dict(sel=torch.where(pick == 1 << 30, -1, pick).to(torch.int32))


def plain_read(st):
    c = st["case"]
    B, H, T = c["B"], c["H"], c["T"]
    first = c["tok0"] // G
    last = min(c["groups"], -(-(c["tok0"] + T) // G))
    if last > first:
        pick = torch.arange(first, last, device=DEV).expand(B, H, -1)
        k, v = dequantized(st, c["mode"], c["bits"], pick)
    else:
        k = v = torch.zeros((B, H, 0, G, D), device=DEV)
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    bk, bv = ring_order(st)
    t = torch.arange(c["tok0"], c["tok0"] + T, device=DEV)
    nq = st["state"][:, 0].long()[:, None] * G
    i_q = (t - first * G).clamp(0, max(0, k.shape[2] - 1))
    i_b = (t - nq).clamp(0, RING - 1)
    in_q, in_b = t < nq, (t >= nq) & (t < nq + st["state"][:, 1:2])

    def rows(x, b, into):
        r = b.gather(2, i_b[:, None, :, None].expand(B, H, T, D))
        if x.shape[2]:
            r = torch.where(in_q[:, None, :, None], x[:, :, i_q], r)
        return torch.where((in_q | in_b)[:, None, :, None], r.half(), into)

    return dict(k=rows(k, bk, st["k_out"]), v=rows(v, bv, st["v_out"]))


def plain_write(st):
    c = st["case"]
    B, H, T = c["B"], c["H"], c["T"]
    L = st["lens"].long()
    ng = torch.where(L > RING, -((RING - L) // G), 0)
    n = prompt_split(T)[0]
    t = torch.arange(T, device=DEV)
    res = {}
    for name, dim in (("k", -2), ("v", -1)):
        x = st[name]
        whole = x[:, :, :n * G].reshape(B, H, n, G, D)
        q, s, z = quantize(whole, dim) if n else (whole, whole, whole)
        deq = (q.float() * s.float() + z.float()).half().reshape(B, H, n * G, D)
        deq = torch.cat([deq, x[:, :, n * G:]], 2)
        quantized = (t < (ng * G)[:, None])[:, None, :, None]
        live = (t < L[:, None])[:, None, :, None]
        res[name] = torch.where(live, torch.where(quantized, deq, x), st[name + "_out"])
    zero = torch.zeros_like(L)
    res["counters"] = torch.stack([ng, L - ng * G, zero, zero], -1).to(torch.int32)
    return res


def plain(st):
    op = st["case"]["op"]
    if op == "select":
        return plain_select(st)
    if op == "sparse":
        ng = st["state"][:, 0].clamp(max=st["case"]["k"])
        return plain_attention(st, st["sel"].clamp(min=0).long(), ng)
    if op == "paged":
        return plain_attention(st, None, st["state"][:, 0])
    return plain_read(st) if op == "read" else plain_write(st)


def run(state):
    if not own:
        return plain(state)
    from hierarchical_quantized_kv_gb300 import qs
    st, c = state, state["case"]
    cache = st["cache"]
    if c["op"] == "select":
        qs.qs_select_groups(cache, st["q"], st["sel"], group=c["group"])
        return dict(sel=st["sel"])
    if c["op"] == "write":
        qs.qs_state_reset(cache)
        qs.qs_prefill_paged(cache, st["k"], st["v"], st["lens"])
        qs.qs_cache_read(cache, qs.QS_VERIFY_INT8, st["k_out"], st["v_out"])
        return dict(k=st["k_out"], v=st["v_out"], counters=cache.state[:, :4])
    mode = qs.QS_DRAFT_UPPER4 if c["mode"] == "draft" else qs.QS_VERIFY_INT8
    if c["op"] == "read":
        qs.qs_cache_read(cache, mode, st["k_out"], st["v_out"], tok0=c["tok0"])
        return dict(k=st["k_out"], v=st["v_out"])
    scale = 1.0 / math.sqrt(D)
    if c["op"] == "sparse":
        qs.qs_attn_decode_sparse(cache, mode, st["sel"], st["q"], scale, st["out"], st["lse"],
                                 st["ws"], group=c["group"])
    else:
        qs.qs_attn_decode_paged(cache, mode, st["q"], scale, st["out"], st["lse"], st["ws"],
                                group=c["group"])
    return dict(out=st["out"], lse=st["lse"])


# ------------------------------------------------- the definition, 64 bits

def nibbles_at(plane, byte, odd):
    """fp64 nibbles of a [..., bytes] plane at byte positions, odd ones high."""
    b = plane.flatten(1)[:, byte.reshape(-1)].to(torch.int64)
    return ((b >> (4 * odd.reshape(-1))) & 15).reshape(-1, *byte.shape)


def exact_groups(st, b, h, groups, mode, bits):
    """fp64 keys and values [n * G, D] of the listed groups of sequence b,
    head h, each code looked up by its address in the stored layout."""
    at = st["table"][b].long()[groups] if "table" in st else groups
    g = {n: (st[n][at, h] if "table" in st else st[n][b, h, at]) for n in PLANES}
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
        sz = torch.empty((len(groups), 2, 128), dtype=torch.float64, device=DEV)
        sz[..., at_pos] = g["meta"][:, row:row + 2].double()
        sz = sz[:, :, None, :] if x == "k" else sz[:, :, :, None]
        res.append((sz[:, 0] * code + sz[:, 1]).reshape(-1, D))
    return res


def exact_quantized(x, per_channel):
    """fp64 dequantized groups of x [n, G, D]."""
    x = x.double()
    dim = 1 if per_channel else 2
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s = torch.from_numpy(up16(((hi - lo) / 255).cpu().numpy())).to(x.device)
    code = torch.where(s > 0, torch.round((x - lo) / torch.where(s > 0, s, 1.0)), 0.0)
    return s * torch.clamp(code, 0, 255) + lo


def up16(x):
    h = x.astype(np.float16)
    return np.where(h.astype(np.float64) < x, np.nextafter(h, np.float16(np.inf)), h).astype(np.float64)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    B, H = c["B"], c["H"]
    if c["op"] == "write":
        res = dict(k=st["k_out"].double(), v=st["v_out"].double())
        counters = torch.zeros((B, 4), dtype=torch.int32)
        for b in range(B):
            L = int(st["lens"][b])
            ng, fill = prompt_split(L)
            counters[b, 0], counters[b, 1] = ng, fill
            for n in ("k", "v"):
                for h in range(H):
                    x = st[n][b, h, :L]
                    res[n][b, h, :L] = x.double()
                    if ng:
                        res[n][b, h, :ng * G] = exact_quantized(x[:ng * G].reshape(ng, G, D),
                                                               n == "k").reshape(-1, D)
        return dict(res, counters=counters)
    state = st["state"].cpu()
    if c["op"] == "read":
        res = dict(k=st["k_out"].double(), v=st["v_out"].double())
        for b in range(B):
            n, fill, half = int(state[b, 0]), int(state[b, 1]), int(state[b, 3])
            lo, hi = c["tok0"], min(c["tok0"] + c["T"], n * G + fill)
            if hi <= lo:
                continue
            slots = (half * G + torch.arange(fill, device=DEV)) % RING
            first, last = min(lo // G, n), min(-(-hi // G), n)
            for h in range(H):
                parts = exact_groups(st, b, h, torch.arange(first, last, device=DEV), c["mode"],
                                     c["bits"]) if last > first else \
                    [torch.zeros((0, D), dtype=torch.float64, device=DEV)] * 2
                for name, x, buf in (("k", parts[0], "buf_k"), ("v", parts[1], "buf_v")):
                    x = torch.cat([x, st[buf][b, h, slots].double()])
                    res[name][b, h, :hi - lo] = x[lo - first * G:hi - first * G]
        return res
    q = st["q"].double().reshape(B, H, c["group"] * c["n_q"], D)
    R = q.shape[2]
    if c["op"] == "select":
        sel = torch.full((B, H, c["k"]), -1, dtype=torch.int32)
        ch = K_CHANNEL
        for b in range(B):
            n = int(state[b, 0])
            for h in range(H):
                at = st["table"][b, :n].long() if "table" in st else None
                m = (st["meta"][at, h] if at is not None else st["meta"][b, h, :n]).double()
                qr = q[b, h][:, ch]
                lo, hi = m[:, 1], m[:, 1] + 255 * m[:, 0]
                box = torch.maximum(qr[:, None] * lo, qr[:, None] * hi).sum(-1).amax(0)
                by = np.lexsort((np.arange(n), -box.cpu().numpy()))[:c["k"]]
                sel[b, h, :len(by)] = torch.from_numpy(np.sort(by)).to(torch.int32)
        return dict(sel=sel)
    if work(c)["flops"] > 4e11:
        return None
    out = torch.zeros((B, H, R, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, H, R), dtype=torch.float64, device=DEV)
    for b in range(B):
        n, fill, half = int(state[b, 0]), int(state[b, 1]), int(state[b, 3])
        slots = (half * G + torch.arange(fill, device=DEV)) % RING
        last = fill - c["n_q"] + torch.arange(R, device=DEV) % c["n_q"]
        for h in range(H):
            groups = torch.arange(n, device=DEV)
            if c["op"] == "sparse":
                groups = st["sel"][b, h].long()
                groups = groups[groups >= 0]
            k, v = exact_groups(st, b, h, groups, c["mode"], c["bits"])
            k = torch.cat([k, st["buf_k"][b, h, slots].double()])
            v = torch.cat([v, st["buf_v"][b, h, slots].double()])
            s = q[b, h] @ k.T / math.sqrt(D)
            i = torch.arange(len(k), device=DEV) - len(groups) * G
            s = s.masked_fill(i > last[:, None], -math.inf)
            lse[b, h] = torch.logsumexp(s, -1)
            out[b, h] = torch.exp(s - lse[b, h][:, None]) @ v
    shape = st["q"].shape
    return dict(out=out.reshape(shape), lse=lse.reshape(shape[:3]))
