"""Elements that are not numbers or not finite in quantized groups, bit for bit:
the minimum and maximum are those of the numbers among a group's elements, an
element that is not a number has code 0 (it reads as the minimum), and every
code of a group with an infinite range is 0.  The other groups see nothing."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests.test_gpu_qs import assert_state_equal, h16, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need CUDA"
    import __graft_entry__
    __graft_entry__.build()
    return t


def spoil(rng, k, v, n, inf):
    """k, v [B, H, T, 128] with some elements of the first n groups NaN (inf: or
    infinite), and the same with those replaced by their groups' minima, plus
    the (group lines) that hold an infinity: keys [B, H, n, 128 channels], values
    [B, H, n, 128 tokens]."""
    out = []
    for x, axis in ((k, 3), (v, 4)):
        g = x[:, :, :128 * n].reshape(x.shape[0], x.shape[1], n, 128, 128).astype(np.float32)
        bad = rng.random(g.shape) < 0.01
        values = [np.nan, np.inf, -np.inf] if inf else [np.nan]
        g[bad] = rng.choice(values, int(bad.sum()))
        infinite = np.isinf(g).any(axis)
        good = np.where(np.isfinite(g), g, np.inf)
        clean = np.where(np.isfinite(g), g, good.min(axis, keepdims=True))
        lows = np.where(np.isnan(g), np.inf, g).min(axis)
        spoilt, cleaned = x.copy(), x.copy()
        spoilt[:, :, :128 * n] = g.reshape(x.shape[0], x.shape[1], -1, 128).astype(np.float16)
        cleaned[:, :, :128 * n] = clean.reshape(x.shape[0], x.shape[1], -1, 128).astype(np.float16)
        out.append((spoilt, cleaned, infinite, lows.astype(np.float16)))
    return out


@pytest.mark.parametrize("ub", [4, 2])
@pytest.mark.parametrize("inf", [False, True])
@pytest.mark.parametrize("H,n", [(1, 1), (2, 40), (40, 20)])  # 16, 8 and 4 warps a CTA
def test_codes_of_what_is_no_number(torch, H, n, inf, ub):
    rng = np.random.default_rng([H, n, inf, ub])
    T = 128 * n + 256
    k, v = h16(rng, (1, H, T, 128), 2.0), h16(rng, (1, H, T, 128))
    (ks, kc, ki, kz), (vs, vc, vi, vz) = spoil(rng, k, v, n, inf)
    lens = np.array([T], np.int32)
    oc = oracle.OracleCache(1, H, 128, 128, n + 1)
    oc.prefill(kc, vc, lens)
    # an infinite range: scale +inf, the zero is the minimum, all codes 0
    oc.ks[:, :, :n][ki] = oc.vs[:, :, :n][vi] = 0x7C00
    oc.kz[:, :, :n][ki] = kz[ki].view(np.uint16)
    oc.vz[:, :, :n][vi] = vz[vi].view(np.uint16)
    oc.kq[:, :, :n].swapaxes(3, 4)[ki] = 0
    oc.vq[:, :, :n][vi] = 0
    if inf:
        assert ki.any() and vi.any() and not ki.all()
    pc = qs.Cache(1, H, n + 1, upper_bits=ub)
    qs.qs_prefill(pc, to_dev(torch, ks), to_dev(torch, vs), to_dev(torch, lens))
    torch.cuda.synchronize()
    assert_state_equal(pc, oc, "prefill")
    if n == 1:  # the flush: sixteen warps a CTA
        fc = qs.Cache(1, H, n + 1, upper_bits=ub)
        qs.qs_buffer_append(fc, to_dev(torch, ks[:, :, :256]), to_dev(torch, vs[:, :, :256]))
        qs.qs_buffer_rollback(fc, torch.zeros(1, dtype=torch.int32, device="cuda"))
        qs.qs_quantize_flush(fc)
        torch.cuda.synchronize()
        for name in ("k_upper", "k_lower", "v_upper", "v_lower", "meta"):
            a, b = (getattr(c, name)[:, :, 0].cpu().numpy().view(np.uint8) for c in (fc, pc))
            assert np.array_equal(a, b), name
