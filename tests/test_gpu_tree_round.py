"""Rounds over a tree as a serving loop makes them: levels drafted, the tree
verified, tokens sampled, a path accepted, halves flushed; after each the cache is
that of a program that had appended the accepted tokens alone."""
import numpy as np
import pytest

import oracle
from hierarchical_quantized_kv_gb300 import qs
from tests import paging, trees
from tests.test_gpu_qs import DRAFT, VERIFY, h16, to_dev
from tests.test_gpu_tree_attn import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,levels", [(1, [1, 3, 6]), (4, [1, 4, 9, 12])])
@pytest.mark.parametrize("paged", [False, True])
def test_rounds(group, levels, paged):
    torch = pytest.importorskip("torch")
    import __graft_entry__
    __graft_entry__.build()
    rng = np.random.default_rng([group, paged])
    B, H, V, D = 2, 2, 500, 128
    T, scale = np.array([390, 380], np.int32), 1 / np.sqrt(D)
    k0, v0 = h16(rng, (B, H, 400, D), 2), h16(rng, (B, H, 400, D))
    cap = 24
    if paged:
        cache = qs.PagedCache(B, H, cap, B * cap)
        cache.table.copy_(torch.from_numpy(rng.permutation(B * cap).reshape(B, cap).astype(np.int32)))
        qs.qs_prefill_paged(cache, to_dev(torch, k0), to_dev(torch, v0), to_dev(torch, T))
    else:
        cache = qs.Cache(B, H, cap)
        qs.qs_prefill(cache, to_dev(torch, k0), to_dev(torch, v0), to_dev(torch, T))
    oc = oracle.OracleCache(B, H, D, 128, cap=cap)
    oc.prefill(k0, v0, T)
    n = sum(levels)
    freq = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    fd = to_dev(torch, freq)
    text = T.copy()
    for step in range(12):
        parent = np.full((B, n), -1, np.int32)
        first = np.concatenate([[0], np.cumsum(levels)])
        for lv in range(1, len(levels)):
            parent[:, first[lv]:first[lv + 1]] = rng.integers(first[lv - 1], first[lv], (B, levels[lv]))
        depth = trees.depths(parent)
        qs.qs_quantize_flush_due_paged(cache, n) if paged else qs.qs_quantize_flush_due(cache, n)
        oc.flush(oc.need_flush(n))
        keys = {}
        for name, parts in (("draft", list(zip(first[:-1], first[1:]))), ("verify", [(0, n)])):
            # what the layers' projections leave: heads of a token side by side
            x = h16(rng, (B, n, (group + 2) * H, D))
            q, k, v = (x[:, :, a:b].transpose(0, 2, 1, 3) for a, b in
                       ((0, group * H), (group * H, group * H + H), (group * H + H, None)))
            pos = text[:, None] + depth
            want_q = trees.rotate(q, pos[:, None], freq, False)
            want_k = trees.rotate(k, pos[:, None], freq, False).astype(np.float16)
            mode = DRAFT if name == "draft" else VERIFY
            oc.append(want_k, np.ascontiguousarray(v))
            for a, b in parts:
                xd = to_dev(torch, x[:, a:b]).transpose(1, 2)
                q_out = torch.empty((B, group * H, b - a, D), dtype=torch.float16, device="cuda")
                qs.qs_buffer_append_rotary(cache, xd[:, group * H:group * H + H], xd[:, group * H + H:], fd,
                                           q=xd[:, :group * H], q_out=q_out,
                                           offset=to_dev(torch, np.ascontiguousarray(depth[:, a:b])))
                out, lse = torch.empty_like(q_out), torch.empty(q_out.shape[:3], device="cuda")
                ws = torch.empty(qs.qs_attn_tree_workspace_size(cache, b - a, group), dtype=torch.uint8,
                                 device="cuda")
                qs.qs_attn_decode_tree(cache, mode, to_dev(torch, np.ascontiguousarray(parent[:, :b])), q_out,
                                       scale, out, lse, ws, group=group)
                torch.cuda.synchronize()
                # (nodes of later levels are nobody's ancestors in this one)
                ref, rl = trees.attention(oc, want_q, parent, mode == DRAFT, group)
                check(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref[:, :, a:b], rl[:, :, a:b],
                      "%s %d" % (name, step))
            keys[name] = want_k, v
            if name == "draft":
                drop = np.full(B, n, np.int32)
                qs.qs_buffer_rollback(cache, to_dev(torch, drop))
                oc.rollback(drop)
        # tokens from the target's logits; drafts that often guess them
        logits = torch.from_numpy(rng.standard_normal((B * n, V)).astype(np.float32) * 3).cuda()
        u = rng.random(B * n).astype(np.float32)
        target = torch.empty((B, n), dtype=torch.int32, device="cuda")
        tk = torch.full((B * n,), 5, dtype=torch.int32, device="cuda")
        qs.qs_sample(logits, to_dev(torch, u), target.view(-1), top_k=tk)
        want_t = np.array([trees.sample(x, y, top_k=5)[0] for x, y in zip(logits.double().cpu().numpy(), u)])
        assert np.array_equal(target.cpu().numpy().reshape(-1), want_t)
        tn = want_t.reshape(B, n)
        draft = np.where(rng.random((B, n)) < 0.7, np.take_along_axis(tn, np.maximum(parent, 0), 1), -1).astype(np.int32)
        keep = torch.empty(B, dtype=torch.int32, device="cuda")
        path, emitted = torch.empty((2, B, n), dtype=torch.int32, device="cuda")
        qs.qs_tree_accept(cache, to_dev(torch, parent), to_dev(torch, draft), target, keep, path, emitted)
        # the oracle takes the tree back and appends the path alone
        oc.rollback(np.full(B, n, np.int32))
        paths = [trees.accept(parent[b], draft[b], tn[b]) for b in range(B)]
        assert keep.tolist() == [len(p) for p in paths]
        longest = max(len(p) for p in paths)
        kk, vv = (np.zeros((B, H, longest, D), np.float16) for _ in range(2))
        for b, p in enumerate(paths):
            kk[b, :, :len(p)], vv[b, :, :len(p)] = keys["verify"][0][b][:, p], keys["verify"][1][b][:, p]
            assert emitted[b, :len(p)].tolist() == tn[b][p].tolist()
        oc.append(kk, vv)
        oc.rollback(np.array([longest - len(p) for p in paths], np.int32))
        text += [len(p) for p in paths]
        assert np.all(qs.qs_get_errors(cache) == 0)
        for b in range(B):
            c = oc.counters(b)
            st = cache.state[b].tolist()
            assert st[:3] == [c["n_groups"], c["fill"], 0] and text[b] == c["n_groups"] * 128 + c["fill"]
            at = (st[3] * 128 + np.arange(st[1])) % 256
            for h in range(H):
                bk, bv = (x.view(np.float16).astype(np.float64) for x in oc.buffer_tokens(b, h))
                # (a rotated key may round to the other side of a step)
                d = np.abs(cache.buf_k[b, h].double().cpu().numpy()[at] - bk)
                assert np.all(d <= 2.0 ** -10 * np.abs(bk) + 2.0 ** -18)
                assert np.array_equal(cache.buf_v[b, h].double().cpu().numpy()[at], bv)
    assert cache.state[1, 0] == 2  # a half was flushed on the way (the prompt left one group)
