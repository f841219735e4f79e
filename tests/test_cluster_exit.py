"""The kernels whose CTAs store to one another's shared memory: no CTA leaves
before its cluster's last barrier, whatever it read in the counters (whether two
CTAs read different ones depends on timing and on a caller that breaks the
order of calls, so the sources are checked)."""
import re

from tests.test_stream_order import code


def body(text, name):
    at = re.search(r"\b%s\s*\([^;{]*\)\s*\{" % name, text).end()
    depth, i = 1, at
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at:i]


def test_selection_meets_every_barrier():
    text = body(code("qs_select.cu"), "select_kernel")
    first = text.index("return;")
    assert text.index("cluster.barrier_arrive()") < text.index("cluster.sync()") < first
    # the way out goes by the CTA, and so does what follows the barriers
    assert len(re.findall(r"QS_ST_N_GROUPS", text)) == 1
    assert "if (__syncthreads_and(n_warp <= k_sel))" in text[:first]
    assert re.match(r"cluster\.sync\(\);\s*if \(rank != 0\) return;\s*n = s_n;", text[text.rindex("cluster.sync()"):])


def test_acceptance_decides_its_second_pass_together():
    text = body(code("qs_spec.cu"), "spec_accept_kernel")
    loop = text[text.index("for (int pass = 0"):]
    assert "if (idx >= 0 || !again) break;" in loop and loop.count("break;") == 1
    assert loop.count("cluster.sync()") == 2 and "return" not in text


def test_clustered_attention_meets_every_barrier():
    text = body(code("qs_split.cuh"), "split_kernel")
    start = text[:text.index("finish_cluster<NW>(")]
    # between the counters and the end the clustered variant has no way out
    # (leave() is a lambda of the split one)
    start = re.sub(r"auto leave = .*?\};", "", start, flags=re.S)
    outs = [m.start() for m in re.finditer(r"\breturn;", start)]
    for o in outs:
        guard = start[:o].rstrip()
        assert re.search(r"if \((?:!CL &&|!chk)[^;]*(?:;[^;}]*)?$", guard[-200:]), guard[-200:]
