"""Kernels that overlap their predecessor in the stream read what it may have
written by plain loads: the read-only path keeps lines that the grid
dependency does not drop.  Whether a stale line is met depends on timing, so
the sources are checked."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(__file__)), "hierarchical_quantized_kv_gb300", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", " ", text, flags=re.S)


@pytest.mark.parametrize("name", SOURCES)
def test_no_load_through_the_read_only_path(name):
    text = code(name)
    assert not re.findall(r"__ldg\w*\s*\(|ld\.global(?:\.\w+)*\.nc|__restrict__", text)


def test_every_kernel_that_starts_early_waits():
    """A kernel launched to overlap its predecessor calls pdl_wait (launches
    and waits are matched by name)."""
    launched = set()
    text = "".join(code(n) for n in SOURCES)
    for m in re.finditer(r"launch_pdl(?:_cluster)?\(\s*(\w+_kernel)", text):
        launched.add(m.group(1))
    assert len(launched) >= 9
    for k in launched:
        body = text[re.search(r"\b%s\s*\([^;{]*\)\s*\{" % k, text).end():]
        assert "pdl_wait()" in body[:6000], k
