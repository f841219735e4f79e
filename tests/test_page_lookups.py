"""A page number is checked and used from one reading of the table: an entry
that somebody changes in between must not become an address (a matter of
timing, so the sources are checked)."""
import re

from tests.test_cluster_exit import body
from tests.test_stream_order import code


def test_the_flush_uses_the_page_it_checked():
    text = body(code("qs_quantize.cu"), "flush_kernel")
    assert text.count("group_slot(") == 1
    assert "(size_t)S.place" in text


def test_the_prefill_checks_the_pages_it_uses():
    text = body(code("qs_quantize.cu"), "prefill_kernel")
    assert re.search(r"own = group_slot\([^;]*\);\s*PS\.place\[tid\] = \(int\)own;\s*\}\s*"
                     r"if \(!pages_good\(own < 0\)\)", text)
    assert text.count("group_slot(") == 2  # those, and the whole prompt's in pages_good


def test_listed_units_use_one_lookup():
    assert body(code("qs_split.cuh"), "unit_place").count("group_slot(") == 1
