"""The kernels' dispatch rules ask the device for its number of SMs."""
import re

import pytest

from tests.test_stream_order import SOURCES, code


@pytest.mark.parametrize("name", SOURCES)
def test_no_number_of_sms_in_the_sources(name):
    """152, the SMs of the GPU they were measured on, stands in comments alone."""
    assert not re.findall(r"\b152\b", code(name))
