"""The debug build's checks of the expert layer's kernels, read from the sources: the
routing checks the places that it computes, the grouped products theirs."""
import os

import pytest

from test_debug_checks_host import CSRC, sites


@pytest.mark.parametrize("name,at_least", [("moe.cu", 2), ("grouped.cu", 3)])
def test_kernels_hold_checks(name, at_least):
    assert len(sites(os.path.join(CSRC, name))) >= at_least
