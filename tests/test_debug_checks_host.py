"""The debug build's checks in the sources, without a GPU: the multi-axis rotary,
cache and attention kernels hold some, and a site number names one check."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rmsnorm_linear_projection_gb300", "csrc")


def sites(path):
    """Site numbers of the RNL_DCHECK calls of a file (their last argument)."""
    text = open(path).read()
    found = []
    for m in re.finditer(r"RNL_DCHECK\(&", text):
        depth, i = 0, text.index("(", m.start())
        for j in range(i, len(text)):
            depth += {"(": 1, ")": -1}.get(text[j], 0)
            if depth == 0:
                break
        found.append(text[i + 1:j].rsplit(",", 1)[1].strip())
    return found


@pytest.mark.parametrize("name,at_least", [("ropeaxes.cu", 2), ("kv4cache.cu", 2), ("kv4attn.cu", 3), ("kv4prompt.cu", 5)])
def test_kernels_hold_checks(name, at_least):
    assert len(sites(os.path.join(CSRC, name))) >= at_least


def test_new_site_numbers_name_one_check():
    files = {}
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        for s in sites(path):
            if s.isdigit() and int(s) >= 100:
                assert s not in files and int(s) < 256
                files[s] = path
    assert len(files) >= 12
