"""CPU: the lists of sources that identify a kernel family's code."""
import os
import re

import pytest

from residual_add_normalization_gb300 import buildlib


def included(name, seen):
    """`name` and the headers of csrc/ that it includes, theirs among them."""
    path = os.path.join(buildlib.CSRC, name)
    if name in seen or not os.path.exists(path):
        return seen
    seen.add(name)
    with open(path) as f:
        for one in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
            included(one, seen)
    return seen


@pytest.mark.parametrize("family", sorted(buildlib.FAMILY_SOURCES))
def test_a_family_lists_every_header_that_its_sources_include(family):
    listed = set(buildlib.FAMILY_SOURCES[family])
    assert all(os.path.exists(os.path.join(buildlib.CSRC, f)) for f in listed)
    needed = set()
    for one in listed:
        included(one, needed)
    assert needed == listed
