"""What the two libraries share: a source compiled once has nothing that PW_CHECK changes."""
import os
import re

import pytest

from any_precision_weight_gb300 import build


def _text(name, seen):
    """A source with the sources it includes."""
    seen.add(name)
    text = open(os.path.join(build.CSRC, name)).read()
    for inc in re.findall(r'#include "(\w+\.\w+)"', text):
        if inc not in seen and os.path.exists(os.path.join(build.CSRC, inc)):
            text += _text(inc, seen)
    return text


@pytest.mark.parametrize("name", sorted(build.SOURCES))
def test_sources_compiled_once_have_no_checked_form(name):
    if name in build.UNCHECKED:
        assert "PW_CHECK" not in _text(name, set())
    elif name in ("pw_decode.cu", "pw_prefill.cu", "pw_kernels.cu"):
        assert "PW_CHECK" in _text(name, set())
