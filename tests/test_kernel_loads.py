"""What the kernels' bulk copies may not be, read as text: none is handed to
several CTAs of a cluster at once.  Such a copy is for memory of this GPU alone,
and an entry point takes any address that the device reads."""
import os
import re

import pytest

from optimizer_state_gb300 import build


def statements(name):
    """The instructions in a source file's string literals."""
    with open(os.path.join(build.CSRC, name)) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    joined = re.sub(r'"\s*"', "", text)                  # adjacent literals are one
    return [x for lit in re.findall(r'"((?:[^"\\]|\\.)*)"', joined) for x in lit.split(";")]


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(build.CSRC)
                                        if n.endswith((".cu", ".cuh", ".h"))))
def test_no_bulk_copy_goes_to_several_ctas(name):
    bulk = [x for x in statements(name) if "cp.async.bulk" in x or "cp.reduce.async.bulk" in x]
    assert [x for x in bulk if "multicast" in x] == []
    if name == "z3_mma.cuh":
        assert any("cp.async.bulk.tensor.2d" in x for x in bulk)      # the text is found at all
