"""What the kernel sources may not hold, read as text.

Kernels are launched with programmatic stream serialisation: one may be
resident while the kernel before it still writes what it will read.  The
non-coherent load path (ld.global.nc, __ldg, which the compiler may also move
across the wait for that kernel) is for memory that nothing writes while the
reading kernel runs, so it is no path for buffers that a library call writes."""
import os
import re

import pytest

from optimizer_state_gb300 import build

NON_COHERENT = re.compile(r"__ldg\b|__ldlu\b|\bld\.global(?:\.\w+)*\.nc\b|\bldu\.global\b")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(build.CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(build.CSRC)
                                        if n.endswith((".cu", ".cuh", ".h"))))
def test_no_non_coherent_loads(name):
    assert NON_COHERENT.findall(code(name)) == []
    # the compiler may load through a const __restrict__ pointer that way
    assert re.findall(r"const\s+\w+\s*\*\s*__restrict__\s*\w+", code(name)) == []


def test_every_kernel_waits_before_it_releases_the_next():
    """The early variants of kernels read before they wait for their primary.
    They may, as long as no kernel lets the next one start before it has
    itself waited: then all that came before the primary is complete."""
    order = [x for name in sorted(os.listdir(build.CSRC)) if name.endswith((".cu", ".cuh", ".h"))
             for x in re.findall(r"griddepcontrol\.(\w+)", code(name))]
    assert order and order == ["wait", "launch_dependents"] * (len(order) // 2)
