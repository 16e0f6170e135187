"""A kernel begins while the grid before it still runs, so what that grid writes
is read behind the wait for it and by coherent loads.  Read-only loads may find
what a line held before; they are for weights, which no launch writes.  (Whether
one finds an old line depends on what shared its SM: this looks at the sources.)"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "iq4_xs_quantized_gb300", "csrc")
FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu*")))


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", FILES)
def test_read_only_loads_are_of_weights(name):
    code = _code(name)
    if name == "internal.cuh":  # the loader of a weight row's sub-block
        at = code.index("void wt_load_sub(")
        code = code[:at] + code[code.index("\n}\n", at):]
    assert "__ldg(" not in code
    assert not re.search(r"ld\.global(\.\w+)*\.nc\b", code)


@pytest.mark.parametrize("name", FILES)
def test_pointers_the_compiler_may_read_so_are_weights(name):
    for pointer in re.findall(r"\bconst\s+\w+\s*\*\s*(?:const\s+)?__restrict__\s+(\w+)", _code(name)):
        assert pointer == "w", pointer
