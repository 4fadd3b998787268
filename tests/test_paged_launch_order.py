"""Order of the launches of the paged attention, read from the kernels' source (CPU).

Both launches begin under the end of the one before.  Nothing that the call is
given is read before the wait, by loads that stay ordinary ones, and others begin only after it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_matmul_gb300", "csrc")
WAIT, TRIGGER = "griddepcontrol.wait", "griddepcontrol.launch_dependents"


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels():
    found, text = {}, source("q4_paged_attention.cu")
    for m in re.finditer(r"__global__\s+void\s+(?:__\w+__\([^)]*\)\s*)*(\w+)\(", text):
        at = text.index("{", text.index(")", m.end()))
        start, depth = at + 1, 1
        while depth:
            at += 1
            depth += {"{": 1, "}": -1}.get(text[at], 0)
        found[m.group(1)] = text[start:at]
    return found


KERNELS = kernels()


def test_the_kernels_are_found():
    assert set(KERNELS) == {"paged_kernel", "paged_join_kernel"}


@pytest.mark.parametrize("name", ["paged_kernel", "paged_join_kernel"])
def test_others_begin_after_the_wait(name):
    body = KERNELS[name]
    assert body.count(WAIT) == 1 and body.count(TRIGGER) == 1 and body.index(WAIT) < body.index(TRIGGER)


@pytest.mark.parametrize("name", ["paged_kernel", "paged_join_kernel"])
def test_nothing_is_read_before_the_wait(name):
    before = KERNELS[name][:KERNELS[name].index(WAIT)]
    assert not re.search(r"ld_int|__ld|load_request|a\.(offsets|slot|pos|table|out|ws|status)\b", before)


def test_loads_stay_ordinary():
    text = source("q4_paged_attention.cu")
    assert "__ldg" not in text
    # numbers of the step come by one kind of load, sums of pieces past the first-level cache
    assert not re.search(r"a\.(offsets|slot|pos|table)\[", text)
    assert not re.search(r"= a\.ws\.(ml|partial|joins)\[", KERNELS["paged_join_kernel"])
