"""Order of the launches of the 4-bit cache, read from the kernels' source (CPU).

A launch that begins early is ordered by its own ``griddepcontrol.wait`` only,
and that wait is for the launch before it.  The join and the weights' launch
read the step's description, the queries and the cache before their waits, so
the first launch of the call may let them begin only when everything ahead of
the call has ended: its trigger comes after its wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_matmul_gb300", "csrc")
WAIT, TRIGGER = "griddepcontrol.wait", "griddepcontrol.launch_dependents"
# launched behind kvq_attention_kernel by the same call: what they read early is older than that launch
BEHIND_THE_FIRST = {"kvq_join_kernel", "kvq_mass_kernel"}


def kernels():
    """Bodies of the cache's kernels by name, without comments."""
    found = {}
    for name in ("q4_kvq.cu", "q4_kvq_attention.cu", "q4_kvq_evict.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__\s+void\s+(?:__\w+__\([^)]*\)\s*)*(\w+)\([^)]*\)\s*\{", text):
            depth, at = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            found[m.group(1)] = text[m.end():at]
    return found


KERNELS = kernels()


def test_all_kernels_are_found():
    assert set(KERNELS) == {"kvq_append_kernel", "kvq_read_kernel", "kvq_read_groups_kernel", "kvq_attention_kernel",
                            "kvq_join_kernel", "kvq_mass_kernel", "evict_select_kernel", "evict_move_kernel"}


@pytest.mark.parametrize("name", sorted(set(KERNELS) - BEHIND_THE_FIRST))
def test_a_launch_that_waits_lets_others_begin_after_its_wait(name):
    body = KERNELS[name]
    if WAIT in body and TRIGGER in body:
        assert body.index(WAIT) < body.index(TRIGGER)


@pytest.mark.parametrize("name", ["kvq_read_kernel", "kvq_read_groups_kernel", "kvq_attention_kernel",
                                  "evict_move_kernel"])
def test_nothing_is_read_before_the_wait_of_a_call(name):
    # up to the wait: no arguments' memory, only shared memory and barriers
    before = KERNELS[name][:KERNELS[name].index(WAIT)]
    assert not re.search(r"__ld|plan_range|kvq_find|kvq_request|load_|a\.(offsets|slot|pos|src|dst|len|new_len|kept)\b",
                         before)


def test_the_join_and_the_weights_wait_on_every_path():
    # the joined rows return from inside a branch that has a wait of its own
    assert KERNELS["kvq_join_kernel"].count(WAIT) == 2
    assert KERNELS["kvq_mass_kernel"].count(WAIT) == 2


# The read-only path (__ldg, and what the compiler may make of a plain load) is for memory that
# nobody writes while the kernel lives; a launch that begins early lives beside its predecessors.
EARLY = ["kvq_read_kernel", "kvq_read_groups_kernel", "kvq_attention_kernel", "kvq_join_kernel", "kvq_mass_kernel",
         "evict_move_kernel"]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_launches_that_begin_early_read_past_the_read_only_path():
    for name in EARLY:
        assert "__ldg" not in KERNELS[name], name
        assert "kvq_find_request(" not in KERNELS[name] and "kvq_request(" not in KERNELS[name], name
    assert "__ldg" not in source("q4_kvq_attention.cu")
    # the shared helpers take the kind of load as an argument, and these kernels ask for an ordinary one
    helpers = source("q4_kvq_attention.cu") + "".join(KERNELS[n] for n in EARLY)
    asked = re.findall(r"kvq_(?:find_request|request|load8)<(\w+)>", helpers)
    assert asked and set(asked) == {"true"}
    assert not re.search(r"kvq_(find_request|request|load8)\(", helpers)


def test_the_move_reads_what_the_select_wrote_by_loads_that_stay_ordinary():
    assert not re.search(r"= a\.(new_len|src|dst|len|kept)\[|\bkept\[|== a\.len\[", KERNELS["evict_move_kernel"])
