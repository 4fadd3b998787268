"""The 4-bit-cache example end to end: prompts, decode steps and eviction."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__

    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_q4_cache

    return decode_q4_cache


def test_serving_is_deterministic_and_within_budget(example):
    lengths, steps, keep = [120, 7, 64, 1], 24, 48
    a, held = example.serve(lengths, steps, keep, recent=8, quiet=True)
    b, _ = example.serve(lengths, steps, keep, recent=8, quiet=True)
    assert torch.equal(a, b)
    assert a.shape == (4, steps + 1) and (a >= 0).all() and (a < example.VOCAB).all()
    for pos in held:
        # thinned out at steps 0 and 12 of the 24: at most keep rows then, one more a step since
        assert (pos <= keep + 12).all() and pos[3] == 1 + steps


def test_steps_without_eviction_hold_every_row(example):
    tokens, held = example.serve([33, 2], 5, keep=500, quiet=True)
    assert [p.tolist() for p in held] == [[38, 7]] * example.LAYERS
