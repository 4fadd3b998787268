"""The paged-cache example end to end: pieces of prompts beside decode rows, pages given out and taken back."""
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
    import serve_paged_cache

    return serve_paged_cache


@pytest.mark.parametrize("budget,pages,page_size", [(96, 64, 16), (17, 30, 16), (500, 8, 128)])
def test_serving_is_deterministic_and_returns_its_pages(example, budget, pages, page_size):
    lengths, new = [120, 7, 64, 1, 200, 33], 9
    a, steps, free = example.serve(lengths, new, pages=pages, page_size=page_size, budget=budget)
    b, again, _ = example.serve(lengths, new, pages=pages, page_size=page_size, budget=budget)
    assert torch.equal(a, b) and steps == again
    assert a.shape == (6, new) and (a >= 0).all() and (a < example.VOCAB).all()
    assert free == pages
