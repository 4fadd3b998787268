"""Sizes that the calls of the paged cache refuse are refused where the cache is made (CPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


@pytest.mark.parametrize("pages,heads,head_dim,page_size", [(0, 1, 64, 16), (-1, 1, 64, 16), (1, 0, 64, 16), (1, 1, 96, 16),
                                                            (1, 1, 0, 16), (1, 1, 256, 16), (1, 1, 64, 24),
                                                            (1, 1, 64, 8), (1, 1, 128, 256)])
def test_sizes_that_are_refused(q4, pages, heads, head_dim, page_size):
    with pytest.raises(ValueError):
        q4.Q4PagedCache(pages, heads, head_dim, page_size, device="cpu")


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
def test_sizes_that_are_taken(q4, head_dim, page_size):
    c = q4.Q4PagedCache(3, 2, head_dim, page_size, dtype=torch.float16, device="cpu")
    assert c.k.shape == c.v.shape == (3, 2, page_size, head_dim) and c.nbytes == 3 * 2 * page_size * head_dim * 4
