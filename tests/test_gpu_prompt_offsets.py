"""Offsets of prompt attention at the ends of 32 bits: rows of sequences that are out of range are zero."""
import pytest
import torch

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


@pytest.mark.parametrize("offsets", [[LOW, HIGH], [LOW, 4], [3, HIGH], [LOW, LOW, HIGH, HIGH], [LOW, 2, 5, HIGH]])
def test_rows_of_sequences_out_of_range_are_zero(q4, offsets):
    x = torch.ones((9, 18, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full((9, 14, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    q4.q4_prompt_attention(x[:, :14], x[:, 14:16], x[:, 16:], off, out=out)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    live = [(b, e) for b, e in zip(offsets, offsets[1:]) if 0 <= b < e <= 9]
    want = torch.zeros_like(out)
    for b, e in live:
        want[b:e] = 1.0  # every V row is ones
    assert torch.equal(out, want)
