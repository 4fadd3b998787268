"""Offsets of the paged attention at the ends of 32 bits: rows of requests that are out of range are zero."""
import pytest
import torch

from test_gpu_paged import Step, _i32

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


@pytest.mark.parametrize("idle", [0, 200])
@pytest.mark.parametrize("offsets", [[LOW, HIGH], [LOW, 4], [3, HIGH], [LOW, LOW, HIGH, HIGH], [LOW, 2, 5, HIGH]])
def test_rows_of_requests_out_of_range_are_zero(q4, offsets, idle):
    # one warp looks through up to 128 requests, all threads through more
    s = Step(q4, 200, [40] + [20] * (2 + idle), [9] + [0] * (2 + idle), 2, 14, 64, 16, torch.bfloat16)
    offsets = offsets + [offsets[-1]] * idle
    out = torch.full((9, 14, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q4.q4_paged_attention(s.cache, s.tables, s.q.cuda(), _i32(offsets), _i32(s.slot[:len(offsets) - 1]),
                          _i32([30] * (len(offsets) - 1)), out=out)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    live = [i for i, (b, e) in enumerate(zip(offsets, offsets[1:])) if 0 <= b < e <= 9]
    rows = sorted(x for i in live for x in range(offsets[i], offsets[i + 1]))
    zero = [x for x in range(9) if x not in rows]
    assert not out[zero].any() and bool(out[rows].ne(7.0).any(-1).all())
