"""Bounded waits of the paged attention at heads of 128, whose copies go another way than those of 64."""
import pytest
import torch

from test_gpu_paged import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


@pytest.mark.parametrize("past,rows", [([3000, 40], [1, 1]), ([500, 900], [300, 1]), ([300], [20])])
def test_waits_that_run_out(q4, past, rows):
    """No copy is issued, so every wait for one runs out: the status says so, and later calls are right."""
    s = Step(q4, 151, past, rows, 4, 28, 128, 16, torch.float16)
    want = s.run().clone()
    assert q4.q4_device_status() == q4.Q4_OK
    q4.q4mm_set_wait_limit_ns(20_000_000)
    q4.q4mm_set_stall_for_test(True)
    try:
        s.run()
        status = q4.q4_device_status()
    finally:
        q4.q4mm_set_stall_for_test(False)
        q4.q4mm_set_wait_limit_ns(0)
    assert status == q4.Q4_ERR_TIMEOUT and q4.q4_device_status() == q4.Q4_OK
    for _ in range(2):
        assert torch.equal(s.run(), want)
    s.check(want)
