"""Prompt attention where weights or scores span many binades, against float64.

Bound.  As in test_gpu_prompt.py, with the term for small weights written out: a
float16 weight is held to half of 2^-24 after it was taken by 2^7 relative to a
reference that is no larger than the row's largest weight, so to 2^-32 of
that, and n keys may all be off the same way:

    |o - o64| <= (4 max ds + u + 2^-16) * sum_j w_j |v_j| + n 2^-32 max |v| + u |o64| (+ 2^-25, float16's half step at 0)."""
import numpy as np
import pytest
import torch

import synthetic

pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _values(q4, q, k, v, scale, dtype):
    """o [rows, d] of one head whose rows q all see all of k, v, and the inputs as the kernel got them."""
    q, k, v = (torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype) for x in (q, k, v))
    o = q4.q4_prompt_attention(q.cuda()[:, None], k.cuda()[:, None], v.cuda()[:, None], _i32(0, len(q)),
                               _i32(0, len(k)), causal=False, scale=scale)
    assert q4.q4_device_status() == q4.Q4_OK
    return o.cpu().double().numpy()[:, 0], [x.double().numpy() for x in (q, k, v)]


def _check(o, q, k, v, scale, dtype):
    s = scale * (q @ k.T)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    want = w @ v
    u = UNIT[dtype]
    ds = 2.0 ** -19 * scale * (np.abs(q) @ np.abs(k).T).max(-1, keepdims=True)
    bound = (4 * ds + u + 2.0 ** -16) * (w @ np.abs(v)) + u * np.abs(want)
    if dtype == torch.float16:
        bound = bound + len(k) * 2.0 ** -32 * np.abs(v).max() + 2.0 ** -25
    err = np.abs(o - want)
    assert np.all(err <= bound), "%.3g of the bound at %s" % ((err / bound).max(),
                                                              np.unravel_index(np.argmax(err / bound), err.shape))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [65, 1000, 16384])
@pytest.mark.parametrize("bits", [12, 18, 21, 24, 26])
@pytest.mark.parametrize("spread", [0.0, 0.02])
def test_one_heavy_key_without_a_value(q4, dtype, d, n, bits, spread):
    # all that counts lies about `bits` binades below the row's largest weight
    q = np.zeros((3, d), np.float32)
    q[:, 0], q[:, 1] = 16.0, [0.3, 1.0, 4.0]
    k, v = synthetic.normal(940, (n, d), sigma=spread), 1 + synthetic.normal(941, (n, d), sigma=0.1)
    k[0], v[0] = 0.0, 0.0
    k[0, 0] = bits * np.log(2.0) / 16
    o, (q, k, v) = _values(q4, q, k, v, 1.0, dtype)
    _check(o, q, k, v, 1.0, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("step", [0.5, 3.0, 7.0, 9.0, 40.0])
@pytest.mark.parametrize("falling", [False, True])
def test_references_that_change_by_little_and_by_much(q4, dtype, step, falling):
    # the scores of each block of keys lie `step` binades above (below) the last one's
    n, d, scale = 1200, 64, 0.125
    q, k, v = np.zeros((5, d), np.float32), synthetic.normal(950, (n, d), sigma=0.05), synthetic.normal(951, (n, d))
    q[:, 0], q[:, 1:] = 8.0, synthetic.normal(952, (5, d - 1))
    k[:, 0] = step * np.log(2.0) * (np.arange(n) // 128)
    if falling:
        k = k[::-1]
    o, (q, k, v) = _values(q4, q, k, v, scale, dtype)
    _check(o, q, k, v, scale, dtype)
