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


@pytest.mark.parametrize("dtype,q0,k0,scale", [
    (torch.float16, 128.0, 128.0, 8.0),         # scores to 2^25
    (torch.float16, 128.0, 128.0, 4096.0),      # 2^34
    (torch.bfloat16, 2.0 ** 20, 2.0 ** 20, 0.125),  # 2^45
    (torch.bfloat16, 2.0 ** 30, 2.0 ** 50, 1.0),    # 2^88
    (torch.float16, 4.0, 4.0, 64.0)])           # 2^18: ordinary ones
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_scores_far_from_one_another_and_from_zero(q4, dtype, q0, k0, scale, order):
    # distinct integers times powers of two: exact scores, the largest far above the others, and one pair of equals
    n, d = 254, 64
    of = np.arange(1, n + 1)
    if order == "falling":
        of = of[::-1]
    if order == "mixed":
        of = np.random.default_rng(3).permutation(n) + 1
    q, k, v = np.zeros((2, d)), np.zeros((n, d)), synthetic.normal(960, (n, d))
    q[:, 0], k[:, 0] = [q0, -q0], k0 * of
    k[7] = k[200] = 0
    k[7, 0] = k[200, 0] = k0 * 255  # the largest, twice
    o, (q, k, v) = _values(q4, q, k, v, scale, dtype)
    least = int(np.argmin(k[:, 0]))
    want = np.stack([(v[7] + v[200]) / 2, v[least]])
    size = np.stack([(np.abs(v[7]) + np.abs(v[200])) / 2, np.abs(v[least])])
    u = UNIT[dtype]  # the weights' rounding and the output's
    assert np.all(np.abs(o - want) <= (u + 2.0 ** -16) * size + u * np.abs(want))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sigma", [300.0, 4000.0, 20000.0])
def test_large_queries_and_keys(q4, dtype, sigma):
    # scores of 10^5 to 10^9: one key has all the weight of its row
    n, d = 500, 128
    q, k, v = (synthetic.normal(970 + i, s, sigma=g) for i, s, g in ((0, (40, d), sigma), (1, (n, d), sigma), (2, (n, d), 1.0)))
    q, k = np.clip(q, -60000, 60000), np.clip(k, -60000, 60000)
    o, (q, k, v) = _values(q4, q, k, v, d ** -0.5, dtype)
    s = q @ k.T * d ** -0.5
    first, second = np.sort(s, -1)[:, -1], np.sort(s, -1)[:, -2]
    # rows where fp32 sums of the scores cannot mix up the first two, nor leave the second any weight
    clear = first - second > 50 + 2.0 ** -18 * d ** -0.5 * (np.abs(q) @ np.abs(k).T).max(-1)
    assert clear.sum() > 20
    want, u = v[np.argmax(s, -1)][clear], UNIT[dtype]
    assert np.all(np.abs(o[clear] - want) <= (2 * u + 2.0 ** -16) * np.abs(want))
    assert np.isfinite(o).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_of_small_and_large_scores_in_one_tile(q4, dtype, d, causal):
    # Row r's scores are 2^(r / 10) times those of row 0, one exact product each, and they grow along the keys; so
    # references grow within a row and rows pass from ordinary ones to those far from zero.  What is left of errors
    # is 2^-12 where the reference's step counts (4096 units of log2), the weights' rounding and the output's.
    n, scale = 700, 1.0
    grow = 2.0 ** (np.arange(n) // 128) * (1 + (np.arange(n) * 37 % 128) / 128)  # 8 significant bits
    q, k, v = np.zeros((n, d)), np.zeros((n, d)), synthetic.normal(980, (n, d))
    q[:, 0] = 2.0 ** (np.arange(n) % 210 // (10 if dtype == torch.bfloat16 else 14)) * np.where(np.arange(n) % 3, 1, -1)
    k[:, 0] = grow / 64
    q, k, v = (torch.from_numpy(np.asarray(x, np.float32)).to(dtype) for x in (q, k, v))
    off = _i32(0, n)
    o = q4.q4_prompt_attention(q.cuda()[:, None], k.cuda()[:, None], v.cuda()[:, None], off, causal=causal, scale=scale)
    assert q4.q4_device_status() == q4.Q4_OK
    o = o.cpu().double().numpy()[:, 0]
    q, k, v = (x.double().numpy() for x in (q, k, v))
    s = np.where(np.tri(n, dtype=bool) | (not causal), q @ k.T * scale, -np.inf)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    u = UNIT[dtype]
    bound = (u + 2.0 ** -12) * (w @ np.abs(v)) + u * np.abs(w @ v) + n * 2.0 ** -32 * np.abs(v).max()
    err = np.abs(o - w @ v)
    assert np.all(err <= bound), "%.3g of the bound at %s" % ((err / bound).max(),
                                                              np.unravel_index(np.argmax(err / bound), err.shape))


@pytest.mark.parametrize("heads,hq,d", [(4, 28, 128), (2, 14, 64), (8, 8, 64)])
def test_output_in_place_of_the_queries(q4, heads, hq, d):
    n = 700
    q, k, v = (torch.from_numpy(synthetic.normal(990 + i, (n, h, d))).bfloat16().cuda()
               for i, h in enumerate((hq, heads, heads)))
    off = _i32(0, 1, 130, 400, n)
    want = q4.q4_prompt_attention(q, k, v, off)
    room = q.clone()
    assert torch.equal(q4.q4_prompt_attention(room, k, v, off, out=room), want)
    if heads == hq:
        for call in (lambda: q4.q4_prompt_attention(q, k, v, off, out=k), lambda: q4.q4_prompt_attention(q, k, v, off, out=v)):
            with pytest.raises(q4.Q4Error) as e:
                call()
            assert e.value.status == q4.Q4_ERR_INVALID_ARG
    assert q4.q4_device_status() == q4.Q4_OK
