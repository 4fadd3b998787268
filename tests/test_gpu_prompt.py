"""Prompt attention on the GPU against the float64 oracle.

Bound per value.  Scores are fp32 sums of exact products: off by less than ds
= 2^-19 scale sum_d |q_d k_d|; weights are rounded to the type (u = 2^-8 for
bfloat16, 2^-11 for float16, and 2^-24 of the largest where float16 has no
normal numbers left) and the output once more; sums over keys are fp32:

    |o - o64| <= (4 max ds + u + 2^-16) * sum_j w_j |v_j| + 2^-22 max |v| + u |o64|."""
import numpy as np
import pytest
import torch

import synthetic
from oracle import attention as ref

pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


def _i32(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")


def _normal(seed, shape, dtype, sigma=1.0):
    return torch.from_numpy(synthetic.normal(seed, shape, sigma=sigma)).to(dtype)


def _check(o, q, k, v, scale, causal, dtype, what):
    """One sequence, vectorised over its rows per head; returns the worst share of the bound."""
    n, hq, d = q.shape
    m, h, _ = k.shape
    worst = 0.0
    if n == 0:
        return worst
    see = (np.arange(m)[None, :] <= np.arange(n)[:, None] + m - n) if causal else np.ones((n, m), bool)
    for x in range(hq):
        kk, vv, qq = k[:, x // (hq // h)], v[:, x // (hq // h)], q[:, x]
        if m == 0:
            assert not o[:, x].any(), what
            continue
        s = np.where(see, scale * (qq @ kk.T), -np.inf)
        top = s.max(-1, keepdims=True)
        e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
        total = e.sum(-1, keepdims=True)
        w = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
        want = w @ vv
        ds = 2.0 ** -19 * scale * np.where(see, np.abs(qq) @ np.abs(kk).T, 0.0).max(-1, keepdims=True)
        u = UNIT[dtype]
        bound = (4 * ds + u + 2.0 ** -16) * (w @ np.abs(vv)) + 2.0 ** -22 * np.abs(vv).max() + u * np.abs(want)
        err = np.abs(o[:, x] - want)
        bad = see.any(-1) == 0
        assert not o[bad, x].any(), "%s: rows that see nothing are zero" % what
        err[bad] = 0
        assert np.all(err <= bound), "%s head %d: %.3g of the bound at %s" % (
            what, x, (err / bound).max(), np.unravel_index(np.argmax(err / bound), err.shape))
        worst = max(worst, float((err / bound).max()))
    return worst


def _run(q4, seed, qlens, klens, heads, hq, d, dtype, causal=True, scale=None, sigma=1.0):
    q = _normal(seed, (sum(qlens), hq, d), dtype, sigma)
    k = _normal(seed + 1, (sum(klens), heads, d), dtype)
    v = _normal(seed + 2, (sum(klens), heads, d), dtype)
    qo, ko = np.concatenate([[0], np.cumsum(qlens)]), np.concatenate([[0], np.cumsum(klens)])
    out = torch.full((sum(qlens), hq, d), 9.0, dtype=dtype, device="cuda")
    q4.q4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), _i32(qo), _i32(ko), causal=causal, scale=scale, out=out)
    assert q4.q4_device_status() == q4.Q4_OK
    o = out.cpu().double().numpy()
    q, k, v = (x.double().numpy() for x in (q, k, v))
    scale = d ** -0.5 if scale is None else scale
    return max(_check(o[qo[s]:qo[s + 1]], q[qo[s]:qo[s + 1]], k[ko[s]:ko[s + 1]], v[ko[s]:ko[s + 1]], scale, causal,
                      dtype, "sequence %d" % s) for s in range(len(qlens)))


HEADS = [(4, 28, 128), (2, 14, 64), (8, 8, 64), (2, 2, 128), (1, 16, 128), (1, 3, 64)]


def test_the_oracles_agree():
    q, k, v = (synthetic.normal(i, s) for i, s in ((1, (5, 4, 8)), (2, (9, 2, 8)), (3, (9, 2, 8))))
    for causal in (True, False):
        o = ref.prompt(q, k, v, 0.3, causal)
        assert _check(o, q.astype(np.float64), k.astype(np.float64), v.astype(np.float64), 0.3, causal,
                      torch.float16, "oracle") < 1e-6


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,hq,d", HEADS)
@pytest.mark.parametrize("causal", [True, False])
def test_packed_prompts(q4, dtype, heads, hq, d, causal):
    lens = [1, 2, 17, 18, 19, 36, 37, 127, 128, 129, 0, 300]
    _run(q4, 10, lens, lens, heads, hq, d, dtype, causal)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,hq,d", HEADS[:3])
def test_one_longer_prompt(q4, dtype, heads, hq, d):
    _run(q4, 20, [1100], [1100], heads, hq, d, dtype)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,hq,d", HEADS[:3])
def test_rows_after_a_past_and_rows_that_see_nothing(q4, heads, hq, d, causal):
    # more keys than rows (a prompt's later piece), fewer (the first rows see nothing), none at all
    _run(q4, 30, [40, 200, 1, 5, 30], [500, 131, 1, 0, 3], heads, hq, d, torch.bfloat16, causal)


@pytest.mark.parametrize("sigma,scale", [(30.0, None), (1.0, 4.0), (1e-3, None)])
def test_sharp_and_flat_weights(q4, sigma, scale):
    _run(q4, 40, [333], [333], 2, 14, 128, torch.float16, sigma=sigma, scale=scale)


def test_rising_scores_rescale_the_sum(q4):
    # each block's scores lie far above the last one's, so the running maximum keeps growing
    n, d = 700, 64
    q = torch.ones((n, 1, d), dtype=torch.float16)
    k = (torch.arange(n).float()[:, None, None] * 0.05).expand(n, 1, d).half()
    v = _normal(51, (n, 1, d), torch.float16)
    off = _i32([0, n])
    o = q4.q4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), off)
    assert q4.q4_device_status() == q4.Q4_OK
    _check(o.cpu().double().numpy(), q.double().numpy(), k.double().numpy(), v.double().numpy(), d ** -0.5, True,
           torch.float16, "rising")


@pytest.mark.parametrize("heads,hq,d", [(4, 28, 128), (2, 14, 64)])
def test_views_of_one_tensor(q4, heads, hq, d):
    n = 150
    qkv = _normal(60, (n, hq + 2 * heads, d), torch.bfloat16).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:]
    off = _i32([0, 70, n])
    a = q4.q4_prompt_attention(q, k, v, off)
    b = q4.q4_prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), off)
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)  # head-major storage
    c = q4.q4_prompt_attention(q, kt, v, off)
    assert torch.equal(a, b) and torch.equal(a, c)
    assert q4.q4_device_status() == q4.Q4_OK


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_values_reach_only_rows_that_see_them(q4, bad, d):
    n, at, other = 300, 140, 31
    q, k, v = (_normal(70 + i, (n + other, h, d), torch.bfloat16) for i, h in enumerate((6, 2, 2)))
    clean = q4.q4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), _i32([0, n, n + other]))
    v[at, 1, 7] = bad                    # one value of one row
    k[n:, :], v[n:, :] = bad, bad        # the whole next sequence
    o = q4.q4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), _i32([0, n, n + other])).cpu()
    clean = clean.cpu()
    assert torch.equal(o[:at], clean[:at])
    assert torch.equal(o[:n, :3], clean[:n, :3])  # the other head's group
    col = o[at:n, 3:, 7].float()
    assert (torch.isnan(col) if np.isnan(bad) else ~torch.isfinite(col)).all()
    rest = [c for c in range(d) if c != 7]
    assert torch.equal(o[at:n, 3:][..., rest], clean[at:n, 3:][..., rest])
    assert not torch.isfinite(o[n:]).any()


def test_bad_key_in_the_future(q4):
    n, d = 200, 64
    q, k, v = (_normal(80 + i, (n, 2, d), torch.float16) for i in range(3))
    clean = q4.q4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), _i32([0, n])).cpu()
    k[150, :, 3] = float("nan")
    o = q4.q4_prompt_attention(q.cuda(), k.cuda(), v.cuda(), _i32([0, n])).cpu()
    assert torch.equal(o[:150], clean[:150]) and torch.isnan(o[150:]).all()


def test_rows_of_no_sequence_are_zero(q4):
    d = 64
    q, k, v = (_normal(90 + i, (50, 2, d), torch.bfloat16).cuda() for i in range(3))
    out = torch.full((50, 2, d), 5.0, dtype=torch.bfloat16, device="cuda")
    q4.q4_prompt_attention(q, k, v, _i32([4, 20, 44]), _i32([0, 16, 40]), out=out)
    assert q4.q4_device_status() == q4.Q4_OK
    assert not out[:4].any() and not out[44:].any() and out[4:44].any(-1).all()
    # a sequence whose keys lie outside is left out
    q4.q4_prompt_attention(q, k, v, _i32([0, 20, 50]), _i32([0, 20, 51]), out=out)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    assert not out[20:].any() and out[:20].any(-1).all()


def test_output_aligned_to_16_bytes_only(q4):
    q, k, v = (_normal(92 + i, (70, h, 128), torch.bfloat16).cuda() for i, h in enumerate((4, 2, 2)))
    off = _i32([0, 70])
    want = q4.q4_prompt_attention(q, k, v, off)
    room = torch.zeros(70 * 4 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    out = room[8:].view(70, 4, 128)
    assert out.data_ptr() % 32 == 16
    assert torch.equal(q4.q4_prompt_attention(q, k, v, off, out=out), want)


def test_one_row_and_no_keys(q4):
    _run(q4, 93, [1], [1], 2, 14, 64, torch.float16)
    _run(q4, 94, [3], [0], 1, 4, 128, torch.bfloat16)


def test_keys_shared_by_stride_zero(q4):
    # an expanded view: every head of k and v is one head's rows
    q, k, v = (_normal(96 + i, (140, h, 64), torch.bfloat16).cuda() for i, h in enumerate((4, 1, 1)))
    off = _i32([0, 140])
    want = q4.q4_prompt_attention(q, k.repeat(1, 2, 1), v.repeat(1, 2, 1), off)
    assert torch.equal(q4.q4_prompt_attention(q, k.expand(-1, 2, -1), v.expand(-1, 2, -1), off), want)


def test_waits_run_out_and_the_next_call_is_right(q4):
    q, k, v = (_normal(98 + i, (700, h, 128), torch.bfloat16).cuda() for i, h in enumerate((8, 2, 2)))
    off = _i32([0, 200, 700])
    want = q4.q4_prompt_attention(q, k, v, off)
    torch.cuda.synchronize()
    q4.q4mm_set_wait_limit_ns(1000000)
    q4.q4mm_set_stall_for_test(True)
    try:
        q4.q4_prompt_attention(q, k, v, off)
        assert q4.q4_device_status() == q4.Q4_ERR_TIMEOUT
    finally:
        q4.q4mm_set_stall_for_test(False)
        q4.q4mm_set_wait_limit_ns(0)
    assert torch.equal(q4.q4_prompt_attention(q, k, v, off), want)
    assert q4.q4_device_status() == q4.Q4_OK


def test_many_short_sequences(q4):
    lens = [1 + (7 * i) % 5 for i in range(700)]
    _run(q4, 95, lens, lens, 1, 4, 64, torch.bfloat16)


def test_deterministic_on_another_stream(q4):
    q, k, v = (_normal(97 + i, (900, h, 128), torch.bfloat16).cuda() for i, h in enumerate((28, 4, 4)))
    off = _i32([0, 333, 900])
    a = q4.q4_prompt_attention(q, k, v, off)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        outs = [q4.q4_prompt_attention(q, k, v, off) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(a, o) for o in outs)


def test_refusals(q4):
    x = torch.zeros((8, 4, 64), dtype=torch.float16, device="cuda")
    off = _i32([0, 8])
    for call in (lambda: q4.q4_prompt_attention(x.float(), x.float(), x.float(), off),
                 lambda: q4.q4_prompt_attention(x, x, x.bfloat16(), off),
                 lambda: q4.q4_prompt_attention(x, x[:, :3], x[:, :3], off),
                 lambda: q4.q4_prompt_attention(x, x, x[:7], off),
                 lambda: q4.q4_prompt_attention(x, x, x, off.long()),
                 lambda: q4.q4_prompt_attention(x, x, x, off, _i32([0])),
                 lambda: q4.q4_prompt_attention(x.cpu(), x.cpu(), x.cpu(), off.cpu())):
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros((8, 4, 68), dtype=torch.float16, device="cuda")[..., :64]  # 136-byte heads
    y = torch.zeros((8, 4, 96), dtype=torch.float16, device="cuda")
    for call, status in ((lambda: q4.q4_prompt_attention(wide, x, x, off), q4.Q4_ERR_ALIGN),
                         (lambda: q4.q4_prompt_attention(y, y, y, off), q4.Q4_ERR_SHAPE),
                         (lambda: q4.q4_prompt_attention(x, x, x, off, scale=-1.0), q4.Q4_ERR_INVALID_ARG)):
        with pytest.raises(q4.Q4Error) as e:
            call()
        assert e.value.status == status
    assert q4.q4_prompt_attention(x[:0], x, x, _i32([0, 0]), off).shape == (0, 4, 64)
