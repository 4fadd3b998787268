"""Attention over the 4-bit cache where V or the weights span many binades, against float64.

Bound.  As in test_gpu_kvq.py, with one term more: a weight times V's scale is
held in two binary16 terms, whose last place is 2^-24 however small they are.
Relative to a weight of 1 (the row's largest is no less) the weight is taken by 2^9 and the
scale by 1 / T, T the largest scale of the request's head so far as a power of two
(2^-14 at least); three roundings of half a place, codes of 8 at most:

    8 * 3 * 2^-25 * 2^-9 * T <= 2^-29 T  per key,

with T <= 2 max |scale|.  So, per value,

    |o - o64| <= (4 max ds + 2^-18 + (n / 16 + 64) 2^-22) * sum_p w_p 16 |s_v| + n 2^-29 T + u |o64|."""
import numpy as np
import pytest
import torch

import synthetic
from oracle import attention as ref

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _check(o, q, k, v, dtype, what):
    """One row o, q [hq, d] over all of k, v [n, heads, d]; every value."""
    n, heads, d = k.shape
    hq = q.shape[0]
    ck, sk = ref.encode(k)
    cv, sv = ref.encode(v)
    k64, v64 = ref.decode(ck, sk), ref.decode(cv, sv)
    wide_k = 16 * np.repeat(np.abs(sk.astype(np.float64)), 32, -1)
    wide_v = 16 * np.repeat(np.abs(sv.astype(np.float64)), 32, -1)
    scale, worst = d ** -0.5, 0.0
    for x in range(hq):
        h = x // (hq // heads)
        s = scale * (k64[:, h] @ q[x])
        w = np.exp(s - s.max())
        w /= w.sum()
        want = w @ v64[:, h]
        ds = 2.0 ** -18 * scale * (wide_k[:, h] @ np.abs(q[x])).max()
        top = max(2 * np.abs(sv[:, h].astype(np.float64)).max(), 2.0 ** -14)
        bound = (4 * ds + 2.0 ** -18 + (n / 16 + 64) * 2.0 ** -22) * (w @ wide_v[:, h])
        bound = bound + n * 2.0 ** -29 * top + UNIT[dtype] * np.abs(want) + 2.0 ** -25 * (dtype == torch.float16)
        err = np.abs(o[x] - want)
        assert np.all(err <= bound), "%s, head %d: %.3g of the bound" % (what, x, (err / bound).max())
        worst = max(worst, float((err / bound).max()))
    return worst


def _attend_all(q4, q, k, v, dtype, what, requests=1):
    """Requests that all cache the rows k, v [n, heads, d] and ask with q [1, hq, d] on the last of them."""
    n, heads, d = k.shape
    cache = q4.Q4KVCache(requests, heads, d, n)
    q, k, v = (torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype) for x in (q, k, v))
    slots = _i32(*range(requests))
    rows = _i32(*[n * i for i in range(requests + 1)])
    q4.q4_kvq_append(cache, k.cuda().repeat(requests, 1, 1), v.cuda().repeat(requests, 1, 1), rows, slots,
                     _i32(*[0] * requests))
    o = q4.q4_kvq_attention(cache, q.cuda().repeat(requests, 1, 1), _i32(*range(requests + 1)), slots,
                            _i32(*[n - 1] * requests)).cpu().double().numpy()
    assert q4.q4_device_status() == q4.Q4_OK
    q, k, v = q.double().numpy()[0], k.float().numpy(), v.float().numpy()
    return max(_check(o[r], q, k, v, dtype, what) for r in {0, requests - 1})


HEADS = [(4, 28, 128), (2, 14, 64)]


@pytest.mark.parametrize("sigma", [1e-6, 1e-5, 1e-3, 3000.0])
@pytest.mark.parametrize("heads,hq,d", HEADS)
@pytest.mark.parametrize("n", [1, 9, 40, 700])
def test_small_and_large_values(q4, sigma, heads, hq, d, n):
    q, k = synthetic.normal(900, (1, hq, d)), synthetic.normal(901, (n, heads, d))
    _attend_all(q4, q, k, synthetic.normal(902, (n, heads, d), sigma=sigma), torch.float32, "sigma %g" % sigma)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,hq,d", HEADS)
@pytest.mark.parametrize("bits", [6, 12, 16, 20])
@pytest.mark.parametrize("n,sigma", [(40, 1.0), (40, 2.0 ** -8), (700, 2.0 ** -8), (5000, 1.0)])
def test_one_heavy_key_without_a_value(q4, dtype, heads, hq, d, bits, n, sigma):
    # all that counts lies `bits` binades below the row's largest weight
    q = np.repeat(synthetic.normal(910, (1, heads, d)), hq // heads, 1) + synthetic.normal(911, (1, hq, d), sigma=0.05)
    k, v = synthetic.normal(912, (n, heads, d), sigma=0.2), synthetic.normal(913, (n, heads, d), sigma=sigma)
    at = n // 3
    k[at] = bits * np.log(2.0) / np.sqrt(d) * q[0].reshape(heads, hq // heads, d)[:, 0]
    v[at] = 0.0
    _attend_all(q4, q, k, v, dtype, "%d binades" % bits)


@pytest.mark.parametrize("heads,hq,d", HEADS)
@pytest.mark.parametrize("falling", [False, True])
def test_values_that_grow_or_shrink_along_the_cache(q4, heads, hq, d, falling):
    # the scales' power of two changes again and again within one warp's tiles
    n = 6000
    q, k, v = (synthetic.normal(920 + i, s) for i, s in enumerate([(1, hq, d), (n, heads, d), (n, heads, d)]))
    v = v * np.float32(2.0) ** np.linspace(-20, 12, n, dtype=np.float32)[:, None, None]
    _attend_all(q4, q, k, v[::-1] if falling else v, torch.float32, "growing")


@pytest.mark.parametrize("falling", [False, True])
def test_several_tiles_of_changing_scales_a_warp(q4, falling):
    # 12,032 tiles: more than the launch has warps, so each takes a run of them
    heads, hq, d, n = 8, 8, 64, 3000
    q, k, v = (synthetic.normal(930 + i, s) for i, s in enumerate([(1, hq, d), (n, heads, d), (n, heads, d)]))
    v = v * np.float32(2.0) ** np.linspace(-18, 6, n, dtype=np.float32)[:, None, None]
    _attend_all(q4, q, k, v[::-1] if falling else v, torch.float32, "runs", requests=16)


@pytest.mark.parametrize("heads,hq,d", HEADS)
@pytest.mark.parametrize("n,order", [(30, "mixed"), (254, "rising"), (254, "falling"), (3000, "mixed"), (3000, "rising")])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_far_from_zero(q4, heads, hq, d, n, order, sign):
    # One exact product each: 8 significant bits of the key, powers of two up to 2^60 of the query, so that scores go
    # from a few to far past 2^24.  A score is off by 2^-23 of itself, which shows in weights only while neighbours
    # are less than 40 apart, so up to scores of about 2^13: by 2^-10, and the weight beside it by as much.
    rng = np.random.default_rng(5)
    of = (128 + np.arange(n) % 128) * 2.0 ** (np.arange(n) * 4 // n)
    of = {"rising": of, "falling": of[::-1], "mixed": rng.permutation(of)}[order]
    powers = 2.0 ** np.round(np.linspace(-2, 60, hq))
    q, k, v = np.zeros((1, hq, d)), np.zeros((n, heads, d)), synthetic.normal(940, (n, heads, d))
    q[0, :, 0], k[:, :, 0] = sign * powers, of[:, None] / 128
    k, v = k.astype(np.float32), np.asarray(v, np.float32)
    cache = q4.Q4KVCache(1, heads, d, n)
    q4.q4_kvq_append(cache, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), _i32(0, n), _i32(0), _i32(0))
    mass = cache.new_mass()
    args = (cache, torch.from_numpy(q).float().cuda(), _i32(0, 1), _i32(0), _i32(n - 1))
    o = q4.q4_kvq_attention(*args, scale=1.0, mass=mass)
    assert torch.equal(o, q4.q4_kvq_attention(*args, scale=1.0))
    assert q4.q4_device_status() == q4.Q4_OK
    want, weights = ref.attention(q, ref.held(k), ref.held(v), n - 1, 1.0)
    assert np.array_equal(ref.held(k), k)
    wide = 16 * np.abs(ref.encode(v)[1].astype(np.float64)).max()
    assert np.abs(o.cpu().double().numpy() - want).max() <= 2.0 ** -9 * wide
    got = mass[0].cpu().numpy()
    assert np.abs(got - weights).max() <= 2.0 ** -9 * hq / heads
    assert np.allclose(got.sum(-1), hq / heads, rtol=1e-3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_blocks_without_a_scale_hold_positive_zeros(q4, dtype, d):
    # all zero, and values whose scale rounds to 0 in binary16 from either side: code 8 with scale 0, so 0 and not -0
    x = torch.zeros((40, 2, d), dtype=torch.float32)
    x[1], x[2] = 1e-8, -1e-8                          # scales -+1.25e-9
    x[3, :, ::2], x[4, :, 1::2] = 2e-7, -2e-7         # half of 2^-24 is 2.98e-8: 2.5e-8 rounds to 0
    if dtype != torch.float16:
        x[5], x[6] = 1e-40, -1e-40                    # no normal number
    x[7] = -0.0
    x = x.to(dtype)
    cache = q4.Q4KVCache(1, 2, d, 40)
    cache.data.fill_(255)
    args = (_i32(0, 40), _i32(0), _i32(0))
    q4.q4_kvq_append(cache, x.cuda(), x.cuda(), *args)
    for got in q4.q4_kvq_read(cache, *args, 40):
        assert not got.any() and not torch.signbit(got).any()
    assert q4.q4_device_status() == q4.Q4_OK
    # the codes as well: the first tile (32 positions) holds nothing but code 8 and scale 0
    tile = cache.data[:32 * (d + d // 8)].cpu()
    half = 32 * (d // 2 + d // 16)
    for part in (tile[:half], tile[half:]):
        assert (part[:16 * d] == 0x88).all() and not part[16 * d:].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,hq,d", HEADS)
def test_output_in_place_of_the_queries(q4, dtype, heads, hq, d):
    lens, news = [3000, 5, 700], [1, 3, 5]
    cache = q4.Q4KVCache(3, heads, d, 3008)
    k, v = (torch.from_numpy(synthetic.normal(950 + i, (sum(lens), heads, d))).cuda() for i in range(2))
    at = np.cumsum([0] + lens).tolist()
    q4.q4_kvq_append(cache, k, v, _i32(*at), _i32(0, 1, 2), _i32(0, 0, 0))
    q = torch.from_numpy(synthetic.normal(952, (9, hq, d))).to(dtype).cuda()
    step = (_i32(0, 1, 4, 9), _i32(0, 1, 2), _i32(*[n - r for n, r in zip(lens, news)]))
    want = q4.q4_kvq_attention(cache, q, *step)
    room = q.clone()
    assert q4.q4_kvq_attention(cache, room, *step, out=room) is room
    assert torch.equal(room, want)
    room = q.clone()
    for call in (lambda: q4.q4_kvq_attention(cache, room, *step, out=room, mass=cache.new_mass()),
                 lambda: q4.q4_kvq_read(cache, *step, 9, k=k[:9], v=k[:9])):
        with pytest.raises(q4.Q4Error) as e:
            call()
        assert e.value.status == q4.Q4_ERR_INVALID_ARG
    assert torch.equal(room, q)
    assert q4.q4_device_status() == q4.Q4_OK
