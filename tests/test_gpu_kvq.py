"""The 4-bit KV cache on the GPU against the float64 oracle: append and read
bit for bit, attention within a bound derived below, eviction exactly.

Attention bound.  A score is a sum of D products accumulated in fp32, code by
code with the offset -8 as a starting value, so with A = scale * sum_d |q_d| *
16 |scale of k_d's block| each of the about ten roundings on its way is within
2^-22 A (tensor-core sums truncate), and the query's two binary16 terms add
2^-21 A: its error is below ds = 2^-18 A.  A weight is then off by a factor of
at most exp(2 ds) and the exponential's own 2^-20.  A sum over n keys rounds
once per 16 keys and a few times at the joins, each within 2^-22 of sum_p w_p
16 |scale of v's block|.  Together, per value,

    |o - o64| <= (4 max ds + 2^-18 + (n / 16 + 64) 2^-22) * sum_p w_p 16 |s_v| + u |o64|,

u = half a unit in the last place of the output type."""
import numpy as np
import pytest
import torch

import synthetic
from oracle import attention as ref

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(seed, shape, dtype, sigma=1.0):
    return torch.from_numpy(synthetic.normal(seed, shape, sigma=sigma)).to(dtype)


def _starts(counts, lead=0):
    return _i32(*(lead + np.concatenate([[0], np.cumsum(counts)]).astype(int)).tolist())


def _filled(q4, seed, lens, heads, d, cap, slots=None, dtype=torch.float32):
    """A cache with lens[s] rows in slot s, and those rows (CPU, fp32)."""
    slots = slots or len(lens)
    cache = q4.Q4KVCache(slots, heads, d, cap)
    cache.data.fill_(255)  # what was never appended must not matter: NaN scales, full codes
    k = _normal(seed, (sum(lens), heads, d), dtype)
    v = _normal(seed + 1, (sum(lens), heads, d), dtype)
    n = len(lens)
    q4.q4_kvq_append(cache, k.cuda(), v.cuda(), _starts(lens), _i32(*range(n)), _i32(*[0] * n))
    at = np.concatenate([[0], np.cumsum(lens)])
    rows = [(k[a:b].float().numpy(), v[a:b].float().numpy()) for a, b in zip(at, at[1:])]
    return cache, rows


# ---------------------------------------------------------------- append, read

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,d", [(4, 128), (2, 64), (1, 128), (3, 64)])
def test_append_and_read_match_the_block_rule(q4, dtype, heads, d):
    lens = [1, 17, 0, 40, 16, 5]
    n, lead = sum(lens), 3  # packed rows before the first request are not cached
    k = _normal(11, (n + lead, heads, d), dtype)
    v = _normal(12, (heads, n + lead, d), dtype).transpose(0, 1)  # a strided view
    k[5, 0, :32] = 0.0                                           # an all-zero block
    k[6, 0, 3], k[6, 0, 9] = 7.5, -7.5                           # equal magnitudes: the first sets the scale
    slots = 8
    cache = q4.Q4KVCache(slots, heads, d, 64)
    slot, pos = [5, 0, 1, 7, 2, 6], [0, 13, 0, 24, 48, 59]
    args = (_starts(lens, lead), _i32(*slot), _i32(*pos))
    q4.q4_kvq_append(cache, k.cuda(), v.cuda(), *args)
    for out_type in TYPES:
        gk, gv = q4.q4_kvq_read(cache, *args, n + lead, dtype=out_type)
        assert q4.q4_device_status() == q4.Q4_OK
        for got, x in ((gk, k), (gv, v)):
            want = torch.from_numpy(ref.held(x.float().numpy())).float().to(out_type)
            want[:lead] = 0
            assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dtype", TYPES)
def test_halves_and_their_neighbours_round_as_the_quotient_does(q4, dtype):
    """Values on half codes, next to them in the type, and scales from the smallest to the largest."""
    rows, heads, d = 400, 2, 128
    g = torch.Generator().manual_seed(15)
    top = torch.randn((rows, heads, d // 32, 1), generator=g)
    top = (top * 2.0 ** torch.randint(-24, 15, top.shape, generator=g)).to(dtype).float()
    x = (top / -8) * torch.randint(-16, 17, (rows, heads, d // 32, 32), generator=g) / 2
    x = x.to(dtype)
    step = torch.randint(-2, 3, x.shape, generator=g)
    ints = x.view(torch.int32 if dtype == torch.float32 else torch.int16)
    near_zero = (ints & (2 ** 31 - 1 if dtype == torch.float32 else 2 ** 15 - 1)) < 4  # a step may pass zero there
    x = torch.where(near_zero, x, (ints + step.to(ints.dtype)).view(dtype)).float()
    x = torch.where(x.abs() > top.abs(), top, x)
    x[..., :1] = top
    x = x.reshape(rows, heads, d).to(dtype)
    cache = q4.Q4KVCache(1, heads, d, rows)
    args = (_i32(0, rows), _i32(0), _i32(0))
    q4.q4_kvq_append(cache, x.cuda(), x.flip(0).cuda(), *args)
    k, v = q4.q4_kvq_read(cache, *args, rows)
    assert q4.q4_device_status() == q4.Q4_OK
    want = torch.from_numpy(ref.held(x.float().numpy())).float()
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want.flip(0))


def test_append_leaves_other_rows_alone(q4):
    heads, d, cap = 2, 64, 37
    cache, rows = _filled(q4, 21, [cap, cap], heads, d, cap)
    new = _normal(23, (2, heads, d), torch.float32)
    q4.q4_kvq_append(cache, new.cuda(), new.cuda(), _i32(0, 2), _i32(1), _i32(15))
    k, v = q4.q4_kvq_read(cache, _i32(0, cap, 2 * cap), _i32(0, 1), _i32(0, 0), 2 * cap)
    for got, which in ((k, 0), (v, 1)):
        want = np.concatenate([ref.held(rows[0][which]), ref.held(rows[1][which])])
        want[cap + 15:cap + 17] = ref.held(new.numpy())
        assert np.array_equal(got.cpu().numpy().astype(np.float64), want)


def test_values_that_have_no_scale_read_back_as_nan(q4):
    cache = q4.Q4KVCache(1, 1, 64, 16)
    x = torch.ones((3, 1, 64))
    x[0, 0, 5], x[1, 0, 40], x[2, 0, 1] = float("nan"), float("-inf"), 1e6
    args = (_i32(0, 3), _i32(0), _i32(0))
    q4.q4_kvq_append(cache, x[:2].cuda(), x[:2].cuda(), _i32(0, 2), _i32(0), _i32(0))
    assert q4.q4_device_status() == q4.Q4_ERR_NONFINITE
    q4.q4_kvq_append(cache, x.cuda()[2:], x.cuda()[2:], _i32(0, 1), _i32(0), _i32(2))
    assert q4.q4_device_status() == q4.Q4_ERR_RANGE
    k, _ = q4.q4_kvq_read(cache, *args, 3)
    nan = torch.isnan(k.cpu()[:, 0])
    assert nan[0, :32].all() and not nan[0, 32:].any()
    assert nan[1, 32:].all() and not nan[1, :32].any()
    assert nan[2, :32].all() and not nan[2, 32:].any()


def test_requests_out_of_range_are_left_out(q4):
    heads, d, cap = 2, 128, 20
    cache, rows = _filled(q4, 31, [cap, cap], heads, d, cap)
    before = cache.data.clone()
    new = _normal(33, (6, heads, d), torch.float32).cuda()
    offsets, slot, pos = _i32(0, 2, 3, 5, 6), _i32(0, 7, 1, -1), _i32(19, 0, -1, 0)  # past the end, no slot, ...
    q4.q4_kvq_append(cache, new, new, offsets, slot, pos)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    assert torch.equal(cache.data, before)
    k, v = q4.q4_kvq_read(cache, offsets, slot, pos, 6)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    assert not k.any() and not v.any()
    out = q4.q4_kvq_attention(cache, _normal(34, (6, 4, d), torch.float32).cuda(), offsets, slot, pos,
                              out=torch.full((6, 4, d), 7.0, device="cuda"))
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    assert not out.any()


# ---------------------------------------------------------------- attention

def _check(o, q, k, v, pos, scale, dtype, what):
    """o [rows, Hq, D] of one request against float64, per value; returns (worst share of the bound, mass)."""
    ck, sk = ref.encode(k)
    cv, sv = ref.encode(v)
    k64, v64 = ref.decode(ck, sk), ref.decode(cv, sv)
    want, mass = ref.attention(q, k64, v64, pos, scale)
    rows, hq, d = q.shape
    g = hq // k.shape[1]
    wide_k = 16 * np.repeat(np.abs(sk.astype(np.float64)), 32, -1)
    wide_v = 16 * np.repeat(np.abs(sv.astype(np.float64)), 32, -1)
    worst = 0.0
    for j in range(rows):
        seen = pos + j + 1
        for x in range(hq):
            h = x // g
            s = scale * (k64[:seen, h] @ q[j, x])
            w = np.exp(s - s.max())
            w /= w.sum()
            ds = 2.0 ** -18 * scale * (wide_k[:seen, h] @ np.abs(q[j, x])).max()
            bound = (4 * ds + 2.0 ** -18 + (seen / 16 + 64) * 2.0 ** -22) * (w @ wide_v[:seen, h])
            bound = bound + UNIT[dtype] * np.abs(want[j, x]) + 1e-30
            err = np.abs(o[j, x] - want[j, x])
            assert np.all(err <= bound), "%s row %d head %d: %.3g of the bound" % (what, j, x, (err / bound).max())
            worst = max(worst, float((err / bound).max()))
    return worst, mass


def _attend(q4, seed, lens, news, heads, hq, d, dtype, cap=None, scale=None, mass=False, sigma=1.0):
    """Fills a cache with lens, appends news rows, attends; everything checked."""
    n = len(lens)
    cap = cap or max(a + b for a, b in zip(lens, news))
    cache, rows = _filled(q4, seed, [max(x, 0) for x in lens], heads, d, cap)
    total = sum(news)
    kn, vn = _normal(seed + 5, (total, heads, d), dtype), _normal(seed + 6, (total, heads, d), dtype)
    q = _normal(seed + 7, (total, hq, d), dtype, sigma)
    args = (_starts(news), _i32(*range(n)), _i32(*lens))
    q4.q4_kvq_append(cache, kn.cuda(), vn.cuda(), *args)
    m = None
    if mass:
        m = torch.from_numpy(np.abs(synthetic.normal(seed + 8, (n, heads, cap)))).cuda()
        m0 = m.cpu().numpy().astype(np.float64)
    o = q4.q4_kvq_attention(cache, q.cuda(), *args, scale=scale, mass=m)
    assert q4.q4_device_status() == q4.Q4_OK
    o = o.cpu().double().numpy()
    at = np.concatenate([[0], np.cumsum(news)])
    scale = 1 / np.sqrt(d) if scale is None else scale
    worst = 0.0
    for s in range(n):
        a, b = at[s], at[s + 1]
        if a == b:
            continue
        k = np.concatenate([rows[s][0], kn[a:b].float().numpy()])
        v = np.concatenate([rows[s][1], vn[a:b].float().numpy()])
        w, want = _check(o[a:b], q[a:b].double().numpy(), k, v, lens[s], scale, dtype, "request %d" % s)
        worst = max(worst, w)
        if mass:
            m0[s, :, lens[s]:lens[s] + b - a] = 0
            m0[s, :, :lens[s] + b - a] += want
    if mass:  # weights within 2^-14 of themselves (scores below 2^7 at 2^-21 relative), sums exact to fp32
        got = m.cpu().numpy()
        assert np.all(np.abs(got - m0) <= 2.0 ** -14 * (b - a + 1) * hq / heads + 2.0 ** -20 * m0)
        for s in range(n):
            if news[s]:
                share = np.abs(got[s] - m0[s])
                assert share.max() < 1e-4
    return worst


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,hq,d", [(4, 28, 128), (2, 14, 64), (8, 8, 64), (1, 16, 128), (2, 2, 128)])
def test_attention_single_rows(q4, dtype, heads, hq, d):
    # one token with nothing before it, lengths around a tile (16) and a CTA's share, and long ones
    _attend(q4, 100, [0, 1, 14, 15, 16, 17, 63, 64, 65, 300, 1031], [1] * 11, heads, hq, d, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,hq,d", [(4, 28, 128), (2, 14, 64), (1, 3, 64)])
def test_attention_several_rows_are_causal(q4, dtype, heads, hq, d):
    _attend(q4, 200, [0, 5, 200, 31, 16, 7], [3, 0, 5, 1, 9, 40], heads, hq, d, dtype)


def test_attention_one_long_request(q4):
    _attend(q4, 300, [9001], [1], 1, 2, 128, torch.float32)
    _attend(q4, 301, [5003], [2], 2, 14, 64, torch.float32)


def test_attention_many_requests(q4):
    lens = [(37 * i) % 91 for i in range(333)]
    _attend(q4, 400, lens, [1 + (i % 7 == 0) for i in range(333)], 1, 4, 64, torch.float32)


@pytest.mark.parametrize("sigma,scale", [(1e-30, None), (1e4, 1e-4), (40.0, None), (1.0, 3.0)])
def test_attention_query_ranges(q4, sigma, scale):
    # tiny, large and sharply peaked queries (float32: the fragment is scaled by a power of two per row)
    _attend(q4, 500, [150, 33], [1, 2], 2, 14, 128, torch.float32, sigma=sigma, scale=scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [2, 8, 70])
def test_attention_sums_that_nearly_cancel(q4, dtype, n):
    # every other value row is the last one's negative and weights are nearly equal: what
    # remains is small, and the output type's own rounding of it hides nothing
    heads, hq, d = 2, 14, 128
    k = _normal(600, (n, heads, d), dtype)
    v = _normal(601, (n, heads, d), dtype)
    v[1::2] = -v[::2]
    q = _normal(602, (1, hq, d), dtype, 1e-3)
    cache = q4.Q4KVCache(1, heads, d, n)
    q4.q4_kvq_append(cache, k.cuda(), v.cuda(), _i32(0, n), _i32(0), _i32(0))
    o = q4.q4_kvq_attention(cache, q.cuda(), _i32(0, 1), _i32(0), _i32(n - 1)).cpu().double().numpy()
    _check(o, q.double().numpy(), k.float().numpy(), v.float().numpy(), n - 1, d ** -0.5, dtype, "%d keys" % n)


@pytest.mark.parametrize("heads,hq,d,news", [(4, 28, 128, [1, 1, 1]), (2, 14, 64, [1, 3, 4]), (1, 16, 64, [2, 0, 1])])
def test_attention_mass(q4, heads, hq, d, news):
    _attend(q4, 600, [70, 0, 515], news, heads, hq, d, torch.float32, mass=True)


def test_mass_sums_to_rows_times_group(q4):
    heads, hq, d = 2, 14, 64
    cache, _ = _filled(q4, 650, [500, 90], heads, d, 512)
    m = cache.new_mass()
    q = _normal(651, (5, hq, d), torch.float32).cuda()
    q4.q4_kvq_attention(cache, q, _i32(0, 3, 5), _i32(0, 1), _i32(497, 88), mass=m)
    got = m.sum(-1).cpu().numpy()
    assert np.allclose(got, [[21, 21], [14, 14]], rtol=1e-5)
    assert not m[0, :, 500:].any() and not m[1, :, 90:].any()


def test_nan_in_masked_rows_stays_there(q4):
    # a NaN row at position 40 (K and V): rows before it do not see it, rows from it on do
    heads, hq, d = 1, 4, 128
    cache, _ = _filled(q4, 700, [40], heads, d, 64)
    bad = torch.full((1, heads, d), float("nan"), device="cuda")
    q4.q4_kvq_append(cache, bad, bad, _i32(0, 1), _i32(0), _i32(40))
    assert q4.q4_device_status() == q4.Q4_ERR_NONFINITE
    q = _normal(701, (6, hq, d), torch.float32).cuda()
    o = q4.q4_kvq_attention(cache, q, _i32(0, 6), _i32(0), _i32(36))
    assert torch.isfinite(o[:4]).all() and torch.isnan(o[4:]).all()


def test_attention_strided_queries_and_gaps(q4):
    heads, hq, d = 2, 14, 64
    cache, rows = _filled(q4, 720, [50, 20], heads, d, 64)
    wide = _normal(721, (9, 2 * hq + 4, d), torch.float32).cuda()
    q = wide[:, 3:3 + 2 * hq:2]  # every second head of a wider tensor
    out = torch.full((9, hq, d), 3.0, device="cuda")
    q4.q4_kvq_attention(cache, q, _i32(2, 5, 7), _i32(1, 0), _i32(17, 48), out=out)
    assert q4.q4_device_status() == q4.Q4_OK
    same = q4.q4_kvq_attention(cache, q.contiguous(), _i32(2, 5, 7), _i32(1, 0), _i32(17, 48))
    assert torch.equal(out, same)
    assert not out[:2].any() and not out[7:].any()
    o, qn = out.cpu().double().numpy(), q.cpu().double().numpy()
    _check(o[2:5], qn[2:5], rows[1][0], rows[1][1], 17, d ** -0.5, torch.float32, "slot 1")
    _check(o[5:7], qn[5:7], rows[0][0], rows[0][1], 48, d ** -0.5, torch.float32, "slot 0")


def test_attention_is_deterministic_and_stream_ordered(q4):
    heads, hq, d = 4, 28, 128
    cache, _ = _filled(q4, 730, [3000, 40, 900], heads, d, 3001)
    q = _normal(731, (3, hq, d), torch.float32).cuda()
    args = (cache, q, _i32(0, 1, 2, 3), _i32(0, 1, 2), _i32(2999, 39, 899))
    a = q4.q4_kvq_attention(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        outs = [q4.q4_kvq_attention(*args) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(a, o) for o in outs)


def test_attention_in_a_cuda_graph(q4):
    heads, hq, d = 2, 14, 64
    cache, _ = _filled(q4, 740, [100], heads, d, 128)
    q = _normal(741, (1, hq, d), torch.float32).cuda()
    offsets, slot, pos = _i32(0, 1), _i32(0), _i32(60)
    out = torch.empty_like(q)
    q4.q4_kvq_attention(cache, q, offsets, slot, pos, out=out)  # sizes the scratch
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.q4_kvq_attention(cache, q, offsets, slot, pos, out=out)
    for p in (99, 3):  # the lengths are read when the graph runs
        pos.fill_(p)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q4.q4_kvq_attention(cache, q, offsets, slot, _i32(p)))


def test_a_captured_step_outlives_the_growth_of_the_scratch(q4):
    cache, _ = _filled(q4, 171, [700, 33], 2, 128, 704)
    q = _normal(173, (2, 8, 128), torch.float32).cuda()
    step = (_starts([1, 1]), _i32(0, 1), _i32(699, 32))
    out = torch.empty_like(q)
    want = q4.q4_kvq_attention(cache, q, *step)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        q4.q4_kvq_attention(cache, q, *step, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.q4_kvq_attention(cache, q, *step, out=out)
    # 131,072 rows of 32 heads with weights: 17 MB of row sums
    wide = q4.Q4KVCache(4096, 1, 64, 32)
    wide.data.zero_()
    rows = torch.zeros((4096 * 32, 32, 64), dtype=torch.bfloat16, device="cuda")
    n = torch.arange(4097, dtype=torch.int32, device="cuda")
    mass = wide.new_mass()
    q4.q4_kvq_attention(wide, rows, n * 32, n[:-1].contiguous(), torch.zeros_like(n[:-1]), mass=mass)
    total = mass.double().sum((1, 2)).cpu()
    assert torch.allclose(total, torch.full_like(total, 32.0 * 32.0), rtol=1e-5, atol=0)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert q4.q4_device_status() == q4.Q4_OK


def test_offsets_past_32_bits(q4):
    # one plane of the cache starts beyond 2^32 bytes
    heads, hq, d = 1, 4, 128
    slots, cap = 34, 1 << 20
    cache = q4.Q4KVCache(slots, heads, d, cap)
    assert cache.nbytes > 1 << 32
    k = _normal(751, (50, heads, d), torch.float32)
    v = _normal(752, (50, heads, d), torch.float32)
    last = cap - 50
    args = (_i32(0, 50), _i32(slots - 1), _i32(last))
    q4.q4_kvq_append(cache, k.cuda(), v.cuda(), *args)
    gk, gv = q4.q4_kvq_read(cache, *args, 50)
    assert np.array_equal(gk.cpu().numpy(), ref.held(k.numpy()).astype(np.float32))
    assert np.array_equal(gv.cpu().numpy(), ref.held(v.numpy()).astype(np.float32))
    # all earlier positions hold zeros: their scores are 0
    q = _normal(753, (1, hq, d), torch.float32)
    o = q4.q4_kvq_attention(cache, q.cuda(), _i32(0, 1), _i32(slots - 1), _i32(cap - 1)).cpu().double().numpy()[0]
    k64, v64 = ref.held(k.numpy())[:, 0], ref.held(v.numpy())[:, 0]
    for x in range(hq):
        e = np.exp(d ** -0.5 * (k64 @ q[0, x].double().numpy()))
        want = e @ v64 / (e.sum() + last)
        assert np.abs(o[x] - want).max() <= 2.0 ** -8 * np.abs(want).max()  # 2^16 sums of 16 keys at 2^-24
    del cache


@pytest.mark.parametrize("mass", [False, True])
def test_waits_run_out_and_the_next_call_is_right(q4, mass):
    # copies withheld: every wait gives up after its bound, and nothing of it is left behind
    heads, hq, d = 2, 14, 64
    cache, _ = _filled(q4, 760, [300, 20], heads, d, 320)
    q = _normal(761, (2, hq, d), torch.float32).cuda()
    args = (cache, q, _i32(0, 1, 2), _i32(0, 1), _i32(299, 19))
    m = cache.new_mass() if mass else None
    want = q4.q4_kvq_attention(*args)
    torch.cuda.synchronize()
    q4.q4mm_set_wait_limit_ns(1000000)
    q4.q4mm_set_stall_for_test(True)
    try:
        q4.q4_kvq_attention(*args, mass=m)
        assert q4.q4_device_status() == q4.Q4_ERR_TIMEOUT
    finally:
        q4.q4mm_set_stall_for_test(False)
        q4.q4mm_set_wait_limit_ns(0)
    assert torch.equal(q4.q4_kvq_attention(*args), want)
    assert q4.q4_device_status() == q4.Q4_OK


# ---------------------------------------------------------------- eviction

def _evict_case(q4, seed, lens, heads, d, cap, keep, recent, in_place, mass_of=None):
    n = len(lens)
    cache, rows = _filled(q4, seed, [max(x, 1) for x in lens], heads, d, cap, slots=2 * n)
    g = np.random.default_rng(seed)
    mass = (g.random((2 * n, heads, cap)) ** 6).astype(np.float32)
    mass[g.random(mass.shape) < 0.3] = 0.0
    if mass_of is not None:
        mass_of(mass)
    src = list(range(n))
    dst = src if in_place else [n + s for s in src]
    m = torch.from_numpy(mass).cuda()
    new_len, kept = q4.q4_kvq_evict(cache, m, _i32(*src), _i32(*dst), _i32(*lens), keep, recent)
    assert q4.q4_device_status() == q4.Q4_OK
    new_len, kept, m = new_len.cpu().numpy(), kept.cpu().numpy(), m.cpu().numpy()
    counts = [min(x, keep) for x in lens]
    assert new_len.tolist() == counts
    k, v = q4.q4_kvq_read(cache, _starts(counts), _i32(*dst), _i32(*[0] * n), sum(counts))
    k, v = k.cpu().numpy(), v.cpu().numpy()
    at = np.concatenate([[0], np.cumsum(counts)])
    for s in range(n):
        for h in range(heads):
            want = ref.evict(mass[src[s], h, :lens[s]], keep, recent)
            c = counts[s]
            assert kept[s, h, :c].tolist() == want.tolist(), (s, h)
            assert (kept[s, h, c:] == -1).all()
            assert np.array_equal(m[dst[s], h, :c], mass[src[s], h][want], equal_nan=True)
            hk, hv = ref.held(rows[s][0][:, h]), ref.held(rows[s][1][:, h])
            assert np.array_equal(k[at[s]:at[s + 1], h], hk[want].astype(np.float32))
            assert np.array_equal(v[at[s]:at[s + 1], h], hv[want].astype(np.float32))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("heads,d", [(2, 128), (3, 64)])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (7, 3), (64, 64), (100, 16), (700, 33)])
def test_evict(q4, in_place, heads, d, keep, recent):
    _evict_case(q4, 800 + keep, [0, 1, 6, 64, 100, 101, 733, 1025], heads, d, 1030, keep, recent, in_place)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_of_a_cache_too_long_for_shared_memory(q4, in_place):
    _evict_case(q4, 840, [49000, 48000], 1, 64, 49001, 5000, 100, in_place)


def test_evict_ties_negative_and_nan_weights(q4):
    def odd(mass):
        mass[0] = 1.0                      # all equal: the lowest positions stay
        mass[1, :, ::2] = -1.0
        mass[2, :, :300] = np.nan          # smallest of all, -inf included
        mass[2, :, 300:400] = -np.inf
        mass[3, :, ::3] = -0.0
        mass[3, :, 1::3] = 0.0
        mass[4, :, 5] = np.inf
    _evict_case(q4, 850, [600] * 5, 2, 64, 640, 250, 20, True, odd)


def test_evict_then_attend(q4):
    # a thinned cache answers like one that was filled with the kept rows
    heads, hq, d, cap = 2, 14, 128, 400
    cache, rows = _filled(q4, 870, [400], heads, d, cap, slots=2)
    m = torch.rand((2, heads, cap), device="cuda")
    new_len, kept = q4.q4_kvq_evict(cache, m, _i32(0), _i32(0), _i32(400), 90, 10)
    q = _normal(871, (1, hq, d), torch.float32)
    o = q4.q4_kvq_attention(cache, q.cuda(), _i32(0, 1), _i32(0), _i32(89)).cpu().double().numpy()
    keep = kept.cpu().numpy()[0]
    k = np.stack([rows[0][0][keep[h], h] for h in range(heads)], 1)
    v = np.stack([rows[0][1][keep[h], h] for h in range(heads)], 1)
    _check(o, q.double().numpy(), k, v, 89, d ** -0.5, torch.float32, "thinned")


@pytest.mark.parametrize("heads,hq,d", [(4, 28, 128), (2, 14, 64), (8, 8, 64)])
def test_calls_in_a_row_see_what_the_last_one_wrote(q4, heads, hq, d):
    """Launches begin under the end of the one before: with a wait for the GPU after every call the results are the same."""
    S, cap, keep, steps = 6, 96, 40, 24
    k = _normal(181, (steps, S, heads, d), torch.float32).cuda()
    v = _normal(182, (steps, S, heads, d), torch.float32).cuda()
    q = _normal(183, (S, hq, d), torch.float32).cuda()
    offsets, slot, zero = _starts([1] * S), _i32(*range(S)), _i32(*[0] * S)
    lens = [70, 41, 66, 90, 40, 55]

    def run(between):
        cache, _ = _filled(q4, 185, lens, heads, d, cap)
        mass = cache.new_mass()
        pos = list(lens)
        out = []
        between()
        for t in range(steps):
            at = _i32(*pos)
            q4.q4_kvq_append(cache, k[t], v[t], offsets, slot, at)
            between()
            # the next query is the last output: nothing comes between the calls
            o = q4.q4_kvq_attention(cache, out[-1] if out else q, offsets, slot, at, mass=mass)
            between()
            o = q4.q4_kvq_attention(cache, o, offsets, slot, at, mass=mass)
            between()
            out.append(o)
            pos = [p + 1 for p in pos]
            if max(pos) > 80:
                n, _ = q4.q4_kvq_evict(cache, mass, slot, slot, _i32(*pos), keep, 8)
                between()
                pos = [min(p, keep) for p in pos]
                rows = q4.q4_kvq_read(cache, _starts(pos), slot, zero, sum(pos))
                between()
                out.extend(rows)
                assert n.tolist() == pos
                out.append(torch.ones((S, hq, d), device="cuda"))  # the next step's query
        out.append(mass)
        torch.cuda.synchronize()
        return [x.cpu() for x in out]

    apart = run(torch.cuda.synchronize)
    for _ in range(3):
        for x, y in zip(run(lambda: None), apart):
            assert torch.equal(x, y)
    assert q4.q4_device_status() == q4.Q4_OK


def test_evict_refuses_slots_that_meet(q4):
    heads, d, cap = 1, 64, 40
    cache, _ = _filled(q4, 880, [40, 40, 40], heads, d, cap, slots=5)
    before, m = cache.data.clone(), torch.rand((5, heads, cap), device="cuda")
    m0 = m.clone()
    # 0 and 1 into one slot; 2 reads a slot out of range
    new_len, kept = q4.q4_kvq_evict(cache, m, _i32(0, 1, 9), _i32(3, 3, 2), _i32(40, 40, 40), 8)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    assert new_len.tolist() == [-1, -1, -1] and (kept == -1).all()
    assert torch.equal(cache.data, before) and torch.equal(m, m0)
    # 1 writes what 0 reads; 2 stands apart and is done
    new_len, _ = q4.q4_kvq_evict(cache, m, _i32(0, 1, 2), _i32(3, 0, 4), _i32(40, 40, 41), 8)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    assert new_len.tolist() == [-1, -1, -1]  # 41 is past the capacity
    new_len, _ = q4.q4_kvq_evict(cache, m, _i32(0, 1, 2), _i32(3, 0, 4), _i32(40, 40, 40), 8)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    assert new_len.tolist() == [-1, -1, 8]


# ---------------------------------------------------------------- refusals

def test_binding_refuses_what_does_not_fit(q4):
    cache = q4.Q4KVCache(2, 2, 64, 32)
    x = torch.zeros((3, 2, 64), device="cuda")
    o, s, p = _i32(0, 3), _i32(0), _i32(0)
    bad = [
        lambda: q4.q4_kvq_append(cache, x, x[:2], o, s, p),                          # rows differ
        lambda: q4.q4_kvq_append(cache, x, x.half(), o, s, p),                       # types differ
        lambda: q4.q4_kvq_append(cache, x[:, :1], x[:, :1], o, s, p),                # heads
        lambda: q4.q4_kvq_append(cache, x.double(), x.double(), o, s, p),            # type
        lambda: q4.q4_kvq_append(cache, x, x, o.long(), s, p),                       # int64 offsets
        lambda: q4.q4_kvq_append(cache, x, x, _i32(0), s, p),                        # offsets too short
        lambda: q4.q4_kvq_append(cache, x.transpose(1, 2).contiguous().transpose(1, 2), x, o, s, p),  # values strided
        lambda: q4.q4_kvq_append(cache, x.cpu(), x.cpu(), o, s, p),
        lambda: q4.q4_kvq_attention(cache, torch.zeros((3, 3, 64), device="cuda"), o, s, p),  # 3 heads over 2
        lambda: q4.q4_kvq_attention(cache, x, o, s, p, out=torch.zeros((3, 2, 64))),
        lambda: q4.q4_kvq_attention(cache, x, o, s, p, mass=torch.zeros((2, 2, 31), device="cuda")),
        lambda: q4.q4_kvq_evict(cache, torch.zeros((2, 2, 32), device="cuda"), s, _i32(0, 1), p, 4),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    shifted = torch.zeros(3 * 2 * 64 + 1, device="cuda")[1:].view(3, 2, 64)  # 4-byte aligned only
    for call, status in [
        (lambda: q4.q4_kvq_append(cache, shifted, x, o, s, p), q4.Q4_ERR_ALIGN),
        (lambda: q4.q4_kvq_attention(cache, shifted, o, s, p), q4.Q4_ERR_ALIGN),
        (lambda: q4.q4_kvq_attention(cache, x, o, s, p, scale=0.0), q4.Q4_ERR_INVALID_ARG),
        (lambda: q4.q4_kvq_attention(cache, x, o, s, p, scale=float("nan")), q4.Q4_ERR_INVALID_ARG),
        (lambda: q4.q4_kvq_evict(cache, cache.new_mass(), s, s, p, 33), q4.Q4_ERR_INVALID_ARG),
        (lambda: q4.q4_kvq_evict(cache, cache.new_mass(), s, s, p, 0), q4.Q4_ERR_INVALID_ARG),
        (lambda: q4.q4_kvq_evict(cache, cache.new_mass(), s, s, p, 4, 5), q4.Q4_ERR_INVALID_ARG),
        (lambda: q4.Q4KVCache(1, 1, 96, 16), q4.Q4_ERR_SHAPE),
        (lambda: q4.Q4KVCache(0, 1, 64, 16), q4.Q4_ERR_INVALID_ARG),
    ]:
        with pytest.raises(q4.Q4Error) as e:
            call()
        assert e.value.status == status
    # nothing to do is not an error
    q4.q4_kvq_append(cache, x[:0], x[:0], _i32(0), _i32(), _i32())
    assert q4.q4_kvq_attention(cache, x[:0], _i32(0, 0), s, p).shape == (0, 2, 64)
    assert q4.q4_device_status() == q4.Q4_OK


# ---------------------------------------------------------------- launches that begin early

@pytest.mark.parametrize("heads,hq,d", [(4, 28, 128), (2, 14, 64), (8, 8, 64)])
@pytest.mark.parametrize("lens,news", [([700, 300, 5, 64], [1, 1, 1, 1]), ([1500, 900], [400, 33]), ([9000], [1])])
def test_a_captured_chain_waits_for_what_it_reads(q4, heads, hq, d, lens, news):
    """Evictions, appends and weighing calls back to back in one CUDA graph, with nothing of the host's pace
    between them, against the same calls with a wait for the GPU after each: bit for bit, many times."""
    S, keep, keep2 = len(lens), 256, 200
    mid = [min(n, keep) for n in lens]                        # rows after the first eviction
    end = [min(n + r, keep2) for n, r in zip(mid, news)]      # and after the second
    cap = max(max(lens), max(m + r for m, r in zip(mid, news)))
    cache, _ = _filled(q4, 190, lens, heads, d, cap)
    full = cache.data.clone()
    mass0 = torch.from_numpy(np.abs(synthetic.normal(192, (S, heads, cap)))).cuda()
    mass = mass0.clone()
    total = sum(news)
    k, v = (_normal(193 + i, (total, heads, d), torch.bfloat16).cuda() for i in range(2))
    q = _normal(195, (total, hq, d), torch.float32).cuda()
    one = _normal(196, (S, hq, d), torch.float32).cuda()
    slot, zero, lens_d, mid_d = _i32(*range(S)), _i32(*[0] * S), _i32(*lens), _i32(*mid)
    grown_d, last_d = _i32(*[m + r for m, r in zip(mid, news)]), _i32(*[e - 1 for e in end])
    rows, single, held = _starts(news), _starts([1] * S), _starts(end)

    def chain(between):
        cache.data.copy_(full)
        mass.copy_(mass0)
        between()
        n1, kept1 = q4.q4_kvq_evict(cache, mass, slot, slot, lens_d, keep, 16)
        between()
        # the lengths that the eviction wrote are the positions of the next calls
        q4.q4_kvq_append(cache, k, v, rows, slot, n1)
        between()
        m1 = q4.q4_kvq_attention(cache, q, rows, slot, n1, mass=mass)
        between()
        o = q4.q4_kvq_attention(cache, m1, rows, slot, n1)
        between()
        p = q4.q4_kvq_attention(cache, o, rows, slot, mid_d, mass=mass)
        between()
        n2, kept2 = q4.q4_kvq_evict(cache, mass, slot, slot, grown_d, keep2, 8)
        between()
        w = q4.q4_kvq_attention(cache, one, single, slot, last_d, mass=mass)
        between()
        kk, vv = q4.q4_kvq_read(cache, held, slot, zero, sum(end))
        between()
        return [n1, kept1, m1, o, p, n2, kept2, w, kk, vv]

    want = [x.clone() for x in chain(torch.cuda.synchronize)] + [mass.clone()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain(lambda: None) + [mass]
    for _ in range(60):
        graph.replay()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(outs, want)):
            assert torch.equal(x, y), i
    assert q4.q4_device_status() == q4.Q4_OK
