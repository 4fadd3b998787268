"""The paged cache on the GPU: pools against the rules on lists, appended rows bit
for bit, attention against float64.

Bound per value of attention, as for prompts: scores are fp32 sums of exact
products, off by less than ds = 2^-19 scale sum_d |q_d k_d|; weights are rounded
to the type (u = 2^-8 for bfloat16, 2^-11 for float16, and 2^-24 of the largest
where float16 has no normal numbers left) and the output once more; sums over
keys, and those of the pieces of a request that is divided (their factors are off by
2^-21), are fp32:

    |o - o64| <= (4 max ds + u + 2^-16) * sum_j w_j |v_j| + 2^-22 max |v| + u |o64|."""
import random

import numpy as np
import pytest
import torch

import synthetic
from oracle import paged

pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.bfloat16, torch.float16]
PAGES = [16, 32, 64, 128]


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


# ---------------------------------------------------------------- reserve

class Pair:
    """A pool on the GPU and its oracle, taken through the same steps."""

    def __init__(self, q4, slots, width, pages, page):
        self.q4, self.gpu, self.ref = q4, q4.Q4PageTable(slots, width, pages, page), paged.Pool(slots, width, pages, page)
        self.same()

    def same(self):
        assert np.array_equal(self.gpu.state.cpu().numpy(), self.ref.state())

    def step(self, offsets, slot, pos, total):
        q4 = self.q4
        m, n = q4.q4_paged_reserve(self.gpu, _i32(offsets), _i32(slot), _i32(pos), total)
        want_m, want_n, short, bad = self.ref.reserve(offsets, slot, pos, total)
        assert m.tolist() == want_m
        assert n.tolist() == want_n
        self.same()
        assert q4.q4_device_status() == (q4.Q4_ERR_INVALID_ARG if bad else q4.Q4_ERR_NOMEM if short else q4.Q4_OK)
        return want_n


def _starts(rows):
    return [0] + [int(x) for x in np.cumsum(rows)]


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("slots,width,pages,most", [(1, 3, 2, 40), (7, 5, 20, 60), (40, 9, 200, 150),
                                                    (300, 40, 2000, 300)])
def test_pools_over_steps(q4, page, slots, width, pages, most):
    rng = random.Random(page * 1000 + slots)
    p, length = Pair(q4, slots, width, pages, page), [0] * slots
    for _ in range(12):
        who = rng.sample(range(slots), rng.randint(1, slots))
        pos = [rng.choice((length[s], length[s], length[s], 0, length[s] // 2)) for s in who]
        rows = [rng.choice((0, 1, 1, rng.randint(0, most))) for _ in who]
        off = _starts(rows)
        for s, n in zip(who, p.step(off, who, pos, off[-1] + rng.choice((0, 0, 5)))):
            length[s] = n if n >= 0 else length[s]


@pytest.mark.parametrize("total,S", [(4095, 1), (4096, 1), (4090, 6), (4091, 6), (20000, 3), (9000, 2000), (0, 5000)])
def test_one_cta_and_a_cluster(q4, total, S):
    rng = random.Random(total + S)
    cuts = sorted(rng.randint(0, total) for _ in range(S - 1))
    p = Pair(q4, S + 2, 20000 // 16 + 2, 20000 // 16 + S + 7, 16)
    slot = rng.sample(range(S + 2), S)
    n = p.step([0] + cuts + [total], slot, [0] * S, total)
    p.step([0] * (S + 1), slot, [x // 2 for x in n], 0)  # cut back
    p.step(list(range(S + 1)), slot, [x // 2 for x in n], S)
    p.step([0] * (S + 1), slot, [0] * S, 0)  # ended
    assert p.ref.count == p.ref.pages


def test_the_most_requests_and_slots(q4):
    S, slots = 8192, 65536
    rng = random.Random(1)
    p = Pair(q4, slots, 2, S + 100, 16)
    slot = rng.sample(range(slots), S)
    p.step(list(range(S + 1)), slot, [0] * S, S)
    p.step(_starts([i % 3 for i in range(S)]), slot, [1] * S, sum(i % 3 for i in range(S)))


def test_requests_that_break_a_rule_are_left_as_they_are(q4):
    p = Pair(q4, 4, 3, 9, 16)
    p.step([0, 20, 30], [0, 1], [0, 0], 30)
    for slot, pos, rows in (
            ([-1, 1], [0, 10], [1, 1]), ([4, 1], [0, 10], [1, 1]), ([2, 2], [0, 0], [5, 5]), ([1, 2, 1], [10, 0, 0], [1, 2, 0]),
            ([0, 2], [-1, 0], [1, 1]), ([0, 3], [20, 0], [29, 3]), ([0, 3], [33, 0], [1, 3]), ([2, 3], [1, 0], [3, 3]),
            ([0, 1], [2 ** 31 - 1, 11], [1, 1])):
        off = _starts(rows)
        p.step(off, slot, pos, off[-1])
    # offsets that decrease, begin below 0 or pass total: nobody's rows can be told
    for off in ([0, 5, 3], [-1, 2, 3], [0, 2, 9]):
        p.step(off, [0, 1], [20, 10], 8)
    # rows before the first request and after the last
    p.step([2, 4, 6], [0, 1], [20, 10], 9)


def test_a_pool_that_is_not_one_is_not_touched(q4):
    for where, value in ((0, -1), (0, 10), (10, 7), (10, -1)):  # the count; the pages of slot 0
        t = q4.Q4PageTable(2, 6, 9, 16)
        q4.q4_paged_reserve(t, _i32([0, 70]), _i32([0]), _i32([0]), 70)
        t.state[where] = value
        before = t.state.clone()
        m, n = q4.q4_paged_reserve(t, _i32([0, 20]), _i32([0]), _i32([70]), 20)
        assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
        assert m.tolist() == [-1] * 20 and n.tolist() == [-1] and torch.equal(t.state, before)
    # more pages given back than there are
    t = q4.Q4PageTable(2, 6, 9, 16)
    q4.q4_paged_reserve(t, _i32([0, 70]), _i32([0]), _i32([0]), 70)
    t.free_count.fill_(6)
    before = t.state.clone()
    m, n = q4.q4_paged_reserve(t, _i32([0, 0]), _i32([0]), _i32([0]), 0)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG and n.tolist() == [-1] and torch.equal(t.state, before)
    # page numbers out of range are not passed on
    t = q4.Q4PageTable(1, 6, 9, 16)
    t.free.fill_(9)
    m, n = q4.q4_paged_reserve(t, _i32([0, 3]), _i32([0]), _i32([0]), 3)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG and m.tolist() == [-1] * 3


def test_reserve_in_a_graph_and_on_another_stream(q4):
    p = Pair(q4, 3, 40, 100, 16)
    p.step([0, 0], [0], [0], 0)  # the first call of a process allocates
    off, slot, pos = _i32([0, 1, 2, 3]), _i32([0, 1, 2]), _i32([0, 0, 0])
    m, n = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        q4.q4_paged_reserve(p.gpu, off, slot, pos, 3, slot_map=m, new_length=n)
        pos.copy_(n)
    for i in range(40):
        g.replay()
        want, _, _, _ = p.ref.reserve([0, 1, 2, 3], [0, 1, 2], [i] * 3, 3)
        torch.cuda.synchronize()
        assert m.tolist() == want
    p.same()
    side.wait_stream(torch.cuda.current_stream())
    q4.q4_paged_reserve(p.gpu, _i32([0, 0]), _i32([1]), _i32([0]), 0, stream=side)
    p.ref.reserve([0, 0], [1], [0], 0)
    torch.cuda.synchronize()
    p.same()
    assert q4.q4_device_status() == q4.Q4_OK


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("cache_dtype,dtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                               (torch.bfloat16, torch.float32), (torch.float16, torch.float32)])
@pytest.mark.parametrize("heads,d,page", [(1, 64, 16), (4, 128, 64), (2, 64, 128), (3, 128, 32)])
@pytest.mark.parametrize("total", [1, 7, 300])
def test_appended_rows(q4, cache_dtype, dtype, heads, d, page, total):
    c = q4.Q4PagedCache(total // page + 9, heads, d, page, dtype=cache_dtype)
    places = c.pages * page
    rng = random.Random(total)
    where = rng.sample(range(places), total)
    if total > 1:
        where[total // 2] = -1
    # K and V side by side; values that round up, to infinity and to 0, NaN
    kv = _normal(3, (total, 2 * heads, d), dtype).cuda()
    kv.view(-1)[::97] *= 1e38 if dtype == torch.float32 else 1.0
    kv.view(-1)[1::97] *= 1e-41 if dtype == torch.float32 else 1.0
    kv.view(-1)[5::211] = float("nan")
    kv.view(-1)[6::211] = float("-inf")
    kv.view(-1)[7::211] = -0.0
    c.k.fill_(5.0)
    c.v.fill_(6.0)
    want = [c.k.clone(), c.v.clone()]
    for x, rows in zip(want, (kv[:, :heads], kv[:, heads:])):
        for t, w in enumerate(where):
            if w >= 0:
                x[w // page, :, w % page] = rows[t].to(cache_dtype)
    q4.q4_paged_append(c, kv[:, :heads], kv[:, heads:], _i32(where))
    assert q4.q4_device_status() == q4.Q4_OK
    for got, x in zip((c.k, c.v), want):
        nan = torch.isnan(x)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got.view(torch.int16)[~nan], x.view(torch.int16)[~nan])


def test_places_out_of_range_are_not_written(q4):
    c = q4.Q4PagedCache(2, 1, 64, 16)
    c.k.zero_()
    k = torch.ones((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    q4.q4_paged_append(c, k, k, _i32([32, -2, 31, 2 ** 31 - 1]))
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    assert int(c.k.ne(0).sum()) == 64 and bool(c.k[1, 0, 15].eq(1).all())
    q4.q4_paged_append(c, k[:0], k[:0], _i32([]))
    assert q4.q4_device_status() == q4.Q4_OK


# ---------------------------------------------------------------- attention

def _check(o, q, k, v, past, scale, dtype, what):
    """One request's rows per head: o, q [n, hq, d], k, v [past + n, h, d], float64; the worst share of the bound."""
    n, hq, d = q.shape
    m, h, _ = k.shape
    worst, u = 0.0, UNIT[dtype]
    see = np.arange(m)[None, :] <= past + np.arange(n)[:, None]
    for x in range(hq):
        kk, vv, qq = k[:, x // (hq // h)], v[:, x // (hq // h)], q[:, x]
        s = np.where(see, scale * (qq @ kk.T), -np.inf)
        e = np.exp(s - s.max(-1, keepdims=True))
        w = e / e.sum(-1, keepdims=True)
        want = w @ vv
        ds = 2.0 ** -19 * scale * np.where(see, np.abs(qq) @ np.abs(kk).T, 0.0).max(-1, keepdims=True)
        bound = (4 * ds + u + 2.0 ** -16) * (w @ np.abs(vv)) + 2.0 ** -22 * np.abs(vv).max() + u * np.abs(want)
        err = np.abs(o[:, x] - want)
        assert np.all(err <= bound), "%s head %d: %.3g of the bound at %s" % (
            what, x, (err / bound).max(), np.unravel_index(np.argmax(err / bound), err.shape))
        worst = max(worst, float((err / bound).max()))
    return worst


class Step:
    """A step over a cache whose unused places hold NaN: requests of past positions and new rows."""

    def __init__(self, q4, seed, past, rows, heads, hq, d, page, dtype, sigma=1.0, gap=0):
        self.q4, self.past, self.rows, self.dtype, self.d = q4, past, rows, dtype, d
        S = len(rows)
        rng = random.Random(seed)
        need = [-(-(p + n) // page) for p, n in zip(past, rows)]
        pages = sum(need) + 3
        self.cache = q4.Q4PagedCache(pages, heads, d, page, dtype=dtype)
        self.tables = q4.Q4PageTable(S + 2, max(need + [1]) + 2, pages, page)
        self.cache.k.fill_(float("nan"))
        self.cache.v.fill_(float("nan"))
        self.slot = rng.sample(range(S + 2), S)
        numbers = rng.sample(range(pages), pages)
        table = np.full((S + 2, self.tables.width), 2 ** 30, np.int64)  # never looked at
        self.k, self.v, where = [], [], []
        for s in range(S):
            n = past[s] + rows[s]
            ids, numbers = numbers[:need[s]], numbers[need[s]:]
            table[self.slot[s], :need[s]] = ids
            self.k.append(_normal(seed + 7 * s, (n, heads, d), dtype))
            self.v.append(_normal(seed + 7 * s + 1, (n, heads, d), dtype))
            where += [ids[p // page] * page + p % page for p in range(n)]
        self.tables.table.copy_(torch.from_numpy(table))
        self.gap = gap  # rows before the first request and after the last
        self.offsets = [gap + x for x in _starts(rows)]
        self.total = sum(rows) + 2 * gap
        self.q = _normal(seed + 5, (self.total, hq, d), dtype, sigma)
        self.where = where
        self.fill()

    def fill(self):
        if self.where:
            self.q4.q4_paged_append(self.cache, torch.cat(self.k).cuda(), torch.cat(self.v).cuda(), _i32(self.where))

    def run(self, scale=None, q=None, out=None, stream=None):
        return self.q4.q4_paged_attention(self.cache, self.tables, self.q.cuda() if q is None else q, _i32(self.offsets),
                                          _i32(self.slot), _i32(self.past), scale=scale, out=out, stream=stream)

    def check(self, out, scale=None):
        assert self.q4.q4_device_status() == self.q4.Q4_OK
        scale = self.d ** -0.5 if scale is None else scale
        o, q = out.cpu().double().numpy(), self.q.double().numpy()
        worst = 0.0
        for s, n in enumerate(self.rows):
            b = self.offsets[s]
            worst = max(worst, _check(o[b:b + n], q[b:b + n], self.k[s].double().numpy(), self.v[s].double().numpy(),
                                      self.past[s], scale, self.dtype, "request %d" % s)) if n else worst
        gap = self.gap
        assert not o[:gap].any() and not o[self.total - gap:].any()
        return worst


HEADS = [(4, 28, 128), (2, 14, 64), (8, 8, 64), (2, 2, 128), (1, 16, 128), (1, 3, 64)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,hq,d", HEADS)
@pytest.mark.parametrize("page", PAGES)
def test_steps_of_all_kinds(q4, dtype, heads, hq, d, page):
    # single tokens with nothing, a page less one, a page, a block and more behind them; drafts; chunks; nothing
    past = [0, 15, 16, 127, 128, 129, 1000, 0, 300, 0, 63, 5, 200, 640]
    rows = [1, 1, 1, 1, 1, 1, 1, 2, 5, 130, 17, 0, 40, 300]
    s = Step(q4, 10, past, rows, heads, hq, d, page, dtype, gap=3)
    out = torch.full((s.total, hq, d), 9.0, dtype=dtype, device="cuda")
    s.check(s.run(out=out))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,hq,d", HEADS[:4])
def test_long_requests_are_divided(q4, dtype, heads, hq, d):
    # one request, so that its blocks go to as many CTAs as there are
    s = Step(q4, 20, [6000], [1], heads, hq, d, 16, dtype)
    s.check(s.run())
    s = Step(q4, 21, [3333], [100], heads, hq, d, 64, dtype)
    s.check(s.run())


@pytest.mark.parametrize("heads,hq,d", HEADS[:2])
def test_many_requests(q4, heads, hq, d):
    rng = random.Random(3)
    past = [rng.choice((0, 1, 31, rng.randint(0, 400))) for _ in range(700)]
    rows = [rng.choice((0, 1, 1, 1, 2)) for _ in past]
    s = Step(q4, 30, past, rows, heads, hq, d, 32, torch.bfloat16, gap=1)
    s.check(s.run())


@pytest.mark.parametrize("S", [1, 31, 32, 33, 64, 65, 127, 128, 129, 640, 641])
def test_counts_of_requests(q4, S):
    # up to 128 one warp looks through them, up to 640 each thread through one
    rng = random.Random(S)
    past = [rng.choice((0, 1, 15, rng.randint(0, 300))) for _ in range(S)]
    rows = [rng.choice((1, 1, 0, 2, 9, 40)) if S < 200 else rng.choice((1, 0)) for _ in past]
    rows[-1] = 3
    s = Step(q4, 31, past, rows, 1, 2, 64, 16, torch.float16, gap=2)
    s.check(s.run())


@pytest.mark.parametrize("S", [100, 5000])
def test_requests_without_rows(q4, S):
    # a padded step: most requests bring nothing, runs of them lie between the others and at both ends
    rows = [0] * S
    for i, n in ((3, 1), (35, 40), (36, 1), (S // 2, 5), (S - 20, 300), (S - 2, 1)):
        rows[i] = n
    past = [(i * 7) % 900 if n else 0 for i, n in enumerate(rows)]
    s = Step(q4, 33, past, rows, 2, 14, 64, 16, torch.bfloat16, gap=1)
    s.check(s.run())


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 64, 126, 127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("heads,hq", [(2, 2), (1, 8), (1, 7)])
def test_rows_at_the_borders_of_tiles(q4, rows, heads, hq):
    # light rows (rows x group up to 8), one tile, two tiles, two pairs; pasts that end at and beside a block
    for past in (0, 127, 128, 700):
        s = Step(q4, 32, [past, 5], [rows, 1], heads, hq, 64, 32, torch.bfloat16)
        s.check(s.run())


@pytest.mark.parametrize("hq,heads", [(128, 1), (64, 1), (40, 1), (33, 1), (130, 2)])
def test_large_groups(q4, hq, heads):
    s = Step(q4, 40, [100, 0, 257], [1, 5, 3], heads, hq, 64, 16, torch.float16)
    s.check(s.run())


@pytest.mark.parametrize("sigma,scale", [(30.0, None), (1.0, 4.0), (1e-3, None)])
@pytest.mark.parametrize("dtype", TYPES)
def test_sharp_and_flat_weights(q4, sigma, scale, dtype):
    s = Step(q4, 50, [900, 0, 2500], [1, 200, 9], 2, 14, 128, 32, dtype, sigma=sigma)
    s.check(s.run(scale=scale), scale)


@pytest.mark.parametrize("slope", [0.05, -0.05, 40.0, -40.0])
def test_rising_and_falling_scores(q4, slope):
    # each block's scores lie far above or below the last one's, in and across the pieces of a request
    n, d = 3000, 64
    s = Step(q4, 60, [n - 150], [150], 1, 1, d, 16, torch.bfloat16)
    k = (torch.arange(n).float() * slope).to(torch.bfloat16)
    s.q.fill_(1.0)
    s.k[0] = k[:, None, None].expand(n, 1, d).contiguous()
    s.fill()
    s.check(s.run())


def test_scores_far_from_zero(q4):
    # references of a size whose steps a weight would show: a large common part, small differences
    n, d = 2000, 128
    s = Step(q4, 61, [n - 20], [20], 1, 2, d, 32, torch.bfloat16)
    s.q[:] = 1.0
    s.k[0][:] = 0.0
    s.k[0][:, :, 0] = 2.0 ** 16
    s.k[0][:, :, 1] = (torch.arange(n) % 7).to(torch.bfloat16)[:, None]
    s.fill()
    s.check(s.run(scale=1.0), 1.0)


@pytest.mark.parametrize("heads,hq,d", HEADS[:2])
@pytest.mark.parametrize("past", [0, 70, 1500])
def test_values_that_a_row_does_not_see(q4, heads, hq, d, past):
    # infinities and NaN in V and K of later rows of the same chunk reach the rows that see them only
    n = 90
    s = Step(q4, 70, [past, 3], [n, 2], heads, hq, d, 16, torch.bfloat16)
    clean = s.run().clone()
    s.v[0][past + 40, :, 5] = float("nan")
    s.v[0][past + 60, :, 6] = float("inf")
    s.v[0][past + 61, :, 7] = float("-inf")
    s.k[0][past + 80] = float("nan")
    s.fill()
    out = s.run()
    assert q4.q4_device_status() == q4.Q4_OK
    o = out.float()
    assert torch.equal(out[:40], clean[:40]) and torch.equal(out[n:], clean[n:])
    assert bool(torch.isnan(o[40:n, :, 5]).all()) and not bool(torch.isnan(o[:40]).any())
    assert bool(torch.isposinf(o[60:80, :, 6]).all()) and bool(torch.isneginf(o[61:80, :, 7]).all())
    assert bool(torch.isfinite(o[40:60, :, 8:]).all()) and bool(torch.isnan(o[80:n]).all())
    assert torch.equal(out[40:80, :, 8:], clean[40:80, :, 8:])


def test_an_infinity_in_a_divided_request(q4):
    s = Step(q4, 71, [5000], [1], 1, 2, 64, 16, torch.float16)
    s.v[0][77, 0, 3] = float("inf")
    s.v[0][4000, 0, 4] = float("nan")
    s.fill()
    o = s.run()[0].float()
    assert bool(torch.isposinf(o[:, 3]).all()) and bool(torch.isnan(o[:, 4]).all())
    assert bool(torch.isfinite(o[:, 5:]).all()) and bool(torch.isfinite(o[:, :3]).all())


@pytest.mark.parametrize("heads,hq,d", [(4, 28, 128), (2, 14, 64)])
def test_views_and_out_in_place(q4, heads, hq, d):
    s = Step(q4, 80, [40, 500, 0], [1, 30, 77], heads, hq, d, 32, torch.bfloat16, gap=2)
    want = s.run()
    wide = torch.randn((s.total, hq + 5, d), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + hq] = s.q.cuda()
    assert torch.equal(s.run(q=wide[:, 2:2 + hq]), want)
    heads_first = s.q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(s.run(q=heads_first), want)
    q = s.q.cuda()
    assert s.run(q=q, out=q) is q and torch.equal(q, want)
    # 16-byte aligned only
    base = torch.zeros(s.total * hq * d + 8, dtype=torch.bfloat16, device="cuda")
    out = base[8:].view(s.total, hq, d)
    assert torch.equal(s.run(out=out), want)
    s.check(want)


def test_the_same_call_gives_the_same_bits(q4):
    s = Step(q4, 90, [3000, 17, 900], [1, 60, 4], 4, 28, 128, 16, torch.float16)
    first = s.run().clone()
    for _ in range(5):
        assert torch.equal(s.run(), first)


def test_requests_out_of_range(q4):
    s = Step(q4, 100, [40, 20, 30], [3, 2, 70], 2, 14, 64, 16, torch.bfloat16)
    want = s.run().clone()
    reach = s.tables.width * 16
    for slot, past in ((-1, 20), (5, 20), (s.slot[1], -1), (s.slot[1], reach - 1)):
        out = torch.full_like(want, 9.0)
        q4.q4_paged_attention(s.cache, s.tables, s.q.cuda(), _i32(s.offsets), _i32([s.slot[0], slot, s.slot[2]]),
                              _i32([40, past, 30]), out=out)
        assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
        assert not out[3:5].any() and torch.equal(out[:3], want[:3])
        s_out = out.cpu().double().numpy()
        assert _check(s_out[5:], s.q.double().numpy()[5:], s.k[2].double().numpy(), s.v[2].double().numpy(), 30, 0.125,
                      torch.bfloat16, "the others") < 1
    # offsets that pass total, and no request at all
    out = torch.full_like(want, 9.0)
    q4.q4_paged_attention(s.cache, s.tables, s.q.cuda(), _i32([0, 3, 200]), _i32(s.slot[:2]), _i32([40, 20]), out=out)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    assert torch.equal(out[:3].isfinite(), torch.ones_like(out[:3], dtype=torch.bool)) and not out[3:].any()
    out = torch.full_like(want, 9.0)
    q4.q4_paged_attention(s.cache, s.tables, s.q.cuda(), _i32([0, 0]), _i32(s.slot[:1]), _i32([0]), out=out)
    assert q4.q4_device_status() == q4.Q4_OK and not out.any()


@pytest.mark.parametrize("page,number", [(16, -1), (32, 2 ** 31 - 1), (128, -2 ** 31)])
def test_page_numbers_out_of_range_read_as_zeros(q4, page, number):
    s = Step(q4, 110, [300], [4], 2, 14, 64, page, torch.bfloat16)
    s.tables.table[s.slot[0], 1] = number
    out = s.run()
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG
    s.k[0][page:2 * page] = 0
    s.v[0][page:2 * page] = 0
    s.check(out)


def test_a_graph_over_growing_requests_and_two_graphs_in_turn(q4):
    heads, hq, d, page = 2, 14, 64, 16
    s = Step(q4, 120, [100, 7], [50, 50], heads, hq, d, page, torch.bfloat16)  # 50 rows each, one a step
    q = torch.zeros((2, hq, d), dtype=torch.bfloat16, device="cuda")
    off, slot, pos = _i32([0, 1, 2]), _i32(s.slot), _i32([100, 7])
    outs = [torch.zeros_like(q), torch.zeros_like(q)]
    graphs = []
    s.run()
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q4.q4_paged_attention(s.cache, s.tables, q, off, slot, pos, out=out)
        graphs.append(g)
    rows = [s.q[:50].cuda(), s.q[50:].cuda()]
    for i in range(0, 50, 7):
        q.copy_(torch.stack([rows[0][i], rows[1][i]]))
        pos.copy_(_i32([100 + i, 7 + i]))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        for r, past in enumerate((100, 7)):
            n = past + i
            _check(outs[0][r:r + 1].cpu().double().numpy(), q[r:r + 1].cpu().double().numpy(),
                   s.k[r][:n + 1].double().numpy(), s.v[r][:n + 1].double().numpy(), n, d ** -0.5, torch.bfloat16, "graph")
    assert q4.q4_device_status() == q4.Q4_OK


def test_another_stream(q4):
    s = Step(q4, 130, [200, 900], [4, 60], 2, 14, 64, 32, torch.float16)
    want = s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q = s.q.cuda()
    side.wait_stream(torch.cuda.current_stream())
    out = s.run(q=q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)


def test_pages_past_32_bits(q4):
    # the cache has more than 2^31 values; the request's pages are its last ones
    page, heads, d = 128, 8, 128
    pages = (2 ** 31 // (page * heads * d)) + 40
    cache = q4.Q4PagedCache(pages, heads, d, page)
    tables = q4.Q4PageTable(1, 4, pages, page)
    tables.table[0] = _i32([pages - 1, pages - 3, pages - 2, pages - 4])
    n = 300
    k, v = _normal(140, (n, heads, d), torch.bfloat16), _normal(141, (n, heads, d), torch.bfloat16)
    where = [int(tables.table[0, p // page]) * page + p % page for p in range(n)]
    q4.q4_paged_append(cache, k.cuda(), v.cuda(), _i32(where))
    assert torch.equal(cache.k[pages - 1, :, 5].cpu(), k[5]) and torch.equal(cache.v[pages - 3, :, 1].cpu(), v[129])
    q = _normal(142, (3, 8, d), torch.bfloat16)
    out = q4.q4_paged_attention(cache, tables, q.cuda(), _i32([0, 3]), _i32([0]), _i32([n - 3]))
    assert q4.q4_device_status() == q4.Q4_OK
    _check(out.cpu().double().numpy(), q.double().numpy(), k.double().numpy(), v.double().numpy(), n - 3, d ** -0.5,
           torch.bfloat16, "last pages")


def test_a_long_chunk_that_fills_its_table(q4):
    n, past, d, page = 40000, 960, 64, 64
    total = n + past
    cache = q4.Q4PagedCache(total // page, 1, d, page)
    tables = q4.Q4PageTable(1, total // page, total // page, page)
    slot_map, length = q4.q4_paged_reserve(tables, _i32([0, total]), _i32([0]), _i32([0]), total)
    assert length.tolist() == [total] and torch.equal(slot_map, torch.arange(total, dtype=torch.int32, device="cuda"))
    k, v, q = (_normal(180 + i, (m, h, d), torch.bfloat16) for i, (m, h) in enumerate(((total, 1), (total, 1), (n, 2))))
    q4.q4_paged_append(cache, k.cuda(), v.cuda(), slot_map)
    out = q4.q4_paged_attention(cache, tables, q.cuda(), _i32([0, n]), _i32([0]), _i32([past])).cpu().double().numpy()
    assert q4.q4_device_status() == q4.Q4_OK
    k, v, q = (x.double().numpy() for x in (k, v, q))
    for i in (0, 1, 63, 64, 127, 128, 5000, 12345, 20031, 39999):
        _check(out[i:i + 1], q[i:i + 1], k[:past + i + 1], v[:past + i + 1], past + i, d ** -0.5, torch.bfloat16, "row %d" % i)


def test_a_whole_step_in_a_graph(q4):
    """Pages, rows and attention of two decoding requests captured once; each replay is a step further."""
    heads, hq, d, page, steps = 2, 14, 64, 16, 40
    tables = q4.Q4PageTable(3, 8, 20, page)
    cache = q4.Q4PagedCache(20, heads, d, page)
    k, v, q = (_normal(190 + i, (steps + 1, 2, h, d), torch.bfloat16).cuda() for i, h in enumerate((heads, heads, hq)))
    off, slot, pos = _i32([0, 1, 2]), _i32([2, 0]), _i32([0, 0])
    now = [torch.empty_like(x[0]) for x in (k, v, q)]

    def step():
        slot_map, length = q4.q4_paged_reserve(tables, off, slot, pos, 2)
        q4.q4_paged_append(cache, now[0], now[1], slot_map)
        out = q4.q4_paged_attention(cache, tables, now[2], off, slot, pos)
        pos.copy_(length)
        return out

    def feed(i):
        for x, y in zip(now, (k, v, q)):
            x.copy_(y[i])

    feed(0)
    first = step().clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    got = [first]
    for i in range(1, steps + 1):
        feed(i)
        g.replay()
        got.append(out.clone())
    assert q4.q4_device_status() == q4.Q4_OK and pos.tolist() == [steps + 1] * 2
    o = torch.stack(got).cpu().double().numpy()
    kk, vv, qq = (x.cpu().double().numpy() for x in (k, v, q))
    for r in range(2):
        _check(o[:, r], qq[:, r], kk[:, r], vv[:, r], 0, d ** -0.5, torch.bfloat16, "request %d" % r)


@pytest.mark.parametrize("past,rows", [([3000, 40], [1, 1]), ([500, 900], [300, 1]), ([300], [20])])
def test_waits_that_run_out(q4, past, rows):
    """No copy is issued, so every wait for one runs out: the status says so, and later calls are right."""
    s = Step(q4, 150, past, rows, 2, 14, 64, 16, torch.bfloat16)
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


def test_beside_the_other_attentions(q4):
    """The calls that share the library's scratch, one after another on a stream and in a graph."""
    heads, hq, d = 2, 14, 64
    s = Step(q4, 160, [2500, 100], [1, 30], heads, hq, d, 16, torch.bfloat16)
    kvq = q4.Q4KVCache(2, heads, d, 4000)
    k, v = (_normal(161 + i, (3000, heads, d), torch.bfloat16).cuda() for i in range(2))
    q4.q4_kvq_append(kvq, k, v, _i32([0, 3000]), _i32([1]), _i32([0]))
    q1 = _normal(163, (1, hq, d), torch.bfloat16).cuda()
    off, slot, pos = _i32([0, 1]), _i32([1]), _i32([2999])
    prompt = _normal(164, (200, hq + 2 * heads, d), torch.bfloat16).cuda()
    poff = _i32([0, 200])
    q, soff, sslot, spos = s.q.cuda(), _i32(s.offsets), _i32(s.slot), _i32(s.past)

    def calls():
        a = q4.q4_paged_attention(s.cache, s.tables, q, soff, sslot, spos)
        b = q4.q4_kvq_attention(kvq, q1, off, slot, pos)
        c = q4.q4_paged_attention(s.cache, s.tables, q, soff, sslot, spos)
        e = q4.q4_prompt_attention(prompt[:, :hq], prompt[:, hq:hq + heads], prompt[:, hq + heads:], poff)
        return a, b, c, e, q4.q4_paged_attention(s.cache, s.tables, q, soff, sslot, spos)

    alone = s.run().clone()
    first = [x.clone() for x in calls()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = calls()
    for _ in range(10):
        g.replay()
        calls()
        torch.cuda.synchronize()
        for x, y in zip(outs, first):
            assert torch.equal(x, y)
    for i in (0, 2, 4):
        assert torch.equal(first[i], alone)
    assert q4.q4_device_status() == q4.Q4_OK


def test_the_binding_refuses(q4):
    s = Step(q4, 170, [10, 3], [1, 2], 2, 4, 64, 16, torch.bfloat16)
    q, off, slot, pos = s.q.cuda(), _i32(s.offsets), _i32(s.slot), _i32(s.past)
    attend = q4.q4_paged_attention
    other = q4.Q4PageTable(4, 3, s.cache.pages, 32)
    for bad in (lambda: attend(s.cache, s.tables, q.half(), off, slot, pos),
                lambda: attend(s.cache, s.tables, s.q, off, slot, pos),
                lambda: attend(s.cache, other, q, off, slot, pos),
                lambda: attend(s.cache, s.tables, q[:, :3], off, slot, pos),
                lambda: attend(s.cache, s.tables, q, off[:2], slot, pos),
                lambda: attend(s.cache, s.tables, q, off, slot.long(), pos),
                lambda: attend(s.cache, s.tables, q.transpose(1, 2), off, slot, pos),
                lambda: attend(s.cache, s.tables, q, off, slot, pos, out=torch.empty_like(q)[:1]),
                lambda: q4.q4_paged_append(s.cache, q[:, :2], q[:, 2:], _i32([0, 1])),
                lambda: q4.q4_paged_append(s.cache, q[:, :2].half(), q[:, 2:].half(), _i32([0, 1, 2])),
                lambda: q4.q4_paged_append(s.cache, q[:, :2], q[:2, 2:], _i32([0, 1, 2])),
                lambda: q4.q4_paged_reserve(s.tables, off, slot, pos[:1], 3),
                lambda: q4.q4_paged_reserve(s.tables, off, slot, pos, 3, slot_map=_i32([0, 0]))):
        with pytest.raises((ValueError, q4.Q4Error)):
            bad()
    assert q4.q4_device_status() == q4.Q4_OK
    s.check(s.run())


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [16, 128])
def test_requests_come_grow_and_end(q4, dtype, page):
    """Steps of prompts in pieces, decode rows and drafts of which some are rejected, as a serving loop makes them."""
    heads, hq, d, slots = 2, 14, 64, 5
    rng = random.Random(page)
    tables = q4.Q4PageTable(slots, 1024 // page + 1, 5 * 1024 // page, page)
    cache = q4.Q4PagedCache(tables.pages, heads, d, page, dtype=dtype)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    held = {}  # slot: its K and V rows so far
    seed = 1000
    for step in range(25):
        slot, pos, rows, gone = [], [], [], []
        for s in range(slots):
            if s not in held:
                if rng.random() < 0.5:
                    held[s] = (torch.zeros((0, heads, d), dtype=dtype), torch.zeros((0, heads, d), dtype=dtype))
                    slot.append(s), pos.append(0), rows.append(rng.choice((1, 16, 100, 200)))
                continue
            n = len(held[s][0])
            if n > 700 or rng.random() < 0.1:
                del held[s]
                slot.append(s), pos.append(0), rows.append(0), gone.append(s)
                continue
            back = rng.choice((0, 0, 0, min(n, 3)))  # rejected drafts
            held[s] = tuple(x[:n - back] for x in held[s])
            slot.append(s), pos.append(n - back), rows.append(rng.choice((1, 1, 5, 60)))
        if not slot:
            continue
        off = _starts(rows)
        total = off[-1]
        k, v, q = (_normal(seed + i, (total, h, d), torch.float32) for i, h in enumerate((heads, heads, hq)))
        seed += 3
        dev = (_i32(off), _i32(slot), _i32(pos))
        slot_map, length = q4.q4_paged_reserve(tables, *dev, total)
        q4.q4_paged_append(cache, k.cuda(), v.cuda(), slot_map)
        out = q4.q4_paged_attention(cache, tables, q.to(dtype).cuda(), *dev)
        assert q4.q4_device_status() == q4.Q4_OK
        assert length.tolist() == [p + n for p, n in zip(pos, rows)]
        o = out.cpu().double().numpy()
        for i, s in enumerate(slot):
            if s in gone or rows[i] == 0:
                continue
            a, b = off[i], off[i + 1]
            held[s] = (torch.cat([held[s][0], k[a:b].to(dtype)]), torch.cat([held[s][1], v[a:b].to(dtype)]))
            _check(o[a:b], q[a:b].to(dtype).double().numpy(), held[s][0].double().numpy(), held[s][1].double().numpy(),
                   pos[i], d ** -0.5, dtype, "step %d slot %d" % (step, s))
    used = sum(-(-len(x[0]) // page) for x in held.values())
    assert int(tables.free_count) == tables.pages - used
