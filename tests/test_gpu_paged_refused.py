"""Steps of the paged cache in which the pool runs out: reserve refuses requests, append leaves their rows out, and
the attention of the same step gives them zeros and the others what they would get without them."""
import random

import pytest
import torch

from oracle import paged
from test_gpu_paged import _check, _i32, _normal, _starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


class Requests:
    """A pool, its oracle, a cache and the rows that each slot has so far; the cache's unused places hold NaN."""

    def __init__(self, q4, heads, hq, d, page, dtype, slots, pages):
        self.q4, self.heads, self.hq, self.d, self.dtype = q4, heads, hq, d, dtype
        self.tables, self.pool = q4.Q4PageTable(slots, pages, pages, page), paged.Pool(slots, pages, pages, page)
        self.cache = q4.Q4PagedCache(pages, heads, d, page, dtype=dtype)
        self.cache.k.fill_(float("nan"))
        self.cache.v.fill_(float("nan"))
        none = torch.zeros((0, heads, d), dtype=dtype)
        self.k, self.v = [none] * slots, [none] * slots
        self.seed = 500

    def step(self, slot, rows, in_place=False):
        """One step: (rows of new_len that were refused, the device's status); all results checked."""
        q4 = self.q4
        pos, off = [len(self.k[s]) for s in slot], _starts(rows)
        total = off[-1]
        k, v, q = (_normal(self.seed + i, (total, h, self.d), self.dtype)
                   for i, h in enumerate((self.heads, self.heads, self.hq)))
        self.seed += 3
        dev = (_i32(off), _i32(slot), _i32(pos))
        slot_map, length = q4.q4_paged_reserve(self.tables, *dev, total)
        want_map, want_length, _, _ = self.pool.reserve(off, slot, pos, total)
        q4.q4_paged_append(self.cache, k.cuda(), v.cuda(), slot_map)
        queries = q.cuda()
        out = queries if in_place else torch.full_like(queries, 9.0)
        q4.q4_paged_attention(self.cache, self.tables, queries, *dev, out=out)
        status = q4.q4_device_status()
        assert slot_map.tolist() == want_map and length.tolist() == want_length
        o = out.cpu().double().numpy()
        for i, s in enumerate(slot):
            a, b = off[i], off[i + 1]
            if want_length[i] < 0:
                assert not o[a:b].any(), "rows of refused request %d" % i
            elif a < b:
                self.k[s], self.v[s] = torch.cat([self.k[s], k[a:b]]), torch.cat([self.v[s], v[a:b]])
                _check(o[a:b], q[a:b].double().numpy(), self.k[s].double().numpy(), self.v[s].double().numpy(), pos[i],
                       self.d ** -0.5, self.dtype, "request %d" % i)
        return [i for i, n in enumerate(want_length) if n < 0], status


@pytest.mark.parametrize("heads,hq,d,page,dtype", [(2, 14, 64, 16, torch.bfloat16), (1, 7, 128, 32, torch.float16),
                                                   (8, 8, 64, 128, torch.bfloat16), (1, 16, 128, 64, torch.bfloat16)])
@pytest.mark.parametrize("idle,in_place", [(0, False), (200, True)])
def test_refused_requests_get_zeros(q4, heads, hq, d, page, dtype, idle, in_place):
    # slots 0-5; `idle` others without rows, so that the step is looked through by one warp or by all threads
    past = [page + 3, 600, 5 * page - 9, 4 * page, -(-2999 // page) * page - 5, -(-3000 // page) * page]
    pages = sum(-(-p // page) for p in past) + 2
    r = Requests(q4, heads, hq, d, page, dtype, 6 + idle, pages)
    assert r.step(list(range(6)), past) == ([], q4.Q4_OK)
    # 0 fits, 1 (a chunk) does not, nor do 3 and 5 (one row each, in a page of their own, few and many positions
    # behind them); 2 and 4 need no further page
    rows = [1, 200 + 2 * page, 5, 1, 1, 1]
    refused, status = r.step(list(range(6)) + list(range(6, 6 + idle)), rows + [0] * idle, in_place)
    assert refused == [1, 3, 5] and status == q4.Q4_ERR_NOMEM
    # the step after it: the chunk waits, a page that is left goes to slot 3
    refused, status = r.step([0, 3, 4, 5], [1, 1, 2, 0])
    assert refused == [] and status == q4.Q4_OK


def test_a_step_of_refused_requests_only(q4):
    page = 16
    r = Requests(q4, 2, 14, 64, page, torch.bfloat16, 3, 20)
    assert r.step([0, 1], [10 * page, 9 * page]) == ([], q4.Q4_OK)
    for rows in ([40, 1], [100, 3], [33, 16]):
        refused, status = r.step([0, 1], rows)
        assert refused == [0, 1] and status == q4.Q4_ERR_NOMEM


def test_a_pool_that_runs_out_step_by_step(q4):
    """Decode rows and chunks until most requests wait; the others go on as if nothing was."""
    rng = random.Random(4)
    r = Requests(q4, 2, 14, 64, 16, torch.float16, 8, 60)
    seen = set()
    for _ in range(14):
        slot = rng.sample(range(8), 6)
        refused, status = r.step(slot, [rng.choice((1, 1, 2, 30, 150)) for _ in slot])
        assert status == (q4.Q4_ERR_NOMEM if refused else q4.Q4_OK)
        seen.add(len(refused))
    assert 0 in seen and len(seen) > 2


def test_a_refused_request_beside_a_page_number_out_of_range(q4):
    page = 16
    r = Requests(q4, 2, 14, 64, page, torch.bfloat16, 3, 12)
    assert r.step([0, 1, 2], [4 * page, 3 * page, 4 * page + 3]) == ([], q4.Q4_OK)
    k, v, q = (_normal(900 + i, (3, h, 64), torch.bfloat16) for i, h in enumerate((2, 2, 14)))
    dev = (_i32([0, 1, 2, 3]), _i32([0, 1, 2]), _i32([4 * page, 3 * page, 4 * page + 3]))
    r.tables.free_count.fill_(0)  # requests 0 and 1 want a page
    slot_map, length = q4.q4_paged_reserve(r.tables, *dev, 3)
    q4.q4_paged_append(r.cache, k.cuda(), v.cuda(), slot_map)
    assert length.tolist() == [-1, -1, 4 * page + 4] and q4.q4_device_status() == q4.Q4_ERR_NOMEM
    r.tables.table[2, 1] = 12
    out = q4.q4_paged_attention(r.cache, r.tables, q.cuda(), *dev)
    assert q4.q4_device_status() == q4.Q4_ERR_INVALID_ARG  # the graver of the two
    assert not out[:2].any()
    k, v = (torch.cat([x[2], y[2:]]) for x, y in ((r.k, k), (r.v, v)))
    k[page:2 * page] = 0
    v[page:2 * page] = 0
    _check(out[2:].cpu().double().numpy(), q[2:].double().numpy(), k.double().numpy(), v.double().numpy(), 4 * page + 3,
           64 ** -0.5, torch.bfloat16, "request 2")


def test_a_pool_that_runs_out_in_a_graph(q4):
    """A captured step replayed past the pool's end: who is refused keeps its place and gets zeros until a page is free."""
    page, d = 16, 64
    tables = q4.Q4PageTable(2, 4, 3, page)
    cache = q4.Q4PagedCache(3, 2, d, page)
    steps = 40
    k, v, q = (_normal(950 + i, (steps, 2, h, d), torch.bfloat16).cuda() for i, h in enumerate((2, 2, 14)))
    off, slot, pos = _i32([0, 1, 2]), _i32([0, 1]), _i32([0, 0])
    now = [torch.empty_like(x[0]) for x in (k, v, q)]
    q4.q4_paged_attention(cache, tables, now[2], _i32([0, 0, 0]), slot, pos)  # the first call allocates
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        slot_map, length = q4.q4_paged_reserve(tables, off, slot, pos, 2)
        q4.q4_paged_append(cache, now[0], now[1], slot_map)
        out = q4.q4_paged_attention(cache, tables, now[2], off, slot, pos)
        pos.copy_(torch.where(length < 0, pos, length))
    rows, got = [[], []], []
    for i in range(steps):
        for x, y in zip(now, (k, v, q)):
            x.copy_(y[i])
        g.replay()
        torch.cuda.synchronize()
        got.append(out.clone())
        for s in range(2):
            if not (i >= 32 or (s == 1 and i >= 16)):
                rows[s].append(i)
        assert pos.tolist() == [len(rows[0]), len(rows[1])]
        assert q4.q4_device_status() == (q4.Q4_ERR_NOMEM if i >= 16 else q4.Q4_OK)
    o = torch.stack(got).cpu().double().numpy()
    kk, vv, qq = (x.cpu().double().numpy() for x in (k, v, q))
    for s in range(2):
        n = len(rows[s])
        _check(o[:n, s], qq[:n, s], kk[:n, s], vv[:n, s], 0, d ** -0.5, torch.bfloat16, "slot %d" % s)
        assert not o[n:, s].any()
