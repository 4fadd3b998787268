"""Paged attention where scores are large: references of any size, rising and falling from block to block, in light rows
(rows times heads of a group up to 8), one tile, two tiles, items that are cut and items that are not.

All scores are integers below 2^22, sums of two products of integers, so fp32 holds them exactly in
whatever order they are summed, and the oracle's weights are those of the very scores.  What is left:

- weights are rounded to the type, u = eps / 2 of each, and where float16 has no normal numbers left 2^-32 of the
  largest (3,000 of them: below 2^-20); the output is rounded once more, u |o|;
- where a row's reference passes 2^12 (in units of log2) on the way, references up to 2^12, rounded by 2^-12 at most each,
  are taken from one another: 2 * 2^-12 ln 2 < 2^-11 of a weight; powers of two and sums in fp32 are far below that.

    |o - o64| <= (u + 2^-11) * sum_j w_j |v_j| + 2^-20 max |v| + u |o64|

Every case asserts that an output of zeros, and the mean of the visible V rows, exceed the bound."""
import numpy as np
import pytest
import torch

from test_gpu_paged import UNIT, _i32, _normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


# (key/value heads, query heads, rows): light, light with a group, eight light rows; one tile; two tiles, two pairs
LAYOUTS = [(1, 1, 1), (2, 14, 1), (1, 1, 8), (1, 1, 20), (2, 14, 5), (1, 1, 150), (2, 14, 30), (1, 1, 300)]


def _far(j):
    # a large common part, differences of 0 to 6
    return 2.0 ** 16 + (j * 5) % 7, ((2.0 ** 6, 1.0), (np.full_like(j, 2 ** 10), (j * 5) % 7))


def _slope(slope):
    def scores(j):
        return slope * j, ((64.0 * slope, slope), (j // 64, j % 64))

    return scores


SCORES = {"far": _far, "40": _slope(40.0), "-40": _slope(-40.0), "2": _slope(2.0), "-2": _slope(-2.0)}
# (requests, positions, head size, page, type): one request is cut between the CTAs; of many alike, over
# the same pages, most items are whole
STEPS = [(1, 3000, 64, 16, torch.bfloat16), (1, 3000, 128, 64, torch.float16), (300, 600, 64, 32, torch.float16),
         (160, 600, 128, 128, torch.bfloat16)]


@pytest.mark.parametrize("heads,hq,rows", LAYOUTS)
@pytest.mark.parametrize("name", list(SCORES))
def test_large_scores(q4, heads, hq, rows, name):
    for step in STEPS:
        _check_step(q4, heads, hq, rows, name, *step)


def _check_step(q4, heads, hq, rows, name, requests, n, d, page, dtype):
    j = np.arange(n)
    score, (qs, ks) = SCORES[name](j)
    k = torch.zeros((n, heads, d), dtype=dtype)
    q = torch.zeros((rows, hq, d), dtype=dtype)
    for i, (a, b) in enumerate(zip(qs, ks)):
        q[:, :, i] = a
        k[:, :, i] = torch.from_numpy(np.asarray(b, np.float32))[:, None].to(dtype)
    exact = q[0, 0].double() @ k[:, 0].double().T
    assert np.array_equal(exact.numpy(), score) and np.abs(score).max() < 2 ** 22
    v = _normal(800, (n, heads, d), dtype)
    pages = -(-n // page)
    cache = q4.Q4PagedCache(pages, heads, d, page, dtype=dtype)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    tables = q4.Q4PageTable(requests, pages, pages, page)
    order = np.random.default_rng(1).permutation(pages)
    tables.table.copy_(torch.from_numpy(order.astype(np.int32)).expand(requests, pages))
    q4.q4_paged_append(cache, k.cuda(), v.cuda(), _i32(order[j // page] * page + j % page))
    out = q4.q4_paged_attention(cache, tables, q.cuda().repeat(requests, 1, 1), _i32(range(0, (requests + 1) * rows, rows)),
                                _i32(range(requests)), _i32([n - rows] * requests), scale=1.0)
    assert q4.q4_device_status() == q4.Q4_OK
    o = out.cpu().double().numpy().reshape(requests, rows, hq, d)
    see = j[None] <= n - rows + np.arange(rows)[:, None]
    s = np.where(see, score, -np.inf)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    u, vv = UNIT[dtype], v.double().numpy()
    want = np.repeat(np.einsum("rj,jhd->rhd", w, vv), hq // heads, 1)
    most = np.repeat(np.einsum("rj,jhd->rhd", w, np.abs(vv)), hq // heads, 1)
    bound = (u + 2.0 ** -11) * most + 2.0 ** -20 * np.abs(vv).max() + u * np.abs(want)
    mean = np.repeat(np.einsum("rj,jhd->rhd", see / see.sum(-1, keepdims=True), vv), hq // heads, 1)
    for wrong in (np.zeros_like(want), mean):
        assert ((np.abs(wrong - want) > bound).any(-1)).all()
    worst = (np.abs(o - want) / bound).max((1, 2, 3))
    assert (worst <= 1).all(), "%d requests of %s: %.3g of the bound, request %d" % (
        requests, dtype, worst.max(), worst.argmax())
