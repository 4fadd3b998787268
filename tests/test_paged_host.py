"""The paged cache's calls: refusals on the host, and the oracle of its pool (CPU)."""
import ctypes
import random

import numpy as np
import pytest

from oracle import paged

I2 = ctypes.c_int64 * 2
A = 1 << 20  # aligned stand-in addresses, far apart: the calls return before any CUDA call


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


def at(i):
    return A * (i + 1)


def reserve(q4, ptr=(), slots=4, width=8, pages=16, page=16, S=2, total=3):
    p = {i: at(i) for i in range(9)}
    p.update(ptr)
    return q4.raw_library().q4_paged_reserve(p[0], p[1], p[2], p[3], slots, width, pages, page, p[4], p[5], p[6], S,
                                             total, p[7], p[8], None)


def test_reserve_arguments(q4):
    bad, shape = q4.Q4_ERR_INVALID_ARG, q4.Q4_ERR_SHAPE
    for page in (0, 8, 17, 48, 256, -16):
        assert reserve(q4, page=page) == shape
    assert reserve(q4, slots=0) == bad and reserve(q4, width=0) == bad and reserve(q4, pages=0) == bad
    assert reserve(q4, slots=65537) == shape and reserve(q4, S=8193) == shape
    assert reserve(q4, S=-1) == bad and reserve(q4, total=-1) == bad
    assert reserve(q4, S=0, total=0) == q4.Q4_OK and reserve(q4, S=0, total=1) == bad
    assert reserve(q4, width=2 ** 27) == bad and reserve(q4, pages=2 ** 27) == bad
    assert reserve(q4, total=2 ** 30) == bad
    for i in range(9):
        assert reserve(q4, {i: None}) == bad, i


def test_reserve_outputs_overlap_nothing(q4):
    for out in (0, 1, 2, 3, 7, 8):
        for other in range(9):
            if other != out:
                assert reserve(q4, {out: at(other)}) == q4.Q4_ERR_INVALID_ARG, (out, other)


def append(q4, ptr=(), cache=2, dtype=2, pages=8, heads=2, d=64, page=16, ks=(128, 64), vs=(128, 64), total=3):
    p = {i: at(i) for i in range(5)}
    p.update(ptr)
    return q4.raw_library().q4_paged_append(p[0], p[1], cache, p[2], p[3], dtype, pages, heads, d, page,
                                            I2(*ks) if ks else None, I2(*vs) if vs else None, p[4], total, None)


def test_append_arguments(q4):
    bad, shape, align = q4.Q4_ERR_INVALID_ARG, q4.Q4_ERR_SHAPE, q4.Q4_ERR_ALIGN
    assert append(q4, page=24) == shape and append(q4, d=96) == shape
    assert append(q4, pages=0) == bad and append(q4, heads=0) == bad
    assert append(q4, cache=0) == bad and append(q4, cache=3) == bad
    assert append(q4, cache=1, dtype=2) == bad and append(q4, cache=2, dtype=1) == bad and append(q4, dtype=7) == bad
    assert append(q4, ks=None) == bad and append(q4, vs=(-1, 64)) == bad
    assert append(q4, total=-1) == bad and append(q4, total=0) == q4.Q4_OK
    assert append(q4, total=2 ** 27) == bad  # 8 pieces a row and head: past 32 bits
    assert append(q4, pages=2 ** 27) == bad and append(q4, pages=2 ** 26, heads=2 ** 10) == bad
    for i in range(5):
        assert append(q4, {i: None}) == bad, i
    for i in range(4):
        assert append(q4, {i: at(i) + 8}) == align, i
    assert append(q4, ks=(100, 64)) == align and append(q4, vs=(128, 4)) == align


def test_append_outputs_overlap_nothing(q4):
    for out in (0, 1):
        for other in range(5):
            if other != out:
                assert append(q4, {out: at(other)}) == q4.Q4_ERR_INVALID_ARG, (out, other)
    # rows whose gaps hold the pages are taken as one piece
    assert append(q4, {0: at(2) + 128}, ks=(1 << 12, 1 << 10)) == q4.Q4_ERR_INVALID_ARG


def attend(q4, ptr=(), dtype=2, pages=8, heads=2, hq=4, d=64, page=16, qs=(256, 64), scale=0.125, slots=3, width=4,
           S=2, total=3):
    p = {i: at(i) for i in range(8)}  # k, v, q, out, table, offsets, slot, pos
    p.update(ptr)
    return q4.raw_library().q4_paged_attention(p[0], p[1], p[2], p[3], dtype, pages, heads, hq, d, page,
                                               I2(*qs) if qs else None, scale, p[4], slots, width, p[5], p[6], p[7],
                                               S, total, None)


def test_attention_arguments(q4):
    bad, shape, align = q4.Q4_ERR_INVALID_ARG, q4.Q4_ERR_SHAPE, q4.Q4_ERR_ALIGN
    assert attend(q4, page=0) == shape and attend(q4, d=32) == shape
    assert attend(q4, dtype=0) == bad and attend(q4, dtype=3) == bad
    assert attend(q4, hq=3) == bad and attend(q4, hq=0) == bad and attend(q4, hq=258) == shape
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert attend(q4, scale=scale) == bad, scale
    assert attend(q4, slots=0) == bad and attend(q4, width=0) == bad and attend(q4, width=2 ** 27) == bad
    assert attend(q4, S=-1) == bad and attend(q4, S=0) == bad and attend(q4, S=0, total=0) == q4.Q4_OK
    assert attend(q4, total=-1) == bad and attend(q4, total=2 ** 30) == bad
    assert attend(q4, total=2 ** 29, hq=8) == shape
    assert attend(q4, qs=None) == bad and attend(q4, qs=(1 << 40, 64)) == bad
    assert attend(q4, qs=(250, 64)) == align
    for i in range(8):
        assert attend(q4, {i: None}) == bad, i
    for i in range(4):
        assert attend(q4, {i: at(i) + 8}) == align, i


def test_attention_output_overlaps_nothing_but_its_own_queries(q4):
    for other in (0, 1, 4, 5, 6, 7):
        assert attend(q4, {3: at(other)}) == q4.Q4_ERR_INVALID_ARG, other
    assert attend(q4, {3: at(2) + 64}) == q4.Q4_ERR_INVALID_ARG
    assert attend(q4, {3: at(2)}, qs=(512, 64)) == q4.Q4_ERR_INVALID_ARG  # rows of a wider tensor


def test_python_checks(q4):
    with pytest.raises(ValueError):
        q4.Q4PageTable(1, 1, 1, 24, device="cpu")
    with pytest.raises(ValueError):
        q4.Q4PageTable(0, 1, 1, 16, device="cpu")
    with pytest.raises(ValueError):
        import torch

        q4.Q4PagedCache(1, 1, 64, 16, dtype=torch.float32, device="cpu")
    t = q4.Q4PageTable(2, 3, 5, 16, device="cpu")
    assert np.array_equal(t.state.numpy(), paged.Pool(2, 3, 5, 16).state())
    assert t.table.shape == (2, 3) and int(t.free_count) == 5


def test_the_pools_oracle():
    # a worked step: two slots, pages of 16
    p = paged.Pool(2, 4, 5, 16)
    m, n, short, bad = p.reserve([0, 17, 18], [1, 0], [0, 0], 18)
    assert (m[0], m[15], m[16], m[17]) == (0, 15, 16, 32) and n == [17, 1] and not short and not bad
    assert p.count == 2 and p.held == [1, 2] and p.table[1][:2] == [0, 1] and p.table[0][0] == 2
    # slot 1 ends, slot 0 grows by 20 rows into two more pages: the last ones that came back
    m, n, short, bad = p.reserve([0, 0, 20], [1, 0], [0, 1], 20)
    assert n == [0, 21] and p.held == [2, 0] and p.table[0][:2] == [2, 1] and m[0] == 33 and m[15] == 16
    assert p.count == 3 and p.free[:3] == [4, 3, 0]


def test_the_pool_keeps_every_page_once():
    rng = random.Random(5)
    for _ in range(200):
        slots, width, page = rng.randint(1, 6), rng.randint(1, 6), rng.choice((16, 32))
        pages = rng.randint(1, slots * width)
        p, length = paged.Pool(slots, width, pages, page), [0] * slots
        for _ in range(12):
            who = rng.sample(range(slots), rng.randint(1, slots))
            pos = [rng.choice((length[s], length[s], 0, length[s] // 2)) for s in who]
            rows = [rng.choice((0, 1, rng.randint(0, page * 2))) for _ in who]
            off = [0] + list(np.cumsum(rows))
            m, n, short, bad = p.reserve([int(x) for x in off], who, pos, int(off[-1]))
            for s, x in zip(who, n):
                if x >= 0:
                    length[s] = x
            owned = [x for s in range(slots) for x in p.table[s][:p.held[s]]] + p.free[:p.count]
            assert sorted(owned) == list(range(pages))
            assert all(p.held[s] == -(-length[s] // page) for s in range(slots) if s in who and n[who.index(s)] >= 0)
            used = [x for x in m if x >= 0]
            assert len(used) == len(set(used))
