"""Pins of the cache and attention oracle (CPU), and the host-side checks of the
calls it stands for."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import synthetic
from oracle import attention as ref


def test_encode_is_the_canonical_block_taken_apart():
    x = synthetic.normal(5, (3, 2, 64))
    codes, scales = ref.encode(x)
    blocks = oracle.quantize(x.reshape(-1, 64))
    assert np.array_equal(oracle.dequantize(blocks).astype(np.float64).reshape(x.shape), ref.decode(codes, scales))
    # hand-derived: -8 is the first value of largest magnitude, so d = 1 and codes are value + 8
    hand = np.zeros((1, 32), np.float32)
    hand[0, :4] = [-8, 3, -2.5, 8]
    codes, scales = ref.encode(hand)
    assert scales[0, 0] == 1.0 and codes[0, :5].tolist() == [0, 11, 5, 15, 8]


def test_attention_of_one_key_is_its_value():
    q, k, v = (synthetic.normal(i, (1, h, 32)) for i, h in ((1, 4), (2, 2), (3, 2)))
    o, mass = ref.attention(q, k.astype(np.float64), v.astype(np.float64), 0, 0.2)
    assert np.allclose(o[0], np.repeat(v[0], 2, 0)) and np.allclose(mass, [[2.0], [2.0]])


def test_equal_scores_average_the_values():
    q = np.zeros((2, 1, 32))
    v = synthetic.normal(4, (5, 1, 32)).astype(np.float64)
    o, mass = ref.attention(q, v, v, 3, 1.0)
    assert np.allclose(o[0, 0], v[:4, 0].mean(0)) and np.allclose(o[1, 0], v[:, 0].mean(0))
    assert np.allclose(mass, [[0.45, 0.45, 0.45, 0.45, 0.2]])
    p = ref.prompt(q, v, v, 1.0)
    assert np.allclose(p, o)
    assert not ref.prompt(np.zeros((7, 1, 32)), v, v, 1.0)[:2].any()  # two rows more than keys


def test_evict_keeps_the_latest_and_the_heaviest():
    w = np.array([0, 5, 1, 1, 0, 1, 9, 0], np.float32)
    assert ref.evict(w, 4, 1).tolist() == [1, 2, 6, 7]       # ties: 2 before 3 and 5
    assert ref.evict(w, 8, 3).tolist() == list(range(8))
    assert ref.evict(np.array([np.nan, -np.inf, -1, 0], np.float32), 2, 0).tolist() == [2, 3]
    assert ref.evict(np.array([np.nan, -np.inf, np.nan, 0], np.float32), 2, 0).tolist() == [1, 3]


@pytest.fixture(scope="module")
def q4():
    import __graft_entry__

    __graft_entry__.build()
    import bit_quantized_matmul_gb300 as q4

    return q4


A = 4096  # an aligned stand-in address: these calls return before any CUDA call
I2 = ctypes.c_int64 * 2


def test_cache_bytes_and_dimensions(q4):
    lib = q4.raw_library()
    n = ctypes.c_size_t(0)
    assert lib.q4_kvq_cache_bytes(3, 2, 128, 33, ctypes.byref(n)) == q4.Q4_OK
    assert n.value == 3 * 2 * 2 * 32 * (128 + 16)  # two tiles of 32 positions, 4.5 bits a value, K and V
    assert lib.q4_kvq_cache_bytes(1, 1, 64, 1, ctypes.byref(n)) == q4.Q4_OK and n.value == 32 * 72
    for dims, status in (((0, 1, 64, 1), q4.Q4_ERR_INVALID_ARG), ((1, 1, 32, 1), q4.Q4_ERR_SHAPE),
                         ((1, 1, 64, 1 << 31), q4.Q4_ERR_INVALID_ARG),
                         ((1 << 30, 1 << 30, 64, 1), q4.Q4_ERR_INVALID_ARG)):
        assert lib.q4_kvq_cache_bytes(*dims, ctypes.byref(n)) == status
    assert lib.q4_kvq_cache_bytes(1, 1, 64, 1, None) == q4.Q4_ERR_INVALID_ARG


def test_append_and_read_arguments_checked_on_host(q4):
    lib = q4.raw_library()

    def append(p=A, dtype=0, d=64, st=(128, 64), off=A, S=1, total=1, heads=2):
        s = I2(*st) if st else None
        return lib.q4_kvq_append(A, p, p, dtype, 2, heads, d, 16, s, s, off, off, off, S, total, None)

    assert append(S=0) == q4.Q4_OK and append(total=0) == q4.Q4_OK
    for bad in (dict(p=None), dict(dtype=3), dict(dtype=-1), dict(st=None), dict(st=(-1, 64)), dict(off=None),
                dict(S=-1), dict(total=-1), dict(heads=0), dict(total=1 << 30, heads=4)):
        assert append(**bad) == q4.Q4_ERR_INVALID_ARG, bad
    assert append(d=96) == q4.Q4_ERR_SHAPE
    assert append(p=A + 4) == q4.Q4_ERR_ALIGN
    assert append(st=(130, 64), total=2) == q4.Q4_ERR_ALIGN

    def read(out=A, dtype=0, S=1, total=1):
        return lib.q4_kvq_read(A, out, out, dtype, 2, 2, 64, 16, A, A, A, S, total, None)

    assert read(total=0) == q4.Q4_OK
    assert read(out=None) == q4.Q4_ERR_INVALID_ARG and read(dtype=7) == q4.Q4_ERR_INVALID_ARG
    assert read(S=0) == q4.Q4_ERR_INVALID_ARG
    assert read(out=A + 8) == q4.Q4_ERR_ALIGN


def test_attention_arguments_checked_on_host(q4):
    lib = q4.raw_library()

    def attend(q=A, out=A, dtype=0, heads=2, hq=14, d=64, st=(896, 64), scale=0.125, S=1, total=1):
        return lib.q4_kvq_attention(A, q, out, None, dtype, 2, heads, hq, d, 16, I2(*st), scale, A, A, A, S, total, None)

    assert attend(total=0) == q4.Q4_OK
    for bad in (dict(q=None), dict(out=None), dict(dtype=3), dict(hq=13), dict(hq=0), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=3e38), dict(S=0)):
        assert attend(**bad) == q4.Q4_ERR_INVALID_ARG, bad
    assert attend(d=80) == q4.Q4_ERR_SHAPE and attend(heads=1, hq=65536) == q4.Q4_ERR_SHAPE
    assert attend(out=A + 4) == q4.Q4_ERR_ALIGN and attend(st=(896, 66)) == q4.Q4_ERR_ALIGN


def test_eviction_arguments_checked_on_host(q4):
    lib = q4.raw_library()

    def evict(mass=A, S=1, keep=4, recent=1, kept=A, heads=2):
        return lib.q4_kvq_evict(A, mass, 2, heads, 64, 16, A, A, A, S, keep, recent, A, kept, None)

    assert evict(S=0) == q4.Q4_OK
    for bad in (dict(mass=None), dict(S=-1), dict(keep=0), dict(keep=17), dict(recent=5), dict(recent=-1),
                dict(kept=None)):
        assert evict(**bad) == q4.Q4_ERR_INVALID_ARG, bad
    assert evict(S=40000) == q4.Q4_ERR_SHAPE


def test_prompt_arguments_checked_on_host(q4):
    lib = q4.raw_library()

    def prompt(q=A, k=A, out=A, dtype=1, hq=14, hk=2, d=64, st=(1152, 64), scale=0.125, off=A, S=1, tq=4, tk=4):
        s = I2(*st)
        return lib.q4_prompt_attention(q, k, k, out, dtype, hq, hk, d, s, s, s, scale, 1, off, off, S, tq, tk, None)

    assert prompt(tq=0) == q4.Q4_OK
    for bad in (dict(q=None), dict(k=None), dict(out=None), dict(dtype=0), dict(hq=13), dict(hk=0), dict(scale=-0.1),
                dict(off=None), dict(S=0), dict(S=-1), dict(tq=-1), dict(tk=1 << 31)):
        assert prompt(**bad) == q4.Q4_ERR_INVALID_ARG, bad
    assert prompt(d=96) == q4.Q4_ERR_SHAPE and prompt(hq=129, hk=1) == q4.Q4_ERR_SHAPE
    assert prompt(q=A + 8) == q4.Q4_ERR_ALIGN and prompt(st=(1150, 64)) == q4.Q4_ERR_ALIGN


# ---------------------------------------------------------------- outputs over inputs

def _accepted(status, q4):
    # past the arguments' checks a call looks for a device: made only where there is none
    return status not in (q4.Q4_ERR_INVALID_ARG, q4.Q4_ERR_SHAPE, q4.Q4_ERR_ALIGN)


def test_outputs_over_inputs_are_refused_on_host(q4):
    lib = q4.raw_library()
    no_device = not torch.cuda.is_available()
    row = 14 * 64 * 4  # bytes of a packed fp32 row

    def attend(q, out, st=(896, 64), mass=None, total=3):
        return lib.q4_kvq_attention(A << 20, q, out, mass, 0, 2, 2, 14, 64, 16, I2(*st), 0.125, A, A, A, 3, total, None)

    B = A << 8
    for bad in (dict(q=B, out=B + 16), dict(q=B, out=B - 16), dict(q=B, out=B + 3 * row - 16),
                dict(q=B, out=B - 3 * row + 16), dict(q=B, out=B, mass=A << 30), dict(q=B, out=B, st=(1024, 64)),
                dict(q=B, out=B, st=(896, 128)), dict(q=B, out=B + 8 * row, st=(4 * 896, 64)),
                dict(q=B, out=B << 4, mass=(B << 4) + row),
                dict(q=B, out=B + 16, st=(0, 64))):
        assert attend(**bad) == q4.Q4_ERR_INVALID_ARG, bad
    if no_device:
        for good in (dict(q=B, out=B), dict(q=B, out=B + 3 * row), dict(q=B, out=B - 3 * row),
                     dict(q=B, out=B + 9 * row, st=(4 * 896, 64)), dict(q=B, out=B + row, st=(8 * 896, 64)),
                     dict(q=B, out=B + row, st=(0, 64)), dict(q=B, out=B << 4, mass=A << 30)):
            assert _accepted(attend(**good), q4), good

    def prompt(q, k, v, out, st=(1152, 64), tq=4, tk=9):
        s = I2(*st)
        return lib.q4_prompt_attention(q, k, v, out, 1, 14, 2, 64, s, s, s, 0.125, 1, A, A, 1, tq, tk, None)

    far, row = A << 20, 14 * 64 * 2
    for bad in (dict(q=B, k=far, v=far, out=B), dict(q=far, k=B, v=far, out=B), dict(q=far, k=far, v=B, out=B),
                dict(q=far, k=B, v=far, out=B + 8 * 1152 * 2 + 16), dict(q=far, k=far, v=B, out=B - 4 * row + 16)):
        assert prompt(**bad) == q4.Q4_ERR_INVALID_ARG, bad
    assert prompt(q=B, k=far, v=far, out=B + 16, st=(896, 64)) == q4.Q4_ERR_INVALID_ARG
    if no_device:
        assert _accepted(prompt(q=B, k=far, v=far, out=B, st=(896, 64)), q4)
        assert _accepted(prompt(q=far, k=B, v=far, out=B + 8 * 1152 * 2 + 256), q4)
        assert _accepted(prompt(q=far, k=0, v=0, out=far * 2, tk=0), q4)

    def read(k, v):
        return lib.q4_kvq_read(far, k, v, 0, 2, 2, 64, 16, A, A, A, 1, 5, None)

    for bad in ((B, B), (B, B + 5 * 2 * 64 * 4 - 16), (B + 16, B)):
        assert read(*bad) == q4.Q4_ERR_INVALID_ARG, bad
    if no_device:
        assert _accepted(read(B, B + 5 * 2 * 64 * 4), q4)

    def evict(length, new_len, kept, src=B, dst=B):
        return lib.q4_kvq_evict(far, far * 2, 4, 2, 64, 16, src, dst, length, 3, 5, 1, new_len, kept, None)

    for bad in ((B, B, A), (B, B + 8, A), (A, B * 2, B - 4), (A, B * 2, B - 3 * 2 * 5 * 4 + 4), (A, A * 2, A * 2 + 8)):
        assert evict(*bad) == q4.Q4_ERR_INVALID_ARG, bad
    if no_device:
        assert _accepted(evict(B, A, A + 12), q4) and _accepted(evict(B, B - 12, B + 12), q4)


def test_sizes_that_32_bit_indexes_would_pass_are_refused_on_host(q4):
    """A loop over rows or positions steps past its end by up to a grid's warps; just below 2^31 that would turn
    negative: an append of 2^30 - 1 rows would never end."""
    lib = q4.raw_library()
    most = 2 ** 31 - 2 ** 17
    n = ctypes.c_size_t(0)
    assert lib.q4_kvq_cache_bytes(1, 1, 64, most, ctypes.byref(n)) == q4.Q4_OK
    for capacity in (most + 1, 2 ** 31 - 1000, 2 ** 31 - 65):
        assert lib.q4_kvq_cache_bytes(1, 1, 64, capacity, ctypes.byref(n)) == q4.Q4_ERR_INVALID_ARG

    def append(S, total, heads):
        return lib.q4_kvq_append(A, A, A, 1, 2, heads, 64, 16, I2(0, 64), I2(0, 64), A, A, A, S, total, None)

    def read(S, total, heads):
        return lib.q4_kvq_read(A, A << 8, A << 60, 1, 2, heads, 64, 16, A, A, A, S, total, None)

    for call in (append, read):
        for S, total, heads in ((1, 2 ** 30 - 1, 1), (1, most // 2 + 1, 1), (1, most // 3 + 1, 3), (most + 1, 1, 1)):
            assert call(S, total, heads) == q4.Q4_ERR_INVALID_ARG, (S, total, heads)

    def attend(total, hq, heads=1, S=1):
        return lib.q4_kvq_attention(A, A, A << 8, None, 1, 2, heads, hq, 64, 16, I2(0, 64), 0.125, A, A, A, S, total,
                                    None)

    assert attend(2 ** 30 - 1, 2) == q4.Q4_ERR_INVALID_ARG
    assert attend((2 ** 31 - 1) // 28, 28) == q4.Q4_ERR_SHAPE and attend(most // 28 + 1, 28) == q4.Q4_ERR_SHAPE
    assert attend(1, 28, S=most + 1) == q4.Q4_ERR_INVALID_ARG

    def prompt(S=1, tq=4, tk=4, hq=1):
        s = I2(0, 64)
        return lib.q4_prompt_attention(A, A, A, A << 8, 1, hq, 1, 64, s, s, s, 0.125, 1, A, A, S, tq, tk, None)

    for bad in (dict(S=most + 1), dict(tq=most + 1), dict(tk=most + 1)):
        assert prompt(**bad) == q4.Q4_ERR_INVALID_ARG, bad
    assert prompt(tq=most // 7 + 1, hq=7) == q4.Q4_ERR_SHAPE
    assert lib.q4_kvq_evict(A, A, 2, 1, 64, 16, A, A, A, most + 1, 4, 1, A, A, None) == q4.Q4_ERR_INVALID_ARG
