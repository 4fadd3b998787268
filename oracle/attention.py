"""CPU oracle for the 4-bit KV cache, attention over it, its eviction, and
prompt attention — test infrastructure only (the CUDA library never reaches
it and shares no code with it).

Written out per request, row and head in numpy float64.  The cache's contents
come from the block rule of ``oracle.quantize`` (the C oracle), so the values
that attention sees are exact; the weights and sums are float64.
"""
from __future__ import annotations

import numpy as np

import oracle


def encode(x):
    """(codes uint8, scales float16) of rows x[..., D]: the canonical blocks, taken apart."""
    x = np.ascontiguousarray(x, np.float32)
    d = x.shape[-1]
    blocks = oracle.quantize(x.reshape(-1, d)).reshape(-1, d // 32, 18)
    scales = np.ascontiguousarray(blocks[:, :, :2]).view(np.float16)[..., 0]
    low, high = blocks[:, :, 2:] & 15, blocks[:, :, 2:] >> 4
    codes = np.concatenate([low, high], -1)
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1] + (d // 32,))


def decode(codes, scales):
    """Float64 values of codes and scales (every product is exact)."""
    c = codes.reshape(codes.shape[:-1] + (-1, 32)).astype(np.float64) - 8
    return (c * scales[..., None].astype(np.float64)).reshape(codes.shape)


def held(x):
    """What a cache holds for rows x, in float64."""
    return decode(*encode(x))


def _softmax(s):
    s = s - s.max(-1, keepdims=True)
    e = np.exp(s)
    return e / e.sum(-1, keepdims=True)


def attention(q, k, v, pos, scale):
    """One request: q [rows, Hq, D], cached values k, v [keys, H, D]; row j sees keys 0 .. pos + j.

    Returns (o [rows, Hq, D], mass [H, keys]: the weight that each key got)."""
    rows, hq, d = q.shape
    h = k.shape[1]
    g = hq // h
    o = np.zeros((rows, hq, d))
    mass = np.zeros((h, k.shape[0]))
    for j in range(rows):
        seen = pos + j + 1
        for x in range(hq):
            w = _softmax(scale * (k[:seen, x // g] @ q[j, x].astype(np.float64)))
            o[j, x] = w @ v[:seen, x // g]
            mass[x // g, :seen] += w
    return o, mass


def evict(mass, keep, recent):
    """Kept positions, ascending, of one head with weights mass[n]."""
    n = len(mass)
    if n <= keep:
        return np.arange(n)
    first = n - recent
    w = np.where(np.isnan(mass[:first]), -np.inf, mass[:first].astype(np.float64))
    nan_last = np.isnan(mass[:first])
    order = np.lexsort((np.arange(first), -w, nan_last))
    return np.sort(np.concatenate([order[:keep - recent], np.arange(first, n)]))


def prompt(q, k, v, scale, causal=True):
    """One sequence: q [n, Hq, D], k, v [m, H, D]; rows that see no key are zero."""
    n, hq, d = q.shape
    m, h, _ = k.shape
    o = np.zeros((n, hq, d))
    for i in range(n):
        seen = min(m, i + m - n + 1) if causal else m
        if seen <= 0:
            continue
        for x in range(hq):
            w = _softmax(scale * (k[:seen, x // (hq // h)].astype(np.float64) @ q[i, x].astype(np.float64)))
            o[i, x] = w @ v[:seen, x // (hq // h)].astype(np.float64)
    return o
