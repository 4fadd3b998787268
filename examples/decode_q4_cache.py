"""Prompts and decode steps of a small decoder on a 4-bit KV cache.

    python examples/decode_q4_cache.py [--steps 48] [--keep 160]

A decoder with random weights, the layer shapes of a 0.5B model (hidden size
896, 14 query and 2 key/value heads of 64) and two layers, serves four requests
the way a serving loop would:

  prompts   q/k/v of all prompts' packed rows in one grouped 4-bit matmul,
            rotary positions, ``q4_prompt_attention``, and the rows into the
            cache (``q4_kvq_append``); the prompts' last rows attend once more
            over the cache with ``mass`` to weigh its positions;
  steps     one row a request: matmul, append, ``q4_kvq_attention`` (which adds
            up the weight that each position gets);
  eviction  when a request's cache has grown past the budget, ``q4_kvq_evict``
            keeps the positions that collected most weight, in place.

Keys are cached after the rotary step, so evicted caches need no positions of
their own: the rotary position of a new row is the request's true length, the
cache position is the number of rows that are kept.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_matmul_gb300 as q4  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, D, FFN, VOCAB, LAYERS = 896, 14, 2, 64, 4864, 4096, 2


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def starts(counts):
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def rotate(x, at):
    """Rotary positions on x [rows, heads, D]; at: the rows' positions."""
    freq = 1e6 ** (-torch.arange(0, D, 2, device=x.device) / D)
    angle = at[:, None].float() * freq
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


class Layer:
    def __init__(self, g, slots, capacity):
        def weight(n, k):
            return q4.q4_quantize(torch.randn((n, k), generator=g, device="cuda") * k ** -0.5)

        self.qkv = [weight(Q_HEADS * D, HIDDEN), weight(KV_HEADS * D, HIDDEN), weight(KV_HEADS * D, HIDDEN)]
        self.o = weight(HIDDEN, Q_HEADS * D)
        self.gate, self.up, self.down = weight(FFN, HIDDEN), weight(FFN, HIDDEN), weight(HIDDEN, FFN)
        self.cache = q4.Q4KVCache(slots, KV_HEADS, D, capacity)
        self.mass = self.cache.new_mass()

    def project(self, x, at):
        q, k, v = q4.q4mm_forward_group(self.qkv, norm(x))
        return (rotate(q.view(-1, Q_HEADS, D), at), rotate(k.view(-1, KV_HEADS, D), at), v.view(-1, KV_HEADS, D))

    def rest(self, x, o):
        x = x + q4.q4mm_forward(self.o, o.reshape(-1, Q_HEADS * D))
        return x + q4.q4mm_forward(self.down, q4.q4mm_forward_gated(self.gate, self.up, norm(x)))


class Decoder:
    def __init__(self, seed, slots, capacity):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn((VOCAB, HIDDEN), generator=g, device="cuda")
        self.layers = [Layer(g, slots, capacity) for _ in range(LAYERS)]
        self.head = q4.q4_quantize(torch.randn((VOCAB, HIDDEN), generator=g, device="cuda") * HIDDEN ** -0.5)

    def prompts(self, tokens, lengths, watch=16):
        """Runs whole prompts (packed tokens) and fills the cache; returns each request's next token.

        The last `watch` rows of every prompt weigh its positions."""
        n = lengths.numel()
        offsets, slot, zero = starts(lengths), torch.arange(n, dtype=torch.int32, device="cuda"), ints([0] * n)
        at = torch.arange(tokens.numel(), device="cuda") - offsets[:-1].repeat_interleave(lengths)
        ends = lengths.cumsum(0)
        rows = lengths.clamp(max=watch)
        last = torch.cat([torch.arange(e - r, e, device="cuda") for e, r in zip(ends.tolist(), rows.tolist())])
        x = self.embed[tokens]
        for layer in self.layers:
            q, k, v = layer.project(x, at)
            q4.q4_kvq_append(layer.cache, k, v, offsets, slot, zero)
            o = q4.q4_prompt_attention(q.bfloat16(), k.bfloat16(), v.bfloat16(), offsets)
            layer.mass.zero_()
            q4.q4_kvq_attention(layer.cache, q[last].contiguous(), starts(rows), slot, (lengths - rows).int(),
                                mass=layer.mass)
            x = layer.rest(x, o.float())
        return self.pick(x[ends - 1])

    def step(self, tokens, true_length, held):
        """One row a request: true_length rows so far, held[layer] of them in the cache."""
        n = tokens.numel()
        offsets, slot = torch.arange(n + 1, dtype=torch.int32, device="cuda"), ints(list(range(n)))
        x = self.embed[tokens]
        for layer, pos in zip(self.layers, held):
            q, k, v = layer.project(x, true_length)
            q4.q4_kvq_append(layer.cache, k, v, offsets, slot, pos)
            x = layer.rest(x, q4.q4_kvq_attention(layer.cache, q, offsets, slot, pos, mass=layer.mass))
        return self.pick(x)

    def pick(self, x):
        idx, _ = q4.q4mm_argmax(self.head, norm(x).contiguous(), want_max=False)
        return idx.long()


def serve(prompt_lengths, steps, keep, recent=32, seed=1, quiet=False):
    """Serves random prompts; returns (tokens [requests, steps + 1], rows held per layer)."""
    n = len(prompt_lengths)
    # a request may grow by a quarter of the budget before it is thinned out again
    room = keep + max(1, keep // 4)
    model = Decoder(seed, n, max(max(prompt_lengths), room) + steps)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    lengths = ints(prompt_lengths).long()
    tokens = torch.randint(0, VOCAB, (sum(prompt_lengths),), generator=g, device="cuda")
    out = [model.prompts(tokens, lengths)]
    slot = ints(list(range(n)))
    held = [lengths.int() for _ in model.layers]
    torch.cuda.synchronize()
    began = time.perf_counter()
    for i in range(steps):
        if max(prompt_lengths) + i >= room and i % max(1, keep // 4) == 0:  # the host knows the lengths' bound
            held = [q4.q4_kvq_evict(layer.cache, layer.mass, slot, slot, pos, keep, recent)[0]
                    for layer, pos in zip(model.layers, held)]
        out.append(model.step(out[-1], lengths + i, held))
        held = [pos + 1 for pos in held]
    torch.cuda.synchronize()
    if not quiet:
        print("%d requests, %d steps: %.0f us a step" % (n, steps, (time.perf_counter() - began) / max(1, steps) * 1e6))
    status = q4.q4_device_status()
    if status != q4.Q4_OK:
        raise q4.Q4Error(status, "serve")
    return torch.stack(out, 1), held


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=48)
    ap.add_argument("--keep", type=int, default=160, help="cached positions a head keeps of each request")
    args = ap.parse_args()
    tokens, held = serve([500, 37, 211, 1], args.steps, args.keep)
    print("rows held after the last step:", held[0].tolist())
    for r, t in enumerate(tokens.tolist()):
        print("request %d: %s" % (r, " ".join(map(str, t[:12]))))


if __name__ == "__main__":
    main()
