"""Prompts in pieces beside decode steps, over a paged 16-bit KV cache.

    python examples/serve_paged_cache.py [--budget 96] [--pages 64]

A decoder with random weights, the layer shapes of a 0.5B model (hidden size
896, 14 query and 2 key/value heads of 64) and two layers, serves requests that
arrive while others decode.  Every step merges one row of each decoding request
with pieces of the prompts that are still being read, up to a budget of rows:

  reserve   ``q4_paged_reserve`` gives the step's requests the pages they grow into
            and takes back those of requests that have ended;
  layers    q/k/v of all rows in one grouped 4-bit matmul, rotary positions,
            ``q4_paged_append``, and ``q4_paged_attention`` for single rows and pieces alike;
  pick      ``q4mm_argmax_rows`` for the rows that need a token.

A request waits while the pool may lack pages for all of it, so that no request is
ever refused on the way.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_matmul_gb300 as q4  # noqa: E402
from decode_q4_cache import D, FFN, HIDDEN, KV_HEADS, LAYERS, Q_HEADS, VOCAB, ints, norm, rotate  # noqa: E402


class Layer:
    def __init__(self, g, pages, page_size):
        def weight(n, k):
            return q4.q4_quantize(torch.randn((n, k), generator=g, device="cuda") * k ** -0.5)

        self.qkv = [weight(Q_HEADS * D, HIDDEN), weight(KV_HEADS * D, HIDDEN), weight(KV_HEADS * D, HIDDEN)]
        self.o = weight(HIDDEN, Q_HEADS * D)
        self.gate, self.up, self.down = weight(FFN, HIDDEN), weight(FFN, HIDDEN), weight(HIDDEN, FFN)
        self.cache = q4.Q4PagedCache(pages, KV_HEADS, D, page_size)

    def __call__(self, x, at, tables, step, slot_map):
        q, k, v = q4.q4mm_forward_group(self.qkv, norm(x))
        q, k = rotate(q.view(-1, Q_HEADS, D), at), rotate(k.view(-1, KV_HEADS, D), at)
        q4.q4_paged_append(self.cache, k, v.view(-1, KV_HEADS, D), slot_map)
        o = q4.q4_paged_attention(self.cache, tables, q.to(self.cache.dtype), *step)
        x = x + q4.q4mm_forward(self.o, o.float().view(-1, Q_HEADS * D))
        return x + q4.q4mm_forward(self.down, q4.q4mm_forward_gated(self.gate, self.up, norm(x)))


class Request:
    def __init__(self, prompt, new_tokens):
        self.prompt, self.new_tokens = prompt, new_tokens
        self.rows = 0    # rows cached so far
        self.tokens = []  # tokens picked so far, one device value each

    @property
    def most(self):
        return self.prompt.numel() + self.new_tokens


def serve(prompt_lengths, new_tokens, slots=4, pages=64, page_size=16, budget=96, seed=1):
    """Serves random prompts in order of arrival; returns (tokens [requests, new_tokens], steps, free pages left)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    embed = torch.randn((VOCAB, HIDDEN), generator=g, device="cuda")
    layers = [Layer(g, pages, page_size) for _ in range(LAYERS)]
    head = q4.q4_quantize(torch.randn((VOCAB, HIDDEN), generator=g, device="cuda") * HIDDEN ** -0.5)
    requests = [Request(torch.randint(0, VOCAB, (n,), generator=g, device="cuda"), new_tokens) for n in prompt_lengths]
    if max(-(-r.most // page_size) for r in requests) > pages:
        raise ValueError("the pool is too small for the longest request")
    tables = q4.Q4PageTable(slots, max(-(-r.most // page_size) for r in requests), pages, page_size)
    waiting, running, ended, steps = list(requests), {}, [], 0
    while waiting or running or ended:
        while waiting and len(running) + len(ended) < slots:
            promised = sum(-(-r.most // page_size) for r in running.values())
            if promised + -(-waiting[0].most // page_size) > pages:
                break
            running[next(s for s in range(slots) if s not in running and s not in ended)] = waiting.pop(0)
        # decoding requests first, then pieces of prompts; requests that ended give their pages back
        room, work = budget, []
        for s, r in sorted(running.items(), key=lambda x: x[1].rows < x[1].prompt.numel()):
            n = min(room, max(1, r.prompt.numel() - r.rows))
            if n:
                work.append((s, r, n))
                room -= n
        slot = [s for s, _, _ in work] + ended
        pos = [r.rows for _, r, _ in work] + [0] * len(ended)
        counts = [n for _, _, n in work] + [0] * len(ended)
        ended = []
        total = sum(counts)
        starts = [sum(counts[:i]) for i in range(len(counts) + 1)]
        step = (ints(starts), ints(slot), ints(pos))
        slot_map, _ = q4.q4_paged_reserve(tables, *step, total)
        if total:
            rows = [r.prompt[r.rows:r.rows + n] if r.rows < r.prompt.numel() else r.tokens[-1] for _, r, n in work]
            at = torch.cat([torch.arange(r.rows, r.rows + n, device="cuda") for _, r, n in work])
            x = embed[torch.cat(rows)]
            for layer in layers:
                x = layer(x, at, tables, step, slot_map)
            picked, _ = q4.q4mm_argmax_rows(head, norm(x).contiguous(), ints([e - 1 for e in starts[1:len(work) + 1]]),
                                            want_max=False)
            for i, (s, r, n) in enumerate(work):
                r.rows += n
                if r.rows >= r.prompt.numel():
                    r.tokens.append(picked[i:i + 1].long())
                if len(r.tokens) == r.new_tokens:
                    del running[s]
                    ended.append(s)
        steps += 1
    status = q4.q4_device_status()
    if status != q4.Q4_OK:
        raise q4.Q4Error(status, "serve")
    return torch.stack([torch.cat(r.tokens) for r in requests]), steps, int(tables.free_count)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--budget", type=int, default=96, help="rows of a step")
    ap.add_argument("--pages", type=int, default=64)
    args = ap.parse_args()
    tokens, steps, free = serve([300, 37, 211, 1, 64, 150], 24, pages=args.pages, budget=args.budget)
    print("%d steps, %d of %d pages free at the end" % (steps, free, args.pages))
    for r, t in enumerate(tokens.tolist()):
        print("request %d: %s" % (r, " ".join(map(str, t[:12]))))


if __name__ == "__main__":
    main()
