"""Measured cases of the paged KV cache.

Three operators of a serving step whose K and V rows live in pages that
requests are given as they grow, in the order in which a step uses them:

- ``reserve``: block tables and the step's slot map from the requests' lengths,
  on the GPU: pages of requests that ended or were cut back return to the pool,
  and requests that grow past their last page get others;
- ``append``: the step's new K and V rows, rounded to the cache's type, into
  the places of the slot map;
- ``attend``: the step's query rows over the pages: single tokens, drafts, and
  chunks of prompts behind what is cached already, in one call.

Each case is a dict of plain values; ``run`` is one call as a serving loop
makes it.  With ``own`` false it is written out in elementary torch
operations; ``exact`` restates each operator in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
NINF = float("-inf")

# (query heads, key/value heads, head size) of the 7B and the 0.5B decoder
SEVEN, HALF = (28, 4, 128), (14, 2, 64)


def _reserve(requests, ended, chunks, rows, longest, page, spread, short=False):
    """A step of `requests`: `ended` of them give all pages back, `chunks` bring up to `rows` rows, the others one
    each; `short`: the pool runs out on the way."""
    return {"op": "reserve", "requests": requests, "ended": ended, "chunks": chunks, "rows": rows,
            "longest": longest, "page": page, "spread": spread, "short": short}


def _cached(op, requests, longest, shortest, chunks, rows, heads, page, dtype, spread, **more):
    """Requests of `shortest` to `longest` cached positions; `chunks` of them bring up to `rows` rows, the others one."""
    q_heads, kv_heads, head_dim = heads
    return dict({"op": op, "requests": requests, "longest": longest, "shortest": shortest, "chunks": chunks,
                 "rows": rows, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
                 "dtype": dtype, "spread": spread}, **more)


def listed():
    return [
        # the smallest call: a decode step of 64 requests, a page or none for each
        dict(_reserve(64, 0, 0, 1, 4096, 64, 1), name="reserve 64 decode rows"),
        # a busy step: prompts come in, requests end, the others decode
        dict(_reserve(512, 40, 24, 3000, 5000, 16, 2), name="reserve 512 mixed"),
        # that decode step's rows, fp32 as the q/k/v matmul leaves them, into a 7B layer's cache
        dict(_cached("append", 64, 4096, 300, 0, 1, SEVEN, 64, "bf16", 3, rows_in="fp32"), name="append 64 decode rows"),
        # 9 prompts cached at once, rows in 16 bits already
        dict(_cached("append", 9, 0, 0, 9, 901, SEVEN, 16, "fp16", 4, rows_in="fp16"), name="append 9 prompts"),
        # the smallest attention: one request of the 0.5B decoder with 2,049 positions behind it
        dict(_cached("attend", 1, 2049, 2049, 0, 1, HALF, 16, "bf16", 5), name="attend 1 at 2049"),
        # an ordinary decode step: 64 requests of very different lengths, 7B
        dict(_cached("attend", 64, 6000, 33, 0, 1, SEVEN, 64, "bf16", 6), name="attend 64 ragged"),
        # few requests with long contexts
        dict(_cached("attend", 8, 32768, 30001, 0, 1, SEVEN, 16, "fp16", 7), name="attend 8 at 32k"),
        # draft verification: up to 5 rows for each of 16 requests
        dict(_cached("attend", 16, 3001, 257, 16, 5, SEVEN, 32, "fp16", 8), name="attend 16 drafts"),
        # a merged step: four pieces of prompts beside 60 decode rows
        dict(_cached("attend", 64, 5000, 33, 4, 700, SEVEN, 16, "bf16", 9), name="attend 4 chunks 60 rows"),
        # a whole short prompt of the 0.5B decoder, nothing cached before it
        dict(_cached("attend", 1, 0, 0, 1, 517, HALF, 32, "bf16", 10), name="attend prompt 517"),
        # one piece of a long prompt
        dict(_cached("attend", 1, 14001, 14001, 1, 2048, SEVEN, 64, "bf16", 11), name="attend 2048 over 14001"),
        # the largest: a large piece of a very long prompt
        dict(_cached("attend", 1, 28672, 28672, 1, 4096, SEVEN, 128, "fp16", 12), name="attend 4096 over 28672"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("reserve", "append", "attend", "attend", "attend", "attend"))
    spread, page = rng.randrange(1 << 20), rng.choice((16, 32, 64, 128))
    if op == "reserve":
        requests = _log(rng, 1, 600)
        chunks = rng.randint(0, min(requests, 30))
        ended = rng.randint(0, requests - chunks)
        return _reserve(requests, ended, chunks, _log(rng, 1, 3000), _log(rng, 1, 8000), page, spread,
                        rng.random() < 0.2)
    heads = rng.choice((SEVEN, HALF, SEVEN, HALF, (8, 8, 64), (32, 8, 128), (16, 1, 128)))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "append":
        requests = _log(rng, 1, 96)
        rows = _log(rng, 1, max(1, 8000 // requests))
        longest = _log(rng, 1, 5000)
        return _cached(op, requests, longest, rng.randint(0, longest), rng.randint(0, requests), rows, heads, page,
                       dtype, spread, rows_in=rng.choice(("fp32", dtype)))
    if rng.random() < 0.5:  # decode and drafts
        longest = _log(rng, 1, 30000)
        requests = _log(rng, 1, max(1, min(96, 250000 // longest)))
        rows = rng.choice((1, 1, rng.randint(2, 8)))
        return _cached(op, requests, longest, _log(rng, 1, longest), requests if rows > 1 else 0, rows, heads, page,
                       dtype, spread)
    chunks = _log(rng, 1, 6)
    rows = _log(rng, 16, max(16, 3000 // chunks))
    longest = rng.choice((0, _log(rng, 1, 9000), _log(rng, 1, 9000)))
    return _cached(op, chunks + rng.choice((0, _log(rng, 1, 20))), longest, rng.randint(0, longest), chunks, rows,
                   heads, page, dtype, spread)


# ---------------------------------------------------------------- sizes of a case

def _lengths(case):
    """Cached positions of each request, the first the longest."""
    r = random.Random(case["spread"])
    rest = [r.randint(case["shortest"], case["longest"]) for _ in range(case["requests"] - 1)]
    return [case["longest"]] + rest


def _new_rows(case):
    """New rows of each request: the first brings most of the chunks, the last requests one row each."""
    r = random.Random(case["spread"] + 1)
    rows = case["rows"]
    chunks = [rows] + [r.randint(1, rows) for _ in range(case["chunks"] - 1)] if case["chunks"] else []
    return chunks + [1] * (case["requests"] - len(chunks))


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _up(n, page):
    return (n + page - 1) // page


def _pool(case):
    """(pages held, first new position, new rows) of each request, slots, table width, pages left, all for a
    step of `reserve`."""
    r = random.Random(case["spread"])
    page, held, pos, rows = case["page"], [], [], []
    for s in range(case["requests"]):
        length = r.randint(1, case["longest"])
        if s < case["chunks"]:
            length = r.choice((0, length))
            held.append(_up(length, page))
            pos.append(length)
            rows.append(r.randint(1, case["rows"]))
        elif s < case["chunks"] + case["ended"]:
            held.append(_up(length, page))
            pos.append(0)
            rows.append(0)
        else:
            # some were cut back by rejected drafts and hold more than they need
            held.append(_up(length + r.choice((0, 0, 0, r.randint(0, 40))), page))
            pos.append(length)
            rows.append(1)
    grow = sum(max(0, _up(p + n, page) - h) for h, p, n in zip(held, pos, rows))
    back = sum(max(0, h - _up(p + n, page)) for h, p, n in zip(held, pos, rows))
    left = max(0, grow * 2 // 3 - back) if case["short"] else grow + 100
    slots = case["requests"] + case["requests"] // 4 + 1
    width = max([_up(p + n, page) for p, n in zip(pos, rows)] + held) + 2
    return held, pos, rows, slots, width, left


def work(case):
    page = case["page"]
    if case["op"] == "reserve":
        held, pos, rows, _, _, _ = _pool(case)
        n = len(held)
        need = [_up(p + k, page) for p, k in zip(pos, rows)]
        moved = sum(abs(a - b) for a, b in zip(need, held))
        named = sum(_up(p + k, page) - p // page for p, k in zip(pos, rows) if k)
        return {"bytes": 4 * (6 * n + 2 * moved + named + sum(rows)), "flops": 4 * n + sum(rows)}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    lens, rows = _lengths(case), _new_rows(case)
    if case["op"] == "append":
        return {"bytes": sum(rows) * (2 * hk * d * (SIZE[case["rows_in"]] + 2) + 4), "flops": sum(rows) * 2 * hk * d}
    keys = sum(lens) + sum(rows)
    seen = sum(k * n + k * (k + 1) // 2 for n, k in zip(lens, rows))
    table = 4 * sum(_up(n + k, page) for n, k in zip(lens, rows))
    return {"bytes": 2 * keys * hk * d * 2 + 2 * sum(rows) * hq * d * 2 + table, "flops": 4 * seen * hq * d}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _rows(g, *shape):
    """Key or value rows: normal, with a few channels of larger spread, as projections give them."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., ::17] *= 3.0
    return x


def _tables(g, slot, held, slots, width, pages):
    """Block tables [slots, width]: pages in no order, and those that nobody holds."""
    order = torch.randperm(pages, generator=g, device="cuda").int()
    first, count = [0] * slots, [0] * slots
    at = 0
    for s, h in zip(slot, held):
        first[s], count[s] = at, h
        at += h
    place = torch.arange(width, device="cuda", dtype=torch.int32)
    index = (_ints(first)[:, None] + place).clamp(max=pages - 1)
    table = torch.where(place < _ints(count)[:, None], order[index.long()], torch.full_like(index, -1))
    return table, _ints(count), order[at:]


def _inputs(case, seed):
    """What the operators are called with, as tensors of this file."""
    g, page, n = _gen(seed), case["page"], case["requests"]
    order = random.Random(case["spread"] + 2)
    if case["op"] == "reserve":
        held, pos, rows, slots, width, left = _pool(case)
        slot = order.sample(range(slots), n)
        pages = sum(held) + left
        table, count, rest = _tables(g, slot, held, slots, width, max(1, pages))
        free = torch.zeros(max(1, pages), dtype=torch.int32, device="cuda")
        free[:left] = rest[:left]
        return {"slot": slot, "pos": pos, "rows": rows, "table": table, "held": count, "free": free, "left": left}
    lens, rows = _lengths(case), _new_rows(case)
    hq, hk, d, t = case["q_heads"], case["kv_heads"], case["head_dim"], TYPES[case["dtype"]]
    slot = order.sample(range(n + 3), n)
    held = [_up(a + b, page) for a, b in zip(lens, rows)]
    pages = sum(held) + 7
    table, _, _ = _tables(g, slot, held, n + 3, max(held) + 1, pages)
    i = {"slot": slot, "pos": lens, "rows": rows, "table": table, "pages": pages}
    shape = (pages, hk, page, d)
    i["k_pages"], i["v_pages"] = _rows(g, *shape).to(t), _rows(g, *shape).to(t)
    if case["op"] == "append":
        kv = _rows(g, sum(rows), 2 * hk, d).to(TYPES[case["rows_in"]])  # K and V of a row side by side: strided views
        i["k"], i["v"] = kv[:, :hk], kv[:, hk:]
        i["map"] = _ints(_places(lens, rows, slot, table.tolist(), page))
    else:
        qkv = torch.randn((sum(rows), hq + 2 * hk, d), generator=g, device="cuda").to(t)
        i["q"] = qkv[:, :hq]  # as the projections' matmul leaves it
        i["scale"] = 1.0 / math.sqrt(d)
    return i


def _places(pos, rows, slot, table, page):
    out = []
    for p, n, s in zip(pos, rows, slot):
        out += [table[s][x // page] * page + x % page for x in range(p, p + n)]
    return out


def prepare(case, seed):
    i = _inputs(case, seed)
    s = {"op": case["op"], "page": case["page"], "total": sum(i["rows"]), "rows": i["rows"], "lens": i["pos"]}
    s["slot"], s["pos"], s["offsets"] = _ints(i["slot"]), _ints(i["pos"]), _ints(_starts(i["rows"]))
    if case["op"] == "reserve":
        before = torch.cat([_ints([i["left"]]), i["free"], i["held"], i["table"].flatten()])
        s.update(before=before, pages=i["free"].numel(), slots=i["table"].shape[0], width=i["table"].shape[1])
        if own:
            import bit_quantized_matmul_gb300 as q4

            s["tables"] = q4.Q4PageTable(s["slots"], s["width"], s["pages"], s["page"])
        return s
    for name in ("k", "v", "q", "map", "scale"):
        if name in i:
            s[name] = i[name]
    if own:
        import bit_quantized_matmul_gb300 as q4

        s["cache"] = q4.Q4PagedCache(i["pages"], case["kv_heads"], case["head_dim"], case["page"],
                                     dtype=TYPES[case["dtype"]])
        s["cache"].k.copy_(i["k_pages"])
        s["cache"].v.copy_(i["v_pages"])
        s["tables"] = q4.Q4PageTable(i["table"].shape[0], i["table"].shape[1], i["pages"], case["page"])
        s["tables"].table.copy_(i["table"])
    else:
        s.update(k_pages=i["k_pages"], v_pages=i["v_pages"], table=i["table"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"reserve": _plain_reserve, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)


def _run_own(s):
    import bit_quantized_matmul_gb300 as q4

    if s["op"] == "reserve":
        tables = s["tables"]
        tables.state.copy_(s["before"])  # every pass begins with the same pool
        slot_map, length = q4.q4_paged_reserve(tables, s["offsets"], s["slot"], s["pos"], s["total"])
        return slot_map, length, tables.state
    if s["op"] == "append":
        q4.q4_paged_append(s["cache"], s["k"], s["v"], s["map"])
        return s["cache"].k, s["cache"].v
    return q4.q4_paged_attention(s["cache"], s["tables"], s["q"], s["offsets"], s["slot"], s["pos"], scale=s["scale"])


def _plain_reserve(s):
    pages, slots, width, page = s["pages"], s["slots"], s["width"], s["page"]
    count, free, held, table = s["before"].split([1, pages, slots, slots * width])
    table = table.view(slots, width)
    slot, offsets = s["slot"].long(), s["offsets"]
    rows = offsets.diff()
    length = s["pos"] + rows
    need, have = (length + page - 1) // page, held[slot]
    place = torch.arange(width, device="cuda", dtype=torch.int32)
    # surplus pages to the end of the free list, in the requests' order
    back = (have - need).clamp(min=0)
    first = count + back.cumsum(0, dtype=torch.int32) - back
    gone = (place >= need[:, None]) & (place < have[:, None])
    to = (first[:, None] + place - need[:, None]).masked_fill(~gone, pages)
    free = torch.cat([free, free[:1]]).scatter(0, to.flatten().long(), table[slot].flatten())
    top = count + back.sum(dtype=torch.int32)
    # missing ones from there
    more = (need - have).clamp(min=0)
    upto = more.cumsum(0, dtype=torch.int32)
    fits = (more == 0) | (upto <= top)
    more = more * fits
    taken = (place >= have[:, None]) & (place < need[:, None]) & fits[:, None]
    at = top - 1 - ((upto - more)[:, None] + place - have[:, None])
    new = torch.where(taken, free[at.clamp(0, pages).long()], table[slot])
    table = table.clone()
    table[slot] = new.masked_fill(gone, -1)
    held = held.clone()
    held[slot] = torch.where(fits, need, have)
    t = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    r = torch.searchsorted(offsets, t, right=True) - 1
    p = s["pos"][r] + t - offsets[r]
    there = table[slot[r], (p // page).long()] * page + p % page
    slot_map = torch.where(fits[r], there, torch.full_like(there, -1))
    length = torch.where(fits, length, torch.full_like(length, -1))
    count = top - more.sum(dtype=torch.int32)
    return slot_map, length, torch.cat([count, free[:pages], held, table.flatten()])


def _plain_append(s):
    where, at = (s["map"] // s["page"]).long(), (s["map"] % s["page"]).long()
    s["k_pages"][where, :, at] = s["k"].to(s["k_pages"].dtype)
    s["v_pages"][where, :, at] = s["v"].to(s["v_pages"].dtype)
    return s["k_pages"], s["v_pages"]


def _softmax_product(x, hidden, v):
    """softmax of x over its last axis, nothing where hidden, times v."""
    x.masked_fill_(hidden, NINF)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True)
    return (x @ v).div_(total)


def _plain_attend(s):
    q, page = s["q"].float(), s["page"]
    total, hq, d = q.shape
    hk = s["k_pages"].shape[1]
    g = hq // hk
    starts, out = _starts(s["rows"]), torch.zeros((total, hq, d), device="cuda")
    few = [r for r, n in enumerate(s["rows"]) if 0 < n <= 8]
    if few:  # requests of a few rows side by side, as long as the longest of them
        n, wide = len(few), max(s["rows"][r] for r in few)
        used = _up(max(s["lens"][r] + s["rows"][r] for r in few), page)
        which = _ints(few).long()
        ids = s["table"][s["slot"][which].long(), :used].clamp(min=0).long()  # [n, used]
        k = s["k_pages"][ids].transpose(1, 2).reshape(n, hk, used * page, d).float()
        v = s["v_pages"][ids].transpose(1, 2).reshape(n, hk, used * page, d).float()
        step = torch.arange(wide, device="cuda")
        row = (s["offsets"][which][:, None] + step).clamp(max=total - 1).long()  # [n, wide]
        live = step < s["offsets"].diff()[which][:, None]
        qs = q[row].view(n, wide, hk, g, d).permute(0, 2, 1, 3, 4).reshape(n, hk, wide * g, d)
        x = (qs @ k.transpose(2, 3)).mul_(s["scale"])
        last = (s["pos"][which][:, None] + step).repeat_interleave(g, 1)  # [n, wide * g]
        hidden = torch.arange(used * page, device="cuda") > last[..., None]
        o = _softmax_product(x, hidden[:, None], v).view(n, hk, wide, g, d).permute(0, 2, 1, 3, 4)
        o = o.reshape(n, wide, hq, d).masked_fill_(~live[..., None, None], 0.0)
        out.index_add_(0, row.flatten(), o.view(-1, hq, d))
    for r, n in enumerate(s["rows"]):
        if n <= 8:
            continue
        past = s["lens"][r]
        ids = s["table"][s["slot"][r].long(), :_up(past + n, page)].long()
        k = s["k_pages"][ids].transpose(0, 1).reshape(hk, -1, d)[:, :past + n].float()
        v = s["v_pages"][ids].transpose(0, 1).reshape(hk, -1, d)[:, :past + n].float()
        qs = q[starts[r]:starts[r] + n].view(n, hk, g, d).permute(1, 2, 0, 3).reshape(hk, g * n, d)
        x = (qs @ k.transpose(1, 2)).mul_(s["scale"])
        last = past + torch.arange(n, device="cuda").repeat(g)
        o = _softmax_product(x, torch.arange(past + n, device="cuda") > last[:, None], v)
        out[starts[r]:starts[r] + n] = o.view(hk, g, n, d).permute(2, 0, 1, 3).reshape(n, hq, d)
    return out.to(s["q"].dtype)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    i = _inputs(case, seed)
    page = case["page"]
    if case["op"] == "reserve":
        return _exact_reserve(i, page)
    if case["op"] == "append":
        out = []
        for pages, rows in ((i["k_pages"], i["k"]), (i["v_pages"], i["v"])):
            x = pages.double()
            for h in range(case["kv_heads"]):
                x[i["map"].long() // page, h, i["map"].long() % page] = rows[:, h].double()
            out.append(x)
        return tuple(out)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    g, out, t = hq // hk, [], 0
    for slot, past, n in zip(i["slot"], i["pos"], i["rows"]):
        ids = i["table"][slot, :_up(past + n, page)].long()
        o = torch.empty((n, hq, d), dtype=torch.float64, device="cuda")
        for h in range(hk):
            k = i["k_pages"][ids, h].reshape(-1, d)[:past + n].double()
            v = i["v_pages"][ids, h].reshape(-1, d)[:past + n].double()
            for a in range(0, n, 512):
                b = min(n, a + 512)
                q = i["q"][t + a:t + b, h * g:(h + 1) * g].double()
                x = torch.einsum("ngd,kd->gnk", q, k[:past + b]) * i["scale"]
                x += torch.full_like(x[0], NINF).triu_(past + a + 1)
                o[a:b, h * g:(h + 1) * g] = torch.einsum("gnk,kd->ngd", torch.softmax(x, -1), v[:past + b])
        out.append(o)
        t += n
    return torch.cat(out)


def _exact_reserve(i, page):
    """The rules one request after another, on lists."""
    table, held, free = i["table"].tolist(), i["held"].tolist(), i["free"].tolist()
    count, slot_map, length = i["left"], [], []
    need = [_up(p + n, page) for p, n in zip(i["pos"], i["rows"])]
    for slot, k in zip(i["slot"], need):
        for at in range(k, held[slot]):
            free[count] = table[slot][at]
            table[slot][at] = -1
            count += 1
        held[slot] = min(held[slot], k)
    wanted, top = 0, count
    for slot, pos, rows, k in zip(i["slot"], i["pos"], i["rows"], need):
        more = k - held[slot]
        wanted += more
        if more > 0 and wanted > top:
            length.append(-1)
            slot_map += [-1] * rows
            continue
        for at in range(held[slot], k):
            count -= 1
            table[slot][at] = free[count]
        held[slot] = k
        length.append(pos + rows)
        slot_map += [table[slot][x // page] * page + x % page for x in range(pos, pos + rows)]
    state = [count] + free + held + [x for row in table for x in row]
    return tuple(_ints(x).double() for x in (slot_map, length, state))
