"""Measured cases of the attention and 4-bit KV-cache operators.

Five operators of a serving step, in the order in which a step uses them:

- ``prompt``: causal attention over the packed rows of whole prompts (16-bit
  types), query heads sharing key/value heads, sequences of different lengths;
- ``append``: the step's new K and V rows into a cache of 4-bit blocks, and
  those rows read back as the values the cache now stands for;
- ``attend``: the step's query rows over that cache (single tokens or a few
  draft rows per request), with or without the attention weight that each
  cached position collects;
- ``evict``: a cache thinned out to the positions that collected most weight.

Each case is a dict of plain values; ``run`` is one call as a serving loop
makes it.  With ``own`` false it is written out in elementary torch
operations in 32 bits; ``exact`` restates each operator in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 32  # values that share one scale
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
NINF = float("-inf")


def _case(op, requests, longest, shortest, rows, heads, dtype, spread, **more):
    q_heads, kv_heads, head_dim = heads
    return dict({"op": op, "requests": requests, "longest": longest, "shortest": shortest, "rows": rows,
                 "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "dtype": dtype,
                 "spread": spread}, **more)


# (query heads, key/value heads, head size) of the 7B and the 0.5B decoder
SEVEN, HALF = (28, 4, 128), (14, 2, 64)


def listed():
    return [
        # one decode step of 64 requests on a 7B layer: fp32 rows, as the q/k/v matmul leaves them
        dict(_case("append", 64, 4096, 300, 1, SEVEN, "fp32", 1), name="append 64 decode rows"),
        # the prompts of 9 requests cached at once, rows in 16 bits
        dict(_case("append", 9, 0, 0, 901, SEVEN, "bf16", 2), name="append 9 prompts"),
        # the smallest call: one request of the 0.5B decoder with 2,049 positions
        dict(_case("attend", 1, 2049, 2049, 1, HALF, "fp32", 3, mass=False), name="attend 1 at 2049"),
        # an ordinary decode step: 64 requests of very different lengths, 7B
        dict(_case("attend", 64, 6000, 33, 1, SEVEN, "fp32", 4, mass=False), name="attend 64 ragged"),
        # few requests, long contexts, 16-bit rows
        dict(_case("attend", 8, 32768, 30001, 1, SEVEN, "bf16", 5, mass=False), name="attend 8 at 32k"),
        # draft verification: up to 5 rows for each of 16 requests
        dict(_case("attend", 16, 3001, 257, 5, SEVEN, "fp16", 6, mass=False), name="attend 16 drafts"),
        # a decode step that also adds up each position's attention weight
        dict(_case("attend", 32, 4500, 2000, 1, SEVEN, "fp32", 7, mass=True), name="attend 32 weighing"),
        # two short contexts of the 0.5B decoder thinned out
        dict(_case("evict", 2, 1500, 1100, 1, HALF, "fp32", 8, keep=513, recent=64), name="evict 2 short"),
        # 32 contexts of a 7B layer cut to a quarter
        dict(_case("evict", 32, 8192, 5000, 1, SEVEN, "bf16", 9, keep=2048, recent=256), name="evict 32 long"),
        # a short prompt of the 0.5B decoder
        dict(_case("prompt", 1, 517, 517, 1, HALF, "bf16", 10, past=0), name="prompt 517"),
        # a step's packed prompts, one token to a few thousand each
        dict(_case("prompt", 9, 2100, 1, 1, SEVEN, "fp16", 11, past=0), name="prompt 9 packed"),
        # one long prompt, 7B
        dict(_case("prompt", 1, 16384, 16384, 1, SEVEN, "bf16", 12, past=0), name="prompt 16k"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "evict", "prompt", "prompt"))
    heads = rng.choice((SEVEN, HALF, SEVEN, HALF, (8, 8, 64), (32, 8, 128), (16, 1, 128)))
    spread = rng.randrange(1 << 20)
    if op == "append":
        requests = _log(rng, 1, 96)
        rows = _log(rng, 1, max(1, 8000 // requests))
        longest = _log(rng, 1, 5000)
        return _case(op, requests, longest, rng.randint(0, longest), rows, heads,
                     rng.choice(("fp32", "bf16", "fp16")), spread)
    if op == "attend":
        longest = _log(rng, 1, 30000)
        requests = _log(rng, 1, max(1, min(96, 250000 // longest)))
        rows = rng.choice((1, 1, 1, rng.randint(2, 8)))
        return _case(op, requests, longest, _log(rng, 1, longest), rows, heads,
                     rng.choice(("fp32", "bf16", "fp16")), spread, mass=rng.random() < 0.3)
    if op == "evict":
        longest = _log(rng, 64, 12000)
        requests = _log(rng, 1, max(1, min(64, 250000 // longest)))
        keep = rng.randint(max(1, longest // 8), longest)
        return _case(op, requests, longest, _log(rng, 1, longest), 1, heads, rng.choice(("fp32", "bf16")), spread,
                     keep=keep, recent=rng.randint(0, keep))
    longest = _log(rng, 16, 9000)
    requests = _log(rng, 1, max(1, min(32, 9000 // longest)))
    return _case(op, requests, longest, _log(rng, 1, longest), 1, heads, rng.choice(("bf16", "fp16")), spread,
                 past=rng.choice((0, 0, _log(rng, 1, 2000))))


# ---------------------------------------------------------------- sizes of a case

def _lengths(case):
    """Cached positions (or prompt rows) of each request, the first the longest."""
    r = random.Random(case["spread"])
    rest = [r.randint(case["shortest"], case["longest"]) for _ in range(case["requests"] - 1)]
    return [case["longest"]] + rest


def _new_rows(case):
    """New rows of each request in this step."""
    r = random.Random(case["spread"] + 1)
    rows = case["rows"]
    low = rows if rows == 1 else 1
    return [rows] + [r.randint(low, rows) for _ in range(case["requests"] - 1)]


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def work(case):
    hq, hk, d, es = case["q_heads"], case["kv_heads"], case["head_dim"], SIZE[case["dtype"]]
    cached = 2 * hk * (d // 2 + d // 16)  # bytes of one position: K and V codes and scales
    lens = _lengths(case)
    if case["op"] == "append":
        total = sum(_new_rows(case))
        return {"bytes": total * (2 * cached + 2 * 2 * hk * d * es), "flops": total * 2 * hk * d * 4}
    if case["op"] == "attend":
        rows = _new_rows(case)
        keys = sum(n + r for n, r in zip(lens, rows))
        seen = sum(r * n + r * (r + 1) // 2 for n, r in zip(lens, rows))
        weigh = keys * hk * 8 if case["mass"] else 0
        return {"bytes": keys * cached + 2 * sum(rows) * hq * d * es + weigh, "flops": 4 * seen * hq * d}
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        # the weights, the kept rows moved, their weights and places written, the rows read back
        return {"bytes": sum(lens) * hk * 4 + kept * (2 * cached + 8 * hk + cached + 2 * hk * d * es),
                "flops": sum(lens) * hk * 4}
    past = case["past"]
    seen = sum(n * past + n * (n + 1) // 2 for n in lens)
    return {"bytes": es * d * (2 * hq * sum(lens) + 2 * hk * (sum(lens) + past * len(lens))),
            "flops": 4 * seen * hq * d}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rows(g, *shape):
    """Key or value rows: normal, with a few channels of larger spread, as projections give them."""
    x = torch.randn(shape, generator=g, device="cuda")
    scale = torch.ones(shape[-2:], device="cuda")
    scale[:, ::17] = 3.0
    return x.mul_(scale)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _encode(x):
    """(codes 0..15, fp16 scales) of the rows' blocks of 32 values: the first value of largest
    magnitude m sets the scale m / -8; codes are round-half-away(x / scale) + 8 in 32 bits."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    at = b.abs().argmax(-1, keepdim=True)
    d = b.gather(-1, at) / -8
    r = torch.where(d == 0, torch.zeros_like(b), b / d)
    a = r.abs()
    whole = a.trunc()
    n = whole + ((a - whole) >= 0.5)
    q = (torch.where(r < 0, -n, n) + 8).clamp(0, 15)
    return q.to(torch.uint8).flatten(-2), d.squeeze(-1).half()


def _decode(codes, scales):
    """The 32-bit values that codes and scales stand for."""
    return ((codes.float() - 8).unflatten(-1, (-1, BLOCK)) * scales.float().unsqueeze(-1)).flatten(-2)


def _inputs(case, seed):
    """What the operator is called with, before any cache is laid out."""
    g = _gen(seed)
    hq, hk, d, t = case["q_heads"], case["kv_heads"], case["head_dim"], TYPES[case["dtype"]]
    lens, n = _lengths(case), case["requests"]
    i = {"lens": lens}
    if case["op"] == "prompt":
        total, past = sum(lens), case["past"]
        klens = [x + past for x in lens]
        i["klens"] = klens
        # one matmul's output holds q, k and v side by side where no past precedes them: strided views
        if past == 0:
            qkv = torch.randn((total, hq + 2 * hk, d), generator=g, device="cuda").to(t)
            i["q"], i["k"], i["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            i["q"] = torch.randn((total, hq, d), generator=g, device="cuda").to(t)
            i["k"] = torch.randn((sum(klens), hk, d), generator=g, device="cuda").to(t)
            i["v"] = torch.randn((sum(klens), hk, d), generator=g, device="cuda").to(t)
        i["scale"] = 1.0 / math.sqrt(d)
        return i
    rows = _new_rows(case) if case["op"] != "evict" else [0] * n
    slots = n if case["op"] != "evict" else 2 * n
    cap = max(x + r for x, r in zip(lens, rows))
    i.update(rows=rows, cap=cap, slots=slots)
    order = list(range(n))
    random.Random(case["spread"] + 2).shuffle(order)
    i["slot"] = order
    if case["op"] == "append":
        total = sum(rows)
        kv = _rows(g, total, 2 * hk, d).to(t)  # K and V of a row side by side: strided views
        i["k"], i["v"] = kv[:, :hk], kv[:, hk:]
        return i
    i["k"], i["v"] = _rows(g, n, cap, hk, d), _rows(g, n, cap, hk, d)
    if case["op"] == "attend":
        i["q"] = torch.randn((sum(rows), hq, d), generator=g, device="cuda").to(t)
        i["scale"] = 1.0 / math.sqrt(d)
        if case["mass"]:
            i["mass"] = torch.rand((slots, hk, cap), generator=g, device="cuda")
        return i
    # weights as a few hundred steps leave them: most small, a few large, many equal (never attended)
    m = torch.rand((slots, hk, cap), generator=g, device="cuda")
    i["mass"] = torch.where(m < 0.2, torch.zeros_like(m), m.pow(8) * 50)
    return i


def _fill(cache, q4, i, case):
    """The cache as earlier steps left it: request r's rows from position 0 on in its slot."""
    n, cap, hk, d = case["requests"], i["cap"], case["kv_heads"], case["head_dim"]
    offsets = _ints([r * cap for r in range(n + 1)])
    k, v = i["k"].view(n * cap, hk, d), i["v"].view(n * cap, hk, d)
    q4.q4_kvq_append(cache, k, v, offsets, _ints(i["slot"]), _ints([0] * n))


def prepare(case, seed):
    i = _inputs(case, seed)
    n, hk, d = case["requests"], case["kv_heads"], case["head_dim"]
    s = {"op": case["op"], "dtype": TYPES[case["dtype"]], "hk": hk, "d": d}
    if case["op"] == "prompt":
        s.update(q=i["q"], k=i["k"], v=i["v"], scale=i["scale"])
        s["q_offsets"], s["k_offsets"] = _ints(_starts(i["lens"])), _ints(_starts(i["klens"]))
        return s
    s.update(slot=_ints(i["slot"]), pos=_ints(i["lens"]), cap=i["cap"], n=n)
    s["offsets"] = _ints(_starts(i["rows"]))
    s["total"] = sum(i["rows"])
    s["longest_row"] = max(i["rows"])
    if own:
        import bit_quantized_matmul_gb300 as q4

        s["cache"] = q4.Q4KVCache(i["slots"], hk, d, i["cap"])
        if case["op"] != "append":
            _fill(s["cache"], q4, i, case)
    else:  # codes and scales by request; one request's rows together
        shape = (i["slots"], hk, i["cap"])
        for name in ("k", "v"):
            codes = torch.zeros(shape + (d,), dtype=torch.uint8, device="cuda")
            scales = torch.zeros(shape + (d // BLOCK,), dtype=torch.float16, device="cuda")
            if case["op"] != "append":
                q, sc = _encode(i[name].transpose(1, 2))
                codes[s["slot"].long()], scales[s["slot"].long()] = q, sc
            s[name + "_codes"], s[name + "_scales"] = codes, scales
    if case["op"] == "append":
        s.update(k=i["k"], v=i["v"])
    elif case["op"] == "attend":
        s.update(q=i["q"], scale=i["scale"], mass=i.get("mass"))
    else:
        keep = case["keep"]
        s.update(mass=i["mass"], keep=keep, recent=case["recent"])
        s["dst"] = _ints([x + n for x in i["slot"]])
        kept = [min(x, keep) for x in i["lens"]]
        s["kept_offsets"], s["kept_total"], s["zero"] = _ints(_starts(kept)), sum(kept), _ints([0] * n)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"prompt": _plain_prompt, "append": _plain_append, "attend": _plain_attend,
            "evict": _plain_evict}[s["op"]](s)


def _run_own(s):
    import bit_quantized_matmul_gb300 as q4

    if s["op"] == "prompt":
        return q4.q4_prompt_attention(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], scale=s["scale"])
    if s["op"] == "append":
        q4.q4_kvq_append(s["cache"], s["k"], s["v"], s["offsets"], s["slot"], s["pos"])
        return q4.q4_kvq_read(s["cache"], s["offsets"], s["slot"], s["pos"], s["total"], dtype=s["dtype"])
    if s["op"] == "attend":
        if s["mass"] is None:
            return q4.q4_kvq_attention(s["cache"], s["q"], s["offsets"], s["slot"], s["pos"], scale=s["scale"])
        mass = s["mass"].clone()
        return q4.q4_kvq_attention(s["cache"], s["q"], s["offsets"], s["slot"], s["pos"], scale=s["scale"],
                                   mass=mass), mass
    mass = s["mass"].clone()
    length, kept = q4.q4_kvq_evict(s["cache"], mass, s["slot"], s["dst"], s["pos"], s["keep"], s["recent"])
    k, v = q4.q4_kvq_read(s["cache"], s["kept_offsets"], s["dst"], s["zero"], s["kept_total"], dtype=s["dtype"])
    return length, kept, mass, k, v


def _plain_prompt(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    tq, hq, d = q.shape
    tk, hk, _ = k.shape
    rows = torch.arange(tq, device="cuda", dtype=torch.int32)
    keys = torch.arange(tk, device="cuda", dtype=torch.int32)
    sq = torch.searchsorted(s["q_offsets"], rows, right=True) - 1
    sk = torch.searchsorted(s["k_offsets"], keys, right=True) - 1
    qlen, klen = s["q_offsets"].diff(), s["k_offsets"].diff()
    last = rows - s["q_offsets"][sq] + (klen - qlen)[sq]  # last key of its sequence that a row sees
    hidden = (sq[:, None] != sk) | ((keys - s["k_offsets"][sk]) > last[:, None])
    p = q.transpose(0, 1).reshape(hk, -1, d) @ k.permute(1, 2, 0)
    p = p.view(hq, tq, tk).mul_(s["scale"]).masked_fill_(hidden, NINF)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == NINF, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(hk, -1, tk) @ v.transpose(0, 1)).view(hq, tq, d)
    return torch.where(total > 0, o / total, torch.zeros_like(o)).transpose(0, 1).to(s["dtype"]).contiguous()


def _places(s):
    """(request, position, slot) of each packed row."""
    t = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    r = torch.searchsorted(s["offsets"], t, right=True) - 1
    return r, (s["pos"][r] + t - s["offsets"][r]).long(), s["slot"][r].long()


def _plain_append(s):
    _, at, slot = _places(s)
    kq, ks = _encode(s["k"])
    vq, vs = _encode(s["v"])
    s["k_codes"][slot, :, at], s["k_scales"][slot, :, at] = kq, ks
    s["v_codes"][slot, :, at], s["v_scales"][slot, :, at] = vq, vs
    return (_decode(s["k_codes"][slot, :, at], s["k_scales"][slot, :, at]).to(s["dtype"]),
            _decode(s["v_codes"][slot, :, at], s["v_scales"][slot, :, at]).to(s["dtype"]))


def _plain_attend(s):
    n, hk, d, cap, wide = s["n"], s["hk"], s["d"], s["cap"], s["longest_row"]
    slot = s["slot"].long()
    k = _decode(s["k_codes"][slot], s["k_scales"][slot])  # [n, hk, cap, d]
    v = _decode(s["v_codes"][slot], s["v_scales"][slot])
    r, at, _ = _places(s)
    j = at - s["pos"][r]  # a row's place among its request's rows
    q = s["q"].float()
    g = q.shape[1] // hk
    wideq = q.new_zeros((n, wide, hk, g, d))
    wideq[r, j] = q.view(-1, hk, g, d)
    p = wideq.permute(0, 2, 1, 3, 4).reshape(n, hk, wide * g, d) @ k.transpose(2, 3)
    p = p.view(n, hk, wide, g, cap).mul_(s["scale"])
    rows = s["offsets"].diff()
    place = torch.arange(cap, device="cuda")
    step = torch.arange(wide, device="cuda")
    hidden = (place > (s["pos"][:, None] + step)[..., None]) | (step >= rows[:, None])[..., None]  # [n, wide, cap]
    p.masked_fill_(hidden[:, None, :, None], NINF)
    top = p.amax(-1, keepdim=True)
    p = (p - torch.where(top == NINF, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    o = (p.view(n, hk, wide * g, cap) @ v).view(n, hk, wide, g, d).permute(0, 2, 1, 3, 4)[r, j]
    o = o.reshape(-1, hk * g, d).to(s["dtype"])
    if s["mass"] is None:
        return o
    weight = p.sum((2, 3))  # [n, hk, cap]
    old = s["mass"][slot]
    new = (place >= s["pos"][:, None]) & (place < (s["pos"] + rows)[:, None])
    mass = s["mass"].clone()
    mass[slot] = torch.where(new[:, None], torch.zeros_like(old), old) + weight
    return o, mass


def _plain_evict(s):
    n, hk, cap, keep = s["n"], s["hk"], s["cap"], s["keep"]
    src, dst = s["slot"].long(), s["dst"].long()
    length = s["pos"]
    place = torch.arange(cap, device="cuda", dtype=torch.int32).expand(n, hk, cap)
    long = length[:, None, None]
    # the latest first, then by weight, then by place; what lies past the end last
    score = s["mass"][src].masked_fill(place >= long - s["recent"], float("inf"))
    score = score.masked_fill(place >= long, -1.0)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    there = torch.arange(best.shape[-1], device="cuda") < long
    kept = best.masked_fill(~there, cap).sort(-1).values
    new_length = length.clamp(max=keep)
    at = kept.clamp(max=cap - 1)
    old = s["mass"]
    mass = old.clone()
    held = torch.where(there, old[src].gather(-1, at), old[dst][..., :at.shape[-1]])
    mass[dst, :, :at.shape[-1]] = held
    rows = (src[:, None, None], torch.arange(hk, device="cuda")[:, None], at)
    k = _decode(s["k_codes"][rows], s["k_scales"][rows])  # [n, hk, keep, d]
    v = _decode(s["v_codes"][rows], s["v_scales"][rows])
    t = torch.arange(s["kept_total"], device="cuda", dtype=torch.int32)
    r = torch.searchsorted(s["kept_offsets"], t, right=True) - 1
    j = (t - s["kept_offsets"][r]).long()
    out = torch.full((n, hk, keep), -1, dtype=torch.int32, device="cuda")
    out[..., :at.shape[-1]] = torch.where(there, kept, torch.full_like(kept, -1)).int()
    return new_length, out, mass, k[r, :, j].to(s["dtype"]), v[r, :, j].to(s["dtype"])


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    i = _inputs(case, seed)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    g = hq // hk
    if case["op"] == "prompt":
        out, q0, k0 = [], 0, 0
        for nq, nk in zip(i["lens"], i["klens"]):
            o = torch.empty((nq, hq, d), dtype=torch.float64, device="cuda")
            for h in range(hq):
                k, v = i["k"][k0:k0 + nk, h // g].double(), i["v"][k0:k0 + nk, h // g].double()
                for a in range(0, nq, 2048):
                    b = min(nq, a + 2048)
                    seen = b + nk - nq
                    x = i["q"][q0 + a:q0 + b, h].double() @ k[:seen].T * i["scale"]
                    x += torch.full_like(x, NINF).triu_(a + nk - nq + 1)
                    o[a:b, h] = torch.softmax(x, -1) @ v[:seen]
            out.append(o)
            q0, k0 = q0 + nq, k0 + nk
        return torch.cat(out)
    if case["op"] == "append":
        return tuple(_exact_values(i[x]) for x in ("k", "v"))
    n, slots, cap = case["requests"], i["slots"], i["cap"]
    if case["op"] == "attend":
        out, t = [], 0
        mass = i["mass"].double() if case["mass"] else None
        for r in range(n):
            old, rows = i["lens"][r], i["rows"][r]
            k = _exact_values(i["k"][r, :old + rows])  # [keys, hk, d]
            v = _exact_values(i["v"][r, :old + rows])
            if mass is not None:
                mass[i["slot"][r], :, old:old + rows] = 0
            for j in range(rows):
                seen = old + j + 1
                q = i["q"][t].double().view(hk, g, d)
                p = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k[:seen]) * i["scale"], -1)
                out.append(torch.einsum("hgn,nhd->hgd", p, v[:seen]).reshape(hq, d))
                if mass is not None:
                    mass[i["slot"][r], :, :seen] += p.sum(1)
                t += 1
        o = torch.stack(out)
        return o if mass is None else (o, mass)
    keep, recent = case["keep"], case["recent"]
    mass, ks, vs = i["mass"].double(), [], []
    for r in range(n):
        length, slot = i["lens"][r], i["slot"][r]
        m = min(length, keep)
        first = max(0, length - recent)
        w = i["mass"][slot, :, :first].double()
        rest = torch.arange(first, length, device="cuda").expand(hk, -1)
        best = w.sort(dim=-1, descending=True, stable=True).indices[:, :m - rest.shape[1]] if m > rest.shape[1] else \
            rest[:, :0]
        kept = torch.cat([best.sort(-1).values, rest[:, rest.shape[1] - min(m, rest.shape[1]):]], 1)
        mass[slot + n, :, :m] = i["mass"][slot].double().gather(-1, kept)
        for got, x in ((ks, "k"), (vs, "v")):
            rows = i[x][r].gather(0, kept.T[..., None].expand(-1, -1, d))
            got.append(_exact_values(rows))
    return None, None, mass, torch.cat(ks), torch.cat(vs)


def _exact_values(x):
    """What a cache of 4-bit blocks holds for rows x, in 64 bits: codes by the format's own 32-bit rule."""
    b = x.float().reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().max(-1, keepdim=True).values
    first = (b.abs() == top).int().argmax(-1, keepdim=True)
    d = torch.take_along_dim(b, first, -1) * -0.125
    r = torch.nan_to_num(b / d).double()
    q = (torch.sign(r) * torch.floor(r.abs() + 0.5) + 8).clamp(0, 15)
    return ((q - 8) * d.half().double()).reshape(x.shape)
