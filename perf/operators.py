"""The paged-cache operators and their plain forms, on cases of real sizes.

Four operators that are used in turn by a serving step of one attention layer:

* ``plan``    block table, slot map and positions of a step's new tokens, from the requests' lengths;
* ``rotary``  rotary position embedding of queries and keys (and its transpose, the gradient);
* ``write``   rotation of queries and keys with the scatter of keys and values to their cache slots;
* ``decode``  exact softmax attention of single query rows over a paged key/value cache.

With ``own`` false ``run`` computes an operator with elementary torch operations in 32 bits (angles and page
arithmetic in 64); with ``own`` true it makes the library's call on the same state. ``exact`` computes it in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def _rope(rotary_dim, layout="half", scaling="none", factor=1.0, base=10000.0, original_len=4096):
    return {"rotary_dim": rotary_dim, "layout": layout, "scaling": scaling, "factor": factor, "base": base,
            "original_len": original_len}


def listed():
    return [
        # one user, the first tokens of an answer: everything is latency
        {"name": "decode 1 x 200, 32/4 heads", "op": "decode", "dtype": "bf16", "rows": 1, "pad": 0, "hq": 32, "hkv": 4,
         "d": 128, "page": 16, "len_min": 200, "len_max": 200, "window": 0, "mapped": False, "shape": 1},
        # a served batch: lengths from a first message to a long document, pages of 16
        {"name": "decode 64 x 16..16384, 32/4 heads", "op": "decode", "dtype": "bf16", "rows": 64, "pad": 0, "hq": 32,
         "hkv": 4, "d": 128, "page": 16, "len_min": 16, "len_max": 16384, "window": 0, "mapped": False, "shape": 2},
        # the long-context configuration of the repository: 4 sequences of 256K tokens
        {"name": "decode 4 x 262144, 32/4 heads", "op": "decode", "dtype": "bf16", "rows": 4, "pad": 0, "hq": 32,
         "hkv": 4, "d": 128, "page": 64, "len_min": 262144, "len_max": 262144, "window": 0, "mapped": False, "shape": 3},
        # a layer with a sliding window and no shared heads, rows mapped to sequences, the batch padded for a graph
        {"name": "decode 13 of 16 x 5000..100000, window 4096, 8/8 heads", "op": "decode", "dtype": "bf16", "rows": 13,
         "pad": 3, "hq": 8, "hkv": 8, "d": 128, "page": 32, "len_min": 5000, "len_max": 100000, "window": 4096,
         "mapped": True, "shape": 4},
        # an fp32 cache (used where decoding is checked), head_dim 64, odd lengths and small pages
        {"name": "decode f32 6 x 1001..20001, 16/2 heads, d 64", "op": "decode", "dtype": "f32", "rows": 6, "pad": 0,
         "hq": 16, "hkv": 2, "d": 64, "page": 8, "len_min": 1001, "len_max": 20001, "window": 0, "mapped": False,
         "shape": 5},
        # the new tokens of a decode step far into a context that was extended eightfold
        {"name": "rotary 4 tokens, 32/4 heads, yarn", "op": "rotary", "dtype": "bf16", "tokens": 4, "hq": 32, "hkv": 4,
         "d": 128, "pos_max": 262144, "transpose": False, "packed": False, "shape": 6,
         **_rope(128, "half", "yarn", 8.0, 500000.0, 32768)},
        # a prompt of 16K tokens, q and k read out of one packed projection
        {"name": "rotary 16384 tokens, 32/4 heads, packed", "op": "rotary", "dtype": "bf16", "tokens": 16384, "hq": 32,
         "hkv": 4, "d": 128, "pos_max": 16384, "transpose": False, "packed": True, "shape": 7, **_rope(128)},
        # the gradient of an interleaved rotation of half the head, fp32, an odd number of tokens
        {"name": "rotary transposed f32 1537 tokens, 16/2 heads, 32 of 64 interleaved", "op": "rotary", "dtype": "f32",
         "tokens": 1537, "hq": 16, "hkv": 2, "d": 64, "pos_max": 8192, "transpose": True, "packed": False, "shape": 8,
         **_rope(32, "interleaved", "linear", 4.0)},
        # one new token for each of 64 sequences into their pages
        {"name": "write 64 tokens, 32/4 heads", "op": "write", "dtype": "bf16", "tokens": 64, "pad": 0, "hq": 32, "hkv": 4,
         "d": 128, "page": 16, "pos_max": 16384, "packed": False, "shape": 9, **_rope(128)},
        # a chunk of prompts in a padded buffer, from a packed projection
        {"name": "write 12001 of 12288 tokens, 32/4 heads, packed", "op": "write", "dtype": "bf16", "tokens": 12001,
         "pad": 287, "hq": 32, "hkv": 4, "d": 128, "page": 64, "pos_max": 32768, "packed": True, "shape": 10,
         **_rope(128, "half", "ntk", 4.0)},
        # the plan of a decode step: one new token each, a page needed now and then
        {"name": "plan 64 requests, one token each", "op": "plan", "requests": 64, "page": 16, "len_max": 16384,
         "new_max": 1, "release": 0.0, "spare": 5, "shape": 11},
        # a busy scheduler: prompts admitted, decodes going on, requests ending, padded token buffers
        {"name": "plan 700 requests, prompts of up to 1024, some ending", "op": "plan", "requests": 700, "page": 16,
         "len_max": 8192, "new_max": 1024, "release": 0.1, "spare": 1000, "shape": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng, d):
    rd = rng.choice([d, d, d, d // 2, d // 4, 2 * rng.randint(2, d // 2)])
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    return _rope(rd, rng.choice(["half", "interleaved"]), scaling, 1.0 if scaling == "none" else rng.uniform(1.5, 16.0),
                 rng.choice([10000.0, 500000.0, 1000000.0]), rng.choice([2048, 4096, 32768]))


def draw(rng):
    op = rng.choice(["decode", "decode", "rotary", "write", "plan"])
    shape = rng.randrange(1 << 30)
    if op == "plan":
        return {"op": op, "requests": _log(rng, 1, 1500), "page": rng.choice([1, 8, 16, 32, 64, 256]),
                "len_max": _log(rng, 16, 16384), "new_max": rng.choice([1, 1, _log(rng, 2, 512)]),
                "release": rng.choice([0.0, 0.1, 0.3]), "spare": _log(rng, 1, 3000), "shape": shape}
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
    if op == "decode":
        rows = _log(rng, 1, 96)
        # the plain form pads every row to the longest: keep that within the largest listed case
        most = min(262144, (1 << 28) // (rows * hkv * d))
        hi = _log(rng, 1, most)
        return {"op": op, "dtype": dtype, "rows": rows, "pad": rng.choice([0, 0, rng.randint(1, 5)]), "hq": hq, "hkv": hkv,
                "d": d, "page": rng.choice([1, 8, 16, 16, 32, 64, 128, 256]), "len_min": _log(rng, 1, hi), "len_max": hi,
                "window": rng.choice([0, 0, 0, _log(rng, 1, 8192)]), "mapped": rng.choice([False, True]), "shape": shape}
    tokens = min(_log(rng, 1, 16384), (1 << 26) // ((hq + 2 * hkv) * d * (2 if dtype == "f32" else 1)))
    case = {"op": op, "dtype": dtype, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "pos_max": _log(rng, tokens, 1 << 20),
            "packed": rng.choice([False, True]), "shape": shape, **_draw_rope(rng, d)}
    if op == "rotary":
        return {**case, "transpose": rng.choice([False, True])}
    return {**case, "pad": rng.choice([0, rng.randint(1, 200)]), "page": rng.choice([1, 8, 16, 32, 64, 256])}


# ---------------------------------------------------------------- shapes that follow from a case alone

def _lengths(case):
    """Lengths of a decode case's rows: spread over their logarithm, the two ends among them."""
    r = random.Random(case["shape"])
    lens = [_log(r, case["len_min"], case["len_max"]) for _ in range(case["rows"])]
    lens[0] = case["len_max"]
    lens[-1] = case["len_min"] if case["rows"] > 1 else case["len_max"]
    return lens


def _requests(case):
    """(length, new tokens or -1 for a request that ends) of a plan case's requests."""
    r = random.Random(case["shape"])
    got = []
    for _ in range(case["requests"]):
        n = _log(r, 1, case["len_max"])
        if r.random() < case["release"]:
            got.append((n, -1))
        elif case["new_max"] == 1 or r.random() < 0.6:
            got.append((n, 1 if r.random() < 0.95 else 0))
        else:
            got.append((0, _log(r, 2, case["new_max"])))
    return got


def _pages(n, page):
    return -(-n // page)


def _plan_sizes(case):
    """(sequences' lengths, new tokens, pages held, pages needed, token buffer, table width, pool) of a plan case."""
    lens, new = zip(*_requests(case))
    page = case["page"]
    held = sum(_pages(n, page) for n in lens)
    need = sum(_pages(n + a, page) - _pages(n, page) for n, a in zip(lens, new) if a > 0)
    tokens = sum(a for a in new if a > 0)
    width = max(_pages(n + max(a, 0), page) for n, a in zip(lens, new)) + 1
    return lens, new, held, need, tokens + 64, width, held + need + case["spare"]


def work(case):
    op = case["op"]
    if op == "plan":
        lens, new, held, need, tokens, width, pool = _plan_sizes(case)
        ended = sum(_pages(n, case["page"]) for n, a in zip(lens, new) if a < 0)
        return {"bytes": 4 * (4 * len(lens) + 2 * need + 2 * ended + 3 * tokens), "flops": 0}
    es = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "decode":
        seen = [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]
        pages = sum(_pages(n, case["page"]) for n in seen)
        return {"bytes": 2 * sum(seen) * hkv * d * es + len(seen) * hq * (2 * d * es + 4) + 4 * pages + 4 * len(seen),
                "flops": 4 * sum(seen) * hq * d}
    heads = hq + hkv + (hkv if op == "write" else 0)
    per = 2 * heads * d * es + (8 if op == "write" else 4)
    return {"bytes": case["tokens"] * per, "flops": 3 * case["tokens"] * (hq + hkv) * case["rotary_dim"]}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _prepare_decode(case, seed):
    g = _gen(seed)
    dt = TYPES[case["dtype"]]
    hq, hkv, d, page, rows = case["hq"], case["hkv"], case["d"], case["page"], case["rows"]
    lens = _lengths(case)
    counts = [_pages(n, page) for n in lens]
    width, used = max(counts) + 1, sum(counts)
    pool = used + 3
    perm = torch.randperm(pool, generator=g, device=DEVICE).to(torch.int32)
    # row b's pages are the next counts[b] of a permutation; the rest of its row of the table is never read
    first = torch.tensor([sum(counts[:b]) for b in range(rows)], device=DEVICE)
    at = first[:, None] + torch.arange(width, device=DEVICE)[None, :]
    held = torch.arange(width, device=DEVICE)[None, :] < torch.tensor(counts, device=DEVICE)[:, None]
    table = torch.where(held, perm[at.clamp(max=pool - 1)], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
    k = _randn(g, pool, hkv, page, d, dtype=dt)
    k += 0.7 * _randn(g, pool, hkv, 1, d, dtype=dt)   # neighbouring keys are alike
    v = _randn(g, pool, hkv, page, d, dtype=dt)
    n = rows + case["pad"]
    s = {"q": 1.5 * _randn(g, n, hq, d, dtype=dt), "k": k, "v": v, "table": table, "lens": _ints(lens),
         "out": torch.zeros((n, hq, d), dtype=dt, device=DEVICE), "lse": torch.zeros((n, hq), device=DEVICE),
         "longest": max(lens), "seq_ids": None, "positions": None}
    if case["mapped"] or case["pad"]:
        order = list(range(rows))
        random.Random(case["shape"] + 1).shuffle(order)
        s["seq_ids"] = _ints(order + [-1] * case["pad"])
        s["positions"] = _ints([lens[b] - 1 for b in order] + [0] * case["pad"])
    return s


def _projected(g, case, n, parts):
    """[n, heads, d] tensors for each of `parts`, of their own or as slices of one packed projection."""
    d, dt = case["d"], TYPES[case["dtype"]]
    if case["packed"]:
        x = _randn(g, n, sum(parts) * d, dtype=dt)
        return [t.unflatten(1, (-1, d)) for t in torch.split(x, [h * d for h in parts], dim=1)]
    return [_randn(g, n, h, d, dtype=dt) for h in parts]


def _prepare_rotary(case, seed):
    g = _gen(seed)
    n = case["tokens"]
    q, k = _projected(g, case, n, [case["hq"], case["hkv"]] + ([case["hkv"]] if case["packed"] else []))[:2]
    start = random.Random(case["shape"]).randint(0, max(case["pos_max"] - n, 0))
    return {"q": q, "k": k, "positions": torch.arange(start, start + n, dtype=torch.int32, device=DEVICE),
            "q_out": torch.empty(q.shape, dtype=q.dtype, device=DEVICE),
            "k_out": torch.empty(k.shape, dtype=k.dtype, device=DEVICE)}


def _prepare_write(case, seed):
    g = _gen(seed)
    n, page, pad = case["tokens"], case["page"], case["pad"]
    q, k, v = _projected(g, case, n + pad, [case["hq"], case["hkv"], case["hkv"]])
    pool = _pages(n, page) + n // (4 * page) + 2
    shape = (pool, case["hkv"], page, case["d"])
    # tokens fill whole pages in a shuffled order of the pages, as prompts and decodes together do
    perm = torch.randperm(pool, generator=g, device=DEVICE)
    i = torch.arange(n, device=DEVICE)
    slots = (perm[i // page] * page + i % page).to(torch.int32)
    pos = torch.randint(0, case["pos_max"], (n,), generator=g, device=DEVICE, dtype=torch.int32)
    return {"q": q, "k_new": k, "v_new": v, "slots": torch.cat([slots, _ints([-1] * pad)]),
            "positions": torch.cat([pos, _ints([0] * pad)]), "k": _randn(g, *shape, dtype=q.dtype),
            "v": _randn(g, *shape, dtype=q.dtype), "q_out": torch.zeros(q.shape, dtype=q.dtype, device=DEVICE)}


def _prepare_plan(case, seed):
    g = _gen(seed)
    lens, new, held, need, tokens, width, pool = _plan_sizes(case)
    page, n = case["page"], len(lens)
    perm = torch.randperm(pool, generator=g, device=DEVICE).to(torch.int32)
    counts = torch.tensor([_pages(x, page) for x in lens], device=DEVICE)
    first = torch.cumsum(counts, 0) - counts
    col = torch.arange(width, device=DEVICE)[None, :]
    at = (first[:, None] + col).clamp(max=pool - 1)
    table = torch.where(col < counts[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
    free = torch.cat([perm[held:], torch.full((held,), -1, dtype=torch.int32, device=DEVICE)])
    empty = lambda m: torch.zeros(m, dtype=torch.int32, device=DEVICE)  # noqa: E731
    return {"lens": _ints(lens), "n_new": _ints(new), "table": table, "free": free, "n_free": _ints([pool - held]),
            "lens_out": empty(n), "n_free_out": empty(1), "positions": empty(tokens), "slots": empty(tokens),
            "seq_ids": empty(tokens), "cu": empty(n + 1)}


def prepare(case, seed):
    s = {"decode": _prepare_decode, "rotary": _prepare_rotary, "write": _prepare_write, "plan": _prepare_plan}[case["op"]](case, seed)
    s["case"] = case
    if own:
        _handles(s, case)
    return s


def _handles(s, case):
    """What a program that uses the library keeps from call to call: configuration, rotation table, workspace, status."""
    from tree_indexed_sparse_02_b200 import zha
    s["zha"] = zha
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEVICE)
    if case["op"] in ("rotary", "write"):
        s["rotary"] = zha.Rotary(case["rotary_dim"], base=case["base"], layout=case["layout"], scaling=case["scaling"],
                                 factor=case["factor"], original_len=case["original_len"])
    if case["op"] == "plan":
        s["cfg"] = zha.paged_config(len(s["lens"]), 1, 1, 128, page_size=case["page"], n_pages=len(s["free"]),
                                    max_pages=s["table"].shape[1])
        s["map"] = {k: s[k] for k in ("positions", "slots", "seq_ids", "cu")}
    if case["op"] in ("write", "decode"):
        table = s.get("table")
        s["cfg"] = zha.paged_config(1 if table is None else table.shape[0], case["hq"], case["hkv"], case["d"],
                                    page_size=case["page"], n_pages=s["k"].shape[0],
                                    max_pages=1 if table is None else table.shape[1], dtype=case["dtype"],
                                    window=case.get("window", 0))
    if case["op"] == "decode":
        s["workspace"] = zha.paged_workspace(s["cfg"], rows=s["q"].shape[0])


# ---------------------------------------------------------------- plain forms

def _frequencies(case):
    """(angle per position of each pair, factor of the rotated values), in 64 bits."""
    rd, base, factor = case["rotary_dim"], case["base"], case["factor"]
    if case["scaling"] == "ntk" and rd > 2:
        base = base * factor ** (rd / (rd - 2))
    f = base ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=DEVICE) / rd)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "yarn":
        turns = case["original_len"] * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return (1 - keep) * f / factor + keep * f, 0.1 * math.log(factor) + 1
    return f, 1.0


def _rotate(x, positions, case, transpose=False):
    f, m = _frequencies(case)
    a = positions.to(torch.float64)[:, None, None] * f
    c, s = (m * torch.cos(a)).float(), (m * torch.sin(a)).float()
    s = -s if transpose else s
    rd = case["rotary_dim"]
    r, rest = x[..., :rd].float(), x[..., rd:]
    if case["layout"] == "half":
        u, w = r[..., :rd // 2], r[..., rd // 2:]
        y = torch.cat([u * c - w * s, u * s + w * c], dim=-1)
    else:
        u, w = r[..., 0::2], r[..., 1::2]
        y = torch.stack([u * c - w * s, u * s + w * c], dim=-1).flatten(-2)
    return torch.cat([y.to(x.dtype), rest], dim=-1)


def _plain_write(s, case):
    q, k = _rotate(s["q"], s["positions"], case), _rotate(s["k_new"], s["positions"], case)
    used = s["slots"] >= 0
    page, off = (s["slots"] // case["page"])[used].long(), (s["slots"] % case["page"])[used].long()
    s["k"][page, :, off] = k[used]
    s["v"][page, :, off] = s["v_new"][used]
    return torch.where(used[:, None, None], q, s["q_out"]), s["k"], s["v"]


def _plain_decode(s, case):
    hkv, d, page = case["hkv"], case["d"], case["page"]
    n = s["q"].shape[0]
    seq = torch.arange(n, device=DEVICE) if s["seq_ids"] is None else s["seq_ids"].long()
    live = seq >= 0
    seq = seq.clamp(min=0)
    lens = s["lens"][seq].long() if s["positions"] is None else s["positions"].long() + 1
    low = (lens - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(lens)
    span = min(s["longest"], case["window"]) if case["window"] else s["longest"]
    at = low[:, None] + torch.arange(span, device=DEVICE)             # [rows, span] cache positions
    seen = at < lens[:, None]
    at = torch.where(seen, at, torch.zeros_like(at))
    pg = s["table"][seq[:, None], at // page].long()
    k = s["k"][pg, :, at % page].float()                              # [rows, span, hkv, d]
    q = s["q"].float().view(n, hkv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(d)         # [rows, hkv, G, span]
    del k
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    lse = torch.logsumexp(x, dim=-1)
    p = torch.exp(x - lse[..., None])
    v = s["v"][pg, :, at % page].float()
    out = torch.matmul(p, v.permute(0, 2, 1, 3)).view(n, -1, d).to(s["q"].dtype)
    return (torch.where(live[:, None, None], out, s["out"]),
            torch.where(live[:, None], lse.view(n, -1), s["lse"]))


def _plain_plan(s, case):
    page = case["page"]
    lens, new, n_free = s["lens"].long(), s["n_new"].long(), s["n_free"].long()
    table, free = s["table"], s["free"]
    pool, width, tokens = free.numel(), table.shape[1], s["slots"].numel()
    col = torch.arange(width, device=DEVICE)[None, :]
    ends, add = new < 0, new.clamp(min=0)
    old = (lens + page - 1) // page
    # pages of the requests that end go on top of the free stack, in order
    back = torch.where(ends, old, 0)
    to = torch.where(col < back[:, None], n_free + (torch.cumsum(back, 0) - back)[:, None] + col, pool)
    grown = torch.cat([free, free.new_zeros(1)])
    grown[to.flatten()] = table.flatten()
    free.copy_(grown[:pool])
    have = n_free + back.sum()
    # pages of the others come off the top, in order; who does not fit gets none
    last = torch.cumsum(add, 0)
    fits = ~ends & (lens + add <= width * page) & (last <= tokens)
    need = torch.where(fits, (lens + add + page - 1) // page - old, 0)
    upto = torch.cumsum(need, 0)
    fits &= (need == 0) | (upto <= have)
    take = torch.where(fits, need, 0)
    k = (upto - need)[:, None] + col - old[:, None]
    fresh = (col >= old[:, None]) & (col < (old + take)[:, None])
    table.copy_(torch.where(fresh, free[(have - 1 - k).clamp(0, pool - 1)], table))
    i = torch.arange(tokens, device=DEVICE)
    b = torch.searchsorted(last, i, right=True).clamp(max=lens.numel() - 1)
    used = (i < last[-1]) & fits[b]
    pos = torch.where(used, lens[b] + i - (last - add)[b], 0)
    slot = torch.where(used, table[b, pos // page].long() * page + pos % page, -1)
    cu = torch.cat([last.new_zeros(1), last]).clamp(max=tokens)
    as32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": table, "free": free, "lens": as32(torch.where(ends, 0, torch.where(fits, lens + add, lens))),
            "n_free": as32(have - take.sum()), "positions": as32(pos), "slots": as32(slot),
            "seq_ids": as32(torch.where(used, b, -1)), "cu": as32(cu)}


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        zha = s["zha"]
        if op == "decode":
            zha.paged_decode(s["cfg"], s["q"], s["k"], s["v"], s["table"], s["lens"], s["out"], s["workspace"],
                             lse=s["lse"], seq_ids=s["seq_ids"], positions=s["positions"], dev_status=s["status"])
            return s["out"], s["lse"]
        if op == "rotary":
            zha.rotary(s["rotary"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], transpose=case["transpose"])
            return s["q_out"], s["k_out"]
        if op == "write":
            zha.paged_write(s["cfg"], s["rotary"], s["q"], s["k_new"], s["v_new"], s["positions"], s["slots"],
                            s["q_out"], s["k"], s["v"], dev_status=s["status"])
            return s["q_out"], s["k"], s["v"]
        zha.paged_plan(s["cfg"], s["table"], s["lens"], s["n_new"], s["free"], s["n_free"], s["map"],
                       lens_out=s["lens_out"], n_free_out=s["n_free_out"], dev_status=s["status"])
        return {"table": s["table"], "free": s["free"], "lens": s["lens_out"], "n_free": s["n_free_out"],
                "positions": s["positions"], "slots": s["slots"], "seq_ids": s["seq_ids"], "cu": s["cu"]}
    if op == "decode":
        return _plain_decode(s, case)
    if op == "rotary":
        return (_rotate(s["q"], s["positions"], case, case["transpose"]),
                _rotate(s["k"], s["positions"], case, case["transpose"]))
    if op == "write":
        return _plain_write(s, case)
    return _plain_plan(s, case)


# ---------------------------------------------------------------- 64 bits

def _exact_rotation(x, positions, case, transpose=False):
    """Each pair as a complex number times m e^(i position theta)."""
    rd = case["rotary_dim"]
    base, factor, m = case["base"], case["factor"], 1.0
    if case["scaling"] == "ntk" and rd > 2:
        base *= factor ** (rd / (rd - 2.0))
    theta = np.exp(-np.log(base) * 2.0 * np.arange(rd // 2) / rd)
    if case["scaling"] == "linear":
        theta = theta / factor
    if case["scaling"] == "yarn":
        share = np.clip((case["original_len"] * theta / (2.0 * np.pi) - 1.0) / 31.0, 0.0, 1.0)
        theta = theta * (share + (1.0 - share) / factor)
        m = 1.0 + 0.1 * math.log(factor)
    angle = positions.double()[:, None] * torch.from_numpy(theta).to(DEVICE)
    turn = torch.polar(torch.full_like(angle, m), -angle if transpose else angle)[:, None, :]
    y = x.double()
    if case["layout"] == "half":
        z = torch.complex(y[..., :rd // 2], y[..., rd // 2:rd]) * turn
        y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:rd:2], y[..., 1:rd:2]) * turn
        y[..., 0:rd:2], y[..., 1:rd:2] = z.real, z.imag
    return y


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    if op == "rotary":
        s = _prepare_rotary(case, seed)
        return tuple(_exact_rotation(s[x], s["positions"], case, case["transpose"]) for x in ("q", "k"))
    if op == "write":
        s = _prepare_write(case, seed)
        n, page, hkv, d = case["tokens"], case["page"], case["hkv"], case["d"]
        q = _exact_rotation(s["q"], s["positions"], case)
        q[n:] = 0.0
        pools = []
        for pool, new in ((s["k"], _exact_rotation(s["k_new"], s["positions"], case)), (s["v"], s["v_new"].double())):
            flat = pool.double().transpose(1, 2).reshape(-1, hkv, d)
            flat[s["slots"][:n].long()] = new[:n]
            pools.append(flat.view(-1, page, hkv, d).transpose(1, 2))
        return (q, *pools)
    s = _prepare_decode(case, seed)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    out, lse = s["out"].double(), s["lse"].double()
    for r in range(out.shape[0]):
        b = r if s["seq_ids"] is None else int(s["seq_ids"][r])
        if b < 0:
            continue
        n = int(s["lens"][b])
        lo = max(0, n - case["window"]) if case["window"] else 0
        pg = s["table"][b, :_pages(n, page)].long()
        pg = pg[lo // page:]
        cut = slice(lo - lo // page * page, n - lo // page * page)
        for h in range(hkv):
            k = s["k"][pg, h].reshape(-1, d)[cut].double()
            v = s["v"][pg, h].reshape(-1, d)[cut].double()
            rows = slice(h * hq // hkv, (h + 1) * hq // hkv)
            x = s["q"][r, rows].double() @ k.T * d ** -0.5
            top = x.max(dim=1, keepdim=True).values
            e = torch.exp(x - top)
            z = e.sum(dim=1, keepdim=True)
            out[r, rows] = e @ v / z
            lse[r, rows] = (top + torch.log(z))[:, 0]
    return out, lse
