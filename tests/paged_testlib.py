"""Plain 64-bit forms of the paged-cache operators and of the rotary positions,
for the tests: the formulas of include/zha.h in numpy, sharing no code with
the library."""
import math

import numpy as np
import torch

# one rounding to t: at most half a step relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=4096):
    """(angle per position, factor of the values) in extended precision."""
    L = np.longdouble
    rd = L(rotary_dim)
    base = L(base)
    if scaling == "ntk" and rotary_dim > 2:
        base = base * L(factor) ** (rd / (rd - 2))
    theta = base ** (-2 * np.arange(rotary_dim // 2, dtype=L) / rd)
    if scaling == "linear":
        theta = theta / L(factor)
    if scaling == "yarn":
        turns = original_len * theta / (2 * L(math.pi))
        g = np.clip((turns - 1) / 31, 0, 1)
        return (1 - g) * theta / L(factor) + g * theta, 0.1 * math.log(factor) + 1
    return theta, 1.0


def rotate(x, positions, rotary_dim, layout, theta, m, transpose=False):
    """x [n, heads, d] float64 at positions [n]."""
    a = (np.asarray(positions, dtype=np.longdouble)[:, None] * theta[None, :])[:, None, :]
    c, s = (m * np.cos(a)).astype(np.float64), (m * np.sin(a)).astype(np.float64)
    s = -s if transpose else s
    y = x.copy()
    if layout == "half":
        u, v = slice(0, rotary_dim // 2), slice(rotary_dim // 2, rotary_dim)
    else:
        u, v = slice(0, rotary_dim, 2), slice(1, rotary_dim, 2)
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., u] * s + x[..., v] * c
    return y


def pair_size(x, rotary_dim, layout):
    """|x| + |y| of each coordinate's pair (the coordinate's own size where it passes through)."""
    p = np.abs(x)
    q = p.copy()
    if layout == "half":
        u, v = slice(0, rotary_dim // 2), slice(rotary_dim // 2, rotary_dim)
    else:
        u, v = slice(0, rotary_dim, 2), slice(1, rotary_dim, 2)
    q[..., u] = q[..., v] = p[..., u] + p[..., v]
    return q


def plan(table, lens, n_new, free, n_free, page_size, max_tokens):
    """zha_paged_plan in plain integers. Returns a dict of lists and the set of error codes it calls for."""
    B, width, n_pages = len(lens), len(table[0]), len(free)
    table, free, errors = [list(r) for r in table], list(free), set()
    pages = lambda n: -(-n // page_size)  # noqa: E731
    valid = [0 <= n <= width * page_size for n in lens]
    if not all(valid):
        errors.add(1)
    ends = [b for b in range(B) if n_new[b] < 0 and valid[b]]
    back = [table[b][c] for b in ends for c in range(pages(lens[b]))]
    ok = 0 <= n_free <= n_pages and n_free + len(back) <= n_pages
    out = list(lens)
    have = n_free
    positions, slots, seq_ids = [0] * max_tokens, [-1] * max_tokens, [-1] * max_tokens
    if not ok:
        errors.add(1)
    else:
        for p in back:
            if not 0 <= p < n_pages:
                errors.add(1)
            free[have] = p
            have += 1
        for b in ends:
            out[b] = 0
    start, asked, top = 0, 0, have
    cu = [0]
    for b in range(B):
        n = max(n_new[b], 0)
        first, start = start, start + n
        cu.append(min(start, max_tokens))
        if n_new[b] < 0 or not valid[b]:
            continue
        fits = ok and lens[b] + n <= width * page_size and start <= max_tokens
        need = pages(lens[b] + n) - pages(lens[b]) if fits else 0
        if fits and need and asked + need > top:
            fits = False
        asked += need
        if not fits:
            if n:
                errors.add(3 if ok else 1)
            continue
        for c in range(pages(lens[b]), pages(lens[b] + n)):
            have -= 1
            table[b][c] = free[have]
            if not 0 <= free[have] < n_pages:
                errors.add(1)
        for i in range(n):
            p = lens[b] + i
            page = table[b][p // page_size]
            if 0 <= page < n_pages:
                positions[first + i], slots[first + i], seq_ids[first + i] = p, page * page_size + p % page_size, b
            else:
                errors.add(1)
        out[b] = lens[b] + n
    return {"table": table, "free": free, "n_free": have, "lens": out, "positions": positions, "slots": slots,
            "seq_ids": seq_ids, "cu": cu}, errors


def attend(q, K, V, scale):
    """q [G, d], K, V [n, d] float64 -> out [G, d], lse [G], and sum_t p_t |v_t| [G, d]."""
    if K.shape[0] == 0:
        return np.zeros_like(q), np.full(q.shape[0], -np.inf), np.zeros_like(q)
    x = scale * (q @ K.T)
    top = x.max(axis=1, keepdims=True)
    e = np.exp(x - top)
    z = e.sum(axis=1, keepdims=True)
    return e @ V / z, (top + np.log(z))[:, 0], e @ np.abs(V) / z


def gather(pool, table_row, lo, hi, kvh, page_size):
    """Cache rows [lo, hi) of one KV head, float64, from a pool [pages, heads, page_size, d] on any device."""
    t = torch.arange(lo, hi)
    pages = table_row.cpu().long()[t // page_size]
    return np64(pool[pages.to(pool.device), kvh, (t % page_size).to(pool.device)]) if hi > lo else \
        np.zeros((0, pool.shape[-1]))
