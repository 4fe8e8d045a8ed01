"""The paged cache on the GPU -- plan, write, decode, and steps of them -- against
plain 64-bit (or integer) forms."""
import random

import numpy as np
import pytest
import torch

import paged_testlib as P

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAME = {BF16: "bf16", F32: "f32"}


@pytest.fixture(scope="module")
def zha():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_indexed_sparse_02_b200 import zha as z
    return z


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- plan

def run_plan(zha, table, lens, n_new, free, n_free, page, tokens, in_place=False):
    cfg = zha.paged_config(len(lens), 1, 1, 64, page, len(free), len(table[0]))
    t, l, f, k = ints(table), ints(lens), ints(free), ints([n_free])
    m = {x: torch.full((tokens,), 7, dtype=torch.int32, device="cuda") for x in ("positions", "slots", "seq_ids")}
    m["cu"] = ints([7] * (len(lens) + 1))
    lo, ko = (l, k) if in_place else (torch.full_like(l, 7), torch.full_like(k, 7))
    status = ints([0])
    zha.paged_plan(cfg, t, l, ints(n_new), f, k, m, lens_out=lo, n_free_out=ko, dev_status=status)
    torch.cuda.synchronize()
    got = {"table": t.tolist(), "free": f.tolist(), "n_free": int(ko), "lens": lo.tolist(), "cu": m["cu"].tolist(),
           **{x: m[x].tolist() for x in ("positions", "slots", "seq_ids")}}
    if not in_place:
        assert l.tolist() == list(lens) and int(k) == n_free
    return got, int(status)


def check_plan(zha, *args):
    want, errors = P.plan(*args)
    for in_place in (False, True):
        got, code = run_plan(zha, *args, in_place=in_place)
        assert (code in errors) if errors else code == 0, (code, errors)
        for x in want:
            assert got[x] == want[x], x
    return want


def holders(rng, lens, page, width, extra):
    """A table whose sequences hold distinct pages of a pool, and the free stack."""
    counts = [-(-max(n, 0) // page) for n in lens]
    pool = list(range(sum(counts) + extra))
    rng.shuffle(pool)
    table = []
    for c in counts:
        table.append([pool.pop() for _ in range(c)] + [-1] * (width - c))
    n_free = len(pool)
    return table, pool + [-5] * sum(counts), n_free


@pytest.mark.parametrize("B,page,tokens", [(1, 16, 1), (1, 1, 40), (5, 8, 64), (64, 16, 64), (300, 4, 5000),
                                           (1025, 32, 1500), (4096, 16, 9000)])
@pytest.mark.parametrize("kind", ["decode", "mixed", "short"])
def test_plan_matches_integers(zha, B, page, tokens, kind):
    rng = random.Random(B + page)
    lens = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, 6 * page)]) for _ in range(B)]
    if kind == "decode":
        new = [1] * B
        tokens = max(tokens, B)
    else:
        new = [rng.choice([-1, 0, 1, 1, page, rng.randint(0, 2 * page)]) for _ in range(B)]
    width = max(-(-(n + max(a, 0)) // page) for n, a in zip(lens, new)) + (0 if kind == "short" else 1)
    width = max(1, width - (2 if kind == "short" else 0))             # some do not fit the table
    lens = [min(n, width * page) for n in lens]
    table, free, n_free = holders(rng, lens, page, width, B if kind != "short" else max(1, B // 4))
    want = check_plan(zha, table, lens, new, free, n_free, page, tokens)
    live = [s for s in want["slots"] if s >= 0]
    assert len(set(live)) == len(live)


def test_plan_steps_conserve_pages(zha):
    """Steps in place over one state: sequences grow, end and start again; every page is in one place."""
    rng = random.Random(9)
    B, page, n_pages, width, tokens = 40, 8, 200, 12, 160
    cfg = zha.paged_config(B, 1, 1, 64, page, n_pages, width)
    cache = zha.PagedCache(cfg, tokens)
    state = (cache.table.tolist(), [0] * B, cache.free_pages.tolist(), n_pages)
    refused = 0
    for _ in range(60):
        table, lens, free, n_free = state
        new = [-1 if n and rng.random() < 0.1 else rng.choice([0, 1, 1, 1, 9]) for n in lens]
        want, errors = P.plan(table, lens, new, free, n_free, page, tokens)
        cache.plan(ints(new))
        code = int(cache.status)
        cache.status.zero_()
        assert code == (3 if errors else 0)
        refused += code == 3
        assert cache.table.tolist() == want["table"] and cache.lens.tolist() == want["lens"]
        assert int(cache.n_free) == want["n_free"] and cache.token_map["slots"].tolist() == want["slots"]
        state = (want["table"], want["lens"], want["free"], want["n_free"])
        held = [want["table"][b][c] for b in range(B) for c in range(-(-want["lens"][b] // page))]
        assert sorted(held + want["free"][:want["n_free"]]) == list(range(n_pages))
    assert refused


def test_plan_refuses_what_does_not_fit(zha):
    page, width = 4, 3
    table = [[0, -1, -1], [1, 2, -1], [3, -1, -1], [4, -1, -1]]
    free = [5, 6, 7, 8, 9, -1, -1, -1, -1, -1]
    # the second asks for more than the table holds: it alone is not served
    check_plan(zha, table, [4, 5, 1, 2], [1, 8, 5, 1], free, 5, page, 20)
    # two pages left: the first takes one, the second needs two, the third one: neither is served, the last needs none
    check_plan(zha, table, [4, 8, 4, 2], [1, 4 + 1 - 1, 1, 1], free, 1, page, 20)
    check_plan(zha, table, [4, 5, 4, 2], [1, 7, 1, 1], free, 2, page, 20)
    # the token buffer ends in the middle of the third
    check_plan(zha, table, [4, 5, 1, 2], [2, 2, 2, 1], free, 5, page, 5)
    # pages that come back in the same step are enough
    check_plan(zha, table, [4, 5, 1, 2], [5, -1, 5, -1], free, 0, page, 20)
    # lengths that cannot be, and counts of free pages that cannot be
    check_plan(zha, table, [-1, 13, 1, 2], [1, 1, -1, 1], free, 5, page, 20)
    for n_free in (-1, 11, 10):
        check_plan(zha, table, [4, 5, 1, 2], [1, -1, 1, 1], free, n_free, page, 20)
    # page numbers outside the pool, in the table and on the stack
    check_plan(zha, [[0, -1, -1], [99, 2, -1], [3, -1, -1], [4, -1, -1]], [3, 3, 4, 4], [1, 1, 1, -1],
               [5, 6, 7, 8, -9, -1, -1, -1, -1, -1], 4, page, 20)
    # far more tokens than any buffer
    check_plan(zha, table, [4, 5, 1, 2], [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1], free, 5, page, 20)


# ---------------------------------------------------------------- write

@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout,rd", [("half", 64), ("half", 20), ("interleaved", 48), (None, 0)])
@pytest.mark.parametrize("page", [1, 16, 256])
def test_write_matches_rotary_and_copies(zha, dt, layout, rd, page):
    """The same bits as the rotation alone and a copy, at each token's slot; everything else stays."""
    g = torch.Generator().manual_seed(page)
    n, hq, hkv, d = 75, 6, 3, 64
    n_pages = -(-4 * n // page)
    cfg = zha.paged_config(1, hq, hkv, d, page, n_pages, 1, dtype=NAME[dt])
    qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g).to(dt).cuda()
    q, k, v = (t.unflatten(1, (-1, d)) for t in torch.split(qkv, [hq * d, hkv * d, hkv * d], dim=1))
    slots = torch.randperm(n_pages * page, generator=g)[:n].to(torch.int32)
    slots[[3, 40, 74]] = torch.tensor([-1, -2 ** 31, -7], dtype=torch.int32)
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32).cuda()
    kp, vp = (torch.randn(n_pages, hkv, page, d, generator=g).to(dt).cuda() for _ in range(2))
    q_out = torch.randn(n, hq, d, generator=g).to(dt).cuda()
    rot = None if layout is None else zha.Rotary(rd, layout=layout)
    want_q, want_k = q.clone(), k.clone()
    if rot is not None:
        zha.rotary(rot, want_q, want_k, pos)
    use = slots >= 0
    s = slots[use].cuda().long()
    wk, wv, wq = kp.clone(), vp.clone(), q_out.clone()
    wk[s // page, :, s % page] = want_k[use.cuda()]
    wv[s // page, :, s % page] = v[use.cuda()]
    wq[use.cuda()] = want_q[use.cuda()]
    status = ints([0])
    zha.paged_write(cfg, rot, q, k, v, pos if rot is not None else None, slots.cuda(), q_out, kp, vp, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.equal(kp, wk) and torch.equal(vp, wv) and torch.equal(q_out, wq)
    # keys and values alone
    kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
    zha.paged_write(cfg, rot, None, k, v, pos, slots.cuda(), None, kp2, vp2, dev_status=status)
    assert torch.equal(kp2[s // page, :, s % page], want_k[use.cuda()])
    assert torch.equal(vp2[s // page, :, s % page], v[use.cuda()])


def test_write_skips_slots_beyond_the_pool(zha):
    cfg = zha.paged_config(1, 1, 1, 64, 4, 3, 1)
    x = torch.ones(3, 1, 64, dtype=BF16, device="cuda")
    kp = torch.zeros(4, 1, 4, 64, dtype=BF16, device="cuda")          # one page more than the pool has
    status, q = ints([0]), torch.zeros_like(x)
    zha.paged_write(cfg, None, x, x, x, None, ints([12, 5, 2 ** 31 - 1]), q, kp[:3], kp[:3].clone(), dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 1
    assert float(kp.float().sum()) == 64 and float(kp[1, 0, 1].float().sum()) == 64
    assert q.float().sum(dim=(1, 2)).tolist() == [0, 64, 0]


# ---------------------------------------------------------------- decode

class Case:
    """A pool whose sequences hold shuffled pages; every cache row that no sequence holds is NaN."""

    def __init__(self, zha, lens, hq, hkv, d, page, dt, window=0, scale=0.0, seed=0, amp=1.0, poison=float("nan"),
                 pool_pages=None):
        g = torch.Generator().manual_seed(seed)
        self.zha, self.lens, self.dt, self.page, self.hkv, self.window = zha, list(lens), dt, page, hkv, window
        self.G, self.d = hq // hkv, d
        counts = [-(-n // page) for n in lens]
        width = max(max(counts), 1) + 1
        n_pages = pool_pages or sum(counts) + 2
        perm = torch.randperm(n_pages, generator=g) if pool_pages is None else torch.arange(n_pages - 1, -1, -1)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        self.k = torch.full((n_pages, hkv, page, d), poison, dtype=dt, device="cuda")
        self.v = torch.full((n_pages, hkv, page, d), poison, dtype=dt, device="cuda")
        at = 0
        for b, n in enumerate(lens):
            for c in range(counts[b]):
                p = int(perm[at])
                at += 1
                self.table[b, c] = p
                rows = min(page, n - c * page)
                for x, s in ((self.k, amp), (self.v, 1.0)):
                    x[p, :, :rows] = (s * torch.randn(hkv, rows, d, generator=g)).to(dt).cuda()
        self.table = self.table.cuda()
        self.dlens = ints(self.lens)
        self.cfg = zha.paged_config(len(lens), hq, hkv, d, page, n_pages, width, dtype=NAME[dt], window=window,
                                    scale=scale)
        self.scale = scale if scale > 0 else d ** -0.5
        self.g = g

    def queries(self, n):
        return torch.randn(n, self.G * self.hkv, self.d, generator=self.g).to(self.dt).cuda()

    def run(self, q, ws=None, status_is=0, **kw):
        out, lse = torch.full_like(q, 77.0), torch.full(q.shape[:2], 77.0, device="cuda")
        status = ints([0])
        ws = self.zha.paged_workspace(self.cfg, max(q.shape[0], 1)) if ws is None else ws
        self.zha.paged_decode(self.cfg, q, self.k, self.v, self.table, self.dlens, out, ws, lse=lse,
                              dev_status=status, **kw)
        torch.cuda.synchronize()
        assert int(status) == status_is
        return out, lse

    def check(self, q, out, lse, rows):
        """rows: (row, sequence, tokens seen). Error bound, with u = 2^-24 (fp32): a score is a sum of d products,
        off by at most d 2u sum|q k| s, and scaled to base 2 (3u |x|); a weight's exponent carries the errors of its own score
        and of the sums' (twice that), 2 ulp of exp2 and the weights' own split into two bf16 (2^-16); a sum of n
        weights or weighted values adds one rounding of at most 2u a tile of 16 or a rescaling: n/8 + 64 units."""
        u = 2.0 ** -24
        for r, b, n in rows:
            lo = max(0, n - self.window) if self.window else 0
            for h in range(self.hkv):
                K = P.gather(self.k, self.table[b], lo, n, h, self.page)
                V = P.gather(self.v, self.table[b], lo, n, h, self.page)
                qs = P.np64(q[r, h * self.G:(h + 1) * self.G])
                want, wl, size = P.attend(qs, K, V, self.scale)
                got, gl = P.np64(out[r, h * self.G:(h + 1) * self.G]), P.np64(lse[r, h * self.G:(h + 1) * self.G])
                if n == lo:
                    assert np.all(got == 0) and np.all(np.isneginf(gl))
                    continue
                x = self.scale * float(np.max(np.abs(qs) @ np.abs(K).T))
                dx = (2 * self.d + 6) * u * x
                rel = 2 * dx + 2.0 ** -16 * (self.dt is BF16) + ((n - lo) / 8 + 64) * u
                tol = P.HALF_STEP[self.dt] * np.abs(want) + rel * size
                assert np.all(np.abs(got - want) <= tol), (r, b, n, h, float(np.max(np.abs(got - want) - tol)))
                assert np.all(np.abs(gl - wl) <= dx + ((n - lo) / 8 + 64) * u + 4 * u * np.abs(wl)), (r, b, n, h)


EDGES = [1, 0, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 1), (8, 4), (15, 3), (36, 4)])
@pytest.mark.parametrize("page", [1, 16, 128])
def test_decode_edge_lengths(zha, dt, d, hq, hkv, page):
    c = Case(zha, EDGES, hq, hkv, d, page, dt, seed=page + hq)
    q = c.queries(len(EDGES))
    c.check(q, *c.run(q), [(b, b, n) for b, n in enumerate(EDGES)])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page", [2, 4, 8, 32, 64, 256, 1024])
def test_decode_page_sizes(zha, dt, page):
    """Every way of copying pages: row by row, whole small pages, parts of large ones; with a window that begins
    inside them, and garbage in the rows around it."""
    lens = [1, 7, 9, 100, 1023, 1025, 2500]
    for window in (0, 77):
        c = Case(zha, lens, 12, 4, 128, page, dt, window=window, seed=page)
        q = c.queries(len(lens))
        c.check(q, *c.run(q), [(b, b, n) for b, n in enumerate(lens)])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens", [[5000], [20011, 3], [777] * 40, [1] * 300, [4097, 0, 0, 9000, 1, 64]],
                         ids=["one", "long+short", "even", "ones", "ragged"])
def test_decode_splits_and_joins(zha, dt, lens):
    """Rows split over many CTAs, CTAs that hold parts of several rows, and rows that are one CTA's."""
    c = Case(zha, lens, 16, 2, 128 if dt is BF16 else 64, 16, dt, seed=len(lens), amp=1.5)
    q = c.queries(len(lens))
    ws = zha.paged_workspace(c.cfg, len(lens))
    out, lse = c.run(q, ws)
    some = range(len(lens)) if len(lens) < 20 else range(0, len(lens), 13)
    c.check(q, out, lse, [(b, b, lens[b]) for b in some])
    again = c.run(q, ws)                                              # the same workspace, the same bits
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 7, 64, 100, 4096])
def test_decode_window(zha, dt, window):
    lens = [1, 6, 7, 8, 63, 64, 65, 100, 101, 1000, 5003]
    c = Case(zha, lens, 8, 2, 64, 16, dt, window=window, seed=window)
    # pages that lie before every window may have been given away
    for b, n in enumerate(lens):
        c.table[b, :max(0, n - window) // 16] = -1 if n > window else c.table[b, 0]
    q = c.queries(len(lens))
    c.check(q, *c.run(q), [(b, b, n) for b, n in enumerate(lens)])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_decode_mapped_rows(zha, dt):
    """Rows in any order, several of one sequence, padding between and behind: padding is left as it is."""
    lens = [300, 1, 77, 2000]
    c = Case(zha, lens, 8, 2, 128, 32, dt, seed=4)
    seq = [3, -1, 0, 3, 3, 1, -2 ** 31, 2, 0, -1, -1]
    pos = [1999, 5, 0, 0, 1024, 0, 0, 76, 255, -9, 2 ** 31 - 1]
    q = c.queries(len(seq))
    out, lse = c.run(q, seq_ids=ints(seq), positions=ints(pos))
    c.check(q, out, lse, [(r, b, p + 1) for r, (b, p) in enumerate(zip(seq, pos)) if b >= 0])
    for r, b in enumerate(seq):
        if b < 0:
            assert torch.all(out[r] == 77) and torch.all(lse[r] == 77)
    out, lse = c.run(q, seq_ids=ints(seq))                            # without positions: whole sequences
    c.check(q, out, lse, [(r, b, lens[b]) for r, b in enumerate(seq) if b >= 0])
    q = c.queries(4)
    out, lse = c.run(q, positions=ints([17, 0, 76, 1234]))            # without sequences: row r is sequence r
    c.check(q, out, lse, [(0, 0, 18), (1, 1, 1), (2, 2, 77), (3, 3, 1235)])


def test_decode_bad_indices_set_status(zha):
    lens = [40, 50, 60]
    c = Case(zha, lens, 4, 2, 64, 16, BF16, seed=5)
    q = c.queries(3)
    good = c.run(q)
    for table_entry in (-1, c.cfg.n_pages, 2 ** 31 - 1, -2 ** 31):    # a page outside the pool: its tokens are skipped
        keep = c.table[1, 1].clone()
        c.table[1, 1] = table_entry
        out, lse = c.run(q, status_is=1)
        c.table[1, 1] = keep
        assert torch.equal(out[0], good[0][0]) and torch.equal(out[2], good[0][2])
        k2, keep_lens = c.table[1].clone(), list(c.lens)
        # the same row over its other pages alone
        c.table[1, 1], c.table[1, 2] = k2[2], k2[3]
        c.dlens[1] = 34
        want = c.run(q)
        c.table[1], c.dlens[1] = k2, keep_lens[1]
        assert torch.allclose(out[1].float(), want[0][1].float(), rtol=2.0 ** -7, atol=2.0 ** -7)
        assert torch.allclose(lse[1], want[1][1], rtol=1e-5, atol=1e-5)
    for bad in (-1, c.cfg.max_pages * 16 + 1, 2 ** 31 - 1):           # a length beyond the table: zeros
        c.dlens[2] = bad
        out, lse = c.run(q, status_is=3)
        assert torch.equal(out[:2], good[0][:2]) and torch.all(out[2] == 0) and torch.all(torch.isneginf(lse[2]))
    c.dlens[2] = 60
    out, lse = c.run(q, status_is=1, positions=ints([-1, 50, 59]))    # positions outside their sequences: zeros
    assert torch.all(out[:2] == 0) and torch.all(torch.isneginf(lse[:2])) and torch.equal(out[2], good[0][2])
    out, lse = c.run(q, status_is=1, seq_ids=ints([0, 3, 2]))         # a sequence beyond the batch: left alone
    assert torch.equal(out[0], good[0][0]) and torch.all(out[1] == 77) and torch.equal(out[2], good[0][2])
    # an empty call, and no optional arrays at all
    c.run(q[:0])
    out = torch.empty_like(q)
    zha.paged_decode(c.cfg, q, c.k, c.v, c.table, c.dlens, out, zha.paged_workspace(c.cfg, 3))
    assert torch.equal(out, good[0])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_decode_special_values(zha, dt):
    """NaN and infinity in attended rows reach the rows that attend them and no others; a key at minus infinity's
    score takes no weight; huge scores do not overflow."""
    lens = [200, 200, 200, 200, 200]
    c = Case(zha, lens, 2, 1, 64, 16, dt, seed=6)
    q = c.queries(5).abs() + 0.1
    good = c.run(q)
    c.k[c.table[0, 3], 0, 5, 7] = float("nan")
    c.v[c.table[1, 3], 0, 5, 7] = float("nan")
    c.k[c.table[2, 3], 0, 5] = -float("inf")                          # score -inf: weight 0
    c.k[c.table[3, 3], 0, 5] = 3e4                                    # a score of ~1e5: takes all the weight
    out, lse = c.run(q)
    assert torch.all(torch.isnan(out[0])) and torch.all(torch.isnan(lse[0]))
    assert torch.all(torch.isnan(out[1, :, 7])) and not torch.any(torch.isnan(out[1, :, :7]))
    assert torch.equal(lse[1], good[1][1])
    assert torch.all(torch.isfinite(out[2])) and torch.all(torch.isfinite(lse[2]))
    want = c.v[c.table[3, 3], 0, 5]
    # bf16: exactly. fp32 values are taken as two tf32 parts of 11 bits: the first leaves at most 2^-11 |v|, the second
    # at most 2^-11 of that; their sum is rounded once more (2^-24): below 2^-21 |v|
    assert torch.all((out[3] - want).abs() <= (0.0 if dt is BF16 else 2.0 ** -21) * want.abs())
    assert torch.equal(out[4], good[0][4])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_keeps_other_results_when_some_are_not_finite(zha, dt, d):
    """An infinite value makes its own coordinate infinite, a head whose query is NaN only itself NaN, and garbage of
    every kind behind the sequence's end does nothing: all other results keep their bits."""
    lens = [150, 151, 40]
    for poison in (0.0, float("nan"), float("inf"), -3e38):
        c = Case(zha, lens, 8, 1, d, 16, dt, seed=16, poison=poison)
        q = c.queries(3)
        out, lse = c.run(q)
        c.check(q, out, lse, [(b, b, n) for b, n in enumerate(lens)])
        if poison == 0.0:
            good = out, lse
        assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
    c.v[c.table[0, 2], 0, 3, 5] = float("inf")
    c.v[c.table[0, 2], 0, 4, 6] = -float("inf")
    q[1, 3] = float("nan")
    out, lse = c.run(q)
    assert torch.all(out[0, :, 5] == float("inf")) and torch.all(out[0, :, 6] == -float("inf"))
    assert torch.all(torch.isnan(out[1, 3])) and torch.isnan(lse[1, 3])
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[0, :, 5:7] = rest[1, 3] = False
    assert torch.equal(out[rest], good[0][rest])
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(lse[keep], good[1][keep])


def test_decode_scale_and_peaked_scores(zha):
    lens = [1500, 90]
    for scale, amp in ((0.5, 4.0), (1.0, 0.01), (1e-3, 1.0)):
        c = Case(zha, lens, 8, 1, 128, 64, BF16, scale=scale, amp=amp, seed=7)
        q = c.queries(2)
        c.check(q, *c.run(q), [(0, 0, 1500), (1, 1, 90)])


def test_decode_far_offsets(zha):
    """Pages beyond 2^31 elements of the pool."""
    hkv, d, page = 8, 128, 64
    n_pages = (2 ** 31) // (hkv * page * d) + 40
    c = Case(zha, [700, 1500], 16, hkv, d, page, BF16, seed=8, poison=0.0, pool_pages=n_pages)
    assert int(c.table[0, 0]) * hkv * page * d > 2 ** 31
    q = c.queries(2)
    c.check(q, *c.run(q), [(0, 0, 700), (1, 1, 1500)])
    slots = ints([int(c.table[1, 3]) * page + 9])
    x = torch.randn(1, hkv, d, generator=c.g).to(BF16).cuda()
    zha.paged_write(c.cfg, None, None, x, x, None, slots, None, c.k, c.v)
    assert torch.equal(c.k[c.table[1, 3], :, 9], x[0]) and torch.equal(c.v[c.table[1, 3], :, 9], x[0])


def test_decode_on_other_streams(zha):
    """Two calls at once, each on a stream and a workspace of its own."""
    c = Case(zha, [3000, 10, 900, 64], 16, 2, 128, 16, BF16, seed=10)
    q1, q2 = c.queries(4), c.queries(4)
    want = [c.run(x) for x in (q1, q2)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws = [zha.paged_workspace(c.cfg, 4) for _ in range(2)]
    outs = [torch.empty_like(q1) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, o, w in ((s1, q1, outs[0], ws[0]), (s2, q2, outs[1], ws[1])):
            zha.paged_decode(c.cfg, q, c.k, c.v, c.table, c.dlens, o, w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0][0]) and torch.equal(outs[1], want[1][0])


def test_decode_many_rows_and_one_workspace(zha):
    """More rows than a warp or a CTA has threads, empty and left-out ones among them; one workspace for calls of
    different row counts, one after the other."""
    rng = random.Random(17)
    lens = [rng.choice([0, 1, 40, 200, 700]) for _ in range(50)]
    c = Case(zha, lens, 8, 4, 64, 16, BF16, seed=18)
    n = 700
    seq = [rng.randint(-1, 49) for _ in range(n)]
    ws = zha.paged_workspace(c.cfg, n)
    q = c.queries(n)
    out, lse = c.run(q, ws, seq_ids=ints(seq))
    c.check(q, out, lse, [(r, seq[r], lens[seq[r]]) for r in range(0, n, 7) if seq[r] >= 0])
    for r in range(n):
        if seq[r] < 0:
            assert torch.all(out[r] == 77)
    few = c.run(q[:20].contiguous(), ws, seq_ids=ints(seq[:20]))
    c.check(q, few[0], few[1], [(r, seq[r], lens[seq[r]]) for r in range(20) if seq[r] >= 0])
    again = c.run(q, ws, seq_ids=ints(seq))
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_decode_configurations_share_a_workspace(zha):
    """Calls of different types, heads and head sizes, all with split rows, one after the other on one workspace."""
    lens = [20000, 5, 7001]
    cases = [Case(zha, lens, hq, hkv, d, 16, dt, seed=30 + i)
             for i, (hq, hkv, d, dt) in enumerate([(16, 1, 128, BF16), (2, 2, 64, BF16), (3, 1, 64, F32), (8, 1, 128, F32)])]
    ws = max((zha.paged_workspace(c.cfg, 3) for c in cases), key=lambda t: t.numel())
    for c in cases + cases:
        q = c.queries(3)
        c.check(q, *c.run(q, ws), [(0, 0, lens[0]), (1, 1, lens[1]), (2, 2, lens[2])])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_empty_calls_and_queries_in_place(zha, dt):
    cfg = zha.paged_config(2, 4, 2, 64, 16, 6, 3, dtype=NAME[dt])
    kp, vp = (torch.zeros(6, 2, 16, 64, dtype=dt, device="cuda") for _ in range(2))
    rot = zha.Rotary(64)
    none = ints([])
    q0, k0 = torch.zeros(0, 4, 64, dtype=dt, device="cuda"), torch.zeros(0, 2, 64, dtype=dt, device="cuda")
    zha.rotary(rot, q0, k0, none)
    zha.paged_write(cfg, rot, q0, k0, k0, none, none, q0, kp, vp)
    zha.paged_decode(cfg, q0, kp, vp, ints([0] * 6), ints([0, 0]), q0, zha.paged_workspace(cfg, 1))
    g = torch.Generator().manual_seed(20)
    q, k = (torch.randn(9, h, 64, generator=g).to(dt).cuda() for h in (4, 2))
    pos, slots = ints(list(range(50, 59))), ints([3, -1, 5, 90, 7, 8, 9, -1, 11])
    want = torch.empty_like(q)
    zha.rotary(rot, q, None, pos, want)
    want[1], want[7] = q[1], q[7]                                     # skipped rows stay
    zha.paged_write(cfg, rot, q, k, k, pos, slots, q, kp, vp)         # q_out is q
    assert torch.equal(q, want)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- steps

@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_the_whole_cache(zha, dt, captured):
    """Prompts, decodes, sequences that end and start again, a padded token buffer: plan, write and decode together,
    called step by step and replayed from one captured graph."""
    rng = random.Random(11)
    B, hq, hkv, d, page, rows = 5, 8, 2, 64, 8, 40
    cfg = zha.paged_config(B, hq, hkv, d, page, 40, 10, dtype=NAME[dt])
    cache = zha.PagedCache(cfg, rows, zha.Rotary(d))
    g = torch.Generator().manual_seed(12)
    bn = torch.zeros(B, dtype=torch.int32, device="cuda")
    bq, bk, bv = (torch.zeros(rows, h, d, dtype=dt, device="cuda") for h in (hq, hkv, hkv))
    graph = None
    if captured:
        cache.step(bn, bq, bk, bv)                                    # nothing new: changes nothing
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            cache.step(bn, bq, bk, bv)
    hist = [([], []) for _ in range(B)]                               # rotated keys and values of each sequence
    for step in range(9):
        lens = [len(h[0]) for h in hist]
        new = [rng.randint(1, 15) if n == 0 else rng.choice([1, 1, 1, 0, -1, 5]) for n in lens]
        while sum(max(a, 0) for a in new) > rows:
            new[new.index(max(new))] = 1
        q, k, v = (torch.randn(rows, h, d, generator=g).to(dt).cuda() for h in (hq, hkv, hkv))
        cache.out.fill_(77)
        bn.copy_(ints(new))
        bq.copy_(q), bk.copy_(k), bv.copy_(v)
        if graph is not None:
            graph.replay()
        else:
            cache.step(bn, bq, bk, bv)
        torch.cuda.synchronize()
        cache.check_status()
        i = 0
        for b in range(B):
            if new[b] < 0:
                hist[b] = ([], [])
            for _ in range(max(new[b], 0)):
                p = len(hist[b][0])
                kr = torch.empty_like(k[i:i + 1])
                qr = torch.empty_like(q[i:i + 1])
                zha.rotary(cache.rot, q[i:i + 1], k[i:i + 1], ints([p]), qr, kr)
                hist[b][0].append(P.np64(kr[0]))
                hist[b][1].append(P.np64(v[i]))
                K, V, qs = np.stack(hist[b][0]), np.stack(hist[b][1]), P.np64(qr[0])
                for h in range(hkv):
                    rs = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                    want, wl, size = P.attend(qs[rs], K[:, h], V[:, h], d ** -0.5)
                    # as in Case.check, with scores below 64 and at most 100 tokens
                    rel = 2.0 ** -16 * (dt is BF16) + (4 * d * 64 + 128) * 2.0 ** -24
                    err = np.abs(P.np64(cache.out[i, rs]) - want)
                    assert np.all(err <= P.HALF_STEP[dt] * np.abs(want) + rel * size), (step, b, i)
                i += 1
        assert torch.all(cache.out[i:] == 77)                         # padding rows are left as they were
        assert cache.lens.tolist() == [len(h[0]) for h in hist]


def test_tables_of_another_width_are_refused(zha):
    """Wider or narrower rows than the configuration's max_pages; flat and longer tables pass."""
    c = Case(zha, [20, 40], 4, 2, 64, 16, BF16, seed=40)
    q, width = c.queries(2), c.table.shape[1]
    assert width == 4
    want, kept = c.run(q), c.table
    m = {x: ints([0, 0]) for x in ("positions", "slots", "seq_ids")}
    m["cu"] = ints([0, 0, 0])
    for bad in (torch.full((2, 5), -1, dtype=torch.int32, device="cuda"), kept.view(4, 2)):
        c.table = bad
        with pytest.raises(ValueError, match="table"):
            c.run(q)
        with pytest.raises(ValueError, match="table"):
            zha.paged_plan(c.cfg, bad, c.dlens, ints([0, 0]), ints([0] * c.k.shape[0]), ints([0]), m)
    for good in (kept.flatten(), torch.cat([kept, kept])):
        c.table = good
        assert torch.equal(c.run(q)[0], want[0])
