"""Calls of the paged cache that are refused or fail, on the GPU: what they leave behind."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def zha():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_indexed_sparse_02_b200 import zha as z
    return z


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled_cache(zha, rows=24, prompts=(9, 4, 8)):
    """A cache of three sequences after a step of their prompts, and the next step's arguments."""
    width = (max(prompts) + 64) // 16
    cfg = zha.paged_config(3, 8, 2, 64, 16, 3 * width, width)
    cache = zha.PagedCache(cfg, rows, zha.Rotary(64))
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(rows, h, 64, generator=g).to(BF16).cuda() for h in (8, 2, 2))
    cache.step(ints(prompts), q, k, v)
    torch.cuda.synchronize()
    cache.check_status()
    return cache, (ints([1, 1, 1]), q, k, v)


def state(cache):
    return {x: getattr(cache, x).clone() for x in ("table", "lens", "free_pages", "n_free", "k_pool", "v_pool", "out", "lse")}


def test_a_refused_step_changes_nothing(zha):
    cache, (n_new, q, k, v) = filled_cache(zha)
    before = state(cache)
    odd = torch.zeros(24 * 8 * 64 + 1, dtype=BF16, device="cuda")[1:].view(24, 8, 64)      # on no 16-byte boundary
    far = zha.Rotary(64, device="cpu")
    for args in ((q[:3], k[:3], v[:3]), (q, k, v[:20]), (q.float(), k, v), (q, k, v.transpose(0, 1)), (q, k[:, :1], v),
                 (q.cpu(), k, v), (odd, k, v)):
        with pytest.raises((ValueError, zha.ZhaError)):
            cache.step(n_new, *args)
    kept = cache.rot
    for rot in (far, zha.Rotary(128)):                       # on another device; more coordinates than the head has
        cache.rot = rot
        with pytest.raises((ValueError, zha.ZhaError)):
            cache.step(n_new, q, k, v)
    cache.rot = kept
    torch.cuda.synchronize()
    after = state(cache)
    for x in before:
        assert torch.equal(before[x], after[x]), x
    cache.step(n_new, q, k, v)                               # and the step itself still counts its tokens once
    torch.cuda.synchronize()
    cache.check_status()
    assert cache.lens.tolist() == [10, 5, 9]


def test_a_step_without_queries_is_refused(zha):
    """write() may put keys and values alone; a step would attend with the queries of the step before."""
    cache, (n_new, q, k, v) = filled_cache(zha)
    before = state(cache)
    with pytest.raises(ValueError):
        cache.step(n_new, None, k, v)
    torch.cuda.synchronize()
    after = state(cache)
    for x in before:
        assert torch.equal(before[x], after[x]), x
    cache.plan(n_new)
    cache.write(None, k, v)
    torch.cuda.synchronize()
    cache.check_status()
    page = int(cache.table[0, 0])
    want = torch.empty_like(k[:1])
    zha.rotary(cache.rot, None, k[:1], ints([9]), None, want)
    assert torch.equal(cache.k_pool[page, :, 9], want[0]) and torch.equal(cache.v_pool[page, :, 9], v[0])


def test_steps_after_a_wait_ran_out(zha):
    """What a call leaves that gave up, written from the host: the step after check_status is right again, on another
    stream too, and as a replay of a graph captured before."""
    for stream, captured in ((None, False), (torch.cuda.Stream(), False), (None, True)):
        prompts = (4000, 300, 8)                             # rows long enough to be split over several CTAs
        cache, (n_new, q, k, v) = filled_cache(zha, 4320, prompts)
        same, _ = filled_cache(zha, 4320, prompts)
        assert torch.equal(cache.out, same.out)
        if captured:
            none = torch.zeros_like(n_new)
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                cache.step(none, q, k, v)
            none.copy_(n_new)
        cache.workspace.view(torch.int32)[:1776] = 2         # every counter
        cache.status.fill_(5)
        with pytest.raises(zha.ZhaError) as e:
            cache.check_status()
        assert e.value.code == 5
        if captured:
            graph.replay()
        else:
            cache.step(n_new, q, k, v, stream)
        want, lse = same.step(n_new, q, k, v)
        torch.cuda.synchronize()
        cache.check_status()
        assert torch.equal(cache.out[:3], want[:3]) and torch.equal(cache.lse[:3], lse[:3])
        assert cache.lens.tolist() == [4001, 301, 9]


def test_arguments_that_raise_enqueue_nothing(zha):
    """A transpose flag without a truth value, a stream whose handle is no number: the error, and nothing written."""
    class Stream:
        cuda_stream = "17"

    x = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(2)).cuda()
    pos, kept = ints([1, 2, 3, 4, 5]), x.clone()
    rot = zha.Rotary(64)
    before = zha.launch_count()
    for kw in (dict(transpose=torch.ones(2)), dict(stream=Stream())):
        with pytest.raises((RuntimeError, TypeError)):
            zha.rotary(rot, x, None, pos, **kw)
    cfg = zha.paged_config(1, 2, 2, 64, 16, 1, 1, dtype="f32")
    pool = torch.zeros(1, 2, 16, 64, device="cuda")
    with pytest.raises(TypeError):
        zha.paged_write(cfg, None, None, x, x, None, pos, None, pool, pool.clone(), stream=Stream())
    with pytest.raises(TypeError):
        zha.paged_decode(cfg, x[:1], pool, pool, ints([0]), ints([3]), x[1:2], zha.paged_workspace(cfg, 1), stream=Stream())
    torch.cuda.synchronize()
    assert torch.equal(x, kept) and not pool.any() and zha.launch_count() == before


def test_arrays_of_another_layout_are_refused(zha):
    """Pools, outputs and lse of the right number of elements in another order (tokens before heads, pages of another
    size, heads before rows) were read and written askew; shapes that only merge neighbours mean the same array."""
    n, hq, hkv, d, page, pages = 3, 8, 4, 64, 16, 6
    cfg = zha.paged_config(n, hq, hkv, d, page, pages, 2)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(pages, hkv, page, d, generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn(n, hq, d, generator=g).to(BF16).cuda()
    kv = torch.randn(n, hkv, d, generator=g).to(BF16).cuda()
    table, lens, slots = ints([[0, 1], [2, 3], [4, 5]]), ints([20, 7, 32]), ints([3, 50, 90])
    ws = zha.paged_workspace(cfg, n)

    def decode(k=k, v=v, out=None, lse=None):
        out = torch.zeros(n, hq, d, dtype=BF16, device="cuda") if out is None else out
        zha.paged_decode(cfg, q, k, v, table, lens, out, ws, lse=lse)
        return out

    def write(k=k, v=v, q_out=None):
        zha.paged_write(cfg, None, q, kv, kv, None, slots, torch.empty_like(q) if q_out is None else q_out, k, v)

    before = k.clone(), v.clone()
    for shape in ((pages, page, hkv, d), (pages * page, hkv, d), (2 * pages, hkv, page // 2, d), (pages // 2, hkv, 2 * page, d),
                  (hkv, pages, page, d), (pages, hkv, d, page), (pages, hkv, page // 3 + 1, d)):
        other = torch.zeros(shape, dtype=BF16, device="cuda")
        for kw in (dict(k=other), dict(v=other)):
            with pytest.raises(ValueError, match="pool"):
                decode(**kw)
            with pytest.raises(ValueError, match="pool"):
                write(**kw)
    with pytest.raises(ValueError, match="out"):
        decode(out=torch.zeros(hq, n, d, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError, match="lse"):
        decode(lse=torch.zeros(hq, n, device="cuda"))
    with pytest.raises(ValueError, match="q_out"):
        write(q_out=torch.zeros(hq, n, d, dtype=BF16, device="cuda"))
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    want = decode()
    for shape in ((pages, hkv, page * d), (pages * hkv, page, d), (pages * hkv * page * d,), (1, pages, 1, hkv, page, 1, d)):
        assert torch.equal(decode(k.view(shape), v.view(shape)), want)
    assert torch.equal(decode(out=torch.zeros(n, hq * d, dtype=BF16, device="cuda")).view(n, hq, d), want)
    flat = torch.zeros(n * hq, device="cuda")
    assert torch.equal(decode(lse=flat), want) and flat.all()
    write(k.view(-1), v.view(pages, hkv, -1), q_out=torch.empty(n, hq * d, dtype=BF16, device="cuda"))
    assert torch.equal(k[0, :, 3], kv[0]) and torch.equal(v[3, :, 2], kv[1])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 1), (16, 1), (6, 2)])
def test_a_token_with_all_the_weight_comes_out_exactly(zha, dt, d, hq, hkv):
    """Its weight is 2^0 = 1; every other score is more than 150 / ln 2 below, so that its weight is 0 in fp32. The sum
    of the weights is 1 and the output is the token's value row, bit for bit, in rows of one CTA and in split ones."""
    lens, at = [200, 9000, 1, 9000], [85, 8999, 0, 3]
    pages = sum(-(-n // 16) for n in lens)
    width = -(-max(lens) // 16)
    cfg = zha.paged_config(4, hq, hkv, d, 16, pages, width, dtype="bf16" if dt is BF16 else "f32")
    g = torch.Generator().manual_seed(d + hq)
    k, v = (torch.randn(pages, hkv, 16, d, generator=g).to(dt).cuda() for _ in range(2))
    table, first = torch.full((4, width), -1, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        count = -(-n // 16)
        table[b, :count] = torch.arange(first, first + count)
        first += count
    table = table.cuda()
    q = (torch.rand(4, hq, d, generator=g) + 0.1).to(dt).cuda()
    want = torch.empty_like(q)
    for b, t in enumerate(at):
        k[table[b, t // 16], :, t % 16] = 3e4                # a score of 3e4 sum(q) / sqrt(d) > 20,000; the others' are below 200
        want[b] = v[table[b, t // 16], :, t % 16].repeat_interleave(hq // hkv, dim=0)
    out, status = torch.zeros_like(q), ints([0])
    zha.paged_decode(cfg, q, k, v, table, ints(lens), out, zha.paged_workspace(cfg, 4), dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.equal(out, want)


def test_a_table_of_the_users_own(zha):
    """Frequencies and factor put into a Rotary in place are what the next calls use. fp32, in units of 2^-24 of the
    pair's size: sine, cosine, the factor and its product 8, two products and a sum 3; the angle 2^-51 of itself."""
    import numpy as np

    import paged_testlib as P
    rot = zha.Rotary(64)
    theta = np.linspace(0.9, 0.001, 32) ** 2
    rot.freq.copy_(torch.from_numpy(theta / (2 * np.pi)))
    rot.desc.mscale = 1.25
    g = torch.Generator().manual_seed(5)
    x = torch.randn(7, 3, 64, generator=g).cuda()
    pos = torch.randint(0, 9000, (7,), generator=g, dtype=torch.int32)
    y = torch.empty_like(x)
    zha.rotary(rot, x, None, pos.cuda(), y)
    xs = P.np64(x)
    want = P.rotate(xs, pos.numpy(), 64, "half", theta, 1.25)
    far = np.tile(pos.numpy()[:, None] * theta[None, :] * 2.0 ** -51, 2)[:, None, :]
    tol = 2.0 ** -24 * np.abs(want) + 1.25 * P.pair_size(xs, 64, "half") * (11 * 2.0 ** -24 + far)
    assert np.all(np.abs(P.np64(y) - want) <= tol)
