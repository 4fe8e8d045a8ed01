"""Rotary positions on the GPU against their formula in extended precision."""
import numpy as np
import pytest
import torch

import paged_testlib as P

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def zha():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_indexed_sparse_02_b200 import zha as z
    return z


def _check(got, x, pos, rd, layout, theta, m, transpose):
    """Per coordinate: one rounding to the type, and in fp32 (in units of 2^-24 of the pair's size) sine and cosine
    (their reduced angle, 2 ulp, the factor m and its own rounding: 8), two products and a sum (3). The angle itself is an fp64 product of
    three roundings: position * theta * 2^-51 radians."""
    xs = P.np64(x)
    want = P.rotate(xs, pos, rd, layout, theta, m, transpose)
    far = np.abs(np.asarray(pos, dtype=np.float64))[:, None] * theta.astype(np.float64)[None, :] * 2.0 ** -51
    ang = np.zeros((len(pos), xs.shape[-1]))
    if layout == "half":
        ang[:, :rd // 2] = ang[:, rd // 2:rd] = far
    else:
        ang[:, 0:rd:2] = ang[:, 1:rd:2] = far
    tol = P.HALF_STEP[x.dtype] * np.abs(want) + m * P.pair_size(xs, rd, layout) * (11 * 2.0 ** -24 + ang[:, None, :])
    err = np.abs(P.np64(got) - want)
    assert np.all(err <= tol), float(np.max(err - tol))
    assert np.array_equal(P.np64(got)[..., rd:], xs[..., rd:])       # the rest of the head passes through


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rd", [(64, 64), (128, 128), (128, 64), (64, 2), (128, 34), (64, 24), (128, 126)])
def test_rotary_matches_formula(zha, dt, layout, d, rd):
    g = torch.Generator().manual_seed(rd + d)
    rot = zha.Rotary(rd, layout=layout)
    theta, m = P.frequencies(rd)
    for n, hq, hk in ((1, 4, 1), (3, 7, 2), (130, 5, 5)):
        q, k = (torch.randn(n, h, d, generator=g).to(dt).cuda() for h in (hq, hk))
        pos = torch.randint(0, 40000, (n,), generator=g, dtype=torch.int32)
        for transpose in (False, True):
            qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
            zha.rotary(rot, q, k, pos.cuda(), qo, ko, transpose=transpose)
            _check(qo, q, pos.numpy(), rd, layout, theta, m, transpose)
            _check(ko, k, pos.numpy(), rd, layout, theta, m, transpose)
        a, b = q.clone(), k.clone()
        zha.rotary(rot, a, b, pos.cuda())                            # in place
        zha.rotary(rot, q, None, pos.cuda(), qo)                     # queries alone, keys alone
        zha.rotary(rot, None, k, pos.cuda(), None, ko)
        assert torch.equal(a, qo) and torch.equal(b, ko)


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("ntk", 4.0), ("yarn", 8.0)])
def test_scaled_and_far_positions(zha, scaling, factor):
    pos = torch.tensor([0, 1, 32767, 1 << 20, (1 << 30) - 1, 2 ** 31 - 1, -1, -12345], dtype=torch.int32)
    rot = zha.Rotary(128, base=500000.0, scaling=scaling, factor=factor, original_len=32768)
    theta, m = P.frequencies(128, 500000.0, scaling, factor, 32768)
    x = torch.randn(len(pos), 3, 128, generator=torch.Generator().manual_seed(1)).cuda()
    y = torch.empty_like(x)
    zha.rotary(rot, x, None, pos.cuda(), y)
    _check(y, x, pos.numpy(), 128, "half", theta, m, False)


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rd", [64, 20])
def test_strided_tokens_and_many_heads(zha, dt, rd):
    """q and k as slices of a packed projection, written back in place and to strided outputs; the rest of the
    projection is left alone. More heads than one CTA's share of a token."""
    n, hq, hk, d = 37, 128, 8, 64
    qkv = torch.randn(n, (hq + 2 * hk) * d, generator=torch.Generator().manual_seed(2)).to(dt).cuda()
    before = qkv.clone()
    q, k, v = (t.unflatten(1, (-1, d)) for t in torch.split(qkv, [hq * d, hk * d, hk * d], dim=1))
    pos = torch.arange(100, 100 + n, dtype=torch.int32)
    rot = zha.Rotary(rd)
    theta, m = P.frequencies(rd)
    qo, ko = torch.empty(n, hq, d, dtype=dt, device="cuda"), torch.empty(n, 2 * hk, d, dtype=dt, device="cuda")[:, :hk]
    zha.rotary(rot, q, k, pos.cuda(), qo, ko)
    assert torch.equal(qkv, before)
    _check(qo, q, pos.numpy(), rd, "half", theta, m, False)
    _check(ko, k, pos.numpy(), rd, "half", theta, m, False)
    zha.rotary(rot, q, k, pos.cuda())
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


def test_transpose_is_the_gradient(zha):
    """<R x, w> differentiated along random directions equals <x', R^T w> (the map is linear, so the difference
    quotient is exact but for fp32 roundings of its terms)."""
    g = torch.Generator().manual_seed(3)
    rot = zha.Rotary(32, layout="interleaved", scaling="yarn", factor=4.0)
    x, w, dx = (torch.randn(50, 4, 64, generator=g).cuda() for _ in range(3))
    pos = torch.randint(0, 9000, (50,), generator=g, dtype=torch.int32).cuda()

    def f(t):
        y = torch.empty_like(t)
        zha.rotary(rot, t, None, pos, y)
        return float((y.double() * w.double()).sum())

    grad = torch.empty_like(w)
    zha.rotary(rot, w, None, pos, grad, transpose=True)
    want = float((grad.double() * dx.double()).sum())
    got = (f(x + dx) - f(x - dx)) / 2
    # every term carries a few fp32 roundings (16 units of 2^-24, as in _check, of twice the pair's size)
    size = float((w.abs().double() * (x.abs() + dx.abs()).double()).sum()) * 4
    assert abs(got - want) <= 16 * 2.0 ** -24 * size


def test_decode_graph_rotates_while_staging(zha):
    """DecodeGraph with a Rotary equals the same steps on queries and keys rotated beforehand."""
    import zha_testlib as T
    from tree_indexed_sparse_02_b200.inputs import decode_stream, make_inputs
    w = T.small_workloads()[1]
    steps = 5
    cap = w.context + steps + 8
    k_new, v_new, qs = (t.cuda() for t in decode_stream(w, steps))
    rot = zha.Rotary(w.head_dim)
    outs = []
    for inside in (True, False):
        inp = T.to_device(make_inputs(w, capacity=cap))
        cfg = T.make_cfg(zha, w, cap)
        buf = zha.Buffers(cfg)
        zha.tree_build(cfg, buf.tree, inp.K, inp.refs, inp.lens, buf.status)
        graph = zha.DecodeGraph(cfg, buf, inp.K, inp.V, inp.refs, inp.lens, w.p, rot=rot if inside else None)
        got = []
        for i in range(steps):
            q, k = qs[i].clone(), k_new[i].clone()
            if not inside:
                zha.rotary(rot, q, k, inp.lens)
            got.append(graph.step(q, k, v_new[i]).clone())
        torch.cuda.synchronize()
        buf.check_status()
        outs.append((torch.stack(got), inp.K.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_copies_of_handles_stand_alone(zha):
    """A deep copy of a Rotary or of a configuration works after the original is gone."""
    import copy
    import gc
    x = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(4)).cuda()
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    rot = zha.Rotary(64)
    want, got = torch.empty_like(x), torch.empty_like(x)
    zha.rotary(rot, x, None, pos, want)
    twin = copy.deepcopy(rot)
    rot.freq.zero_()
    del rot
    gc.collect()
    zha.rotary(twin, x, None, pos, got)
    assert torch.equal(got, want)
    cfg = zha.paged_config(1, 2, 1, 64, 16, 4, 4, dtype="f32")
    other = copy.copy(cfg)
    del cfg
    gc.collect()
    k = torch.zeros(4, 1, 16, 64, device="cuda")
    zha.paged_write(other, None, None, x[:, :1].contiguous(), x[:, 1:].contiguous(), None, pos, None, k, k.clone())
    assert torch.equal(k[0, 0, :5], x[:, 0])


@pytest.mark.parametrize("stride", [0, 64])
def test_overlapping_tokens_are_refused(zha, stride):
    """A broadcast token (stride 0, which the C call takes for contiguous) or tokens that share coordinates."""
    n, h, d = 6, 2, 64
    one = torch.zeros(n + 1, h, d, dtype=torch.bfloat16, device="cuda")
    odd = one.as_strided((n, h, d), (stride, d, 1))
    whole = one[:n].clone()
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    rot = zha.Rotary(d)
    for kw in (dict(q=odd, q_out=whole), dict(k=odd, k_out=whole), dict(q=odd), dict(q=whole, q_out=odd),
               dict(k=whole, k_out=odd)):
        with pytest.raises(ValueError, match="overlap"):
            zha.rotary(rot, kw.pop("q", None), kw.pop("k", None), ids, **kw)
    cfg = zha.paged_config(1, h, h, d, 16, 1, 1)
    pool = torch.zeros(1, h, 16, d, dtype=torch.bfloat16, device="cuda")
    for q, k, v in ((odd, whole, whole), (whole, odd, whole), (whole, whole, odd)):
        with pytest.raises(ValueError, match="overlap"):
            zha.paged_write(cfg, rot, q, k, v, ids, ids, whole, pool, pool)
    # one token alone overlaps nothing, whatever its stride
    zha.rotary(rot, odd[:1], None, ids)
    torch.cuda.synchronize()
