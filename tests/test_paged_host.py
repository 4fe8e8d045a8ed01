"""The paged cache's and rotary positions' host side: layouts, refusals and the
frequency tables, without a GPU (nothing here launches)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_testlib as P


@pytest.fixture(scope="module")
def zha():
    from tree_indexed_sparse_02_b200 import build
    build.build()
    from tree_indexed_sparse_02_b200 import zha as z
    return z


BASE = dict(batch=3, n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, max_pages=4)
PTR = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.mark.parametrize("change,code", [
    (dict(batch=0), 1), (dict(n_kv_heads=3), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(window=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(page_size=0), 1),
    (dict(head_dim=96), 2), (dict(n_q_heads=34), 2), (dict(dtype=5), 2), (dict(page_size=24), 2),
    (dict(page_size=2048), 2), (dict(batch=4097), 2), (dict(n_pages=(1 << 26) + 1), 2),
    (dict(max_pages=(1 << 26) + 1), 2)])
def test_config_refusals(zha, change, code):
    zha.paged_config(**BASE)
    with pytest.raises(zha.ZhaError) as e:
        zha.paged_config(**{**BASE, **change})
    assert e.value.code == code


def test_reserved_words_are_zero(zha):
    cfg = zha.paged_config(**BASE)
    cfg.reserved[1] = 1
    assert zha.lib().zha_paged_check_config(ctypes.byref(cfg)) == 1
    assert zha.lib().zha_paged_check_config(None) == 1


def test_workspace_bytes(zha):
    cfg = zha.paged_config(**BASE)
    assert zha.paged_workspace_bytes(cfg, 3) > 0
    assert zha.paged_workspace_bytes(cfg, 0) == 0
    assert zha.paged_workspace_bytes(cfg, 3) <= zha.paged_workspace_bytes(cfg, 300)
    with pytest.raises(zha.ZhaError):
        zha.paged_workspace(cfg, 0, device="cpu")


def _with(args, i, v):
    return [v if k == i else a for k, a in enumerate(args)]


def test_plan_refusals(zha):
    cfg = zha.paged_config(**BASE)
    L = zha.lib()
    good = zha.TokenMap(PTR, PTR, PTR, PTR, 8, 0)
    args = [ctypes.byref(cfg), PTR, PTR, PTR, PTR, PTR, PTR, PTR, ctypes.byref(good), None, None]
    for i in range(9):                                    # any missing argument
        assert L.zha_paged_plan(*_with(args, i, None)) == 1, i
    for m in (zha.TokenMap(None, PTR, PTR, PTR, 8, 0), zha.TokenMap(PTR, None, PTR, PTR, 8, 0),
              zha.TokenMap(PTR, PTR, None, PTR, 8, 0), zha.TokenMap(PTR, PTR, PTR, None, 8, 0),
              zha.TokenMap(PTR, PTR, PTR, PTR, 0, 0), zha.TokenMap(PTR, PTR, PTR, PTR, 8, 1)):
        assert L.zha_paged_plan(*_with(args, 8, ctypes.byref(m))) == 1


def _desc(zha, **kw):
    d = dict(rotary_dim=64, layout=0, mscale=1.0, reserved=0, freq=1 << 20)
    d.update(kw)
    return zha.RotaryDesc(d["rotary_dim"], d["layout"], d["mscale"], d["reserved"], d["freq"])


BAD_ROTARY = [dict(rotary_dim=0), dict(rotary_dim=63), dict(rotary_dim=66), dict(layout=2), dict(reserved=1),
              dict(mscale=float("nan")), dict(mscale=float("inf")), dict(freq=None), dict(freq=(1 << 20) + 4)]


def test_rotary_refusals(zha):
    L = zha.lib()
    r = _desc(zha)
    args = [ctypes.byref(r), 64, 0, 5, 8, 2, PTR, 0, PTR, 0, PTR, PTR, 0, PTR, 0, 0, None]
    for i in (0, 6, 8, 10, 11, 13):                       # one of a pair missing, no positions, no table
        assert L.zha_rotary_apply(*_with(args, i, None)) == 1, i
    assert L.zha_rotary_apply(*_with(_with(_with(_with(args, 6, None), 8, None), 11, None), 13, None)) == 1
    for i in (6, 8, 11, 13):
        assert L.zha_rotary_apply(*_with(args, i, ODD)) == 1, i
    assert L.zha_rotary_apply(*_with(args, 1, 96)) == 2
    assert L.zha_rotary_apply(*_with(args, 2, 7)) == 2
    assert L.zha_rotary_apply(*_with(args, 3, -1)) == 1
    assert L.zha_rotary_apply(*_with(args, 4, 0)) == 1
    assert L.zha_rotary_apply(*_with(args, 4, 1025)) == 2
    for i, row in ((7, 512), (9, 128), (12, 512), (14, 128)):
        for stride in (row - 8, row + 4, -row):           # overlapping tokens, not 16 bytes, backwards
            assert L.zha_rotary_apply(*_with(args, i, stride)) == 1, (i, stride)
    for bad in BAD_ROTARY:
        assert L.zha_rotary_apply(*_with(args, 0, ctypes.byref(_desc(zha, **bad)))) == 1, bad
    assert L.zha_rotary_apply(*_with(args, 3, 0)) == 0    # no tokens: nothing to do


def test_write_refusals(zha):
    cfg = zha.paged_config(**BASE)
    L = zha.lib()
    r = _desc(zha)
    args = [ctypes.byref(cfg), ctypes.byref(r), 5, PTR, 0, PTR, 0, PTR, 0, PTR, PTR, PTR, PTR, PTR, None, None]
    for i in (0, 3, 5, 7, 9, 10, 11, 12, 13):
        assert L.zha_paged_write(*_with(args, i, None)) == 1, i
    for i in (3, 5, 7, 11, 12, 13):
        assert L.zha_paged_write(*_with(args, i, ODD)) == 1, i
    for i, row in ((4, 512), (6, 128), (8, 128)):
        for stride in (row - 8, row + 4, -row):
            assert L.zha_paged_write(*_with(args, i, stride)) == 1, (i, stride)
    for bad in BAD_ROTARY:
        assert L.zha_paged_write(*_with(args, 1, ctypes.byref(_desc(zha, **bad)))) == 1, bad
    assert L.zha_paged_write(*_with(args, 2, -1)) == 1
    assert L.zha_paged_write(*_with(args, 2, 0)) == 0


def test_decode_refusals(zha):
    cfg = zha.paged_config(**BASE)
    L = zha.lib()
    args = [ctypes.byref(cfg), 3, PTR, PTR, PTR, PTR, PTR, None, None, PTR, PTR, PTR, None, None]
    for i in (0, 2, 3, 4, 5, 6, 9, 11):
        assert L.zha_paged_decode(*_with(args, i, None)) == 1, i
    for i in (2, 3, 4, 9, 11):
        assert L.zha_paged_decode(*_with(args, i, ODD)) == 1, i
    assert L.zha_paged_decode(*_with(args, 1, -1)) == 1
    assert L.zha_paged_decode(*_with(args, 1, 4)) == 1    # more rows than sequences, no mapping
    assert L.zha_paged_decode(*_with(_with(args, 1, 1 << 22), 7, PTR)) == 2
    assert L.zha_paged_decode(*_with(args, 1, 0)) == 0


def test_binding_refuses_tensors_it_cannot_pass_on(zha):
    cfg = zha.paged_config(**BASE)
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    pool = torch.zeros(10, 2, 16, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(12, dtype=torch.int32)
    ws = torch.zeros(zha.paged_workspace_bytes(cfg, 3), dtype=torch.uint8)

    def decode(**kw):
        a = dict(q=q, k_pool=pool, v_pool=pool, table=i32, lens=i32[:3], out=q, workspace=ws)
        a.update(kw)
        with pytest.raises(ValueError):
            zha.paged_decode(cfg, **a)

    decode()                                              # not on a GPU
    for kw in (dict(q=q.float()), dict(q=q[:, :4]), dict(q=q.transpose(0, 1)), dict(k_pool=pool[:9]),
               dict(v_pool=pool.transpose(1, 2)), dict(table=i32[:11]), dict(lens=i32[:2]), dict(lens=i32.long()),
               dict(out=q.float()), dict(workspace=ws[:16]), dict(lse=torch.zeros(3, 8, dtype=torch.float64)),
               dict(seq_ids=i32[:2]), dict(positions=i32.long())):
        decode(**kw)
    rot = zha.Rotary(64, device="cpu")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for kw in (dict(q=q.half()), dict(q=q[:2]), dict(k=k[..., :32]), dict(q=q.transpose(1, 2)), dict(positions=i32[:2]),
               dict(positions=i32.long()), dict(q_out=q[:2]), dict(q=None, k=None), dict()):
        a = dict(q=q, k=k, positions=i32)
        a.update(kw)
        with pytest.raises(ValueError):
            zha.rotary(rot, **a)
    for kw in (dict(q_out=None), dict(v_new=k[:2]), dict(k_new=k.float()), dict(slots=i32[:2]), dict(k_pool=pool[1:]),
               dict(positions=i32.long()), dict()):
        a = dict(q=q, k_new=k, v_new=k, positions=i32, slots=i32, q_out=q.clone(), k_pool=pool, v_pool=pool)
        a.update(kw)
        with pytest.raises(ValueError):
            zha.paged_write(cfg, rot, **a)
    m = {"positions": i32, "slots": i32, "seq_ids": i32, "cu": i32}
    for kw in (dict(table=i32[:5]), dict(lens=i32[:2]), dict(n_new=i32.long()), dict(free_pages=i32[:9]),
               dict(token_map={**m, "cu": i32[:3]}), dict(token_map={**m, "positions": i32[:5]}), dict()):
        a = dict(table=i32, lens=i32, n_new=i32, free_pages=i32, n_free=i32, token_map=m)
        a.update(kw)
        with pytest.raises(ValueError):
            zha.paged_plan(cfg, **a)


@pytest.mark.filterwarnings("ignore::UserWarning")
def test_binding_refuses_what_is_no_tensor(zha):
    cfg = zha.paged_config(**BASE)
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    for bad in (None, 5, [1.0], np.zeros((3, 8, 64)), torch.sparse_coo_tensor(size=(3, 8, 64), check_invariants=False)):
        with pytest.raises(ValueError):
            zha.paged_decode(cfg, bad, q, q, q, q, q, q)
        with pytest.raises(ValueError):
            zha.rotary(zha.Rotary(64, device="cpu"), bad, bad, q)
        with pytest.raises(ValueError):
            zha.paged_write(cfg, None, q, q, q, None, q, q, bad, q)
        with pytest.raises(ValueError):
            zha.paged_plan(cfg, bad, q, q, q, q, {"positions": q, "slots": q, "seq_ids": q, "cu": q})


@pytest.mark.parametrize("rd", [2, 4, 34, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 1.0), ("yarn", 16.0)])
def test_rotary_frequencies(zha, rd, scaling, factor):
    """Against extended precision: a few fp64 roundings (power, two quotients, a blend)."""
    r = zha.Rotary(rd, base=500000.0, scaling=scaling, factor=factor, original_len=8192, device="cpu")
    theta, m = P.frequencies(rd, 500000.0, scaling, factor, 8192)
    want = (theta / (2 * np.longdouble(math.pi))).astype(np.float64)
    assert np.allclose(r.freq.numpy(), want, rtol=16 * 2.0 ** -53, atol=0)
    assert abs(r.desc.mscale - m) <= 2.0 ** -24 * m


def test_rotary_frequency_refusals(zha):
    L = zha.lib()
    out, m = (ctypes.c_double * 128)(), ctypes.c_float()
    good = [64, 10000.0, 3, 2.0, 4096, out, ctypes.byref(m)]
    assert L.zha_rotary_freqs(*good) == 0
    for i, v in ((0, 0), (0, 63), (0, 258), (1, 1.0), (1, math.nan), (1, math.inf), (2, 4), (2, -1), (3, 0.0),
                 (3, math.nan), (3, math.inf), (3, 0.5), (4, 0), (5, None), (6, None)):
        assert L.zha_rotary_freqs(*_with(good, i, v)) == 1, (i, v)
