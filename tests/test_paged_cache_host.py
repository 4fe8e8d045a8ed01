"""PagedCache and the binding's argument handling without a GPU (nothing here launches): a refused call changes nothing."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def zha():
    from tree_indexed_sparse_02_b200 import build
    build.build()
    from tree_indexed_sparse_02_b200 import zha as z
    return z


BASE = dict(batch=3, n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, max_pages=4)
PTR = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


# ---------------------------------------------------------------- a step is refused before anything moves

def test_a_refused_step_enqueues_nothing(zha, monkeypatch):
    """step() looks at q, k_new and v_new before its first launch (here they are refused for not being on a GPU)."""
    cache = zha.PagedCache(zha.paged_config(**BASE), 6, device="cpu")
    launched = []
    for name in ("paged_plan", "paged_write", "paged_decode"):
        monkeypatch.setattr(zha, name, lambda *a, _n=name, **kw: launched.append(_n))
    q, kv = torch.zeros(6, 8, 64, dtype=torch.bfloat16), torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    n_new = torch.ones(3, dtype=torch.int32)
    for args in ((q, kv, kv), (q[:4], kv[:4], kv[:4]), (q.float(), kv, kv), (q, kv, kv[:, :1])):
        with pytest.raises(ValueError):
            cache.step(n_new, *args)
        assert not launched


def test_a_step_without_queries_is_refused(zha, monkeypatch):
    """With every call of the library let through, a step without queries still is refused, before the first of them."""
    cache = zha.PagedCache(zha.paged_config(**BASE), 6, device="cpu")
    launched = []
    for name in ("paged_write_check", "paged_plan", "paged_write", "paged_decode"):
        monkeypatch.setattr(zha, name, lambda *a, _n=name, **kw: launched.append(_n))
    kv = torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must be"):
        cache.step(torch.ones(3, dtype=torch.int32), None, kv, kv)
    assert not launched


@pytest.mark.parametrize("at,bad", [(0, None), (1, "desc"), (2, -1), (3, None), (3, ODD), (4, 504), (5, None), (5, ODD), (6, 132), (7, None), (8, -128),
                                    (9, None), (10, None), (11, ODD), (12, None), (13, ODD)])
def test_write_check_refuses_what_write_refuses(zha, at, bad):
    cfg = zha.paged_config(**BASE)
    rot = zha.RotaryDesc(64, 0, 1.0, 0, 1 << 20)
    good = [ctypes.byref(cfg), ctypes.byref(rot), 5, PTR, 0, PTR, 0, PTR, 0, PTR, PTR, PTR, PTR, PTR]
    L = zha.lib()
    assert L.zha_paged_write_check(*good) == 0
    if bad == "desc":
        bad = ctypes.byref(zha.RotaryDesc(128, 0, 1.0, 0, 1 << 20))      # rotates more than the head has
    args = good[:at] + [bad] + good[at + 1:]
    assert L.zha_paged_write_check(*args) == L.zha_paged_write(*args, None, None) == 1
    wide = zha.paged_config(**{**BASE, "n_q_heads": 1032, "n_kv_heads": 129})
    args = [ctypes.byref(wide)] + good[1:]
    assert L.zha_paged_write_check(*args) == L.zha_paged_write(*args, None, None) == 2


# ---------------------------------------------------------------- limits that every step would meet

def test_a_cache_that_no_step_could_use_is_refused(zha):
    """Rows and tables beyond zha_paged_decode's limits, heads beyond zha_paged_write's, a rotation of more than a head."""
    L = zha.lib()
    big = zha.paged_config(4, 16, 8, 64, page_size=64, n_pages=1, max_pages=8193)         # 16,384 x 8 x 524,352 > 2^35
    args = [ctypes.byref(big), 16384, PTR, PTR, PTR, PTR, PTR, PTR, None, PTR, None, PTR, None, None]
    assert L.zha_paged_decode(*args) == 2
    assert zha.paged_workspace_bytes(big, 16384) == 0
    wide = zha.paged_config(4, 2048, 128, 64, page_size=1, n_pages=1, max_pages=1)
    for cfg, rows, rot in ((big, 16384, None), (wide, 1, None), (zha.paged_config(**BASE), 1 << 22, None)):
        with pytest.raises(zha.ZhaError) as e:
            zha.PagedCache(cfg, rows, rot, device="cpu")
        assert e.value.code == 2
    with pytest.raises(zha.ZhaError) as e:
        zha.PagedCache(zha.paged_config(**BASE), 4, zha.Rotary(128, device="cpu"), device="cpu")
    assert e.value.code == 1
    for rows in (0, -1):
        with pytest.raises(zha.ZhaError) as e:
            zha.PagedCache(zha.paged_config(**BASE), rows, device="cpu")
        assert e.value.code == 1


@pytest.mark.parametrize("hq,hkv,page,width,most", [(2, 2, 1024, 1 << 14, 1024), (16, 1, 1, 1, 1 << 20), (5, 5, 64, 4096, 26214)])
def test_workspace_and_decode_draw_one_line(zha, hq, hkv, page, width, most):
    cfg = zha.paged_config(1, hq, hkv, 64, page, 1, width)
    assert zha.paged_workspace_bytes(cfg, most) > 0 and zha.paged_workspace_bytes(cfg, most + 1) == 0
    args = lambda n, ws: [ctypes.byref(cfg), n, PTR, PTR, PTR, PTR, PTR, PTR, None, PTR, None, ws, None, None]  # noqa: E731
    assert zha.lib().zha_paged_decode(*args(most + 1, PTR)) == 2
    assert zha.lib().zha_paged_decode(*args(most, None)) == 1             # as far as the missing workspace


# ---------------------------------------------------------------- errors on the device

@pytest.mark.parametrize("code", [5, 3, 1])
def test_an_error_clears_the_workspace(zha, code):
    """A wait that ran out leaves counters behind; the status may show an earlier error instead of it."""
    cache = zha.PagedCache(zha.paged_config(**BASE), 6, device="cpu")
    cache.workspace.view(torch.int32)[[0, 7, 500]] = 3
    cache.check_status()                                     # no error: nothing is touched
    assert cache.workspace.any()
    cache.status.fill_(code)
    with pytest.raises(zha.ZhaError) as e:
        cache.check_status("step")
    assert e.value.code == code
    assert not cache.workspace.any() and not cache.status.any()


# ---------------------------------------------------------------- configurations and rotations of another type

def test_structures_of_another_type_are_refused(zha):
    """The calls take a structure's address: any other one would be read field by field as a paged configuration."""
    import types
    cfg, rot = zha.paged_config(**BASE), zha.Rotary(64, device="cpu")
    other = zha.config(3, 8, 2, 64, 16, 2, 1)
    q, kv = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pool, i32 = torch.zeros(10, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(12, dtype=torch.int32)
    m = {"positions": i32, "slots": i32, "seq_ids": i32, "cu": i32}
    for bad in (other, rot.desc, ctypes.c_int32(3), 1 << 20, None, ctypes.byref(cfg), "cfg"):
        with pytest.raises(TypeError, match="PagedConfig"):
            zha.paged_plan(bad, i32, i32, i32, i32, i32, m)
        for call in (zha.paged_write, zha.paged_write_check):
            with pytest.raises(TypeError, match="PagedConfig"):
                call(bad, rot, q, kv, kv, i32, i32, q, pool, pool)
        with pytest.raises(TypeError, match="PagedConfig"):
            zha.paged_decode(bad, q, pool, pool, i32, i32, q, i32)
    like = types.SimpleNamespace(address=ctypes.addressof(cfg), device=-1, desc=cfg)
    for bad in (cfg, rot.desc, like, 64):
        with pytest.raises(TypeError, match="Rotary"):
            zha.rotary(bad, q, kv, i32)
        for call in (zha.paged_write, zha.paged_write_check):
            with pytest.raises(TypeError, match="Rotary"):
                call(cfg, bad, q, kv, kv, i32, i32, q, pool, pool)
    with pytest.raises(TypeError, match="Rotary"):
        zha.rotary(None, q, kv, i32)


# ---------------------------------------------------------------- the binding's module and what it was built for

def test_the_module_is_rebuilt_for_another_torch_or_python(monkeypatch, tmp_path):
    """As file times alone would not: it is compiled against one torch's C++ headers and one Python's."""
    import sysconfig

    from tree_indexed_sparse_02_b200 import build
    made = []

    def compiler(cmd):
        made.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")

    monkeypatch.setattr(build.subprocess, "check_call", compiler)
    monkeypatch.setattr(build, "BIND", str(tmp_path / "_bind.so"))
    monkeypatch.setattr(build, "BIND_KEY", str(tmp_path / "at" / "_bind.key"), raising=False)
    config_var = sysconfig.get_config_var

    def builds():
        n = len(made)
        assert build.build_bind() == build.BIND and os.path.exists(build.BIND)
        return len(made) - n

    assert [builds(), builds()] == [1, 0]
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".1")
    assert [builds(), builds()] == [1, 0]
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda x: ".other.so" if x == "EXT_SUFFIX" else config_var(x))
    assert [builds(), builds()] == [1, 0]
    os.remove(build.BIND)
    assert [builds(), builds()] == [1, 0]
    os.utime(build.BIND, (1, 1))                             # older than its source
    assert builds() == 1
    n = len(made)
    build.build_bind(force=True)
    assert len(made) == n + 1


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_a_module_of_another_torch_is_not_used(zha):
    """It would load, and read tensors of another layout."""
    r = python("""
import torch
torch.__version__ = "1.0.another"
try:
    from tree_indexed_sparse_02_b200 import zha
    zha.rotary(zha.Rotary(64, device="cpu"), torch.zeros(1, 1, 64), None, torch.zeros(1, dtype=torch.int32))
except ImportError as e:
    assert "1.0.another" in str(e) and "build.py" in str(e), e
    print("refused")
""")
    assert r.stdout.strip() == "refused", r.stdout + r.stderr


def test_the_sparse_path_does_not_need_the_module(zha):
    r = python("""
import sys
sys.modules["tree_indexed_sparse_02_b200._bind"] = None
import torch
from tree_indexed_sparse_02_b200 import zha
assert zha.workspace_bytes(zha.config(2, 8, 2, 64, 16, 2, 1)) > 0
cfg, rot, x, i = zha.paged_config(1, 1, 1, 64, 16, 1, 1), zha.Rotary(64, device="cpu"), torch.zeros(1, 1, 64), torch.zeros(9, dtype=torch.int32)
m = {"positions": i, "slots": i, "seq_ids": i, "cu": i}
for call in (lambda: zha.rotary(rot, x, None, i), lambda: zha.paged_plan(cfg, i, i, i, i, i, m),
             lambda: zha.paged_write(cfg, rot, x, x, x, i, i, x, x, x), lambda: zha.paged_decode(cfg, x, x, x, i, i, x, i)):
    try:
        call()
    except ImportError as e:
        print("build.py" in str(e))
""")
    assert r.stdout.split() == ["True"] * 4, r.stdout + r.stderr
