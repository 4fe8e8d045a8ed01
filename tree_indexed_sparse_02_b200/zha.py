"""Thin Python binding of libzha's C ABI (``include/zha.h``).

Argument marshalling only: every function forwards device pointers of torch
tensors and a CUDA stream to the library, and raises ``ZhaError`` on a
non-zero status. Nothing here computes any step of the method; if libzha.so
is missing the import fails loudly (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzha.so")

ZHA_BF16, ZHA_F32 = 0, 1
ZHA_FLAG_TAIL_ONLY = 1
ZHA_FLAG_TCGEN05 = 2
ZHA_FLAG_FUSED_ROUTE = 4
ZHA_P_FIXED, ZHA_P_DEPTH_ROOT = 0, 1
ZHA_WAIT_ROW_BARRIER, ZHA_WAIT_MBARRIER = 0, 1
ZHA_SUMMARY_NATIVE, ZHA_SUMMARY_MXFP8 = 0, 1
ZHA_ROPE_HALF, ZHA_ROPE_INTERLEAVED = 0, 1
ZHA_ROPE_PLAIN, ZHA_ROPE_LINEAR, ZHA_ROPE_NTK, ZHA_ROPE_YARN = 0, 1, 2, 3
ZHA_MAX_LEVELS = 8
_DTYPES = {torch.bfloat16: ZHA_BF16, torch.float32: ZHA_F32}
STATUS_NAMES = {0: "ZHA_OK", 1: "ZHA_ERR_INVALID_ARG", 2: "ZHA_ERR_UNSUPPORTED",
                3: "ZHA_ERR_CAPACITY", 4: "ZHA_ERR_CUDA", 5: "ZHA_ERR_TIMEOUT"}


class ZhaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} ({_lib.zha_status_string(code).decode()})")


class Config(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("chunk", ctypes.c_int32), ("levels", ctypes.c_int32),
                ("n_refs", ctypes.c_int32), ("dtype", ctypes.c_int32), ("max_len", ctypes.c_int64),
                ("scale", ctypes.c_float), ("flags", ctypes.c_int32), ("attn_splits", ctypes.c_int32),
                ("summary", ctypes.c_int32), ("queries", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    @property
    def group(self) -> int:
        return self.n_q_heads // self.n_kv_heads

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == ZHA_BF16 else torch.float32


class Selection(ctypes.Structure):
    _fields_ = [("leaf_idx", ctypes.c_void_p), ("head_mask", ctypes.c_void_p), ("count", ctypes.c_void_p),
                ("level_kept", ctypes.c_void_p)]


class LevelView(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_int64), ("cand_idx", ctypes.c_size_t), ("cand_mask", ctypes.c_size_t),
                ("scores", ctypes.c_size_t), ("kept_mask", ctypes.c_size_t), ("count", ctypes.c_size_t)]


class PagedConfig(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("scale", ctypes.c_float),
                ("window", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]

    # What the calls need of a configuration every time, made once (a configuration is not changed after its first
    # call: make another).
    @functools.cached_property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == ZHA_BF16 else torch.float32

    @functools.cached_property
    def ref(self):
        return ctypes.byref(self)

    @functools.cached_property
    def pool_elements(self):
        return self.n_pages * self.n_kv_heads * self.page_size * self.head_dim

    def decode_workspace(self, rows):
        known = self.__dict__.setdefault("_workspace", {})
        if rows not in known:
            known[rows] = int(_lib.zha_paged_workspace_bytes(self.ref, rows)) if rows else 0
        return known[rows]


class TokenMap(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("seq_ids", ctypes.c_void_p),
                ("cu_new", ctypes.c_void_p), ("max_tokens", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("freq", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libzha.so not built at {LIB_PATH}; run tree_indexed_sparse_02_b200/build.py")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    CP = ctypes.POINTER(Config)
    SP = ctypes.POINTER(Selection)
    PP, RP, MP = ctypes.POINTER(PagedConfig), ctypes.POINTER(RotaryDesc), ctypes.POINTER(TokenMap)
    f64 = ctypes.c_double
    sig = {
        "zha_status_string": ([i32], ctypes.c_char_p),
        "zha_check_config": ([CP], i32),
        "zha_level_nodes": ([CP, i64, i32], i64),
        "zha_route_fused": ([CP, i32, ctypes.POINTER(i32)], i32),
        "zha_tree_bytes": ([CP], sz),
        "zha_tree_level_offsets": ([CP, i32, ctypes.POINTER(sz), ctypes.POINTER(sz)], i32),
        "zha_tree_level_scales": ([CP, i32, ctypes.POINTER(sz)], i32),
        "zha_tree_level_logmass": ([CP, i32, ctypes.POINTER(sz)], i32),
        "zha_workspace_bytes": ([CP], sz),
        "zha_workspace_level_view": ([CP, i32, ctypes.POINTER(LevelView)], i32),
        "zha_workspace_level_view_block": ([CP, i32, i32, ctypes.POINTER(LevelView)], i32),
        "zha_tree_build": ([CP, P, P, P, P, P, P], i32),
        "zha_tree_append": ([CP, P, P, P, P, i32, P, P], i32),
        "zha_route": ([CP, P, P, P, P, SP, P, P, P], i32),
        "zha_sparse_attn": ([CP, P, P, P, P, SP, P, P, P, P], i32),
        "zha_decode": ([CP, P, P, P, P, P, P, P, P, P, SP, P, P, P, P], i32),
        "zha_decode_block": ([CP, i32, P, P, P, P, P, P, P, P, P, SP, P, P, P, P], i32),
        "zha_dense_decode": ([CP, P, P, P, P, P, P, P, P], i32),
        "zha_topp_select": ([P, P, i32, i64, f32, P, P, P], i32),
        "zha_p_schedule": ([f32, i32, i32, ctypes.POINTER(f32)], i32),
        "zha_wait_expiry_check": ([i32, i64, P, P], i32),
        "zha_paged_check_config": ([PP], i32),
        "zha_paged_plan": ([PP, P, P, P, P, P, P, P, MP, P, P], i32),
        "zha_rotary_freqs": ([i32, f64, i32, f64, i64, ctypes.POINTER(f64), ctypes.POINTER(f32)], i32),
        "zha_rotary_apply": ([RP, i32, i32, i32, i32, i32, P, i64, P, i64, P, P, i64, P, i64, i32, P], i32),
        "zha_paged_write": ([PP, RP, i32, P, i64, P, i64, P, i64, P, P, P, P, P, P, P], i32),
        "zha_paged_workspace_bytes": ([PP, i32], sz),
        "zha_paged_decode": ([PP, i32, P, P, P, P, P, P, P, P, P, P, P, P], i32),
        "zha_launch_count": ([], ctypes.c_uint64),
        "zha_profile_enable": ([i32], i32),
        "zha_profile_read": ([ctypes.c_char_p, i32, ctypes.POINTER(ctypes.c_double),
                              ctypes.POINTER(ctypes.c_int64), i32], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


_lib = _load()
_rotary_apply, _paged_plan = _lib.zha_rotary_apply, _lib.zha_paged_plan
_paged_write, _paged_decode = _lib.zha_paged_write, _lib.zha_paged_decode


def lib():
    return _lib


def config(batch, n_q_heads, n_kv_heads, head_dim, chunk, levels, n_refs, dtype="bf16", max_len=4096,
           scale=0.0, flags=0, attn_splits=0, summary="native", queries=0) -> Config:
    dt = {"bf16": ZHA_BF16, "f32": ZHA_F32}.get(dtype, dtype)
    sm = {"native": ZHA_SUMMARY_NATIVE, "mxfp8": ZHA_SUMMARY_MXFP8}.get(summary, summary)
    c = Config(batch, n_q_heads, n_kv_heads, head_dim, chunk, levels, n_refs, dt, max_len, scale, flags,
               attn_splits, sm, queries)
    check(_lib.zha_check_config(ctypes.byref(c)), "zha_check_config")
    return c


def check(code: int, where: str):
    if code != 0:
        raise ZhaError(code, where)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def level_nodes(cfg: Config, n_tokens: int, level: int) -> int:
    return int(_lib.zha_level_nodes(ctypes.byref(cfg), int(n_tokens), int(level)))


def route_fused(cfg: Config, T: int = 1) -> bool:
    """True if routing with cfg (T query positions) runs the fused launch."""
    out = ctypes.c_int32(0)
    check(_lib.zha_route_fused(ctypes.byref(cfg), int(T), ctypes.byref(out)), "zha_route_fused")
    return bool(out.value)


def tree_bytes(cfg: Config) -> int:
    return int(_lib.zha_tree_bytes(ctypes.byref(cfg)))


def workspace_bytes(cfg: Config) -> int:
    return int(_lib.zha_workspace_bytes(ctypes.byref(cfg)))


def tree_level_offsets(cfg: Config, level: int):
    mu, b = ctypes.c_size_t(), ctypes.c_size_t()
    check(_lib.zha_tree_level_offsets(ctypes.byref(cfg), level, ctypes.byref(mu), ctypes.byref(b)),
          "zha_tree_level_offsets")
    return mu.value, b.value


def workspace_level_view(cfg: Config, level: int, T: int = 1) -> LevelView:
    v = LevelView()
    check(_lib.zha_workspace_level_view_block(ctypes.byref(cfg), int(T), level, ctypes.byref(v)),
          "zha_workspace_level_view_block")
    return v


def _plevels(cfg: Config, p):
    if isinstance(p, (int, float)):
        p = [float(p)] * cfg.levels
    arr = (ctypes.c_float * cfg.levels)(*[float(x) for x in p])
    return arr


def p_schedule(p: float, levels: int, schedule=ZHA_P_FIXED) -> list[float]:
    """Per-level fractions (index l-1 is level l) from libzha's schedule rule."""
    schedule = {"fixed": ZHA_P_FIXED, "root": ZHA_P_DEPTH_ROOT}.get(schedule, schedule)
    out = (ctypes.c_float * max(int(levels), 1))()
    check(_lib.zha_p_schedule(float(p), int(levels), int(schedule), out), "zha_p_schedule")
    return [float(x) for x in out[:levels]]


def _sel(sel) -> Selection:
    return Selection(sel["leaf_idx"].data_ptr(), sel["head_mask"].data_ptr(), sel["count"].data_ptr(),
                     None if sel.get("level_kept") is None else sel["level_kept"].data_ptr())


def tree_build(cfg, tree, K, refs, lens, dev_status=None, stream=None):
    check(_lib.zha_tree_build(ctypes.byref(cfg), _p(tree), _p(K), _p(refs), _p(lens), _p(dev_status),
                              _stream(stream)), "zha_tree_build")


def tree_append(cfg, tree, K, refs, lens, n_new, dev_status=None, stream=None):
    check(_lib.zha_tree_append(ctypes.byref(cfg), _p(tree), _p(K), _p(refs), _p(lens), int(n_new),
                               _p(dev_status), _stream(stream)), "zha_tree_append")


def route(cfg, tree, q, lens, p, sel, workspace, dev_status=None, stream=None):
    s = _sel(sel)
    check(_lib.zha_route(ctypes.byref(cfg), _p(tree), _p(q), _p(lens), _plevels(cfg, p), ctypes.byref(s),
                         _p(workspace), _p(dev_status), _stream(stream)), "zha_route")


def sparse_attn(cfg, q, K, V, lens, sel, out, workspace, dev_status=None, stream=None):
    s = _sel(sel)
    check(_lib.zha_sparse_attn(ctypes.byref(cfg), _p(q), _p(K), _p(V), _p(lens), ctypes.byref(s), _p(out),
                               _p(workspace), _p(dev_status), _stream(stream)), "zha_sparse_attn")


def decode(cfg, tree, K, V, refs, lens, q, k_new, v_new, p, sel, out, workspace, dev_status=None,
           stream=None):
    s = _sel(sel)
    check(_lib.zha_decode(ctypes.byref(cfg), _p(tree), _p(K), _p(V), _p(refs), _p(lens), _p(q), _p(k_new),
                          _p(v_new), _plevels(cfg, p), ctypes.byref(s), _p(out), _p(workspace),
                          _p(dev_status), _stream(stream)), "zha_decode")


def decode_block(cfg, T, tree, K, V, refs, lens, q, k_new, v_new, p, sel, out, workspace, dev_status=None,
                 stream=None):
    """T query positions per sequence: q, out [B, T, Hq, d]; k_new, v_new [B, T, Hkv, d]."""
    s = _sel(sel)
    check(_lib.zha_decode_block(ctypes.byref(cfg), int(T), _p(tree), _p(K), _p(V), _p(refs), _p(lens), _p(q),
                                _p(k_new), _p(v_new), _plevels(cfg, p), ctypes.byref(s), _p(out),
                                _p(workspace), _p(dev_status), _stream(stream)), "zha_decode_block")


def dense_decode(cfg, q, K, V, lens, out, workspace, dev_status=None, stream=None):
    check(_lib.zha_dense_decode(ctypes.byref(cfg), _p(q), _p(K), _p(V), _p(lens), _p(out), _p(workspace),
                                _p(dev_status), _stream(stream)), "zha_dense_decode")


def topp_select(scores, counts, p, kept, dev_status=None, stream=None):
    n_sets, stride = scores.shape
    check(_lib.zha_topp_select(_p(scores), _p(counts), int(n_sets), int(stride), float(p), _p(kept),
                               _p(dev_status), _stream(stream)), "zha_topp_select")


# ---------------------------------------------------------------- paged caches and rotary positions

def paged_config(batch, n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_pages, dtype="bf16", scale=0.0,
                 window=0) -> PagedConfig:
    dt = {"bf16": ZHA_BF16, "f32": ZHA_F32}.get(dtype, dtype)
    c = PagedConfig(batch, n_q_heads, n_kv_heads, head_dim, dt, page_size, n_pages, max_pages, scale, window)
    check(_lib.zha_paged_check_config(ctypes.byref(c)), "zha_paged_check_config")
    return c


def paged_workspace_bytes(cfg: PagedConfig, rows: int) -> int:
    return int(_lib.zha_paged_workspace_bytes(ctypes.byref(cfg), int(rows)))


def paged_workspace(cfg: PagedConfig, rows: int, device="cuda"):
    """Zeroed scratch of paged_decode calls of up to `rows` rows (one call at a time)."""
    n = paged_workspace_bytes(cfg, rows)
    if n == 0:
        raise ZhaError(1, "zha_paged_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


# The checks below are on the path of every call, whose kernels can take less time than their launch: they read
# few tensor attributes, and the messages are made only where one fails. `dev` is a device index (-1: not CUDA).

def _refuse(where: str, what: str, t=None):
    got = "" if t is None else f", got {t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}"
    raise ValueError(f"{where}: {what}{got}")


def _rows(t, where, name, n, heads, d, dtype, dev):
    """The address and the token stride (elements) of a [n, heads, d] tensor whose heads are packed; any other layout
    is refused."""
    if t.shape != (n, heads, d) or t.dtype is not dtype or t.get_device() != dev:
        _refuse(where, f"{name} must be a {dtype} tensor [{n}, {heads}, {d}] on device {dev}", t)
    s0, s1, s2 = t.stride()
    if (s2 != 1 or (s1 != d and heads > 1)) and n > 0:
        _refuse(where, f"{name}'s heads must be packed", t)
    return t.data_ptr(), s0 if n > 1 else heads * d


def _int32(t, where, name, n, dev):
    """The address of an int32 array of at least n entries; None passes."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        _refuse(where, f"{name} must be a contiguous int32 tensor of at least {n} entries on device {dev}", t)
    return t.data_ptr()


def _block(t, where, name, n, dtype, dev):
    """The address of a contiguous array of n elements."""
    if t.dtype is not dtype or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        _refuse(where, f"{name} must be a contiguous {dtype} tensor of {n} elements on device {dev}", t)
    return t.data_ptr()


def _call(where, fn, dev, stream, *args):
    """fn(*args, stream) with device `dev` current, on its current stream by default."""
    if dev < 0:
        _refuse(where, "tensors must be on a CUDA device")
    here = torch._C._cuda_getDevice()
    if dev != here:
        with torch.cuda.device(dev):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    else:
        code = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if code != 0:
        raise ZhaError(code, where)


class Rotary:
    """A rotary embedding: its frequency table (turns per position, fp64) on the device.

    layout "half" pairs coordinates (i, i + rotary_dim/2), "interleaved" (2i, 2i + 1); scaling "none",
    "linear", "ntk" or "yarn" by `factor` (from a context of original_len for YaRN)."""

    def __init__(self, rotary_dim, base=10000.0, layout="half", scaling="none", factor=1.0, original_len=4096,
                 device="cuda"):
        kind = {"none": ZHA_ROPE_PLAIN, "linear": ZHA_ROPE_LINEAR, "ntk": ZHA_ROPE_NTK, "yarn": ZHA_ROPE_YARN}
        lay = {"half": ZHA_ROPE_HALF, "interleaved": ZHA_ROPE_INTERLEAVED}
        table = (ctypes.c_double * max(int(rotary_dim) // 2, 1))()
        m = ctypes.c_float()
        check(_lib.zha_rotary_freqs(int(rotary_dim), float(base), kind.get(scaling, scaling), float(factor),
                                    int(original_len), table, ctypes.byref(m)), "zha_rotary_freqs")
        self.freq = torch.tensor(list(table), dtype=torch.float64).to(device)
        self.desc = RotaryDesc(int(rotary_dim), lay.get(layout, layout), m.value, 0, self.freq.data_ptr())
        self.ref = ctypes.byref(self.desc)
        self.device = self.freq.get_device()


def rotary(rot: Rotary, q, k, positions, q_out=None, k_out=None, transpose=False, stream=None):
    """Rotate q [n, Hq, d] and k [n, Hk, d] (either may be None; tokens may be strided) at int32 positions [n].
    The outputs default to the inputs (in place); transpose applies the gradient's map. Returns (q_out, k_out)."""
    where = "zha_rotary_apply"
    one = k if q is None else q
    if one is None or one.ndim != 3:
        _refuse(where, "q or k [n, heads, d] is needed", one)
    (n, heads, d), dt, dev = one.shape, one.dtype, one.get_device()
    code = _DTYPES.get(dt)
    if code is None:
        _refuse(where, "bf16 or fp32 is needed", one)
    hq = hk = qs = ks = qos = kos = 0
    qp = kp = qo = ko = None
    if q is not None:
        hq = heads
        qp, qs = _rows(q, where, "q", n, hq, d, dt, dev)
        if q_out is None:
            q_out, qo, qos = q, qp, qs
        else:
            qo, qos = _rows(q_out, where, "q_out", n, hq, d, dt, dev)
    if k is not None:
        hk = k.shape[1] if k.ndim == 3 else 0
        kp, ks = _rows(k, where, "k", n, hk, d, dt, dev)
        if k_out is None:
            k_out, ko, kos = k, kp, ks
        else:
            ko, kos = _rows(k_out, where, "k_out", n, hk, d, dt, dev)
    if rot.device != dev:
        _refuse(where, f"the rotary table is on device {rot.device}, the tensors on {dev}")
    _call(where, _rotary_apply, dev, stream, rot.ref, d, code, n, hq, hk, qp, qs, kp, ks,
          _int32(positions, where, "positions", n, dev), qo, qos, ko, kos, 1 if transpose else 0)
    return q_out, k_out


def paged_plan(cfg: PagedConfig, table, lens, n_new, free_pages, n_free, token_map, lens_out=None, n_free_out=None,
               dev_status=None, stream=None):
    """Block tables, slots and lengths of a step with n_new[b] new tokens of sequence b (< 0: it ends).
    token_map: {"positions", "slots", "seq_ids"} (one entry per row of the token buffer) and "cu" [batch + 1];
    lens_out and n_free_out default to lens and n_free (in place)."""
    where, dev, B = "zha_paged_plan", table.get_device(), cfg.batch
    slots = token_map["slots"]
    rows = slots.numel()
    m = TokenMap(_int32(token_map["positions"], where, "positions", rows, dev), _int32(slots, where, "slots", rows, dev),
                 _int32(token_map["seq_ids"], where, "seq_ids", rows, dev),
                 _int32(token_map["cu"], where, "cu", B + 1, dev), rows, 0)
    lens_p, free_p = _int32(lens, where, "lens", B, dev), _int32(n_free, where, "n_free", 1, dev)
    _call(where, _paged_plan, dev, stream, cfg.ref, _int32(table, where, "table", B * cfg.max_pages, dev),
          lens_p, _int32(n_new, where, "n_new", B, dev), _int32(free_pages, where, "free_pages", cfg.n_pages, dev), free_p,
          lens_p if lens_out is None else _int32(lens_out, where, "lens_out", B, dev),
          free_p if n_free_out is None else _int32(n_free_out, where, "n_free_out", 1, dev), ctypes.byref(m),
          _int32(dev_status, where, "dev_status", 1, dev))


def paged_write(cfg: PagedConfig, rot, q, k_new, v_new, positions, slots, q_out, k_pool, v_pool, dev_status=None,
                stream=None):
    """Rotate q and k_new [n, heads, d] and write k_new, v_new to their cache slots [n] (negative: skipped).
    rot None: no rotation; q None: keys and values only."""
    where, dev, dt, d, hkv = "zha_paged_write", k_pool.get_device(), cfg.torch_dtype, cfg.head_dim, cfg.n_kv_heads
    n = k_new.shape[0]
    kp, ks = _rows(k_new, where, "k_new", n, hkv, d, dt, dev)
    vp, vs = _rows(v_new, where, "v_new", n, hkv, d, dt, dev)
    qs, qp, qo = 0, None, None
    if q is not None:
        hq = cfg.n_q_heads
        qp, qs = _rows(q, where, "q", n, hq, d, dt, dev)
        if q_out is None:
            _refuse(where, "q_out is needed with q")
        qo = _block(q_out, where, "q_out", n * hq * d, dt, dev)
    if rot is not None and rot.device != dev:
        _refuse(where, f"the rotary table is on device {rot.device}, the tensors on {dev}")
    size = cfg.pool_elements
    _call(where, _paged_write, dev, stream, cfg.ref, None if rot is None else rot.ref, n, qp, qs, kp, ks, vp, vs,
          _int32(positions, where, "positions", n, dev), _int32(slots, where, "slots", n, dev), qo,
          _block(k_pool, where, "k_pool", size, dt, dev), _block(v_pool, where, "v_pool", size, dt, dev),
          _int32(dev_status, where, "dev_status", 1, dev))
    return q_out


def paged_decode(cfg: PagedConfig, q, k_pool, v_pool, table, lens, out, workspace, lse=None, seq_ids=None,
                 positions=None, dev_status=None, stream=None):
    """Attention of rows q [n, Hq, d] over the paged cache into out (and lse [n, Hq] fp32). Row r is of sequence
    seq_ids[r] (default r; negative: left as it is) and attends tokens 0 .. positions[r] (default: all)."""
    where, dev, dt, hq, d = "zha_paged_decode", q.get_device(), cfg.torch_dtype, cfg.n_q_heads, cfg.head_dim
    n, size, batch = q.shape[0], cfg.pool_elements, cfg.batch
    if q.ndim != 3 or (seq_ids is None and n > batch):
        _refuse(where, f"q must be [n, {hq}, {d}] with a sequence for each row", q)
    qp, op = _block(q, where, "q", n * hq * d, dt, dev), _block(out, where, "out", n * hq * d, dt, dev)
    if workspace.get_device() != dev or not workspace.is_contiguous() or workspace.nbytes < cfg.decode_workspace(n):
        _refuse(where, f"the workspace must be contiguous and hold paged_workspace_bytes(cfg, {n}) bytes on device {dev}",
                workspace)
    _call(where, _paged_decode, dev, stream, cfg.ref, n, qp,
          _block(k_pool, where, "k_pool", size, dt, dev), _block(v_pool, where, "v_pool", size, dt, dev),
          _int32(table, where, "table", batch * cfg.max_pages, dev), _int32(lens, where, "lens", batch, dev),
          _int32(seq_ids, where, "seq_ids", n, dev), _int32(positions, where, "positions", n, dev), op,
          None if lse is None else _block(lse, where, "lse", n * hq, torch.float32, dev), workspace.data_ptr(),
          _int32(dev_status, where, "dev_status", 1, dev))
    return out


class PagedCache:
    """Device state of one layer's paged cache: pools, block table, lengths, free pages, a step's token map and
    buffers, status. max_tokens is the size of a step's token buffer; shorter steps leave its tail unused.

    step() runs plan, write and decode; everything stays on the device, so a step can be captured into a CUDA
    graph (n_new, q, k_new, v_new are then the captured buffers). The cache serves one step at a time."""

    def __init__(self, cfg: PagedConfig, max_tokens: int, rot: Rotary | None = None, device="cuda"):
        self.cfg, self.rot = cfg, rot
        kw = dict(dtype=torch.int32, device=device)
        shape = (cfg.n_pages, cfg.n_kv_heads, cfg.page_size, cfg.head_dim)
        self.k_pool = torch.zeros(shape, dtype=cfg.torch_dtype, device=device)
        self.v_pool = torch.zeros(shape, dtype=cfg.torch_dtype, device=device)
        self.table = torch.full((cfg.batch, cfg.max_pages), -1, **kw)
        self.lens = torch.zeros(cfg.batch, **kw)
        self.free_pages = torch.arange(cfg.n_pages - 1, -1, -1, **kw)     # page 0 is on top
        self.n_free = torch.full((1,), cfg.n_pages, **kw)
        self.token_map = {"positions": torch.zeros(max_tokens, **kw), "slots": torch.full((max_tokens,), -1, **kw),
                          "seq_ids": torch.full((max_tokens,), -1, **kw), "cu": torch.zeros(cfg.batch + 1, **kw)}
        rows = (max_tokens, cfg.n_q_heads, cfg.head_dim)
        self.q = torch.zeros(rows, dtype=cfg.torch_dtype, device=device)
        self.out = torch.zeros(rows, dtype=cfg.torch_dtype, device=device)
        self.lse = torch.zeros(rows[:2], dtype=torch.float32, device=device)
        self.workspace = paged_workspace(cfg, max_tokens, device)
        self.status = torch.zeros(1, **kw)

    def plan(self, n_new, stream=None):
        """Room for n_new[b] more tokens of each sequence (< 0: it ends); fills the token map."""
        paged_plan(self.cfg, self.table, self.lens, n_new, self.free_pages, self.n_free, self.token_map,
                   dev_status=self.status, stream=stream)

    def write(self, q, k_new, v_new, stream=None):
        """Rotated queries into self.q, rotated keys and values into the cache, for the planned token rows."""
        m = self.token_map
        paged_write(self.cfg, self.rot, q, k_new, v_new, m["positions"], m["slots"], self.q, self.k_pool, self.v_pool,
                    dev_status=self.status, stream=stream)

    def attend(self, stream=None):
        """Each planned token's attention over its sequence up to itself: (out, lse), rows as in the token map."""
        m = self.token_map
        paged_decode(self.cfg, self.q, self.k_pool, self.v_pool, self.table, self.lens, self.out, self.workspace,
                     lse=self.lse, seq_ids=m["seq_ids"], positions=m["positions"], dev_status=self.status,
                     stream=stream)
        return self.out, self.lse

    def step(self, n_new, q, k_new, v_new, stream=None):
        """q [max_tokens, Hq, d], k_new, v_new [max_tokens, Hkv, d]: the step's token rows, before rotation."""
        self.plan(n_new, stream)
        self.write(q, k_new, v_new, stream)
        return self.attend(stream)

    def check_status(self, where="device"):
        code = int(self.status.item())
        if code:
            self.status.zero_()
            raise ZhaError(code, where)


def wait_expiry_check(kind: int, limit_cycles: int, dev_status, stream=None):
    """Run one of the library's bounded device waits on a condition nothing
    satisfies (ZHA_WAIT_ROW_BARRIER or ZHA_WAIT_MBARRIER), giving up after
    limit_cycles SM cycles with ZHA_ERR_TIMEOUT in dev_status."""
    check(_lib.zha_wait_expiry_check(int(kind), int(limit_cycles), _p(dev_status), _stream(stream)),
          "zha_wait_expiry_check")


def launch_count() -> int:
    """Kernels libzha has launched since it was loaded."""
    return int(_lib.zha_launch_count())


def profile_enable(on: bool = True):
    check(_lib.zha_profile_enable(1 if on else 0), "zha_profile_enable")


def profile_read(max_kernels: int = 64) -> dict:
    """{kernel name: (total ms, launches)} of the launches recorded since the last read."""
    names = ctypes.create_string_buffer(8192)
    ms = (ctypes.c_double * max_kernels)()
    ln = (ctypes.c_int64 * max_kernels)()
    n = _lib.zha_profile_read(names, 8192, ms, ln, max_kernels)
    if n < 0:
        raise ZhaError(4, "zha_profile_read")
    keys = names.value.decode().split("\n")[:n]
    return {k: (ms[i], ln[i]) for i, k in enumerate(keys)}


class DecodeGraph:
    """zha_decode captured once into a CUDA graph and replayed per step.

    Every pointer, grid size and p is fixed at capture; the cache lengths live
    on the device, so one graph serves every later step. Inputs are copied into
    the graph's own q / k_new / v_new buffers before each replay. With `rot` (a
    Rotary) q and k_new are given before rotation: staging them turns them to
    the new token's position, lens[b]."""

    def __init__(self, cfg, buf, K, V, refs, lens, p, rot=None):
        B, Hq, Hkv, d = cfg.batch, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim
        dt = cfg.torch_dtype
        dev = K.device
        self.rot, self.lens = rot, lens
        self.q = torch.zeros((B, Hq, d), dtype=dt, device=dev)
        self.k_new = torch.zeros((B, Hkv, d), dtype=dt, device=dev)
        self.v_new = torch.zeros((B, Hkv, d), dtype=dt, device=dev)
        self.out = torch.zeros((B, Hq, d), dtype=dt, device=dev)
        # one ordinary (state-free) launch first, so per-device kernel attributes
        # are set outside the capture
        dense_decode(cfg, self.q, K, V, lens, self.out, buf.workspace, buf.status)
        before = launch_count()
        self.graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(self.graph):
            decode(cfg, buf.tree, K, V, refs, lens, self.q, self.k_new, self.v_new, p, buf.sel, self.out,
                   buf.workspace, buf.status)
        self.kernels_per_step = launch_count() - before

    def stage(self, q, k_new, v_new):
        """Put a step's inputs into the graph's own buffers (one multi-tensor
        copy, or the rotation and a copy of v_new); a caller that produces them
        there directly skips this."""
        if self.rot is not None:
            rotary(self.rot, q, k_new, self.lens, self.q, self.k_new)
            self.v_new.copy_(v_new, non_blocking=True)
            return
        torch._foreach_copy_([self.q, self.k_new, self.v_new], [q, k_new, v_new], non_blocking=True)

    def replay(self):
        """One decode step on the inputs in the graph's buffers."""
        self.graph.replay()
        return self.out

    def step(self, q, k_new, v_new):
        self.stage(q, k_new, v_new)
        return self.replay()


class Buffers:
    """Device buffers one configuration needs: tree, workspace, selection, status."""

    def __init__(self, cfg: Config, device="cuda", level_kept: bool = True):
        self.cfg = cfg
        cap1 = max(level_nodes(cfg, cfg.max_len, 1), 1)
        G = cfg.n_kv_heads * cfg.batch
        self.tree = torch.empty(tree_bytes(cfg), dtype=torch.uint8, device=device)
        self.workspace = torch.zeros(workspace_bytes(cfg), dtype=torch.uint8, device=device)
        self.sel = {
            "leaf_idx": torch.zeros((cfg.batch, cfg.n_kv_heads, cap1), dtype=torch.int32, device=device),
            "head_mask": torch.zeros((cfg.batch, cfg.n_kv_heads, cap1), dtype=torch.int32, device=device),
            "count": torch.zeros((cfg.batch, cfg.n_kv_heads), dtype=torch.int32, device=device),
            # [B, Hq, L] for single queries; a block call writes [B, Hkv, T, G, L]
            "level_kept": (torch.zeros((cfg.batch, cfg.n_q_heads * max(cfg.queries, 1), cfg.levels),
                                       dtype=torch.int32, device=device) if level_kept else None),
        }
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        del G

    def check_status(self, where="device"):
        code = int(self.status.item())
        if code:
            self.status.zero_()
            raise ZhaError(code, where)

    # views of the tree buffer (for inspection and tests)
    def tree_level(self, level: int):
        """(mu, bias) views of one level; with MX-FP8 summaries mu is the E4M3
        byte array and tree_level_scales() gives the block scales."""
        cfg = self.cfg
        mu_off, b_off = tree_level_offsets(cfg, level)
        cap = level_nodes(cfg, cfg.max_len, level)
        shape = (cfg.batch, cfg.n_kv_heads, cap, cfg.n_refs, cfg.head_dim)
        n_mu = cfg.batch * cfg.n_kv_heads * cap * cfg.n_refs * cfg.head_dim
        if cfg.summary == ZHA_SUMMARY_MXFP8:
            mu = self.tree[mu_off:mu_off + n_mu].view(*shape)
        else:
            es = 2 if cfg.dtype == ZHA_BF16 else 4
            mu = self.tree[mu_off:mu_off + n_mu * es].view(cfg.torch_dtype).view(*shape)
        n_b = cfg.batch * cfg.n_kv_heads * cap * cfg.n_refs
        bias = self.tree[b_off:b_off + n_b * 4].view(torch.float32).view(cfg.batch, cfg.n_kv_heads, cap, cfg.n_refs)
        return mu, bias

    def tree_level_scales(self, level: int):
        """Block-scale bytes [B, Hkv, cap, R, d/32] of an MX-FP8 level (2^(byte-127))."""
        cfg = self.cfg
        off = ctypes.c_size_t()
        check(_lib.zha_tree_level_scales(ctypes.byref(cfg), level, ctypes.byref(off)), "zha_tree_level_scales")
        cap = level_nodes(cfg, cfg.max_len, level)
        n = cfg.batch * cfg.n_kv_heads * cap * cfg.n_refs * (cfg.head_dim // 32)
        return self.tree[off.value:off.value + n].view(cfg.batch, cfg.n_kv_heads, cap, cfg.n_refs,
                                                        cfg.head_dim // 32)

    def tree_level_logmass(self, level: int):
        """Log-masses F [B, Hkv, cap, R] of one level (each plane's log attention
        mass at its own reference)."""
        cfg = self.cfg
        off = ctypes.c_size_t()
        check(_lib.zha_tree_level_logmass(ctypes.byref(cfg), level, ctypes.byref(off)), "zha_tree_level_logmass")
        cap = level_nodes(cfg, cfg.max_len, level)
        n = cfg.batch * cfg.n_kv_heads * cap * cfg.n_refs
        return self.tree[off.value:off.value + n * 4].view(torch.float32).view(cfg.batch, cfg.n_kv_heads, cap,
                                                                               cfg.n_refs)

    def level_state(self, level: int, T: int = 1):
        """Routing state of one level from the last route/decode call (T: query
        positions of the last decode_block call; its rows are t * G + head)."""
        cfg = self.cfg
        v = workspace_level_view(cfg, level, T)
        cap = v.cap
        BG = cfg.batch * cfg.n_kv_heads
        G = cfg.group * T
        ws = self.workspace

        def arr(off, n, dt):
            return ws[off:off + n * 4].view(dt)

        return {
            "cap": cap,
            "cand_idx": arr(v.cand_idx, BG * cap, torch.int32).view(cfg.batch, cfg.n_kv_heads, cap),
            "cand_mask": arr(v.cand_mask, BG * cap, torch.int32).view(cfg.batch, cfg.n_kv_heads, cap),
            "scores": arr(v.scores, BG * G * cap, torch.float32).view(cfg.batch, cfg.n_kv_heads, G, cap),
            "kept_mask": arr(v.kept_mask, BG * cap, torch.int32).view(cfg.batch, cfg.n_kv_heads, cap),
            "count": arr(v.count, BG, torch.int32).view(cfg.batch, cfg.n_kv_heads),
        }
