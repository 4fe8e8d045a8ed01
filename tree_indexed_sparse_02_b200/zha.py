"""Thin Python binding of libzha's C ABI (``include/zha.h``).

Argument marshalling only: every function forwards device pointers of torch
tensors and a CUDA stream to the library, and raises ``ZhaError`` on a
non-zero status. Nothing here computes any step of the method; if libzha.so
is missing the import fails loudly, and without _bind.so, the marshalling of
the paged and rotary calls, those calls do (there is no fallback path).
"""
from __future__ import annotations

import copy
import ctypes
import os

import torch

from .build import bind_key

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

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == ZHA_BF16 else torch.float32


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
        "zha_paged_write_check": ([PP, RP, i32, P, i64, P, i64, P, i64, P, P, P, P, P], i32),
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
        check(_lib.zha_paged_check_config(ctypes.byref(cfg)), "zha_paged_check_config")
        raise ZhaError(1 if rows < 1 else 2, "zha_paged_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


class Rotary:
    """A rotary embedding: its frequency table (turns per position, fp64) on the device.

    layout "half" pairs coordinates (i, i + rotary_dim/2), "interleaved" (2i, 2i + 1); scaling "none",
    "linear", "ntk" or "yarn" by `factor` (from a context of original_len for YaRN). Another table is put into `freq`
    in place (rotary_dim / 2 turns per position; desc.mscale for another factor of the values)."""

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
        self.device = self.freq.get_device()

    @property
    def address(self):
        return ctypes.addressof(self.desc)

    def __deepcopy__(self, memo):
        twin = copy.copy(self)
        twin.freq = self.freq.clone()
        d = self.desc
        twin.desc = RotaryDesc(d.rotary_dim, d.layout, d.mscale, 0, twin.freq.data_ptr())
        return twin


# The calls below check their arguments (tensors' type, shape, layout, device: ValueError; PagedConfig and Rotary:
# TypeError) and pass them on in csrc/zha_bind.cpp: on the GPU they can take less time than Python takes to look at
# the tensors' attributes.
# Where that module cannot be loaded, they raise; the calls of the sparse path need ctypes alone.

class _NoBind:
    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"_bind.so {self._why}; run tree_indexed_sparse_02_b200/build.py")


def _load_bind():
    try:
        from . import _bind
    except ImportError as e:
        return _NoBind(f"not built or not loadable ({e})")
    if getattr(_bind, "built_for", None) != bind_key():
        return _NoBind(f"was built for {getattr(_bind, 'built_for', 'another version')}, this is {bind_key()}")
    _bind.init(*(ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value
                 for name in ("zha_rotary_apply", "zha_paged_plan", "zha_paged_write", "zha_paged_decode",
                              "zha_paged_workspace_bytes", "zha_paged_write_check")), PagedConfig, Rotary)
    return _bind


_bind = _load_bind()


def rotary(rot: Rotary, q, k, positions, q_out=None, k_out=None, transpose=False, stream=None):
    """Rotate q [n, Hq, d] and k [n, Hk, d] (either may be None; tokens may be strided) at int32 positions [n].
    The outputs default to the inputs (in place); transpose applies the gradient's map. Returns (q_out, k_out).
    Nothing is recorded for autograd (as in every call here): a backward pass calls this with transpose."""
    code = _bind.rotary(rot, q, k, positions, q_out, k_out, transpose,
                        None if stream is None else stream.cuda_stream)
    if code:
        raise ZhaError(code, "zha_rotary_apply")
    return q if q_out is None else q_out, k if k_out is None else k_out


def paged_plan(cfg: PagedConfig, table, lens, n_new, free_pages, n_free, token_map, lens_out=None, n_free_out=None,
               dev_status=None, stream=None):
    """Block tables, slots and lengths of a step with n_new[b] new tokens of sequence b (< 0: it ends).
    token_map: {"positions", "slots", "seq_ids"} (one entry per row of the token buffer) and "cu" [batch + 1];
    lens_out and n_free_out default to lens and n_free (in place)."""
    m = token_map
    code = _bind.paged_plan(cfg, table, lens, n_new, free_pages, n_free, m["positions"], m["slots"], m["seq_ids"],
                            m["cu"], lens_out, n_free_out, dev_status, None if stream is None else stream.cuda_stream)
    if code:
        raise ZhaError(code, "zha_paged_plan")


def paged_write(cfg: PagedConfig, rot, q, k_new, v_new, positions, slots, q_out, k_pool, v_pool, dev_status=None,
                stream=None):
    """Rotate q and k_new [n, heads, d] and write k_new, v_new to their cache slots [n] (negative: skipped).
    rot None: no rotation; q None: keys and values only."""
    code = _bind.paged_write(cfg, rot, q, k_new, v_new, positions, slots, q_out, k_pool, v_pool, dev_status,
                             None if stream is None else stream.cuda_stream, False)
    if code:
        raise ZhaError(code, "zha_paged_write")
    return q_out


def paged_write_check(cfg: PagedConfig, rot, q, k_new, v_new, positions, slots, q_out, k_pool, v_pool, dev_status=None):
    """Raise what paged_write raises for these arguments; nothing is launched."""
    code = _bind.paged_write(cfg, rot, q, k_new, v_new, positions, slots, q_out, k_pool, v_pool, dev_status, None, True)
    if code:
        raise ZhaError(code, "zha_paged_write")


def paged_decode(cfg: PagedConfig, q, k_pool, v_pool, table, lens, out, workspace, lse=None, seq_ids=None,
                 positions=None, dev_status=None, stream=None):
    """Attention of rows q [n, Hq, d] over the paged cache into out (and lse [n, Hq] fp32). Row r is of sequence
    seq_ids[r] (default r; negative: left as it is) and attends tokens 0 .. positions[r] (default: all)."""
    code = _bind.paged_decode(cfg, q, k_pool, v_pool, table, lens, out, workspace, lse, seq_ids, positions,
                              dev_status, None if stream is None else stream.cuda_stream)
    if code:
        raise ZhaError(code, "zha_paged_decode")
    return out


class PagedCache:
    """Device state of one layer's paged cache: pools, block table, lengths, free pages, a step's token map and
    buffers, status. max_tokens is the size of a step's token buffer: q, k_new and v_new always have that many rows,
    and a step of fewer tokens leaves the last ones unused.

    step() runs plan, write and decode; everything stays on the device, so a step can be captured into a CUDA
    graph (n_new, q, k_new, v_new are then the captured buffers). The cache serves one step at a time."""

    def __init__(self, cfg: PagedConfig, max_tokens: int, rot: Rotary | None = None, device="cuda"):
        self.cfg, self.rot = cfg, rot
        kw = dict(dtype=torch.int32, device=device)
        # what no step's attention or write would take is refused here (16: an address that the check does not read)
        self.workspace = paged_workspace(cfg, max_tokens, device)
        check(_lib.zha_paged_write_check(ctypes.byref(cfg), None if rot is None else ctypes.byref(rot.desc), max_tokens,
                                         *[16, 0] * 3, *[16] * 5), "zha_paged_write")
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
        """q [max_tokens, Hq, d], k_new, v_new [max_tokens, Hkv, d]: the step's token rows, before rotation.

        Returns the cache's own out [max_tokens, Hq, d] and lse [max_tokens, Hq]. Rows that belong to no token, or to a
        sequence that was not served (pages or table full: check_status raises ZHA_ERR_CAPACITY), keep what an
        earlier step left in them. A step whose arguments are refused changes nothing: they are checked before the
        plan moves lengths and pages."""
        if q is None:
            raise ValueError("PagedCache.step: q must be a tensor (write() puts keys and values alone)")
        m = self.token_map
        paged_write_check(self.cfg, self.rot, q, k_new, v_new, m["positions"], m["slots"], self.q, self.k_pool, self.v_pool,
                          self.status)
        self.plan(n_new, stream)
        self.write(q, k_new, v_new, stream)
        return self.attend(stream)

    def check_status(self, where="device"):
        """Raise what steps of the current stream have set since the last look. The workspace is cleared then: a call
        that gave up on a wait leaves counters in it, and a status that was set before hides that."""
        code = int(self.status.item())
        if code:
            on_gpu = self.status.is_cuda
            if on_gpu:
                torch.cuda.synchronize(self.status.device)
            self.status.zero_()
            self.workspace.zero_()
            if on_gpu:                                       # before a step on any stream
                torch.cuda.synchronize(self.status.device)
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
        copy, or the rotation, of q and k_new on the device, and a copy of v_new);
        a caller that produces them there directly skips this."""
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
