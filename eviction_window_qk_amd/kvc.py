"""Thin Python binding over libkvc (include/kvc.h): argument marshalling only.

Every step of the event runs in the HIP library; this module checks tensor
dtypes, devices, shapes and contiguity, passes raw device pointers and the
current HIP stream, and turns status codes into exceptions.  PyTorch is used
for device memory and streams only.  There is no fallback: if the library is
missing or fails to load, every call raises.

Tensor conventions (see include/kvc.h for the full layouts):
  bf16 data     torch.bfloat16 (or torch.uint16 / torch.int16 bit views)
  u64 credit    torch.int64 holding the unsigned bit pattern
  i32 indices   torch.int32
  8-bit codes   torch.float8_e4m3fn or torch.int8 (the dtype is the format)
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from dataclasses import dataclass, fields

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvc.so")

OK, NOOP = 0, 1
ESCRATCH = -6
NOALLOC_SCRATCH_BYTES = 64 << 20   # KVC_NOALLOC_SCRATCH_BYTES
POOL_AVG, POOL_MAX = 0, 1
AGG_SUM, AGG_MAX = 0, 1
QUOTA_MASS, QUOTA_UNIFORM = 0, 1
Q8_E4M3, Q8_INT8 = 0, 1


class KvcError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn}: status {status}: {strerror(status)}")


class _CParams(ctypes.Structure):
    _fields_ = [
        ("n_heads", ctypes.c_int32), ("group", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("T", ctypes.c_int32), ("t_stride", ctypes.c_int32), ("window", ctypes.c_int32),
        ("budget", ctypes.c_int32), ("seg_min", ctypes.c_int32), ("seg_max", ctypes.c_int32),
        ("q_min", ctypes.c_int32), ("sinks", ctypes.c_int32), ("recent", ctypes.c_int32),
        ("pool_kernel", ctypes.c_int32), ("pool_mode", ctypes.c_int32),
        ("head_agg", ctypes.c_int32), ("ema", ctypes.c_int32), ("n_prev", ctypes.c_int32),
        ("scale", ctypes.c_float), ("delta", ctypes.c_double), ("lambda_", ctypes.c_double),
        ("beta", ctypes.c_double), ("eps", ctypes.c_double),
        ("seg_fixed", ctypes.c_int32), ("quota_mode", ctypes.c_int32),
        ("valid_len", ctypes.c_void_p),
    ]


class _CQ8Cache(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32), ("table_blocks", ctypes.c_int32),
        ("max_len", ctypes.c_int32), ("format", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("n_blocks", ctypes.c_int64),
        ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
    ]


class _CPageTable(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("table_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32), ("n_blocks", ctypes.c_int32),
        ("table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p), ("refs", ctypes.c_void_p),
    ]


class _CPageBuffer(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64)]


class _CPagedCache(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32), ("table_blocks", ctypes.c_int32),
        ("max_len", ctypes.c_int32), ("n_blocks", ctypes.c_int64),
        ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("table", ctypes.c_void_p),
        ("seq_len", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("pos", ctypes.c_void_p),
    ]


class _CRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _CRopePlan(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


@dataclass
class Params:
    """Mirror of kvc_params (names follow the pages' quantities)."""
    n_heads: int
    T: int
    window: int
    budget: int
    group: int = 1
    head_dim: int = 128
    t_stride: int = 0          # 0 => T
    delta: float = 0.1
    seg_min: int = 16
    seg_max: int = 256
    q_min: int = 1
    sinks: int = 4
    recent: int = 64
    pool_kernel: int = 7
    pool_mode: int = POOL_AVG
    head_agg: int = AGG_SUM
    ema: bool = False
    lam: float = 0.9
    beta: float = 0.9
    eps: float = 1e-6
    n_prev: int = 0
    scale: float = 0.0
    seg_fixed: int = 0         # ablation: > 0 => fixed-length raw segments
    quota_mode: int = QUOTA_MASS
    valid_len: object = None   # None or int32 device tensor [n_heads] (left padding)

    @classmethod
    def from_dict(cls, d: dict, **over) -> "Params":
        names = {f.name for f in fields(cls)}
        kw = {k: v for k, v in {**d, **over}.items() if k in names}
        return cls(**kw)

    def to_c(self) -> _CParams:
        c = _CParams()
        for f in fields(self):
            v = getattr(self, f.name)
            if f.name == "lam":
                c.lambda_ = float(v)
            elif f.name == "t_stride":
                c.t_stride = int(v) if v else int(self.T)
            elif f.name == "ema":
                c.ema = 1 if v else 0
            elif f.name == "valid_len":
                c.valid_len = None if v is None else _ptr(v, (torch.int32,), (self.n_heads,),
                                                          "valid_len")
            elif f.name in ("delta", "beta", "eps", "scale"):
                setattr(c, f.name, float(v))
            else:
                setattr(c, f.name, int(v))
        return c

    @property
    def stride(self) -> int:
        return self.t_stride or self.T


# The struct layouts and entry-point signatures this binding marshals
# (KVC_ABI_VERSION in include/kvc.h); a library of another version is refused, and
# one of this version that lacks an entry point added since it was built.
ABI_VERSION = 3

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it is missing (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libkvc.so not found at {LIB_PATH}: build it with "
                           "`python -m eviction_window_qk_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(_CParams)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    sig = {
        "kvc_score_window": [P, vp, vp, vp, vp, sz, vp],
        "kvc_mass_segment": [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "kvc_select": [P, vp, vp, vp, vp, vp, vp, sz, vp],
        "kvc_gather_compact": [P, vp, vp, vp, vp, vp, vp, vp, vp],
        "kvc_gather_paged": [P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, vp, vp, vp, vp,
                             ctypes.c_int32, vp, ctypes.c_int32, vp, vp, vp, vp, vp],
        "kvc_compress_event": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "kvc_compress_event_noalloc": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
        "kvc_qc_trigger": [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp,
                           ctypes.c_double, ctypes.c_int32, vp, vp, vp],
        "kvc_partial_init": [P, vp, vp, vp, vp, vp],
        "kvc_partial_append": [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp,
                               vp, vp, ctypes.c_int32, vp, vp],
        "kvc_full_sync": [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp, vp,
                          ctypes.c_int32, ctypes.c_int32, vp, vp, vp],
        "kvc_q8_store": [vp, ctypes.c_int32, ctypes.c_int32, vp, ctypes.c_int32, vp, vp, vp],
        "kvc_q8_load": [vp, ctypes.c_int32, ctypes.c_int32, vp, vp, vp],
        "kvc_q8_append": [vp, ctypes.c_int32, vp, vp, vp, vp],
        "kvc_q8_attend": [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_float, vp, vp, vp, vp, sz,
                          vp],
        "kvc_q8_attend_workspace_bytes": [vp, ctypes.c_int32, ctypes.c_int32],
        "kvc_pages_alloc": [vp, vp, vp, vp, sz, vp],
        "kvc_pages_fork": [vp, ctypes.c_int32, vp, vp, vp, ctypes.c_int32, vp, vp, sz, vp],
        "kvc_pages_free": [vp, ctypes.c_int32, vp, vp],
        "kvc_pages_copy": [ctypes.c_int32, ctypes.c_int32, vp, vp, vp, ctypes.c_int32, vp],
        "kvc_pages_compact": [vp, vp, ctypes.c_int32, vp, vp, vp, vp, vp, sz, vp],
        "kvc_pages_workspace_bytes": [vp, ctypes.c_int32],
        "kvc_pages_trim": [vp, vp],
        "kvc_rope": [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, ctypes.c_int32, vp, vp, vp,
                     vp],
        "kvc_paged_append": [vp, ctypes.c_int32, vp, vp, vp, ctypes.c_int32, vp, vp, vp, vp, vp],
        "kvc_paged_attend": [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp,
                             ctypes.c_float, vp, vp, vp, vp, sz, vp],
        "kvc_paged_attend_workspace_bytes": [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32],
        "kvc_prompt_attend": [ctypes.c_int32] * 5 + [vp, ctypes.c_float, vp, vp, vp, vp, vp, vp],
        "kvc_paged_evict": [vp, vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, sz, vp],
        "kvc_paged_evict_workspace_bytes": [vp, ctypes.c_int32],
        "kvc_workspace_bytes": [P],
        "kvc_segment_capacity": [P],
        "kvc_check_params": [P],
        "kvc_strerror": [ctypes.c_int],
        "kvc_abi_version": [],
    }
    rebuild = "rebuild with `python -m eviction_window_qk_amd.build`"
    for name in ("kvc_abi_version", *sig):
        if not hasattr(L, name):
            raise RuntimeError(f"{LIB_PATH} has no {name}: {rebuild}")
        fn = getattr(L, name)
        fn.argtypes = sig[name]
        fn.restype = ctypes.c_int
        if name == "kvc_abi_version" and fn() != ABI_VERSION:   # before any other name
            raise RuntimeError(f"{LIB_PATH} has ABI version {fn()}, this binding expects "
                               f"{ABI_VERSION}: {rebuild}")
    for name in ("kvc_workspace_bytes", "kvc_q8_attend_workspace_bytes",
                 "kvc_pages_workspace_bytes", "kvc_paged_attend_workspace_bytes",
                 "kvc_paged_evict_workspace_bytes"):
        getattr(L, name).restype = ctypes.c_size_t
    L.kvc_strerror.restype = ctypes.c_char_p
    _lib = L
    return L


def strerror(status: int) -> str:
    return lib().kvc_strerror(status).decode()


def abi_version() -> int:
    return lib().kvc_abi_version()


def check_params(p: Params) -> int:
    c = p.to_c()
    return lib().kvc_check_params(ctypes.byref(c))


def workspace_bytes(p: Params) -> int:
    c = p.to_c()
    return int(lib().kvc_workspace_bytes(ctypes.byref(c)))


def segment_capacity(p: Params) -> int:
    c = p.to_c()
    rc = lib().kvc_segment_capacity(ctypes.byref(c))
    if rc < 0:
        raise KvcError(rc, "kvc_segment_capacity")
    return rc


# ---------------------------------------------------------------------------
# tensor plumbing
# ---------------------------------------------------------------------------

_BF16_LIKE = (torch.bfloat16, torch.uint16, torch.int16)


def _ptr(t, dtypes, shape, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a GPU tensor, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, fn: str) -> int:
    if rc < 0:
        raise KvcError(rc, fn)
    return rc


def _device(*ts):
    for t in ts:
        if isinstance(t, torch.Tensor):
            return t.device
    raise ValueError("no tensor argument")


def new_workspace(p: Params, device) -> torch.Tensor:
    n = workspace_bytes(p)
    if n == 0:
        raise KvcError(_check_params_rc(p), "kvc_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _check_params_rc(p: Params) -> int:
    rc = check_params(p)
    return rc if rc < 0 else -1


def _ws(p, ws, device):
    if ws is None:
        ws = new_workspace(p, device)
    if ws.dtype != torch.uint8 or ws.device.type != "cuda" or not ws.is_contiguous():
        raise ValueError("workspace: contiguous uint8 GPU tensor expected")
    return ws


def score_window(p: Params, q, k, u=None, ws=None, stream=None):
    """Step 1.  q [NH,G,W,d] bf16, k [NH,t_stride,d] bf16 -> u [NH,T] fp32."""
    dev = _device(q, k)
    if u is None:
        u = torch.empty((p.n_heads, p.T), dtype=torch.float32, device=dev)
    ws = _ws(p, ws, dev)
    c = p.to_c()
    rc = lib().kvc_score_window(
        ctypes.byref(c),
        _ptr(q, _BF16_LIKE, (p.n_heads, p.group, p.window, p.head_dim), "q_win"),
        _ptr(k, _BF16_LIKE, (p.n_heads, p.stride, p.head_dim), "k"),
        _ptr(u, (torch.float32,), (p.n_heads, p.T), "u"), ws.data_ptr(), ws.numel(),
        _stream(stream))
    _check(rc, "kvc_score_window")
    return u


def mass_segment(p: Params, u, credit_in=None, ws=None, stream=None, out=None):
    """Steps 2-3.  Returns dict(score, credit_upd, seg_start, seg_quota, n_seg, status)."""
    dev = _device(u)
    S = segment_capacity(p)
    o = dict(out or {})
    o.setdefault("score", torch.empty((p.n_heads, p.T), dtype=torch.float32, device=dev))
    if p.ema:
        o.setdefault("credit_upd", torch.empty((p.n_heads, p.T), dtype=torch.int64, device=dev))
    o.setdefault("seg_start", torch.empty((p.n_heads, S), dtype=torch.int32, device=dev))
    o.setdefault("seg_quota", torch.empty((p.n_heads, S), dtype=torch.int32, device=dev))
    o.setdefault("n_seg", torch.empty((p.n_heads,), dtype=torch.int32, device=dev))
    ws = _ws(p, ws, dev)
    c = p.to_c()
    rc = lib().kvc_mass_segment(
        ctypes.byref(c), _ptr(u, (torch.float32,), (p.n_heads, p.T), "u"),
        _ptr(credit_in, (torch.int64,), (p.n_heads, p.n_prev), "credit_in"),
        _ptr(o["score"], (torch.float32,), (p.n_heads, p.T), "score"),
        _ptr(o.get("credit_upd"), (torch.int64,), (p.n_heads, p.T), "credit_upd"),
        _ptr(o["seg_start"], (torch.int32,), (p.n_heads, S), "seg_start"),
        _ptr(o["seg_quota"], (torch.int32,), (p.n_heads, S), "seg_quota"),
        _ptr(o["n_seg"], (torch.int32,), (p.n_heads,), "n_seg"), ws.data_ptr(), ws.numel(),
        _stream(stream))
    o["status"] = _check(rc, "kvc_mass_segment")
    return o


def select(p: Params, score, seg_start, seg_quota, n_seg, kept=None, ws=None, stream=None):
    """Step 4.  Returns kept [NH, budget] int32 (ascending, -1 padded)."""
    dev = _device(score)
    S = segment_capacity(p)
    if kept is None:
        kept = torch.empty((p.n_heads, p.budget), dtype=torch.int32, device=dev)
    ws = _ws(p, ws, dev)
    c = p.to_c()
    rc = lib().kvc_select(
        ctypes.byref(c), _ptr(score, (torch.float32,), (p.n_heads, p.T), "score"),
        _ptr(seg_start, (torch.int32,), (p.n_heads, S), "seg_start"),
        _ptr(seg_quota, (torch.int32,), (p.n_heads, S), "seg_quota"),
        _ptr(n_seg, (torch.int32,), (p.n_heads,), "n_seg"),
        _ptr(kept, (torch.int32,), (p.n_heads, p.budget), "kept"), ws.data_ptr(), ws.numel(),
        _stream(stream))
    _check(rc, "kvc_select")
    return kept


def gather_compact(p: Params, kept, k, v, credit_upd=None, k_out=None, v_out=None,
                   credit_out=None, stream=None):
    """Step 5.  Returns (k_out, v_out, credit_out)."""
    dev = _device(kept)
    shp = (p.n_heads, p.budget, p.head_dim)
    if k_out is None:
        k_out = torch.empty(shp, dtype=k.dtype, device=dev)
    if v_out is None:
        v_out = torch.empty(shp, dtype=v.dtype, device=dev)
    if credit_upd is not None and credit_out is None:
        credit_out = torch.empty((p.n_heads, p.budget), dtype=torch.int64, device=dev)
    c = p.to_c()
    rc = lib().kvc_gather_compact(
        ctypes.byref(c), _ptr(kept, (torch.int32,), (p.n_heads, p.budget), "kept"),
        _ptr(k, _BF16_LIKE, (p.n_heads, p.stride, p.head_dim), "k"),
        _ptr(v, _BF16_LIKE, (p.n_heads, p.stride, p.head_dim), "v"),
        _ptr(credit_upd, (torch.int64,), (p.n_heads, p.T), "credit_upd"),
        _ptr(k_out, _BF16_LIKE, shp, "k_out"), _ptr(v_out, _BF16_LIKE, shp, "v_out"),
        _ptr(credit_out, (torch.int64,), (p.n_heads, p.budget), "credit_out"), _stream(stream))
    _check(rc, "kvc_gather_compact")
    return k_out, v_out, credit_out


def gather_paged(p: Params, kept, k_pool, v_pool, table_in, table_out, kv_heads: int,
                 k_pool_out=None, v_pool_out=None, credit_upd=None, credit_out=None,
                 stream=None):
    """Step 5 on a paged cache: pools [n_blocks, kv_heads, block_size, d],
    tables int32 [B, blocks].  Writes the compacted rows into the blocks of
    table_out of k_pool_out / v_pool_out (default: the source pools
    themselves).  Returns (k_pool_out, v_pool_out, credit_out)."""
    dev = _device(kept)
    n_blocks, H, bs, d = k_pool.shape
    B = p.n_heads // kv_heads
    k_pool_out = k_pool if k_pool_out is None else k_pool_out
    v_pool_out = v_pool if v_pool_out is None else v_pool_out
    if credit_upd is not None and credit_out is None:
        credit_out = torch.empty((p.n_heads, p.budget), dtype=torch.int64, device=dev)
    pshape = (n_blocks, kv_heads, bs, p.head_dim)
    c = p.to_c()
    rc = lib().kvc_gather_paged(
        ctypes.byref(c), kv_heads, bs, n_blocks,
        _ptr(kept, (torch.int32,), (p.n_heads, p.budget), "kept"),
        _ptr(k_pool, _BF16_LIKE, pshape, "k_pool"), _ptr(v_pool, _BF16_LIKE, pshape, "v_pool"),
        _ptr(table_in, (torch.int32,), (B, table_in.shape[1]), "table_in"), table_in.shape[1],
        _ptr(table_out, (torch.int32,), (B, table_out.shape[1]), "table_out"),
        table_out.shape[1],
        _ptr(k_pool_out, _BF16_LIKE, pshape, "k_pool_out"),
        _ptr(v_pool_out, _BF16_LIKE, pshape, "v_pool_out"),
        _ptr(credit_upd, (torch.int64,), (p.n_heads, p.T), "credit_upd"),
        _ptr(credit_out, (torch.int64,), (p.n_heads, p.budget), "credit_out"), _stream(stream))
    _check(rc, "kvc_gather_paged")
    return k_pool_out, v_pool_out, credit_out


def compress_event(p: Params, q, k, v, credit_in=None, ws=None, out=None, want_u=False,
                   stream=None):
    """The whole event.  Returns dict(k_out, v_out, credit_out, kept, u, status)."""
    dev = _device(q, k, v)
    shp = (p.n_heads, p.budget, p.head_dim)
    o = dict(out or {})
    o.setdefault("k_out", torch.empty(shp, dtype=k.dtype, device=dev))
    o.setdefault("v_out", torch.empty(shp, dtype=v.dtype, device=dev))
    o.setdefault("kept", torch.empty((p.n_heads, p.budget), dtype=torch.int32, device=dev))
    if p.ema:
        o.setdefault("credit_out", torch.empty((p.n_heads, p.budget), dtype=torch.int64, device=dev))
    if want_u:
        o.setdefault("u", torch.empty((p.n_heads, p.T), dtype=torch.float32, device=dev))
    ws = _ws(p, ws, dev)
    c = p.to_c()
    rc = lib().kvc_compress_event(
        ctypes.byref(c),
        _ptr(q, _BF16_LIKE, (p.n_heads, p.group, p.window, p.head_dim), "q_win"),
        _ptr(k, _BF16_LIKE, (p.n_heads, p.stride, p.head_dim), "k"),
        _ptr(v, _BF16_LIKE, (p.n_heads, p.stride, p.head_dim), "v"),
        _ptr(credit_in, (torch.int64,), (p.n_heads, p.n_prev), "credit_in"),
        _ptr(o["k_out"], _BF16_LIKE, shp, "k_out"), _ptr(o["v_out"], _BF16_LIKE, shp, "v_out"),
        _ptr(o.get("credit_out"), (torch.int64,), (p.n_heads, p.budget), "credit_out"),
        _ptr(o["kept"], (torch.int32,), (p.n_heads, p.budget), "kept"),
        _ptr(o.get("u"), (torch.float32,), (p.n_heads, p.T), "u_out"), ws.data_ptr(),
        ws.numel(), _stream(stream))
    o["status"] = _check(rc, "kvc_compress_event")
    return o


def compress_event_noalloc(p: Params, q, k, v, credit_in=None, out=None, want_u=False,
                           stream=None):
    """The whole event through kvc_compress_event_noalloc (library-held scratch,
    no workspace).  Returns dict(k_out, v_out, credit_out, kept, u, status)."""
    dev = _device(q, k, v)
    shp = (p.n_heads, p.budget, p.head_dim)
    o = dict(out or {})
    o.setdefault("k_out", torch.empty(shp, dtype=k.dtype, device=dev))
    o.setdefault("v_out", torch.empty(shp, dtype=v.dtype, device=dev))
    o.setdefault("kept", torch.empty((p.n_heads, p.budget), dtype=torch.int32, device=dev))
    if p.ema:
        o.setdefault("credit_out", torch.empty((p.n_heads, p.budget), dtype=torch.int64, device=dev))
    if want_u:
        o.setdefault("u", torch.empty((p.n_heads, p.T), dtype=torch.float32, device=dev))
    c = p.to_c()
    rc = lib().kvc_compress_event_noalloc(
        ctypes.byref(c),
        _ptr(q, _BF16_LIKE, (p.n_heads, p.group, p.window, p.head_dim), "q_win"),
        _ptr(k, _BF16_LIKE, (p.n_heads, p.stride, p.head_dim), "k"),
        _ptr(v, _BF16_LIKE, (p.n_heads, p.stride, p.head_dim), "v"),
        _ptr(credit_in, (torch.int64,), (p.n_heads, p.n_prev), "credit_in"),
        _ptr(o["k_out"], _BF16_LIKE, shp, "k_out"), _ptr(o["v_out"], _BF16_LIKE, shp, "v_out"),
        _ptr(o.get("credit_out"), (torch.int64,), (p.n_heads, p.budget), "credit_out"),
        _ptr(o["kept"], (torch.int32,), (p.n_heads, p.budget), "kept"),
        _ptr(o.get("u"), (torch.float32,), (p.n_heads, p.T), "u_out"), _stream(stream))
    o["status"] = _check(rc, "kvc_compress_event_noalloc")
    return o


# ---------------------------------------------------------------------------
# RefreshKV decode-loop pieces (include/kvc.h documents each call)
# ---------------------------------------------------------------------------

def qc_trigger(q, q_ref, threshold: float, update_ref: bool = True, want_cos: bool = False,
               stream=None):
    """Query comparison: q bf16 [rows, Hq, d], q_ref float64 [rows, d] (updated in
    place where a row fires).  Returns full (int32 [rows]) or (full, cos)."""
    rows, Hq, d = q.shape
    dev = _device(q)
    full = torch.empty((rows,), dtype=torch.int32, device=dev)
    cos = torch.empty((rows,), dtype=torch.float64, device=dev) if want_cos else None
    rc = lib().kvc_qc_trigger(rows, Hq, d, _ptr(q, _BF16_LIKE, (rows, Hq, d), "q"),
                              _ptr(q_ref, (torch.float64,), (rows, d), "q_ref"), float(threshold),
                              1 if update_ref else 0, _ptr(full, (torch.int32,), (rows,), "full"),
                              _ptr(cos, (torch.float64,), (rows,), "cos"), _stream(stream))
    _check(rc, "kvc_qc_trigger")
    return (full, cos) if want_cos else full


def partial_init(p: Params, kept, score, stream=None):
    """C_p bookkeeping after a refresh.  Returns (part_score, part_pos)."""
    dev = _device(kept)
    ps = torch.empty((p.n_heads, p.budget), dtype=torch.float32, device=dev)
    pp = torch.empty((p.n_heads, p.budget), dtype=torch.int32, device=dev)
    c = p.to_c()
    rc = lib().kvc_partial_init(ctypes.byref(c),
                                _ptr(kept, (torch.int32,), (p.n_heads, p.budget), "kept"),
                                _ptr(score, (torch.float32,), (p.n_heads, p.T), "score"),
                                ps.data_ptr(), pp.data_ptr(), _stream(stream))
    _check(rc, "kvc_partial_init")
    return ps, pp


def partial_append(part_score, part_pos, k_part, v_part, k_new, v_new, t_new: int, stream=None):
    """One partial step for every head (in place).  Returns the evicted slots."""
    NH, K, d = k_part.shape
    dev = _device(k_part)
    ev = torch.empty((NH,), dtype=torch.int32, device=dev)
    rc = lib().kvc_partial_append(
        NH, K, d, _ptr(part_score, (torch.float32,), (NH, K), "part_score"),
        _ptr(part_pos, (torch.int32,), (NH, K), "part_pos"),
        _ptr(k_part, _BF16_LIKE, (NH, K, d), "k_part"), _ptr(v_part, _BF16_LIKE, (NH, K, d), "v_part"),
        _ptr(k_new, _BF16_LIKE, (NH, d), "k_new"), _ptr(v_new, _BF16_LIKE, (NH, d), "v_new"),
        int(t_new), ev.data_ptr(), _stream(stream))
    _check(rc, "kvc_partial_append")
    return ev


def full_sync(part_pos, k_part, v_part, k_full, v_full, t_from: int, stream=None):
    """Write the C_p entries decoded since t_from into the full cache (in place)."""
    NH, K, d = k_part.shape
    TS = k_full.shape[1]
    rc = lib().kvc_full_sync(
        NH, K, d, _ptr(part_pos, (torch.int32,), (NH, K), "part_pos"),
        _ptr(k_part, _BF16_LIKE, (NH, K, d), "k_part"), _ptr(v_part, _BF16_LIKE, (NH, K, d), "v_part"),
        int(t_from), TS, _ptr(k_full, _BF16_LIKE, (NH, TS, d), "k_full"),
        _ptr(v_full, _BF16_LIKE, (NH, TS, d), "v_full"), _stream(stream))
    _check(rc, "kvc_full_sync")


# ---------------------------------------------------------------------------
# 8-bit paged cache and page tables (include/kvc.h documents each call)
# ---------------------------------------------------------------------------

_Q8_FORMAT = {torch.float8_e4m3fn: Q8_E4M3, torch.int8: Q8_INT8}


def _here(device, stream):
    """Raw handle of the stream a call runs on, or None when the call has to be
    made again under `_there`: a stream was given, or another device is current.
    (torch.cuda.current_stream would build a Stream object: 3 us a call.)"""
    if stream is None and torch._C._cuda_getDevice() == device.index:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return None


def _there(device, stream):
    """Context in which the stream (or the device's current one) and its device are
    current, so that what a call allocates belongs to them."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    return torch.cuda.stream(stream)


def _at(t, dtypes, shape, device, name):
    """_ptr for a tensor that has to be on `device`."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape
            and t.device == device and t.is_contiguous() and device.type == "cuda"):
        return t.data_ptr()
    p = _ptr(t, dtypes, shape, name)
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    return p


_I32, _F32 = (torch.int32,), (torch.float32,)


def _int(x, name):
    """A C int32: ctypes would keep the low 32 bits of a larger one."""
    n = int(x)
    if n != x or not -0x80000000 <= n <= 0x7fffffff:
        raise ValueError(f"{name}: {x} is no 32-bit integer")
    return n


def _scratch(ws, n, device):
    """A call's workspace: the given one, or n new bytes of the current stream."""
    if ws is None:
        return torch.empty(n, dtype=torch.uint8, device=device) if n else None
    if ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace: contiguous uint8 tensor on {device} expected")
    return ws


def _new(like, n=None, dtype=None):
    """A new tensor beside a checked one: same shape and type, or those given."""
    t = torch.empty_like(like) if n is None else like.new_empty(n, dtype=dtype)
    return t, t.data_ptr()


def _given(t, dtypes, shape, device, name):
    return t, _at(t, dtypes, shape, device, name)


def _span(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel())


class _Handle:
    """A C structure over tensors that were checked when it was made: another
    tensor needs another handle."""

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name}: a handle keeps its tensors, copy into "
                                 "them or make a new one")
        super().__setattr__(name, value)


class Q8Cache(_Handle):
    """An 8-bit paged cache: k_pool, v_pool [n_blocks, kv_heads, block_size, d]
    (torch.float8_e4m3fn or torch.int8), k_scale, v_scale fp32 [n_blocks,
    kv_heads], table int32 [n_seqs, table_blocks], seq_len int32 [n_seqs].
    A handle that the calls below share: the tensors are checked once, here,
    and kept; change their contents freely, not the handle nor where they lie
    (resize_, set_).  max_len bounds
    seq_len (0: the table's room) and sizes the launches."""

    def __init__(self, k_pool, v_pool, k_scale, v_scale, table, seq_len, max_len: int = 0):
        max_len = _int(max_len, "max_len")
        if k_pool.dtype not in _Q8_FORMAT:
            raise TypeError(f"k_pool: dtype {k_pool.dtype} not in {tuple(_Q8_FORMAT)}")
        if k_pool.dim() != 4 or table.dim() != 2:
            raise ValueError("k_pool: 4 dimensions expected, table: 2")
        n, H, bs, d = k_pool.shape
        B, tb = table.shape
        dev, code = k_pool.device, (k_pool.dtype,)
        c = _CQ8Cache(n_seqs=B, kv_heads=H, head_dim=d, block_size=bs, table_blocks=tb,
                      max_len=max_len, format=_Q8_FORMAT[k_pool.dtype], reserved=0, n_blocks=n)
        c.k_pool = _at(k_pool, code, (n, H, bs, d), dev, "k_pool")
        c.v_pool = _at(v_pool, code, (n, H, bs, d), dev, "v_pool")
        c.k_scale = _at(k_scale, _F32, (n, H), dev, "k_scale")
        c.v_scale = _at(v_scale, _F32, (n, H), dev, "v_scale")
        c.table = _at(table, _I32, (B, tb), dev, "table")
        c.seq_len = _at(seq_len, _I32, (B,), dev, "seq_len")
        self.device = dev
        self.k_pool, self.v_pool, self.k_scale, self.v_scale = k_pool, v_pool, k_scale, v_scale
        self.table, self.seq_len = table, seq_len
        self.heads, self.head_dim = B * H, d
        self._c, self._ws, self._ref = c, {}, ctypes.addressof(c)

    def attend_workspace_bytes(self, group: int, window: int = 1) -> int:
        """Bytes q8_attend needs for `group` query heads and `window` queries."""
        n = self._ws.get((group, window))
        if n is None:
            n = int(lib().kvc_q8_attend_workspace_bytes(self._ref, _int(group, "group"),
                                                        _int(window, "window")))
            if n == ctypes.c_size_t(-1).value:
                raise KvcError(-4 if group > 64 else -1, "kvc_q8_attend_workspace_bytes")
            self._ws[(group, window)] = n
        return n


def q8_store(cache: Q8Cache, k, v, kept=None, T: int = 0, stream=None):
    """Writes rows of k, v (bf16 [heads, t_stride, d], T of them valid, 0 = all)
    into the cache's pages: the rows kept (int32 [heads, n_kept]), or the last
    seq_len.  Returns the cache."""
    dev = cache.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return q8_store(cache, k, v, kept, T)
    if k.dim() != 3 or (kept is not None and kept.dim() != 2):
        raise ValueError("k: 3 dimensions expected, kept: 2")
    shp = (cache.heads, k.shape[1], cache.head_dim)
    n_kept = 0 if kept is None else kept.shape[1]
    rc = lib().kvc_q8_store(cache._ref, _int(T, "T") or _int(shp[1], "t_stride"),
                            _int(shp[1], "t_stride"),
                            _at(kept, _I32, (cache.heads, n_kept), dev, "kept"),
                            _int(n_kept, "n_kept"),
                            _at(k, _BF16_LIKE, shp, dev, "k"), _at(v, _BF16_LIKE, shp, dev, "v"), s)
    _check(rc, "kvc_q8_store")
    return cache


def q8_load(cache: Q8Cache, T: int, k_out=None, v_out=None, want_v: bool = True, stream=None):
    """The last T positions as bf16 rows, left-padded with zeros: returns (k, v),
    [heads, t_stride >= T, d] (want_v false and v_out None: (k, None))."""
    dev = cache.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return q8_load(cache, T, k_out, v_out, want_v)
    T = _int(T, "T")
    rows = T if k_out is None and v_out is None else (v_out if k_out is None else k_out).shape[1]
    shp = (cache.heads, rows, cache.head_dim)
    k_out, k_ptr = (_new(cache.table, shp, torch.bfloat16) if k_out is None else
                    _given(k_out, _BF16_LIKE, shp, dev, "k_out"))
    v_out, v_ptr = (_new(k_out) if v_out is None and want_v else
                    _given(v_out, _BF16_LIKE, shp, dev, "v_out"))
    rc = lib().kvc_q8_load(cache._ref, T, _int(rows, "t_stride"), k_ptr, v_ptr, s)
    _check(rc, "kvc_q8_load")
    return k_out, v_out


def q8_append(cache: Q8Cache, k_new, v_new, n_new=None, stream=None):
    """Appends k_new, v_new (bf16 [heads, window, d]) as the last `window`
    positions of every sequence (seq_len counts them already), or with n_new
    (int32 [n_seqs]) the last n_new rows of each only.  Returns the cache."""
    dev = cache.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return q8_append(cache, k_new, v_new, n_new)
    if k_new.dim() != 3:
        raise ValueError("k_new: 3 dimensions expected")
    shp = (cache.heads, k_new.shape[1], cache.head_dim)
    rc = lib().kvc_q8_append(cache._ref, _int(shp[1], "window"),
                             _at(n_new, _I32, cache.seq_len.shape, dev, "n_new"),
                             _at(k_new, _BF16_LIKE, shp, dev, "k_new"),
                             _at(v_new, _BF16_LIKE, shp, dev, "v_new"), s)
    _check(rc, "kvc_q8_append")
    return cache


def q8_attend(cache: Q8Cache, q, out=None, lse=None, want_lse: bool = False, scale: float = 0.0,
              ws=None, stream=None):
    """Attention of the last `window` positions' queries q (bf16 [heads, group,
    window, d]) over the cache, scores times scale (0: 1 / sqrt(d)).  Returns out
    (bf16, like q), or (out, lse) with want_lse or an lse tensor (fp32 [heads,
    group, window])."""
    dev = cache.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return q8_attend(cache, q, out, lse, want_lse, scale, ws)
    if q.dim() != 4:
        raise ValueError("q: 4 dimensions expected")
    if scale != 0.0 and abs(scale) < 2.0 ** -149:
        raise ValueError(f"scale: {scale} is zero in fp32, which stands for 1 / sqrt(d)")
    G, W = q.shape[1], q.shape[2]
    shp = (cache.heads, G, W, cache.head_dim)
    q_ptr = _at(q, _BF16_LIKE, shp, dev, "q")
    ws = _scratch(ws, cache.attend_workspace_bytes(G, W), dev)
    out, out_ptr = _new(q) if out is None else _given(out, _BF16_LIKE, shp, dev, "out")
    lse, lse_ptr = (_new(q, shp[:3], torch.float32) if lse is None and want_lse else
                    _given(lse, _F32, shp[:3], dev, "lse"))
    rc = lib().kvc_q8_attend(cache._ref, G, W, scale, q_ptr, out_ptr, lse_ptr,
                             *_span(ws), s)
    _check(rc, "kvc_q8_attend")
    return out if lse is None else (out, lse)


class PageTable(_Handle):
    """Who owns which page: table int32 [n_seqs, table_blocks], seq_len int32
    [n_seqs], refs int32 [n_blocks], pages of block_size positions.  A handle
    like Q8Cache."""

    def __init__(self, table, seq_len, refs, block_size: int):
        block_size = _int(block_size, "block_size")
        if table.dim() != 2 or refs.dim() != 1:
            raise ValueError("table: 2 dimensions expected, refs: 1")
        B, tb = table.shape
        dev = table.device
        c = _CPageTable(n_seqs=B, table_blocks=tb, block_size=block_size,
                        n_blocks=_int(refs.shape[0], "n_blocks"))
        c.table = _at(table, _I32, (B, tb), dev, "table")
        c.seq_len = _at(seq_len, _I32, (B,), dev, "seq_len")
        c.refs = _at(refs, _I32, (refs.shape[0],), dev, "refs")
        self.device = dev
        self.table, self.seq_len, self.refs = table, seq_len, refs
        self.block_size, self.n_blocks = block_size, refs.shape[0]
        self._c, self._ws, self._ref = c, {}, ctypes.addressof(c)

    def workspace_bytes(self, n_pairs: int = 0) -> int:
        """Bytes pages_alloc, pages_fork (n_pairs pairs) and pages_compact need."""
        n = self._ws.get(n_pairs)
        if n is None:
            n = int(lib().kvc_pages_workspace_bytes(self._ref, _int(n_pairs, "n_pairs")))
            if n == 0:
                raise KvcError(-1, "kvc_pages_workspace_bytes")
            self._ws[n_pairs] = n
        return n


class PageBuffers(_Handle):
    """Tensors indexed by page in their first dimension (pools, scales): what a
    page id stands for in every one of them."""

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        self._c = (_CPageBuffer * max(1, len(self.tensors)))()
        self.n_blocks = self.tensors[0].shape[0] if self.tensors else 0
        self.device = self.tensors[0].device if self.tensors else None
        for i, t in enumerate(self.tensors):
            shp = (self.n_blocks,) + tuple(t.shape[1:])
            self._c[i].base = _at(t, (t.dtype,), shp, self.device, f"buffer {i}")
            self._c[i].page_bytes = t[:1].numel() * t.element_size()
        self._ref = ctypes.addressof(self._c)

    def _for(self, n_blocks: int, device):
        if self.tensors and (self.n_blocks != n_blocks or self.device != device):
            raise ValueError(f"buffers of {self.n_blocks} pages on {self.device}, the table has "
                             f"{n_blocks} on {device}")
        return self._ref, len(self.tensors)


def pages_alloc(pages: PageTable, want_len, status=None, ws=None, stream=None):
    """Gives every sequence pages for want_len (int32 [n_seqs]) positions.
    Returns status (int32 [n_seqs]: 0 served, 1 no room, 2 refused)."""
    dev = pages.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return pages_alloc(pages, want_len, status, ws)
    shp = (pages.table.shape[0],)
    w_ptr = _at(want_len, _I32, shp, dev, "want_len")
    status, st_ptr = _new(want_len) if status is None else _given(status, _I32, shp, dev, "status")
    ws = _scratch(ws, pages.workspace_bytes(), dev)
    rc = lib().kvc_pages_alloc(pages._ref, w_ptr, st_ptr, *_span(ws), s)
    _check(rc, "kvc_pages_alloc")
    return status


def pages_fork(pages: PageTable, src, dst, bufs: PageBuffers, status=None, ws=None, stream=None):
    """Sequence dst[i] becomes a copy of src[i] (int32 [n_pairs]), its open page
    copied in `bufs`.  Returns status (int32 [n_pairs])."""
    dev = pages.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return pages_fork(pages, src, dst, bufs, status, ws)
    n = src.shape[0]
    ref, n_bufs = bufs._for(pages.n_blocks, dev)
    s_ptr, d_ptr = _at(src, _I32, (n,), dev, "src"), _at(dst, _I32, (n,), dev, "dst")
    status, st_ptr = _new(src) if status is None else _given(status, _I32, (n,), dev, "status")
    ws = _scratch(ws, pages.workspace_bytes(n), dev)
    rc = lib().kvc_pages_fork(pages._ref, n, s_ptr, d_ptr, ref, n_bufs, st_ptr, *_span(ws), s)
    _check(rc, "kvc_pages_fork")
    return status


def pages_free(pages: PageTable, ids, stream=None):
    """Frees the sequences ids (int32 [n])."""
    dev = pages.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return pages_free(pages, ids)
    n = _int(ids.shape[0], "ids")
    _check(lib().kvc_pages_free(pages._ref, n, _at(ids, _I32, (n,), dev, "ids"), s),
           "kvc_pages_free")


def pages_trim(pages: PageTable, stream=None):
    """Gives up the pages behind each sequence's length."""
    s = _here(pages.device, stream)
    if s is None:
        with _there(pages.device, stream):
            return pages_trim(pages)
    _check(lib().kvc_pages_trim(pages._ref, s), "kvc_pages_trim")


def pages_copy(src, dst, bufs: PageBuffers, stream=None):
    """Copies page src[i] to page dst[i] (int32 [n_pairs]) in every buffer."""
    dev = src.device
    if dev.type != "cuda":
        raise ValueError(f"src: must be a GPU tensor, got {dev}")
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return pages_copy(src, dst, bufs)
    n = _int(src.shape[0], "src")
    ref, n_bufs = bufs._for(bufs.n_blocks, dev)
    _check(lib().kvc_pages_copy(max(1, _int(bufs.n_blocks, "n_blocks")), n, _at(src, _I32, (n,), dev, "src"),
                                _at(dst, _I32, (n,), dev, "dst"), ref, n_bufs, s),
           "kvc_pages_copy")


def pages_compact(pages: PageTable, bufs: PageBuffers, out=None, ws=None, stream=None):
    """Moves the live pages to the front of every buffer.  Returns dict(table,
    refs, remap, n_live): new tensors (or those of `out`), the handle's own are
    left as they were."""
    dev = pages.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return pages_compact(pages, bufs, out, ws)
    ref, n_bufs = bufs._for(pages.n_blocks, dev)
    o, ptr, n = dict(out or {}), {}, (pages.n_blocks,)
    for name, like, shp in (("table", pages.table, pages.table.shape), ("refs", pages.refs, n),
                            ("remap", pages.refs, n), ("n_live", pages.refs, (1,))):
        t = o.get(name)
        o[name], ptr[name] = (_given(t, _I32, shp, dev, name) if t is not None else
                              _new(like) if name != "n_live" else _new(like, 1, torch.int32))
    ws = _scratch(ws, pages.workspace_bytes(), dev)
    rc = lib().kvc_pages_compact(pages._ref, ref, n_bufs, ptr["table"], ptr["refs"], ptr["remap"],
                                 ptr["n_live"], *_span(ws), s)
    _check(rc, "kvc_pages_compact")
    return o


# ---------------------------------------------------------------------------
# bf16 paged cache: rotation, append, attention, eviction (include/kvc.h documents
# each call)
# ---------------------------------------------------------------------------

_F64 = (torch.float64,)


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = None, factor: float = 1.0,
                     trained: int = 0, slow: float = 1.0, fast: float = 4.0):
    """Radians a position of the rot_dim / 2 pairs (fp64, CPU), base^(-2i / rot_dim),
    and the factor on the rotated values (mscale), stretched to `factor` times the
    `trained` positions:
      None      as they are
      "linear"  all divided by factor
      "ntk"     of the base times factor^(rot_dim / (rot_dim - 2)): the fastest pair
                keeps its frequency, the slowest is divided by factor
      "banded"  a pair that turns more than `fast` times in `trained` positions keeps
                its frequency, one that turns less than `slow` times is divided by factor, in
                between a blend, linear in the turns
      "yarn"    the same with a blend linear in the pair's index (between those that
                turn `fast` and `slow` times, rounded outwards; usually 32 and 1), and mscale
                0.1 ln(factor) + 1"""
    rot_dim = _int(rot_dim, "rot_dim")
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim: {rot_dim} is no positive even number")
    if not base > 1.0 or not factor >= 1.0 or math.isinf(base) or math.isinf(factor):
        raise ValueError(f"base {base} and factor {factor}: above 1, at least 1, finite")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot_dim == 2:
            raise ValueError("scaling ntk: needs more than one pair")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = base ** (-2.0 * i / rot_dim)
    if scaling in (None, "ntk"):
        return freq, 1.0
    if scaling == "linear":
        return freq / factor, 1.0
    if scaling not in ("banded", "yarn"):
        raise ValueError(f"scaling: {scaling!r} is none of None, linear, ntk, banded, yarn")
    if trained < 1 or not 0.0 < slow < fast:
        raise ValueError(f"scaling {scaling}: trained {trained} >= 1 and 0 < slow {slow} < fast {fast} expected")
    if scaling == "banded":
        keep = ((trained * freq / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        return freq * (keep + (1 - keep) / factor), 1.0
    pair = lambda turns: rot_dim * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    first, last = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot_dim - 1)
    gone = ((i - first) / max(last - first, 0.001)).clamp(0, 1)
    if pair(slow) < 0:                  # the fastest pair turns less than slow times already
        gone = torch.ones_like(i)
    return freq * (1 - gone + gone / factor), 0.1 * math.log(factor) + 1.0


class Rope(_Handle):
    """A rotation: freq fp64 [rot_dim / 2] on the GPU (rope_frequencies), pairs (i, i +
    rot_dim / 2) or, interleaved, (2i, 2i + 1), rotated values times mscale."""

    def __init__(self, freq, interleaved: bool = False, mscale: float = 1.0):
        if freq.dim() != 1:
            raise ValueError("freq: 1 dimension expected")
        c = _CRopePlan(rot_dim=_int(2 * freq.shape[0], "rot_dim"), interleaved=1 if interleaved else 0,
                       mscale=float(mscale), reserved=0)
        c.freq = _at(freq, _F64, (freq.shape[0],), freq.device, "freq")
        self.device, self.freq = freq.device, freq
        self._c, self._ref = c, ctypes.addressof(c)


def _rows(t, shape, device, name):
    """kvc_rows of a bf16 tensor [n_tokens, heads, d] on a GPU, any strides with whole rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not torch.bfloat16 and t.dtype not in _BF16_LIKE:
        raise TypeError(f"{name}: dtype {t.dtype} not in {_BF16_LIKE}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    ts, hs, one = t.stride()
    if one != 1 and t.numel():
        raise ValueError(f"{name}: rows must be contiguous")
    # a stride that no step is taken by may be anything
    return _pack_rows(t.data_ptr(), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0)


# A _CRows as bytes, in a third of the time a structure takes.
_pack_rows = struct.Struct("=Qqq").pack


def _new_rows(like, n, heads, d):
    """New contiguous rows beside checked ones, and their kvc_rows."""
    t = like.new_empty((n, heads, d))
    return t, _pack_rows(t.data_ptr(), heads * d, d)


def _count(n, name):
    """A dimension as a C int32 (expanded tensors may have more than memory holds)."""
    return n if n <= 0x7fffffff else _int(n, name)


class _Rotate(torch.autograd.Function):
    """The rotation of a tensor that requires a gradient: the other way round on its way back."""

    @staticmethod
    def forward(ctx, x, plan, positions, backward):
        ctx.plan, ctx.back = plan, backward
        ctx.save_for_backward(positions)
        return rope(plan, x, positions, backward=backward)

    @staticmethod
    def backward(ctx, g):
        g = g.contiguous()                       # of a sum it is one value, expanded
        g = g if g.data_ptr() % 16 == 0 else g.clone()
        return rope(ctx.plan, g, ctx.saved_tensors[0], backward=not ctx.back), None, None, None


def rope(plan: Rope, x, positions, y=None, backward: bool = False, stream=None):
    """Rotates x (bf16 [n_tokens, heads, d], rows contiguous) by positions (int32
    [n_tokens]) into y (None: a new tensor; x itself: in place).  backward: by the
    transposed map.  A new tensor of an x that requires a gradient passes it on; into a
    given y such an x is refused.  Returns y."""
    dev = plan.device
    if (x.requires_grad or (y is not None and y.requires_grad)) and torch.is_grad_enabled():
        if y is not None:
            raise ValueError("y: no gradient passes through a given tensor; leave it out, or use torch.no_grad()")
        with _there(dev, stream):
            return _Rotate.apply(x, plan, positions, bool(backward))
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return rope(plan, x, positions, y, backward)
    if x.dim() != 3:
        raise ValueError("x: 3 dimensions expected")
    n, heads, d = x.shape
    cx = _rows(x, (n, heads, d), dev, "x")
    p_ptr = _ints(positions, (n,), dev, "positions")
    if y is None:
        y, cy = _new_rows(x, n, heads, d)
    else:
        cy = cx if y is x else _rows(y, (n, heads, d), dev, "y")
    rc = lib().kvc_rope(_count(n, "n_tokens"), _count(heads, "heads"), _count(d, "head_dim"), plan._ref,
                        1 if backward else 0, p_ptr, cx, cy, s)
    _check(rc, "kvc_rope")
    return y


class PagedCache(_Handle):
    """A bf16 paged cache: k_pool, v_pool [n_blocks, kv_heads, block_size, d], table int32
    [n_seqs, table_blocks], seq_len int32 [n_seqs]; weight fp32 and pos int32 [n_seqs *
    kv_heads, table_blocks * block_size], both or neither: what the attention has
    given each slot, and the position it holds.  A handle like Q8Cache."""

    def __init__(self, k_pool, v_pool, table, seq_len, weight=None, pos=None, max_len: int = 0):
        max_len = _int(max_len, "max_len")
        if k_pool.dim() != 4 or table.dim() != 2:
            raise ValueError("k_pool: 4 dimensions expected, table: 2")
        if (weight is None) != (pos is None):
            raise ValueError("weight and pos: both or neither")
        n, H, bs, d = k_pool.shape
        B, tb = table.shape
        dev, slots = k_pool.device, (B * H, tb * bs)
        c = _CPagedCache(n_seqs=B, kv_heads=H, head_dim=d, block_size=bs, table_blocks=tb,
                         max_len=max_len, n_blocks=n)
        c.k_pool = _at(k_pool, _BF16_LIKE, (n, H, bs, d), dev, "k_pool")
        c.v_pool = _at(v_pool, _BF16_LIKE, (n, H, bs, d), dev, "v_pool")
        c.table = _at(table, _I32, (B, tb), dev, "table")
        c.seq_len = _at(seq_len, _I32, (B,), dev, "seq_len")
        c.weight = _at(weight, _F32, slots, dev, "weight")
        c.pos = _at(pos, _I32, slots, dev, "pos")
        self.device = dev
        self.k_pool, self.v_pool, self.table, self.seq_len = k_pool, v_pool, table, seq_len
        self.weight, self.pos = weight, pos
        self.kv_heads, self.head_dim, self._starts_shape = H, d, (B + 1,)
        self._c, self._ws, self._ref = c, {}, ctypes.addressof(c)

    def attend_workspace_bytes(self, group: int, n_tokens: int, max_new: int = 0) -> int:
        """Bytes paged_attend needs for n_tokens new tokens, max_new of a sequence at most."""
        key = (group, n_tokens, max_new)
        n = self._ws.get(key)
        if n is None:
            n = int(lib().kvc_paged_attend_workspace_bytes(
                self._ref, _int(group, "group"), _int(n_tokens, "n_tokens"), _int(max_new, "max_new")))
            if n == ctypes.c_size_t(-1).value:
                raise KvcError(-4 if group > 64 else -1, "kvc_paged_attend_workspace_bytes")
            if len(self._ws) > 4096:    # prompts bring ever new counts of tokens
                self._ws.clear()
            self._ws[key] = n
        return n

    def evict_workspace_bytes(self, budget: int) -> int:
        """Bytes paged_evict needs."""
        n = self._ws.get(budget)
        if n is None:
            n = int(lib().kvc_paged_evict_workspace_bytes(self._ref, _int(budget, "budget")))
            if n == 0:
                raise KvcError(-1, "kvc_paged_evict_workspace_bytes")
            self._ws[budget] = n
        return n


def _ints(t, shape, device, name):
    """_at for int32 tensors beside ones that are known to lie on a GPU."""
    if (t is not None and t.dtype is torch.int32 and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return t.data_ptr()
    return _at(t, _I32, shape, device, name)


def _group(q, kv_heads, name):
    if q.dim() != 3:
        raise ValueError(f"{name}: 3 dimensions expected")
    if kv_heads < 1 or q.shape[1] % kv_heads:
        raise ValueError(f"{name}: {q.shape[1]} heads are no multiple of {kv_heads}")
    return _int(q.shape[1] // kv_heads, "group")


def paged_append(cache: PagedCache, k, v, starts, positions=None, rope: Rope = None, q=None,
                 q_out=None, stream=None):
    """Writes k, v (bf16 [n_tokens, kv_heads, d], rows contiguous) of the new tokens, packed
    by sequence (starts int32 [n_seqs + 1]), into their slots, k rotated by `rope` at
    positions (int32 [n_tokens]; None: the slots).  q ([n_tokens, heads, d], with rope) is
    rotated into q_out (None: a new tensor; q itself: in place).  Returns q_out, or the cache
    without q."""
    dev = cache.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return paged_append(cache, k, v, starts, positions, rope, q, q_out)
    if k.dim() != 3:
        raise ValueError("k: 3 dimensions expected")
    n = k.shape[0]
    shp = (n, cache.kv_heads, cache.head_dim)
    ck, cv = _rows(k, shp, dev, "k"), _rows(v, shp, dev, "v")
    st_ptr = _ints(starts, cache._starts_shape, dev, "starts")
    p_ptr = _ints(positions, (n,), dev, "positions")
    if rope is not None and rope.device != dev:
        raise ValueError(f"rope: on {rope.device}, expected {dev}")
    G, cq, co = 0, None, None
    if q is not None:
        G = _group(q, cache.kv_heads, "q")
        q_shp = (n, q.shape[1], cache.head_dim)
        cq = _rows(q, q_shp, dev, "q")
        if q_out is None:
            q_out, co = _new_rows(q, *q_shp)
        else:
            co = cq if q_out is q else _rows(q_out, q_shp, dev, "q_out")
    elif q_out is not None:
        raise ValueError("q_out: without q")
    rc = lib().kvc_paged_append(cache._ref, _count(n, "n_tokens"), st_ptr, p_ptr,
                                None if rope is None else rope._ref, G, cq, co,
                                ck, cv, s)
    _check(rc, "kvc_paged_append")
    return cache if q is None else q_out


def _scale(scale):
    if scale != 0.0 and abs(scale) < 2.0 ** -149:
        raise ValueError(f"scale: {scale} is zero in fp32, which stands for 1 / sqrt(d)")
    return scale


def paged_attend(cache: PagedCache, q, starts, max_new: int = 0, out=None, lse=None,
                 want_lse: bool = False, scale: float = 0.0, ws=None, stream=None):
    """Attention of the new tokens' queries q (bf16 [n_tokens, heads, d], rows contiguous,
    packed by sequence: starts int32 [n_seqs + 1]) over the cache; in a cache with
    weight and pos the slots' weights grow by what they receive.  max_new bounds the new
    tokens of a sequence (0: n_tokens).  Returns out (bf16, like q), or (out, lse) with
    want_lse or an lse tensor (fp32 [n_tokens, heads])."""
    dev = cache.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return paged_attend(cache, q, starts, max_new, out, lse, want_lse, scale, ws)
    G = _group(q, cache.kv_heads, "q")
    shp = (q.shape[0], q.shape[1], cache.head_dim)
    cq = _rows(q, shp, dev, "q")
    st_ptr = _ints(starts, cache._starts_shape, dev, "starts")
    ws = _scratch(ws, cache.attend_workspace_bytes(G, shp[0], max_new), dev)
    if out is None:
        out, co = _new_rows(q, *shp)
    else:
        co = _rows(out, shp, dev, "out")
    lse, lse_ptr = (_new(q, shp[:2], torch.float32) if lse is None and want_lse else
                    _given(lse, _F32, shp[:2], dev, "lse"))
    rc = lib().kvc_paged_attend(cache._ref, G, shp[0], _int(max_new, "max_new"), st_ptr, _scale(scale),
                                cq, co, lse_ptr, *_span(ws), s)
    _check(rc, "kvc_paged_attend")
    return out if lse is None else (out, lse)


def prompt_attend(q, k, v, starts, out=None, lse=None, want_lse: bool = False, scale: float = 0.0,
                  stream=None):
    """Causal attention within packed prompts: q (bf16 [n_tokens, heads, d]), k, v ([n_tokens,
    kv_heads, d]), rows contiguous, packed by sequence (starts int32 [n_seqs + 1]).  Returns out
    (bf16, like q), or (out, lse) with want_lse or an lse tensor (fp32 [n_tokens, heads])."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"q: must be a GPU tensor, got {dev}")
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return prompt_attend(q, k, v, starts, out, lse, want_lse, scale)
    if k.dim() != 3 or starts.dim() != 1 or starts.shape[0] < 1 or k.shape[1] < 1:
        raise ValueError("k: 3 dimensions and a head expected, starts: 1 dimension with an entry")
    G = _group(q, k.shape[1], "q")
    n, heads, d = q.shape
    kv = (n, k.shape[1], d)
    cq, ck, cv = _rows(q, (n, heads, d), dev, "q"), _rows(k, kv, dev, "k"), _rows(v, kv, dev, "v")
    st_ptr = _ints(starts, starts.shape, dev, "starts")
    if out is None:
        out, co = _new_rows(q, n, heads, d)
    else:
        co = _rows(out, (n, heads, d), dev, "out")
    lse, lse_ptr = (_new(q, (n, heads), torch.float32) if lse is None and want_lse else
                    _given(lse, _F32, (n, heads), dev, "lse"))
    rc = lib().kvc_prompt_attend(_count(starts.shape[0] - 1, "n_seqs"), _count(kv[1], "kv_heads"), G,
                                 _count(d, "head_dim"), _count(n, "n_tokens"), st_ptr, _scale(scale),
                                 cq, ck, cv, co, lse_ptr, s)
    _check(rc, "kvc_prompt_attend")
    return out if lse is None else (out, lse)


def paged_evict(cache: PagedCache, seen, budget: int, sinks: int = 4, recent: int = 64, ws=None,
                stream=None):
    """Cuts every sequence to `budget` slots a head: positions below sinks, the last
    `recent` of the seen ones (int32 [n_seqs]), then the largest weights.  A sequence that
    shares one of its pages below the budget (a fork) is left as it is, its length too.
    Returns the cache."""
    dev = cache.device
    s = _here(dev, stream)
    if s is None:
        with _there(dev, stream):
            return paged_evict(cache, seen, budget, sinks, recent, ws)
    if cache.weight is None:
        raise ValueError("cache: has no weight and pos")
    seen_ptr = _ints(seen, cache.seq_len.shape, dev, "seen")
    ws = _scratch(ws, cache.evict_workspace_bytes(budget), dev)
    rc = lib().kvc_paged_evict(cache._ref, seen_ptr, _int(budget, "budget"), _int(sinks, "sinks"),
                               _int(recent, "recent"), *_span(ws), s)
    _check(rc, "kvc_paged_evict")
    return cache
