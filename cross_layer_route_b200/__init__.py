"""B200-native RouteRelay router: Python binding of librr.so (include/rr.h).

Method: "RouteRelay: Event-Triggered Cross-Layer Route Reuse for Efficient
Dynamic Sparse Attention" (arXiv 2609.07306).  Anchor layers fully route
every query chunk (S = Qc Kc^T, top-k, §2.1 Eq. 1-2); intermediate layers
rescore each row's ledger candidates, test alpha > beta + gamma (§3.2 Eq.
5-8) and fully re-route only the rows that fail (§4.1-4.2).  The routes feed
a sparse attention over their chunks' tokens (§2.1, Eq. 3; sparse_attention,
RouteLedger.sparse_attention).

This module only marshals arguments: every step of the routing path runs in
the CUDA kernels of librr.so.  There is no CPU fallback; importing it without
the built library raises.  PyTorch supplies device memory and streams.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librr.so")

RR_OK, RR_EINVAL, RR_ESTATE, RR_ENOMEM, RR_ECUDA, RR_EDEVICE, RR_ECAPACITY = range(7)
RR_F32, RR_BF16, RR_F16 = 0, 1, 2
RR_E4M3, RR_E2M1 = 0, 1
CNT_ROWS, CNT_PAIRS, CNT_ERROR, CNT_ROWS_TOTAL, CNT_PAIRS_TOTAL, CNT_LAYERS, CNT_LAST_LAYER, \
    CNT_DRAW_CAP, CNT_FULL_PAIRS, CNT_FULL_PAIRS_TOTAL, CNT_RETRY_TOTAL = range(11)
NUM_COUNTERS = 16


class rr_config(ctypes.Structure):
    _fields_ = [("bh", ctypes.c_int32), ("nq", ctypes.c_int32), ("nk", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("k", ctypes.c_int32),
                ("m_near", ctypes.c_int32), ("r_rand", ctypes.c_int32),
                ("anchor_interval", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("gamma", ctypes.c_float), ("bh_offset", ctypes.c_int32), ("seed", ctypes.c_uint64),
                ("g_sink", ctypes.c_int32), ("g_recent", ctypes.c_int32)]


class rr_ledger_view(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
                ("anchor_layer", ctypes.c_void_p), ("flags", ctypes.c_void_p),
                ("counters", ctypes.c_void_p)]


class rr_attn_config(ctypes.Structure):
    _fields_ = [("bh", ctypes.c_int32), ("nq_tokens", ctypes.c_int32), ("nk_tokens", ctypes.c_int32),
                ("dh", ctypes.c_int32), ("chunk", ctypes.c_int32), ("width", ctypes.c_int32),
                ("route_stride", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float)]


class rr_masked_attn_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "q_heads", "kv_heads", "route_heads", "nq_tokens", "nk_tokens", "dh", "chunk", "width",
                 "route_stride", "causal", "dtype", "q_offset")] + \
               [("scale", ctypes.c_float), ("soft_cap", ctypes.c_float)] + \
               [(n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "v_stride", "out_stride")]


class rr_masked_attn_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("q", "k", "v", "route", "slopes", "doc_q", "doc_k", "prefix", "out", "lse")]


class rr_cache_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("pages", "heads", "dh", "chunk", "format")]


class rr_cache_pool(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class rr_cache_rows(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("rows", ctypes.c_int32), ("cu", ctypes.c_void_p),
                ("start", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("table_width", ctypes.c_int32),
                ("table_stride", ctypes.c_int32)]


class rr_cached_attn_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "q_tokens", "q_heads", "dtype", "table_width", "table_stride", "width", "route_stride")] + \
               [("scale", ctypes.c_float), ("soft_cap", ctypes.c_float), ("q_stride", ctypes.c_int64 * 3)]


class rr_cached_attn_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "seq_lens", "page_table", "route", "slopes", "out", "lse")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"librr.so is not built ({LIB_PATH}); run python cross_layer_route_b200/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    lib.rr_ledger_workspace_bytes.argtypes = [ctypes.POINTER(rr_config)]
    lib.rr_ledger_workspace_bytes.restype = ctypes.c_size_t
    lib.rr_ledger_create.argtypes = [ctypes.POINTER(rr_config), P, ctypes.c_size_t, ctypes.POINTER(P)]
    lib.rr_ledger_create.restype = ctypes.c_int
    lib.rr_ledger_destroy.argtypes = [P]
    lib.rr_ledger_destroy.restype = ctypes.c_int
    for name in ("rr_full_route", "rr_relay_layer", "rr_relay_rescore", "rr_relay_refresh"):
        f = getattr(lib, name)
        f.argtypes = [P, P, P, ctypes.c_int32, P]
        f.restype = ctypes.c_int
    lib.rr_relay_compact.argtypes = [P, ctypes.c_int32, P]
    lib.rr_relay_compact.restype = ctypes.c_int
    lib.rr_ledger_read.argtypes = [P, ctypes.POINTER(rr_ledger_view), P]
    lib.rr_ledger_read.restype = ctypes.c_int
    lib.rr_ledger_device_view.argtypes = [P, ctypes.POINTER(rr_ledger_view)]
    lib.rr_ledger_device_view.restype = ctypes.c_int
    lib.rr_ledger_set_guard.argtypes = [P, P, ctypes.c_int32]
    lib.rr_ledger_set_guard.restype = ctypes.c_int
    lib.rr_ledger_set_hysteresis.argtypes = [P, ctypes.c_int32]
    lib.rr_ledger_set_hysteresis.restype = ctypes.c_int
    lib.rr_ledger_set_wait_budget.argtypes = [P, ctypes.c_int64]
    lib.rr_ledger_set_wait_budget.restype = ctypes.c_int
    lib.rr_ledger_set_hysteresis_margin.argtypes = [P, ctypes.c_float]
    lib.rr_ledger_set_hysteresis_margin.restype = ctypes.c_int
    lib.rr_route_layer_static.argtypes = [ctypes.POINTER(rr_config), P, P, ctypes.c_int32, P, P, P, P, P, P]
    lib.rr_route_layer_static.restype = ctypes.c_int
    lib.rr_sparse_attention.argtypes = [ctypes.POINTER(rr_attn_config), P, P, P, P, P, P]
    lib.rr_sparse_attention.restype = ctypes.c_int
    # structures of the calls below go as addresses of packed bytes
    lib.rr_masked_attention.argtypes = [P, P, P]
    lib.rr_masked_attention.restype = ctypes.c_int
    for name in ("rr_cache_codes_bytes", "rr_cache_scales_bytes"):
        f = getattr(lib, name)
        f.argtypes = [P]
        f.restype = ctypes.c_size_t
    for name in ("rr_cache_write", "rr_cache_read"):
        f = getattr(lib, name)
        f.argtypes = [P, P, P, P, P, P, P, ctypes.c_int32, P]
        f.restype = ctypes.c_int
    lib.rr_cached_attention_workspace_bytes.argtypes = [P, P, ctypes.c_int32]
    lib.rr_cached_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.rr_cached_attention.argtypes = [P, P, P, P, P, ctypes.c_size_t, P]
    lib.rr_cached_attention.restype = ctypes.c_int
    lib.rr_status_string.argtypes = [ctypes.c_int]
    lib.rr_status_string.restype = ctypes.c_char_p
    return lib


_lib = _load()


class RRError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {rr_status_string(status)}")


def _check(status: int, what: str):
    if status != RR_OK:
        raise RRError(status, what)


# ---- the C ABI, name for name ---------------------------------------------
def rr_status_string(status: int) -> str:
    return _lib.rr_status_string(status).decode()


def rr_ledger_workspace_bytes(cfg: rr_config) -> int:
    return int(_lib.rr_ledger_workspace_bytes(ctypes.byref(cfg)))


def rr_ledger_create(cfg: rr_config, d_workspace: int, nbytes: int) -> ctypes.c_void_p:
    out = ctypes.c_void_p()
    _check(_lib.rr_ledger_create(ctypes.byref(cfg), ctypes.c_void_p(d_workspace), nbytes,
                                 ctypes.byref(out)), "rr_ledger_create")
    return out


def rr_ledger_destroy(handle) -> None:
    _check(_lib.rr_ledger_destroy(handle), "rr_ledger_destroy")


def rr_full_route(handle, d_qc: int, d_kc: int, layer: int, stream: int) -> None:
    _check(_lib.rr_full_route(handle, ctypes.c_void_p(d_qc), ctypes.c_void_p(d_kc), layer,
                              ctypes.c_void_p(stream)), "rr_full_route")


def rr_relay_layer(handle, d_qc: int, d_kc: int, layer: int, stream: int) -> None:
    _check(_lib.rr_relay_layer(handle, ctypes.c_void_p(d_qc), ctypes.c_void_p(d_kc), layer,
                               ctypes.c_void_p(stream)), "rr_relay_layer")


def rr_relay_rescore(handle, d_qc: int, d_kc: int, layer: int, stream: int) -> None:
    _check(_lib.rr_relay_rescore(handle, ctypes.c_void_p(d_qc), ctypes.c_void_p(d_kc), layer,
                                 ctypes.c_void_p(stream)), "rr_relay_rescore")


def rr_relay_compact(handle, layer: int, stream: int) -> None:
    _check(_lib.rr_relay_compact(handle, layer, ctypes.c_void_p(stream)), "rr_relay_compact")


def rr_relay_refresh(handle, d_qc: int, d_kc: int, layer: int, stream: int) -> None:
    _check(_lib.rr_relay_refresh(handle, ctypes.c_void_p(d_qc), ctypes.c_void_p(d_kc), layer,
                                 ctypes.c_void_p(stream)), "rr_relay_refresh")


def rr_ledger_read(handle, view: rr_ledger_view, stream: int) -> None:
    _check(_lib.rr_ledger_read(handle, ctypes.byref(view), ctypes.c_void_p(stream)), "rr_ledger_read")


def rr_ledger_device_view(handle) -> rr_ledger_view:
    v = rr_ledger_view()
    _check(_lib.rr_ledger_device_view(handle, ctypes.byref(v)), "rr_ledger_device_view")
    return v


def rr_ledger_set_guard(handle, d_gamma_rows: int, max_age: int) -> None:
    _check(_lib.rr_ledger_set_guard(handle, ctypes.c_void_p(d_gamma_rows), max_age), "rr_ledger_set_guard")


def rr_ledger_set_hysteresis(handle, min_reuse: int) -> None:
    _check(_lib.rr_ledger_set_hysteresis(handle, min_reuse), "rr_ledger_set_hysteresis")


def rr_ledger_set_hysteresis_margin(handle, gamma_h: float) -> None:
    _check(_lib.rr_ledger_set_hysteresis_margin(handle, float(gamma_h)), "rr_ledger_set_hysteresis_margin")


def rr_ledger_set_wait_budget(handle, cycles: int) -> None:
    """Test hook (include/rr.h): the budget of the selection kernel's
    epilogue waits, in SM cycles (0: the default, about a second)."""
    _check(_lib.rr_ledger_set_wait_budget(handle, int(cycles)), "rr_ledger_set_wait_budget")


def rr_route_layer_static(cfg: rr_config, d_qc: int, d_kc: int, layer: int, d_ids: int, d_alpha: int,
                          d_anchor_layer: int, d_flags: int, d_counters: int, stream: int) -> None:
    """One layer on caller-held ledger arrays with no workspace and no
    allocation, for callers that cannot allocate device memory (their host
    framework owns every allocation).  See rr_route_layer_static in
    include/rr.h for its fixed capacity and its shared static scratch."""
    _check(_lib.rr_route_layer_static(ctypes.byref(cfg), ctypes.c_void_p(d_qc), ctypes.c_void_p(d_kc), layer,
                                      ctypes.c_void_p(d_ids), ctypes.c_void_p(d_alpha),
                                      ctypes.c_void_p(d_anchor_layer), ctypes.c_void_p(d_flags),
                                      ctypes.c_void_p(d_counters), ctypes.c_void_p(stream)),
           "rr_route_layer_static")


def rr_sparse_attention(cfg: rr_attn_config, d_q: int, d_k: int, d_v: int, d_route: int, d_out: int,
                        stream: int) -> None:
    """Sparse attention over a route (include/rr_attention.h)."""
    _check(_lib.rr_sparse_attention(ctypes.byref(cfg), ctypes.c_void_p(d_q), ctypes.c_void_p(d_k),
                                    ctypes.c_void_p(d_v), ctypes.c_void_p(d_route), ctypes.c_void_p(d_out),
                                    ctypes.c_void_p(stream)), "rr_sparse_attention")


def rr_masked_attention(cfg: rr_masked_attn_config, args: rr_masked_attn_args, stream: int) -> None:
    """Masked attention over a route (include/rr_attention.h)."""
    _check(_lib.rr_masked_attention(ctypes.byref(cfg), ctypes.byref(args), stream), "rr_masked_attention")


def rr_cache_codes_bytes(cfg: rr_cache_config) -> int:
    return int(_lib.rr_cache_codes_bytes(ctypes.byref(cfg)))


def rr_cache_scales_bytes(cfg: rr_cache_config) -> int:
    return int(_lib.rr_cache_scales_bytes(ctypes.byref(cfg)))


def rr_cache_write(cfg: rr_cache_config, pool: rr_cache_pool, rows: rr_cache_rows, d_k: int, k_stride, d_v: int,
                   v_stride, dtype: int, stream: int) -> None:
    """Quantised store into the paged cache (include/rr_cache.h)."""
    pair = ctypes.c_int64 * 2
    _check(_lib.rr_cache_write(ctypes.byref(cfg), ctypes.byref(pool), ctypes.byref(rows), d_k, pair(*k_stride), d_v,
                               pair(*v_stride), dtype, stream), "rr_cache_write")


def rr_cache_read(cfg: rr_cache_config, pool: rr_cache_pool, rows: rr_cache_rows, d_k: int, k_stride, d_v: int,
                  v_stride, dtype: int, stream: int) -> None:
    """Rows of the paged cache read back (include/rr_cache.h)."""
    pair = ctypes.c_int64 * 2
    _check(_lib.rr_cache_read(ctypes.byref(cfg), ctypes.byref(pool), ctypes.byref(rows), d_k, pair(*k_stride), d_v,
                              pair(*v_stride), dtype, stream), "rr_cache_read")


def rr_cached_attention_workspace_bytes(cfg: rr_cache_config, attn: rr_cached_attn_config, routed: bool) -> int:
    return int(_lib.rr_cached_attention_workspace_bytes(ctypes.byref(cfg), ctypes.byref(attn), int(bool(routed))))


def rr_cached_attention(cfg: rr_cache_config, pool: rr_cache_pool, attn: rr_cached_attn_config,
                        args: rr_cached_attn_args, workspace: int, workspace_bytes: int, stream: int) -> None:
    """Attention over the paged cache (include/rr_cache.h)."""
    _check(_lib.rr_cached_attention(ctypes.byref(cfg), ctypes.byref(pool), ctypes.byref(attn), ctypes.byref(args),
                                    workspace, workspace_bytes, stream), "rr_cached_attention")


# ---- convenience wrapper over torch memory --------------------------------
@dataclass
class Config:
    """Problem statement of one ledger (see rr_config in include/rr.h)."""
    bh: int
    nq: int
    nk: int
    d: int
    k: int
    m_near: int
    r_rand: int
    dtype: str = "f32"          # "f32" | "bf16"
    anchor_interval: int = 0
    causal: bool = False
    gamma: float = 0.0
    seed: int = 0
    bh_offset: int = 0
    g_sink: int = 0             # mandatory global sentinels: sink chunks
    g_recent: int = 0           # ... and recent chunks per row

    @property
    def c(self) -> int:
        return self.k + self.m_near + self.r_rand + self.g_sink + self.g_recent

    @property
    def torch_dtype(self) -> torch.dtype:
        return torch.bfloat16 if self.dtype == "bf16" else torch.float32

    def to_c(self) -> rr_config:
        return rr_config(self.bh, self.nq, self.nk, self.d, RR_BF16 if self.dtype == "bf16" else RR_F32,
                         self.k, self.m_near, self.r_rand, self.anchor_interval, int(bool(self.causal)),
                         float(self.gamma), self.bh_offset, int(self.seed) & 0xFFFFFFFFFFFFFFFF,
                         self.g_sink, self.g_recent)


def _stream_handle(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def sparse_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, route: torch.Tensor, chunk: int,
                     causal: bool = False, width: int | None = None, scale: float | None = None,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of every query token over the tokens of its chunk's route
    (RouteRelay §2.1, Eq. 3).  q [bh, nq_tokens, dh], k and v [bh, nk_tokens,
    dh]: contiguous bf16 on one CUDA device; route: contiguous int32 [bh,
    nq_tokens // chunk, stride] of key-chunk ids, of which the first `width`
    (default: all) are read.  Returns (or fills) fp32 [bh, nq_tokens, dh]."""
    bh, nq_tok, dh = q.shape
    nk_tok = k.shape[1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3 \
                or t.shape[0] != bh or t.shape[2] != dh or t.device != q.device:
            raise ValueError(f"{name}: expected contiguous bf16 [bh, tokens, {dh}] on {q.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    if tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"v {tuple(v.shape)} must match k {tuple(k.shape)}")
    if route.dtype != torch.int32 or not route.is_contiguous() or route.device != q.device or route.dim() != 3 \
            or route.shape[0] != bh or route.shape[1] * chunk != nq_tok:
        raise ValueError(f"route: expected contiguous int32 [{bh}, {nq_tok // max(chunk, 1)}, stride] on "
                         f"{q.device}, got {route.dtype} {tuple(route.shape)} on {route.device}")
    stride = route.shape[2]
    width = stride if width is None else int(width)
    if out is None:
        out = torch.empty((bh, nq_tok, dh), dtype=torch.float32, device=q.device)
    elif out.dtype != torch.float32 or not out.is_contiguous() or tuple(out.shape) != (bh, nq_tok, dh) \
            or out.device != q.device:
        raise ValueError("out: expected contiguous float32 [bh, nq_tokens, dh] on the inputs' device")
    cfg = rr_attn_config(bh, nq_tok, nk_tok, dh, chunk, width, max(stride, 1), int(bool(causal)),
                         0.0 if scale is None else float(scale))
    rr_sparse_attention(cfg, q.data_ptr(), k.data_ptr(), v.data_ptr(), route.data_ptr(), out.data_ptr(),
                        _stream_handle(stream))
    return out


_DTYPES = {torch.float32: RR_F32, torch.bfloat16: RR_BF16, torch.float16: RR_F16}
_HALVES = (torch.bfloat16, torch.float16)


def _describe(t) -> str:
    return f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}" if isinstance(t, torch.Tensor) else repr(t)


# The structures of include/rr_attention.h and rr_cache.h as struct formats: a call
# packs them in one step, a third of the time that filling ctypes fields takes.
_MASKED_CFG, _MASKED_ARGS = struct.Struct("@13i2f12q"), struct.Struct("@10P")
_CACHE_CFG, _CACHE_POOL, _CACHE_ROWS = struct.Struct("@5i"), struct.Struct("@2P"), struct.Struct("@2i3P2i")
_CACHED_CFG, _CACHED_ARGS, _TWO = struct.Struct("@8i2f3q"), struct.Struct("@7P"), struct.Struct("@2q")
for _fmt, _structure in ((_MASKED_CFG, rr_masked_attn_config), (_MASKED_ARGS, rr_masked_attn_args),
                         (_CACHE_CFG, rr_cache_config), (_CACHE_POOL, rr_cache_pool), (_CACHE_ROWS, rr_cache_rows),
                         (_CACHED_CFG, rr_cached_attn_config), (_CACHED_ARGS, rr_cached_attn_args)):
    assert _fmt.size == ctypes.sizeof(_structure), _structure


def _pack(fmt, *values):
    """A structure's bytes; ValueError where a value is no number of its field's type."""
    try:
        return fmt.pack(*values)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"an argument is out of range: {e}") from None


def _on_stream(index: int, stream, call, *args):
    """call(stream handle, *args) with CUDA device `index` current and, where the
    caller names a stream, that stream too, so that what the call allocates
    belongs to it."""
    if stream is None:
        if torch._C._cuda_getDevice() == index:
            return call(torch._C._cuda_getCurrentRawStream(index), *args)
        with torch.cuda.device(index):
            return call(torch._C._cuda_getCurrentRawStream(index), *args)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=index) if stream else torch.cuda.default_stream(index)
    if stream.device.index != index:
        raise ValueError(f"stream: expected a stream of cuda:{index}, got one of {stream.device}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream, *args)


def _int32(name, t, shape, index):
    """Address of a contiguous int32 tensor of this shape."""
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous int32 {shape} on cuda:{index}, got {_describe(t)}")
    return t.data_ptr()


def _dim(name, t, dims, i):
    """Size i of a tensor that should have `dims` dimensions."""
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got {_describe(t)}")
    return shape[i]


def _slopes(t, heads, index):
    if t is None:
        return 0
    if t.dtype is not torch.float32 or t.get_device() != index or t.shape != (heads,) or not t.is_contiguous():
        raise ValueError(f"slopes: expected contiguous float32 [{heads}] on cuda:{index}, got {_describe(t)}")
    return t.data_ptr()


def _rows_like(name, t, dtype, shape, index):
    """Strides, all but the last, of a tensor of this type and shape whose rows are contiguous."""
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or st[-1] != 1 or t.get_device() != index:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on cuda:{index}, the last dimension contiguous, "
                         f"got {_describe(t)}")
    return st[:-1]


def masked_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, route: torch.Tensor, chunk: int,
                     causal: bool = False, width: int | None = None, scale: float | None = None,
                     soft_cap: float = 0.0, slopes: torch.Tensor | None = None, doc_q: torch.Tensor | None = None,
                     doc_k: torch.Tensor | None = None, prefix: torch.Tensor | None = None, q_offset: int = 0,
                     out: torch.Tensor | None = None, return_lse: bool = False, stream=None):
    """Attention over a route with capped scores (`soft_cap`), a bias by
    distance (`slopes` [q_heads] float32), a document mask (`doc_q` [batch,
    nq_tokens] and `doc_k` [batch, nk_tokens] int32) and a prefix that the
    causal rule leaves visible (`prefix` [batch] int32); the formulas stand in
    include/rr_attention.h.

    q [batch, q_heads, nq_tokens, dh], k and v [batch, kv_heads, nk_tokens, dh]:
    bf16 or f16 on one CUDA device, any strides that are multiples of 8 with dh
    contiguous.  route: contiguous int32 [batch, route_heads, query chunks,
    stride] of key-chunk ids, of which the first `width` (default: all) are
    read.  q_offset: position of query token 0.  Returns (or fills) `out` like
    q, with return_lse also the float32 [batch, q_heads, nq_tokens] logarithms
    of the softmax sums.  With a `stream`, the results belong to it."""
    dtype, index, shape = q.dtype, q.get_device(), q.shape
    if len(shape) != 4 or k.dim() != 4 or dtype not in _HALVES or index < 0:
        raise ValueError(f"q: expected bf16 or f16 [batch, heads, tokens, dh] on a CUDA device, got {_describe(q)}")
    batch, q_heads, nq, dh = shape
    kv_heads, nk = k.shape[1], k.shape[2]
    kv_shape = (batch, kv_heads, nk, dh)
    strides = _rows_like("q", q, dtype, shape, index) + _rows_like("k", k, dtype, kv_shape, index) \
        + _rows_like("v", v, dtype, kv_shape, index)
    route_heads, stride = _dim("route", route, 4, 1), route.shape[3]
    d_route = _int32("route", route, (batch, route_heads, -(-nq // chunk) if chunk > 0 else 0, stride), index)
    width = stride if width is None else int(width)
    if width > stride:
        raise ValueError(f"width {width} is larger than the route's {stride} entries")
    if (doc_q is None) != (doc_k is None):
        raise ValueError("doc_q and doc_k go together")
    ints = (batch, q_heads, kv_heads, route_heads, nq, nk, dh, chunk, width, max(stride, 1), 1 if causal else 0,
            _DTYPES[dtype], q_offset, 0.0 if scale is None else scale, soft_cap) + strides
    ptrs = (q.data_ptr(), k.data_ptr(), v.data_ptr(), d_route, _slopes(slopes, q_heads, index),
            0 if doc_q is None else _int32("doc_q", doc_q, (batch, nq), index),
            0 if doc_k is None else _int32("doc_k", doc_k, (batch, nk), index),
            0 if prefix is None else _int32("prefix", prefix, (batch,), index))
    if out is not None:
        _rows_like("out", out, dtype, shape, index)
    return _on_stream(index, stream, _masked_attention, q, out, return_lse, ints, ptrs)


def _masked_attention(handle, q, out, return_lse, ints, ptrs):
    shape = q.shape
    if out is None:
        out = torch.empty_like(q)
    lse = q.new_empty(tuple(shape[:3]), dtype=torch.float32) if return_lse else None
    status = _lib.rr_masked_attention(_pack(_MASKED_CFG, *ints, *out.stride()[:-1]),
                                      _MASKED_ARGS.pack(*ptrs, out.data_ptr(), lse.data_ptr() if return_lse else 0),
                                      handle)
    if status:
        raise RRError(status, "rr_masked_attention")
    return (out, lse) if return_lse else out


def _cache(codes, scales, dh):
    """(config, pool, device index, heads) of a cache's two arrays, for rows of dh elements."""
    index, shape = codes.get_device(), codes.shape
    if codes.dtype is not torch.uint8 or index < 0 or len(shape) != 5 or shape[2] != 2 or not codes.is_contiguous():
        raise ValueError(f"codes: expected contiguous uint8 [pages, heads, 2, chunk, bytes] on a CUDA device, "
                         f"got {_describe(codes)}")
    pages, heads, _, chunk, row = shape
    if row == dh:
        fmt, groups = RR_E4M3, 1
    elif 2 * row == dh:
        fmt, groups = RR_E2M1, dh // 32
    else:
        raise ValueError(f"codes: rows of {row} bytes hold no {dh} elements (e4m3: {dh} bytes, e2m1: {dh // 2})")
    if scales.dtype is not torch.uint8 or scales.get_device() != index or not scales.is_contiguous() \
            or scales.shape != (pages, heads, 2, chunk, groups):
        raise ValueError(f"scales: expected contiguous uint8 {(pages, heads, 2, chunk, groups)} on cuda:{index}, "
                         f"got {_describe(scales)}")
    return _CACHE_CFG.pack(pages, heads, dh, chunk, fmt), _CACHE_POOL.pack(codes.data_ptr(), scales.data_ptr()), \
        index, heads


def cache_empty(pages: int, heads: int, chunk: int, dh: int, fmt: str = "e4m3", device=None):
    """(codes, scales) of a cache of `pages` pages of `chunk` tokens, zeroed
    (every row reads as zeros); fmt "e4m3" or "e2m1"."""
    if fmt not in ("e4m3", "e2m1"):
        raise ValueError(f'fmt: expected "e4m3" or "e2m1", got {fmt!r}')
    if rr_cache_scales_bytes(rr_cache_config(1, heads, dh, chunk, RR_E4M3)) == 0 or pages < 0:
        raise RRError(RR_EINVAL, f"cache_empty(pages={pages}, heads={heads}, chunk={chunk}, dh={dh})")
    row, groups = (dh, 1) if fmt == "e4m3" else (dh // 2, dh // 32)
    mk = lambda n: torch.zeros((pages, heads, 2, chunk, n), dtype=torch.uint8, device="cuda" if device is None else device)
    return mk(row), mk(groups)


def _ragged(rows, cu, start, table, index):
    batch, width = _dim("table", table, 2, 0), table.shape[1]
    d_table = _int32("table", table, (batch, width), index)
    return _pack(_CACHE_ROWS, batch, rows, _int32("cu", cu, (batch + 1,), index),
                 _int32("start", start, (batch,), index), d_table, width, max(width, 1))


def cache_write(codes: torch.Tensor, scales: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor,
                start: torch.Tensor, table: torch.Tensor, stream=None) -> None:
    """Quantises keys and values into the paged cache (include/rr_cache.h).
    codes uint8 [pages, heads, 2, chunk, dh] (e4m3) or [..., dh // 2] (e2m1),
    scales uint8 [pages, heads, 2, chunk, 1] or [..., dh // 32]; k and v [rows,
    heads, dh] of one type (f32, bf16, f16), any strides that keep rows 16-byte
    aligned; rows cu[b]..cu[b+1]-1 are sequence b's at positions start[b]...;
    table [batch, width]: pages of each sequence's chunks (-1: none)."""
    dtype, shape = k.dtype, k.shape
    if len(shape) != 3 or dtype not in _DTYPES:
        raise ValueError(f"k: expected f32, bf16 or f16 [rows, heads, dh], got {_describe(k)}")
    cfg, pool, index, heads = _cache(codes, scales, shape[2])
    want = (shape[0], heads, shape[2])
    args = (cfg, pool, _ragged(shape[0], cu, start, table, index), k.data_ptr(),
            _TWO.pack(*_rows_like("k", k, dtype, want, index)), v.data_ptr(),
            _TWO.pack(*_rows_like("v", v, dtype, want, index)), _DTYPES[dtype])
    _on_stream(index, stream, _cache_write, args)


def _cache_write(handle, args):
    _check(_lib.rr_cache_write(*args, handle), "rr_cache_write")


def cache_read(codes: torch.Tensor, scales: torch.Tensor, cu: torch.Tensor, start: torch.Tensor,
               table: torch.Tensor, rows: int, dh: int, dtype: torch.dtype = torch.bfloat16,
               out: tuple | None = None, stream=None):
    """The cached keys and values of a ragged batch, as (k, v) [rows, heads,
    dh] of `dtype`; see cache_write for the arguments.  Rows that belong to no
    sequence are not written: they keep what `out` (a pair of tensors to fill)
    held, and are unspecified without it."""
    cfg, pool, index, heads = _cache(codes, scales, dh)
    if dtype not in _DTYPES:
        raise ValueError(f"dtype: expected float32, bfloat16 or float16, got {dtype}")
    if rows < 0:
        raise ValueError(f"rows: expected 0 or more, got {rows}")
    args = (cfg, pool, _ragged(rows, cu, start, table, index))
    return _on_stream(index, stream, _cache_read, args, out, (rows, heads, dh), dtype, codes.device, index)


def _cache_read(handle, args, out, shape, dtype, device, index):
    k, v = out if out is not None else (torch.empty(shape, dtype=dtype, device=device),
                                        torch.empty(shape, dtype=dtype, device=device))
    _check(_lib.rr_cache_read(*args, k.data_ptr(), _TWO.pack(*_rows_like("out k", k, dtype, shape, index)),
                              v.data_ptr(), _TWO.pack(*_rows_like("out v", v, dtype, shape, index)), _DTYPES[dtype],
                              handle), "rr_cache_read")
    return k, v


def cached_attention(codes: torch.Tensor, scales: torch.Tensor, q: torch.Tensor, seq_lens: torch.Tensor,
                     table: torch.Tensor, route: torch.Tensor | None = None, width: int | None = None,
                     scale: float | None = None, soft_cap: float = 0.0, slopes: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, return_lse: bool = False,
                     workspace: torch.Tensor | None = None, stream=None):
    """Attention of each sequence's newest tokens over the paged cache
    (include/rr_cache.h).  q [batch, q_tokens, q_heads, dh] bf16 or f16, dh
    contiguous; seq_lens [batch] int32: cached tokens, the query tokens among
    them; table [batch, width] int32; route: None (every chunk) or contiguous
    int32 [batch, cache heads, stride] of chunk ids, of which the first `width`
    (default: all) are read; where there are none the result is zero. Returns (or
    fills) out like q, contiguous, with return_lse also float32 [batch, q_tokens,
    q_heads]. `workspace`: uint8 device memory of
    rr_cached_attention_workspace_bytes, for callers that hold their own; two calls
    that can run at once need one each. With a `stream`, the results belong to it."""
    dtype, shape = q.dtype, q.shape
    if len(shape) != 4 or dtype not in _HALVES:
        raise ValueError(f"q: expected bf16 or f16 [batch, tokens, heads, dh], got {_describe(q)}")
    batch, q_tokens, q_heads, dh = shape
    cfg, pool, index, heads = _cache(codes, scales, dh)
    q_strides = _rows_like("q", q, dtype, shape, index)
    table_width = _dim("table", table, 2, 1)
    d_table = _int32("table", table, (batch, table_width), index)
    stride, d_route = 1, 0
    if route is not None:
        stride = _dim("route", route, 3, 2)
        # (a route of no entries has no address, which would stand for no route at all; it is not read)
        d_route = _int32("route", route, (batch, heads, stride), index) or seq_lens.data_ptr()
        width = stride if width is None else int(width)
        if width > stride:
            raise ValueError(f"width {width} is larger than the route's {stride} entries")
    elif width:
        raise ValueError("width goes with a route")
    if out is not None and (_rows_like("out", out, dtype, shape, index) is None or not out.is_contiguous()):
        raise ValueError(f"out: expected contiguous {dtype} {tuple(shape)} on cuda:{index}, got {_describe(out)}")
    if workspace is not None and (workspace.dtype is not torch.uint8 or workspace.get_device() != index
                                  or not workspace.is_contiguous()):
        raise ValueError(f"workspace: expected contiguous uint8 on cuda:{index}, got {_describe(workspace)}")
    attn = _pack(_CACHED_CFG, batch, q_tokens, q_heads, _DTYPES[dtype], table_width, max(table_width, 1), width or 0,
                            max(stride, 1), 0.0 if scale is None else scale, soft_cap, *q_strides)
    ptrs = (q.data_ptr(), _int32("seq_lens", seq_lens, (batch,), index), d_table, d_route,
            _slopes(slopes, q_heads, index))
    return _on_stream(index, stream, _cached_attention, q, out, return_lse, workspace, cfg, pool, attn, ptrs)


def _cached_attention(handle, q, out, return_lse, workspace, cfg, pool, attn, ptrs):
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = q.new_empty(tuple(q.shape[:3]), dtype=torch.float32) if return_lse else None
    if workspace is None:
        need = _lib.rr_cached_attention_workspace_bytes(cfg, attn, 1 if ptrs[3] else 0)
        if need:
            workspace = q.new_empty((need,), dtype=torch.uint8)
    d_work, size = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _check(_lib.rr_cached_attention(cfg, pool, attn,
                                    _CACHED_ARGS.pack(*ptrs, out.data_ptr(), lse.data_ptr() if return_lse else 0),
                                    d_work, size, handle), "rr_cached_attention")
    return (out, lse) if return_lse else out


class RouteLedger:
    """One ledger (RouteRelay Eq. 4) in a torch-allocated device workspace."""

    def __init__(self, cfg: Config, device=None):
        self.cfg = cfg
        self._c = cfg.to_c()
        dev = torch.device(device if device is not None else "cuda")
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        nbytes = rr_ledger_workspace_bytes(self._c)
        if nbytes == 0:
            raise RRError(RR_EINVAL, "rr_ledger_workspace_bytes (invalid config)")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.handle = rr_ledger_create(self._c, self.workspace.data_ptr(), nbytes)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.rr_ledger_destroy(h)
            self.handle = None

    def _args(self, qc: torch.Tensor, kc: torch.Tensor):
        c = self.cfg
        for name, t, n in (("qc", qc, c.nq), ("kc", kc, c.nk)):
            if t.device != self.device or t.dtype != c.torch_dtype or not t.is_contiguous() \
                    or tuple(t.shape) != (c.bh, n, c.d):
                raise ValueError(f"{name}: expected contiguous {c.torch_dtype} [{c.bh}, {n}, {c.d}] on "
                                 f"{self.device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
        return qc.data_ptr(), kc.data_ptr()

    def full_route(self, qc, kc, layer: int, stream=None):
        q, k = self._args(qc, kc)
        rr_full_route(self.handle, q, k, layer, _stream_handle(stream))

    def relay_layer(self, qc, kc, layer: int, stream=None):
        q, k = self._args(qc, kc)
        rr_relay_layer(self.handle, q, k, layer, _stream_handle(stream))

    def relay_rescore(self, qc, kc, layer: int, stream=None):
        q, k = self._args(qc, kc)
        rr_relay_rescore(self.handle, q, k, layer, _stream_handle(stream))

    def relay_compact(self, layer: int, stream=None):
        rr_relay_compact(self.handle, layer, _stream_handle(stream))

    def relay_refresh(self, qc, kc, layer: int, stream=None):
        q, k = self._args(qc, kc)
        rr_relay_refresh(self.handle, q, k, layer, _stream_handle(stream))

    def is_anchor(self, layer: int) -> bool:
        H = self.cfg.anchor_interval
        return layer == 0 or (H > 0 and layer % H == 0)

    def read(self, device="cpu", stream=None, check: bool = True) -> dict:
        """Copies the ledger out (ids [bh, nq, c], alpha, anchor_layer, flags,
        counters), synchronises the stream and raises on a device error."""
        c = self.cfg
        pin = torch.device(device).type == "cpu"
        mk = lambda shape, dt: torch.empty(shape, dtype=dt, device=device, pin_memory=pin)
        out = {"ids": mk((c.bh, c.nq, c.c), torch.int32), "alpha": mk((c.bh, c.nq), torch.float32),
               "anchor_layer": mk((c.bh, c.nq), torch.int32), "flags": mk((c.bh, c.nq), torch.uint8),
               "counters": mk((NUM_COUNTERS,), torch.int64)}
        v = rr_ledger_view(out["ids"].data_ptr(), out["alpha"].data_ptr(), out["anchor_layer"].data_ptr(),
                           out["flags"].data_ptr(), out["counters"].data_ptr())
        rr_ledger_read(self.handle, v, _stream_handle(stream))
        torch.cuda.synchronize(self.device)
        if check and int(out["counters"][CNT_ERROR]) != 0:
            raise RRError(RR_EDEVICE, f"device error word {int(out['counters'][CNT_ERROR]):#x}")
        return out

    def set_guard(self, gamma_rows=None, max_age: int = 0) -> None:
        """Per-row relay trigger: gamma_rows, a float32 device tensor of bh*nq
        guard margins (or None for cfg.gamma on every row), and the per-row
        lifetime bound max_age (0: off).  The tensor is kept referenced."""
        ptr = 0
        if gamma_rows is not None:
            c = self.cfg
            assert gamma_rows.dtype == torch.float32 and gamma_rows.is_contiguous()
            assert gamma_rows.numel() == c.bh * c.nq and gamma_rows.device == self.workspace.device
            ptr = gamma_rows.data_ptr()
        rr_ledger_set_guard(self.handle, ptr, int(max_age))
        self._gamma_rows = gamma_rows

    def set_hysteresis(self, min_reuse: int) -> None:
        """Minimum reuse horizon after a row is rebuilt (0: off)."""
        rr_ledger_set_hysteresis(self.handle, int(min_reuse))

    def set_hysteresis_margin(self, gamma_h: float) -> None:
        """Larger guard margin of a row rebuilt at a relay layer, until its
        test first passes (0: off; the mark is bit 1 of the flags)."""
        rr_ledger_set_hysteresis_margin(self.handle, float(gamma_h))

    def device_view(self) -> dict:
        """Zero-copy torch views of the ledger inside the workspace."""
        v = rr_ledger_device_view(self.handle)
        c = self.cfg
        base = self.workspace.data_ptr()
        ws = self.workspace

        def view(ptr, nbytes, dt, shape):
            off = ptr - base
            return ws[off:off + nbytes].view(dt).view(shape)

        rows = c.bh * c.nq
        return {"ids": view(v.ids, rows * c.c * 4, torch.int32, (c.bh, c.nq, c.c)),
                "alpha": view(v.alpha, rows * 4, torch.float32, (c.bh, c.nq)),
                "anchor_layer": view(v.anchor_layer, rows * 4, torch.int32, (c.bh, c.nq)),
                "flags": view(v.flags, rows, torch.uint8, (c.bh, c.nq)),
                "counters": view(v.counters, NUM_COUNTERS * 8, torch.int64, (NUM_COUNTERS,))}

    def sparse_attention(self, q, k, v, chunk: int, out=None, stream=None) -> torch.Tensor:
        """Attention over the ledger's current routes (the first k ids of each
        row, read in place): q [bh, nq * chunk, dh], k and v [bh, nk * chunk,
        dh] bf16 token tensors of the same layer, with the ledger's causal rule
        applied at token level."""
        c = self.cfg
        if q.shape[0] != c.bh or q.shape[1] != c.nq * chunk or k.shape[1] != c.nk * chunk:
            raise ValueError(f"q/k: expected [{c.bh}, {c.nq * chunk}, dh] / [{c.bh}, {c.nk * chunk}, dh], "
                             f"got {tuple(q.shape)} / {tuple(k.shape)}")
        ids = self.device_view()["ids"]
        return sparse_attention(q, k, v, ids, chunk, causal=c.causal, width=c.k, out=out, stream=stream)

    def _route_of(self, heads: int, chunk: int, nq_tokens: int, nk_tokens: int):
        """The ledger's ids in place, as [batch, route heads, query chunks, c]:
        its bh heads are `heads` route heads of each batch entry."""
        c = self.cfg
        if chunk < 1:
            raise ValueError(f"chunk: expected 1 or more, got {chunk}")
        if heads < 1 or c.bh % heads != 0:
            raise ValueError(f"route_heads: expected a divisor of the ledger's {c.bh} heads, got {heads}")
        if -(-nq_tokens // chunk) != c.nq or -(-nk_tokens // chunk) > c.nk:
            raise ValueError(f"expected {c.nq} query chunks and at most {c.nk} key chunks of {chunk} tokens, got "
                             f"{nq_tokens} and {nk_tokens} tokens")
        return self.device_view()["ids"].view(c.bh // heads, heads, c.nq, c.c)

    def masked_attention(self, q, k, v, chunk: int, route_heads: int | None = None, **options):
        """masked_attention over the ledger's current routes, read in place:
        q [batch, q_heads, nq_tokens, dh], k and v [batch, kv_heads, nk_tokens,
        dh] of the same layer, the last chunk possibly short; route_heads
        (default: kv_heads) of the ledger's heads belong to each batch entry.
        The ledger's causal rule is applied at token level; options as there."""
        if "causal" in options or "width" in options:
            raise ValueError("causal and width are the ledger's")
        heads = k.shape[1] if route_heads is None else route_heads
        ids = self._route_of(heads, chunk, q.shape[2], k.shape[2])
        return masked_attention(q, k, v, ids, chunk, causal=self.cfg.causal, width=self.cfg.k, **options)

    def cached_attention(self, codes, scales, q, seq_lens, table, **options):
        """cached_attention over the ledger's current routes, read in place: a
        ledger of one query chunk (nq = 1) whose heads are the cache's heads of
        each sequence, batch-major."""
        c, heads = self.cfg, codes.shape[1]
        if c.nq != 1 or c.bh != q.shape[0] * heads:
            raise ValueError(f"expected a ledger of one query chunk for {q.shape[0]} x {heads} heads, got nq {c.nq}, "
                             f"bh {c.bh}")
        if "route" in options or "width" in options:
            raise ValueError("route and width are the ledger's")
        ids = self.device_view()["ids"].view(q.shape[0], heads, c.c)
        return cached_attention(codes, scales, q, seq_lens, table, route=ids, width=c.k, **options)

    def layer(self, qc, kc, layer: int, stream=None):
        """Layer l of a sequence: an anchor at l == 0, else rr_relay_layer
        (which itself turns forced-anchor layers into full routing)."""
        if layer == 0:
            self.full_route(qc, kc, layer, stream)
        else:
            self.relay_layer(qc, kc, layer, stream)
