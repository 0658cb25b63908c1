"""Thin Python binding of the GB300 decode-step MoE library (``libmoe_gb300.so``).

The binding only marshals arguments: it takes torch tensors (device memory
and streams come from PyTorch), checks their shapes, dtypes and devices, and
passes raw pointers to the C ABI declared in ``include/moe.h``.  Every step
of the block runs in the library's CUDA kernels; there is no Python or CPU
fallback, and importing this package fails loudly if the library is missing.

Functions carry the C names (``moe_router_topk``, ``moe_decode_forward``,
``moe_grouped_forward``, ...); errors raise ``MoeError`` with the library's
``moe_last_error()`` text.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
import struct
import warnings
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

MOE_F16, MOE_BF16, MOE_F32, MOE_E4M3 = 1, 2, 3, 4
_DT = {MOE_F16: torch.float16, MOE_BF16: torch.bfloat16, MOE_F32: torch.float32}
_DT_CODE = {torch.float16: MOE_F16, torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_DEVICE"}

# Every symbol include/moe.h declares.
EXPORTS = ("moe_abi_version", "moe_workspace_bytes", "moe_workspace_init", "moe_router_topk",
           "moe_decode_forward", "moe_grouped_forward", "moe_query_status", "moe_last_error",
           "moe_get_stats", "moe_reset_stats", "moe_set_wait_timeout_ns", "moe_test_wait_timeout",
           "moe_decode_forward_noalloc", "moe_sum_partials", "moe_add_rmsnorm", "moe_rope_append",
           "moe_attention_workspace_bytes", "moe_attention_form", "moe_paged_attention")


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{STATUS.get(code, code)}: {what}")
        self.code = code


class moe_cfg_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("hidden", "n_experts", "top_k", "inter", "shared_inter", "dtype",
                                              "out_dtype", "norm_topk", "has_shared_gate", "flags")]


class moe_topk_t(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("weights", ctypes.c_void_p)]


class moe_stats_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("decode_fused_calls", "router_calls", "grouped_calls",
                                               "grouped_tc_calls", "kernels_launched", "decode_general_calls")]


MOE_FLAG_GROUPED_SIMT = 1
MOE_FLAG_GROUPED_TC = 2
MOE_FLAG_STATIC_WEIGHTS = 4
MOE_FLAG_RESIDUAL = 8
MOE_FLAG_GROUPED_SINGLE = 16


@dataclass(frozen=True)
class MoeCfg:
    hidden: int
    n_experts: int
    top_k: int
    inter: int
    shared_inter: int = 0
    dtype: int = MOE_BF16
    out_dtype: int | None = None
    norm_topk: int = 1
    has_shared_gate: int = 0
    flags: int = 0

    def c(self) -> moe_cfg_t:
        return moe_cfg_t(self.hidden, self.n_experts, self.top_k, self.inter, self.shared_inter, self.dtype,
                         self.dtype if self.out_dtype is None else self.out_dtype, self.norm_topk,
                         self.has_shared_gate, self.flags)

    @property
    def torch_dtype(self):
        return _DT[self.dtype]

    @property
    def out_torch_dtype(self):
        return _DT[self.dtype if self.out_dtype is None else self.out_dtype]


_lib = None


def use_library(path: str):
    """Load another build of this library (the phase-trace variant) instead of
    ``libmoe_gb300.so``; must come before the first call."""
    global LIB_PATH
    if _lib is not None:
        raise RuntimeError("the library is already loaded")
    LIB_PATH = path


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                          "(the MoE block has no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, u64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_uint64
    cfgp = ctypes.POINTER(moe_cfg_t)
    sig = {
        "moe_abi_version": ([], i32),
        "moe_workspace_bytes": ([cfgp, i32], sz),
        "moe_workspace_init": ([vp, sz, vp], ctypes.c_int),
        "moe_router_topk": ([cfgp, vp, vp, i32, moe_topk_t, vp, vp, sz, vp], ctypes.c_int),
        "moe_decode_forward": ([cfgp, vp, vp, vp, vp, vp, vp, vp, moe_topk_t, vp, vp, sz, vp], ctypes.c_int),
        "moe_grouped_forward": ([cfgp, vp, vp, vp, vp, vp, vp, vp, moe_topk_t, vp, vp, sz, i32, vp],
                                ctypes.c_int),
        "moe_query_status": ([vp, vp], ctypes.c_int),
        "moe_last_error": ([], ctypes.c_char_p),
        "moe_get_stats": ([ctypes.POINTER(moe_stats_t)], ctypes.c_int),
        "moe_reset_stats": ([], None),
        "moe_set_wait_timeout_ns": ([u64], ctypes.c_int),
        "moe_test_wait_timeout": ([vp, sz, vp], ctypes.c_int),
        "moe_decode_forward_noalloc": ([cfgp, vp, vp, vp, vp, vp, vp, vp, moe_topk_t, vp, vp], ctypes.c_int),
        "moe_sum_partials": ([vp, i32, ctypes.c_int64, vp, i32, vp, i32, vp], ctypes.c_int),
        # the structs below travel as packed bytes (struct.Struct with C alignment)
        "moe_add_rmsnorm": ([ctypes.c_char_p, vp], ctypes.c_int),
        "moe_rope_append": ([ctypes.c_char_p, ctypes.c_char_p, vp, sz, vp], ctypes.c_int),
        "moe_attention_workspace_bytes": ([ctypes.c_char_p, i32], sz),
        "moe_attention_form": ([ctypes.c_char_p, i32, i32, i32, i32], i32),
        "moe_paged_attention": ([ctypes.c_char_p, ctypes.c_char_p, vp, sz, vp], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    _bind_fast_call(lib)
    return lib


# The compiled form of the layer operators' checks (csrc/fast_call.cpp): returns
# the entry's status, or -1 for arguments that the Python form is to explain.
_fast = None


def _bind_fast_call(lib):
    global _fast
    try:
        from . import _fast_call
    except ImportError:  # not built here: the Python form does the same
        return
    entries = (lib.moe_add_rmsnorm, lib.moe_rope_append, lib.moe_paged_attention)
    structs = (_NORM_T, _CACHE_T, _ROPE_T, _ATTN_T)
    if getattr(_fast_call, "built_for", None) != torch.__version__ or not _fast_call.bind(
            *(ctypes.cast(f, ctypes.c_void_p).value for f in entries), *(t.size for t in structs)):
        warnings.warn("the compiled argument checks were built for another PyTorch or header and are not used: "
                      "build them with __graft_entry__.build()")
        return
    _fast = _fast_call


def library():
    """The loaded ctypes library (raises if it was not built)."""
    return _load()


def _check(rc: int):
    if rc != 0:
        raise MoeError(rc, _load().moe_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t, name, shape, dtype, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ------------------------------------------------------------------ helpers
def moe_abi_version() -> int:
    return _load().moe_abi_version()


def moe_workspace_bytes(cfg: MoeCfg, T: int) -> int:
    c = cfg.c()
    return int(_load().moe_workspace_bytes(ctypes.byref(c), int(T)))


def alloc_workspace(cfg: MoeCfg, T: int, device) -> torch.Tensor:
    """A zero-filled, 256-byte aligned workspace for up to T tokens of cfg."""
    n = moe_workspace_bytes(cfg, T)
    if n == 0:
        raise MoeError(1, "invalid cfg")
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def moe_workspace_init(ws: torch.Tensor, stream=None):
    _check(_load().moe_workspace_init(_ptr(ws), ws.numel(), _stream(stream)))


def moe_query_status(ws: torch.Tensor | None, stream=None):
    """Synchronise the stream, then read and clear the device status word of
    ``ws`` (None: the built-in array of moe_decode_forward_noalloc)."""
    _check(_load().moe_query_status(_ptr(ws), _stream(stream)))


def moe_last_error() -> str:
    return _load().moe_last_error().decode(errors="replace")


def moe_get_stats() -> dict:
    s = moe_stats_t()
    _check(_load().moe_get_stats(ctypes.byref(s)))
    return {n: int(getattr(s, n)) for n, _ in moe_stats_t._fields_}


def moe_reset_stats():
    _load().moe_reset_stats()


def moe_set_wait_timeout_ns(ns: int):
    _check(_load().moe_set_wait_timeout_ns(int(ns)))


def moe_test_wait_timeout(ws: torch.Tensor, stream=None):
    _check(_load().moe_test_wait_timeout(_ptr(ws), ws.numel(), _stream(stream)))


# --------------------------------------------------------------- the block
def moe_router_topk(cfg: MoeCfg, x, router_w, ids, weights, ws, logits=None, stream=None):
    """Router logits, softmax and top-k for x [T, H]; fills ids/weights [T, k]."""
    T = x.shape[0]
    dev = x.device
    dt = cfg.torch_dtype
    _need(x, "x", (T, cfg.hidden), dt, dev)
    _need(router_w, "router_w", (cfg.n_experts, cfg.hidden), dt, dev)
    _need(ids, "ids", (T, cfg.top_k), torch.int32, dev)
    _need(weights, "weights", (T, cfg.top_k), torch.float32, dev)
    if logits is not None:
        _need(logits, "logits", (T, cfg.n_experts), torch.float32, dev)
    c = cfg.c()
    _check(_load().moe_router_topk(ctypes.byref(c), _ptr(x), _ptr(router_w), T,
                                   moe_topk_t(ids.data_ptr(), weights.data_ptr()), _ptr(logits),
                                   _ptr(ws), ws.numel(), _stream(stream)))


def _block_args(cfg, x, router_w, w13, w2, shared_w13, shared_w2, shared_gate_w, ids, weights, out, T):
    dev = x.device
    dt = cfg.torch_dtype
    H, E, k, I, Is = cfg.hidden, cfg.n_experts, cfg.top_k, cfg.inter, cfg.shared_inter
    _need(x, "x", (T, H), dt, dev)
    _need(router_w, "router_w", (E, H), dt, dev)
    _need(w13, "w13", (E, 2 * I, H), dt, dev)
    _need(w2, "w2", (E, H, I), dt, dev)
    if Is:
        _need(shared_w13, "shared_w13", (2 * Is, H), dt, dev)
        _need(shared_w2, "shared_w2", (H, Is), dt, dev)
    if cfg.has_shared_gate:
        _need(shared_gate_w, "shared_gate_w", (H,), dt, dev)
    _need(ids, "ids", (T, k), torch.int32, dev)
    _need(weights, "weights", (T, k), torch.float32, dev)
    _need(out, "out", (T, H), cfg.out_torch_dtype, dev)
    return (_ptr(x), _ptr(router_w), _ptr(w13), _ptr(w2), _ptr(shared_w13), _ptr(shared_w2),
            _ptr(shared_gate_w), moe_topk_t(ids.data_ptr(), weights.data_ptr()), _ptr(out))


def moe_decode_forward(cfg: MoeCfg, x, router_w, w13, w2, shared_w13, shared_w2, shared_gate_w, ids, weights,
                       out, ws, stream=None):
    """One decode token (x [1, H]) through the whole block in one kernel launch."""
    args = _block_args(cfg, x, router_w, w13, w2, shared_w13, shared_w2, shared_gate_w, ids, weights, out, 1)
    c = cfg.c()
    _check(_load().moe_decode_forward(ctypes.byref(c), *args, _ptr(ws), ws.numel(), _stream(stream)))


def moe_decode_forward_noalloc(cfg: MoeCfg, x, router_w, w13, w2, shared_w13, shared_w2, shared_gate_w, ids,
                               weights, out, stream=None):
    """moe_decode_forward for callers that cannot allocate a workspace: the
    scratch is a fixed array inside the library (see include/moe.h)."""
    args = _block_args(cfg, x, router_w, w13, w2, shared_w13, shared_w2, shared_gate_w, ids, weights, out, 1)
    c = cfg.c()
    _check(_load().moe_decode_forward_noalloc(ctypes.byref(c), *args, _stream(stream)))


def moe_grouped_forward(cfg: MoeCfg, x, router_w, w13, w2, shared_w13, shared_w2, shared_gate_w, ids, weights,
                        out, ws, stream=None):
    """T tokens (x [T, H]) through the block; T > 1 groups (token, expert) pairs by expert."""
    T = x.shape[0]
    args = _block_args(cfg, x, router_w, w13, w2, shared_w13, shared_w2, shared_gate_w, ids, weights, out, T)
    c = cfg.c()
    _check(_load().moe_grouped_forward(ctypes.byref(c), *args, _ptr(ws), ws.numel(), T, _stream(stream)))


def moe_sum_partials(partials, out, residual=None, stream=None):
    """out = sum over dim 0 of fp32 ``partials`` [n_parts, ...] (+ residual),
    rounded once to out's dtype; the sum runs in part order."""
    if partials.dtype != torch.float32 or not partials.is_contiguous():
        raise ValueError("partials must be contiguous fp32")
    n = out.numel()
    if partials.numel() != partials.shape[0] * n or not out.is_contiguous():
        raise ValueError("partials must be [n_parts, *out.shape], out contiguous")
    if out.device != partials.device:
        raise ValueError("partials and out must be on one device")
    rdt = 0
    if residual is not None:
        if residual.numel() != n or not residual.is_contiguous() or residual.dtype not in (torch.float16,
                                                                                           torch.bfloat16):
            raise ValueError("residual must be a contiguous fp16/bf16 tensor shaped like out")
        rdt = _DT_CODE[residual.dtype]
    _check(_load().moe_sum_partials(_ptr(partials), partials.shape[0], n, _ptr(residual), rdt, _ptr(out),
                                    _DT_CODE[out.dtype], _stream(stream)))


# ------------------------------------------- the layer's attention half
# Packed forms of moe_norm_t, moe_kv_cache_t, moe_rope_t and moe_attention_t.
_NORM_T = struct.Struct("@6P4q5if")
_CACHE_T = struct.Struct("@4P6q5i0q")
_ROPE_T = struct.Struct("@9P8q5if0q")
_ATTN_T = struct.Struct("@5P5q5if0q")


# A decode step makes these calls dozens of times per token and their kernels
# take a few microseconds, so their checks are made in compiled code where that
# is built, and here in single comparisons, with the stream asked for as a number.
_FLOATS = {torch.float16: MOE_F16, torch.bfloat16: MOE_BF16}


def _launch_stream(index, stream):
    """The raw stream a call on tensors of CUDA device `index` goes to."""
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    # (private, so asked for here: a PyTorch without CUDA has neither and still imports this)
    current = torch._C._cuda_getDevice()
    if index != current:
        raise ValueError(f"tensors are on cuda:{index}, the current device is cuda:{current}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is required, got {type(t).__name__}")
    return t


def _int32(v, name):
    try:
        v = operator.index(v)
    except TypeError:
        raise ValueError(f"{name}: an integer is required, got {type(v).__name__}") from None
    if not -0x80000000 <= v <= 0x7fffffff:
        raise ValueError(f"{name}: {v} does not fit 32 bits")
    return v


def _fp32(v, name):
    if not hasattr(v, "__float__"):
        raise ValueError(f"{name}: a number is required, got {type(v).__name__}")
    v = float(v)
    if 3.4028235e38 < abs(v) < math.inf:
        raise ValueError(f"{name}: {v} does not fit fp32")
    return v


def _explain(t, name, shape, dtype, index):
    """Raises for the first thing wrong with an argument (contiguous rows asked for)."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, expected {f'cuda:{index}' if index >= 0 else 'cpu'}")
    raise ValueError(f"{name}: the last dimension must be contiguous")


def _rows(t, name, shape, dtype, index):
    """Strides of a tensor of this shape, type and device with contiguous rows."""
    st = _tensor(t, name).stride()
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or (st[-1] != 1 and shape[-1] > 1):
        _explain(t, name, shape, dtype, index)
    return st


def _flat(t, name, shape, dtype, index):
    """Address of a contiguous tensor of this shape, type and device."""
    if _tensor(t, name).shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _explain(t, name, shape, dtype, index)
    return t.data_ptr()


def _workspace(ws, cache, q):
    """Address and bytes of a workspace on the cache's and the queries' device, whose
    elements lie one after the other (an expanded tensor counts more than it has)."""
    if not _tensor(ws, "ws").is_contiguous():
        raise ValueError("ws must be a contiguous tensor")
    if cache._dev != q.get_device() or ws.get_device() != cache._dev:
        raise ValueError(f"cache on {cache.device} and ws on {ws.device}, expected both on {q.device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def moe_add_rmsnorm(x, weight, out, residual=None, residual_out=None, scales=None, group=0, eps=1e-6, stream=None):
    """RMS norm of ``x (+ residual)`` [T, H] times ``weight`` [H] into ``out``:
    x's dtype, or float8_e4m3fn with ``scales`` [T, 1] (one per row) or
    [T, ceil(H / group)].  ``residual_out`` receives the rounded sum (may be
    ``residual`` itself).  Rows may be strided; see include/moe.h."""
    if _fast is not None:
        rc = _fast.norm(x, weight, out, residual, residual_out, scales, group, eps, stream)
        if rc == 0:
            return
        if rc > 0:
            _check(rc)
    shape, dt, dev = _tensor(x, "x").shape, x.dtype, x.get_device()
    if len(shape) != 2:
        raise ValueError(f"x: shape {tuple(shape)}, expected [T, H]")
    T, H = shape
    code = _FLOATS.get(dt)
    if code is None:
        raise ValueError(f"x: dtype {dt}, expected float16 or bfloat16")
    e4m3 = _tensor(out, "out").dtype is torch.float8_e4m3fn
    group, eps = _int32(group, "group"), _fp32(eps, "eps")
    xs = _rows(x, "x", shape, dt, dev)[0]
    os_ = _rows(out, "out", shape, out.dtype if e4m3 else dt, dev)[0]
    _rows(weight, "weight", (H,), dt, dev)
    r = ro = s = rs = ros = 0
    if residual is not None:
        rs = _rows(residual, "residual", shape, dt, dev)[0]
        r = residual.data_ptr()
    if residual_out is not None:
        if residual is None:
            raise ValueError("residual_out without residual")
        ros = _rows(residual_out, "residual_out", shape, dt, dev)[0]
        ro = residual_out.data_ptr()
    if T == 1:  # a single row's stride says nothing
        xs = os_ = rs = ros = H
    if (scales is not None) != e4m3:
        raise ValueError("scales goes with a float8_e4m3fn out, and only with it")
    if e4m3:
        if group < 0:
            raise ValueError("group must be >= 0")
        s = _flat(scales, "scales", (T, -(-H // group) if group else 1), torch.float32, dev)
    args = _NORM_T.pack(x.data_ptr(), r, weight.data_ptr(), out.data_ptr(), ro, s, xs, rs, os_, ros, T, H, code,
                        MOE_E4M3 if e4m3 else code, group, eps)
    rc = (_lib or _load()).moe_add_rmsnorm(args, _launch_stream(dev, stream))
    if rc:
        _check(rc)


class MoeKvCache:
    """A paged key/value cache as the library takes it: ``k`` and ``v``
    [n_pages, page_size, n_kv_heads, head_dim] in float16, bfloat16 or
    float8_e4m3fn (then with optional fp32 ``k_scale`` and ``v_scale`` per
    kv head).  Any order of pages, tokens and heads in memory (permuted views
    are fine) with contiguous rows.  Holds the tensors; checked once here."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if _tensor(k, "k").dim() != 4:
            raise ValueError(f"k: shape {tuple(k.shape)}, expected [pages, page, kv heads, head_dim]")
        if k.dtype not in (torch.float16, torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"k: dtype {k.dtype}, expected float16, bfloat16 or float8_e4m3fn")
        dev = k.get_device()
        _rows(k, "k", k.shape, k.dtype, dev)
        _rows(v, "v", k.shape, k.dtype, dev)
        e4m3 = k.dtype is torch.float8_e4m3fn
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                if not e4m3:
                    raise ValueError(f"{name} goes with a float8_e4m3fn cache only")
                _flat(t, name, (k.shape[2],), torch.float32, dev)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = k.shape
        self.dtype, self.device, self._dev = k.dtype, k.device, dev
        if max(self.n_pages, self.page_size, self.n_kv_heads) > 0x7fffffff:
            raise ValueError("cache sizes must be below 2^31")
        self._c = _CACHE_T.pack(k.data_ptr(), v.data_ptr(), 0 if k_scale is None else k_scale.data_ptr(),
                                0 if v_scale is None else v_scale.data_ptr(), *k.stride()[:3], *v.stride()[:3],
                                self.n_pages, self.page_size, self.n_kv_heads, self.head_dim,
                                MOE_E4M3 if e4m3 else _DT_CODE[k.dtype])


def moe_attention_workspace_bytes(cache: MoeKvCache, n_q_heads: int) -> int:
    return int(_load().moe_attention_workspace_bytes(cache._c, int(n_q_heads)))


def moe_attention_form(cache: MoeKvCache, B: int, n_q_heads: int, max_pages: int, window: int = 0) -> str | None:
    """Which kernels serve a batch of these sizes: "ctas" or "teams" (None: refused)."""
    return (None, "ctas", "teams")[_load().moe_attention_form(cache._c, B, n_q_heads, max_pages, window)]


def alloc_attention_workspace(cache: MoeKvCache, n_q_heads: int) -> torch.Tensor:
    """A zero-filled, 256-byte aligned workspace for moe_paged_attention (any
    batch and lengths) and moe_rope_append on this cache."""
    n = moe_attention_workspace_bytes(cache, n_q_heads)
    if n == 0:
        raise MoeError(1, "n_q_heads must be a positive multiple of the cache's kv heads")
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=cache.device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def moe_rope_append(cache: MoeKvCache, q, k, v, positions, slots, inv_freq, q_out, ws, q_norm_w=None, k_norm_w=None,
                    eps=1e-6, interleaved=False, stream=None):
    """Rotates new ``q`` [T, Hq, D] (into ``q_out``) and ``k`` [T, Hkv, D] by
    ``positions`` [T] int64 and ``inv_freq`` [rot_dim / 2] fp32, after a per-head
    RMS norm when ``q_norm_w`` and ``k_norm_w`` [D] are given, and stores k and v
    in the cache's ``slots`` [T] int64 (page * page_size + place; negative:
    not stored)."""
    if _fast is not None and isinstance(cache, MoeKvCache):
        rc = _fast.rope(cache._c, cache._dev, q, k, v, positions, slots, inv_freq, q_out, ws, q_norm_w, k_norm_w, eps,
                        interleaved, stream)
        if rc == 0:
            return
        if rc > 0:
            _check(rc)
    if not isinstance(cache, MoeKvCache):
        raise ValueError("cache: a MoeKvCache is required")
    shape, dt, dev = _tensor(q, "q").shape, q.dtype, q.get_device()
    code = _FLOATS.get(dt)
    if code is None:
        raise ValueError(f"q: dtype {dt}, expected float16 or bfloat16")
    D = cache.head_dim
    if len(shape) != 3 or shape[2] != D:
        raise ValueError(f"q: shape {tuple(shape)}, expected [T, heads, {D}]")
    T, hq, _ = shape
    kv = (T, cache.n_kv_heads, D)
    qs = _rows(q, "q", shape, dt, dev)
    ks = _rows(k, "k", kv, dt, dev)
    vs = _rows(v, "v", kv, dt, dev)
    os_ = _rows(q_out, "q_out", shape, dt, dev)
    pos = _flat(positions, "positions", (T,), torch.int64, dev)
    slot = _flat(slots, "slots", (T,), torch.int64, dev)
    n_freq = _tensor(inv_freq, "inv_freq").numel()
    freq = _flat(inv_freq, "inv_freq", (n_freq,), torch.float32, dev)
    ws_p, ws_bytes = _workspace(ws, cache, q)
    qn = kn = 0
    if q_norm_w is not None or k_norm_w is not None:
        if q_norm_w is None or k_norm_w is None:
            raise ValueError("q_norm_w and k_norm_w go together")
        qn = _flat(q_norm_w, "q_norm_w", (D,), dt, dev)
        kn = _flat(k_norm_w, "k_norm_w", (D,), dt, dev)
    args = _ROPE_T.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), pos, slot, freq, qn, kn,
                        qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os_[0], os_[1], T, hq, 2 * n_freq, code,
                        1 if interleaved else 0, _fp32(eps, "eps"))
    rc = (_lib or _load()).moe_rope_append(cache._c, args, ws_p, ws_bytes, _launch_stream(dev, stream))
    if rc:
        _check(rc)


def moe_paged_attention(cache: MoeKvCache, q, block_table, seq_lens, out, ws, scale=None, window=0, lse=None,
                        stream=None):
    """Attention of one new token per sequence: ``q`` [B, Hq, D] over the
    ``seq_lens`` [B] int32 cached tokens that ``block_table`` [B, max_pages]
    int32 places, into ``out`` [B, Hq, D] (and ``lse`` [B, Hq] fp32).  ``scale``
    defaults to D ** -0.5; ``window`` > 0 keeps the last ``window`` tokens."""
    if _fast is not None and isinstance(cache, MoeKvCache):
        rc = _fast.attention(cache._c, cache._dev, q, block_table, seq_lens, out, ws, scale, window, lse, stream)
        if rc == 0:
            return
        if rc > 0:
            _check(rc)
    if not isinstance(cache, MoeKvCache):
        raise ValueError("cache: a MoeKvCache is required")
    shape, dt, dev = _tensor(q, "q").shape, q.dtype, q.get_device()
    code = _FLOATS.get(dt)
    if code is None:
        raise ValueError(f"q: dtype {dt}, expected float16 or bfloat16")
    D = cache.head_dim
    if len(shape) != 3 or shape[2] != D:
        raise ValueError(f"q: shape {tuple(shape)}, expected [B, heads, {D}]")
    B, hq, _ = shape
    qs = _rows(q, "q", shape, dt, dev)
    os_ = _rows(out, "out", shape, dt, dev)
    pages = block_table.shape[-1] if _tensor(block_table, "block_table").dim() else 0
    bs = _rows(block_table, "block_table", (B, pages), torch.int32, dev)
    lens = _flat(seq_lens, "seq_lens", (B,), torch.int32, dev)
    lse_p = 0 if lse is None else _flat(lse, "lse", (B, hq), torch.float32, dev)
    ws_p, ws_bytes = _workspace(ws, cache, q)
    args = _ATTN_T.pack(q.data_ptr(), out.data_ptr(), lse_p, block_table.data_ptr(), lens, qs[0], qs[1], os_[0], os_[1],
                        bs[0], B, hq, pages, _int32(window, "window"), code,
                        D ** -0.5 if scale is None else _fp32(scale, "scale"))
    rc = (_lib or _load()).moe_paged_attention(cache._c, args, ws_p, ws_bytes, _launch_stream(dev, stream))
    if rc:
        _check(rc)


def cfg_from_workload(wl, out_dtype=None, flags=0) -> MoeCfg:
    """MoeCfg for a synthetic workload description (moe_synth.Workload)."""
    return MoeCfg(wl.hidden, wl.n_experts, wl.top_k, wl.inter, wl.shared_inter, wl.dtype, out_dtype,
                  wl.norm_topk, wl.has_shared_gate, flags)
