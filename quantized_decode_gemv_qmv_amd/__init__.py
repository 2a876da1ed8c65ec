"""Quantized decode matvec for AMD MI355X (gfx950).

Python binding of ``libqmv.so`` (the C ABI declared in ``include/qmv.h``).
This module only marshals arguments: every step of the computation runs in
the library's HIP kernels.  PyTorch supplies device memory and the stream; the
calls are enqueued on ``torch.cuda.current_stream()`` unless a stream is
given, and never synchronize.

If the library has not been built, importing works but the first call raises
``RuntimeError`` -- there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re

import torch

__all__ = [
    "Q8_0", "Q4_K", "IQ4_XS", "Q5_K", "Q6_K", "Q8G128", "QmvError", "lib", "library_path", "symbols",
    "row_bytes", "act_bytes", "act_offsets", "act_fields", "matvec_workspace_bytes",
    "moe_workspace_bytes", "quantize_act", "matvec", "matvec_x", "matvec_batch", "moe_matvec", "moe_matvec_noalloc",
    "moe_gate_up_swiglu",
    "block_dots",
    "block_dots_mx", "moe_block_dots", "stream_read",
    "rmsnorm_quantize", "kv_append", "kv_attn", "kv_attn_workspace_bytes", "KV_BLOCK",
    "set_tuning", "swiglu_quantize", "router_topk", "variant_name", "variants", "pick_variant", "matvec_plan", "MAX_TOKENS", "MAX_MOE_TOKENS",
]

Q8_0, Q4_K, IQ4_XS, Q5_K, Q6_K, Q8G128 = 0, 1, 2, 3, 4, 5
MAX_TOKENS = 16
MAX_MOE_TOKENS = 64
MAX_BATCH = 8
KV_BLOCK = 64

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
_LIB = os.path.join(_PKG, "libqmv.so")
_HEADER = os.path.join(_ROOT, "include", "qmv.h")
_lib = None


class _Item(ctypes.Structure):
    """qmv_matvec_item of include/qmv.h."""
    _fields_ = [("w", ctypes.c_void_p), ("n_rows", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64), ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64)]


class _Kv(ctypes.Structure):
    """qmv_kv of include/qmv.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("n_blocks", ctypes.c_int64),
                ("n_kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("block_table", ctypes.c_void_p),
                ("table_width", ctypes.c_int64), ("seq_lens", ctypes.c_void_p), ("tok_start", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int64), ("n_tok", ctypes.c_int64), ("max_q", ctypes.c_int64)]


class QmvError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = _lib.qmv_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{what}: {msg}")
        self.status = status


def library_path() -> str:
    return _LIB


def symbols() -> list[str]:
    """Function names declared in include/qmv.h."""
    with open(_HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(qmv_\w+)\s*\(", text)))


def lib():
    """The loaded library; raises if it was never built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB):
        raise RuntimeError(f"{_LIB} is missing: build it with __graft_entry__.build() "
                           "(or python quantized_decode_gemv_qmv_amd/build.py)")
    L = ctypes.CDLL(_LIB)
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sig = {
        "qmv_abi_version": ([], I),
        "qmv_last_hip_error": ([], I),
        "qmv_last_hip_error_name": ([], ctypes.c_char_p),
        "qmv_status_string": ([I], ctypes.c_char_p),
        "qmv_row_bytes": ([I, I64], SZ),
        "qmv_act_bytes": ([I64, I64], SZ),
        "qmv_act_offset_d": ([I64, I64], SZ),
        "qmv_act_offset_s": ([I64, I64], SZ),
        "qmv_quantize_act": ([P, I64, I64, I64, P, P], I),
        "qmv_swiglu_quantize": ([P, I64, I64, I64, P, P, P], I),
        "qmv_router_topk": ([P, I64, I64, I64, P, I64, I64, P, P, P, P, P], I),
        "qmv_matvec_workspace_bytes": ([I, I64, I64, I64], SZ),
        "qmv_matvec": ([I, P, I64, I64, P, I64, P, I64, P, SZ, P], I),
        "qmv_matvec_batch": ([I, ctypes.POINTER(_Item), I64, I64, P, I64, P], I),
        "qmv_matvec_x": ([I, P, I64, I64, P, I64, I64, P, I64, P, P, SZ, P], I),
        "qmv_moe_workspace_bytes": ([I, I64, I64, I64, I64, I64], SZ),
        "qmv_moe_matvec": ([I, P, I64, I64, I64, P, I, P, P, I64, I64, P, P, SZ, P], I),
        "qmv_moe_matvec_noalloc": ([I, P, I64, I64, I64, P, I, P, P, I64, I64, P, P], I),
        "qmv_moe_gate_up_swiglu": ([I, P, I64, I64, I64, P, P, I64, I64, P, P, P, SZ, P], I),
        "qmv_rmsnorm_quantize": ([P, I64, P, I64, I64, I64, P, ctypes.c_float, P, I64, P, I64, P, P], I),
        "qmv_kv_append": ([ctypes.POINTER(_Kv), P, I64, P, I64, P], I),
        "qmv_kv_attn_workspace_bytes": ([I64, I64, I64, I64, I64, I64, I64], SZ),
        "qmv_kv_attn": ([ctypes.POINTER(_Kv), P, I64, I64, ctypes.c_float, I64, P, I64, P, P, SZ, P], I),
        "qmv_block_dots": ([I, P, I64, I64, P, I64, P, P], I),
        "qmv_block_dots_mx": ([I, P, I64, I64, P, I64, I64, I, P, P], I),
        "qmv_moe_block_dots": ([I, P, I64, I64, I64, P, I, P, I64, I64, I64, P, P, SZ, P], I),
        "qmv_stream_read": ([P, I64, P, P], I),
        "qmv_set_tuning": ([ctypes.c_char_p, I64], I),
        "qmv_variant_name": ([I64], ctypes.c_char_p),
        "qmv_pick_variant": ([I, I64, I64, I64], I64),
        "qmv_matvec_plan": ([I, I64, I64, I64, I, ctypes.POINTER(I64), ctypes.POINTER(I)], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


# ------------------------------------------------------------------ helpers
def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without a Stream object around it (0.1 us
# against 3 us for torch.cuda.current_stream())
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        if _raw_stream is not None:
            return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, what: str) -> None:
    if status != 0:
        if status == 5:  # QMV_ERR_HIP: name the runtime's error
            what = f"{what} ({lib().qmv_last_hip_error_name().decode()})"
        raise QmvError(status, what)


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")


# ------------------------------------------------------------------- sizes
def row_bytes(fmt: int, k: int) -> int:
    return int(lib().qmv_row_bytes(fmt, k))


@functools.lru_cache(maxsize=4096)
def act_bytes(n_tok: int, k: int) -> int:
    return int(lib().qmv_act_bytes(n_tok, k))


@functools.lru_cache(maxsize=4096)
def act_offsets(n_tok: int, k: int) -> tuple[int, int]:
    L = lib()
    return int(L.qmv_act_offset_d(n_tok, k)), int(L.qmv_act_offset_s(n_tok, k))


def act_fields(xq: torch.Tensor, n_tok: int, k: int):
    """Views (qs int8 [T][K], d fp32 [T][K/32], s int32 [T][K/32]) of a Q8
    activation buffer."""
    od, os_ = act_offsets(n_tok, k)
    nb = k // 32
    if xq.numel() < os_ + 4 * n_tok * nb:  # the fields' end; what pads the buffer behind it may be missing
        raise ValueError("activation buffer too small")
    if xq.numel() % 4 == 0 and xq.storage_offset() % 4 == 0 and xq.dim() == 1 and xq.stride(0) == 1:
        # two tensor operations a field
        d, s = xq.view(torch.float32), xq.view(torch.int32)
        at, shape, st = d.storage_offset(), (n_tok, nb), (nb, 1)
        return (xq.view(torch.int8).as_strided((n_tok, k), (k, 1)), d.as_strided(shape, st, at + od // 4),
                s.as_strided(shape, st, at + os_ // 4))
    qs = xq[: n_tok * k].view(torch.int8).view(n_tok, k)
    d = xq[od: od + 4 * n_tok * nb].view(torch.float32).view(n_tok, nb)
    s = xq[os_: os_ + 4 * n_tok * nb].view(torch.int32).view(n_tok, nb)
    return qs, d, s


def swiglu_quantize(gu: torch.Tensor, n_ff: int, out: torch.Tensor | None = None,
                    h_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gu fp32 [R][>= 2 n_ff] (gate | up) -> Q8 activation buffer of
    h = silu(gate) * up [R][n_ff]; h_out (fp32 [R][n_ff]) receives h."""
    _need(gu, torch.float32, "gu")
    if gu.dim() != 2 or gu.stride(1) != 1:
        raise ValueError("gu must be a 2-D tensor with unit column stride")
    rows = gu.shape[0]
    if out is None:
        out = torch.empty(act_bytes(rows, n_ff), dtype=torch.uint8, device=gu.device)
    if h_out is not None:
        _need(h_out, torch.float32, "h_out")
    ldg = gu.stride(0) if rows > 1 else gu.shape[1]  # a single row's stride is arbitrary
    _check(lib().qmv_swiglu_quantize(_ptr(gu), ldg, rows, n_ff, _ptr(out), _ptr(h_out),
                                     _stream(stream)), "qmv_swiglu_quantize")
    return out


def router_topk(x: torch.Tensor, wr: torch.Tensor, top_k: int, ids: torch.Tensor | None = None,
                weights: torch.Tensor | None = None, logits: torch.Tensor | None = None,
                xq: torch.Tensor | None = None, stream=None):
    """x fp32 [T][K], router weights fp32 [E][K] -> (ids int32 [T][top_k],
    weights fp32 [T][top_k]); logits (fp32 [T][E], allocated when None)
    receives the router logits, xq (optional) the Q8 blocks of x.  x may
    have a row stride beyond K (a multiple of 4)."""
    if x.dim() == 1:
        x = x.view(1, -1)
    if x.dtype != torch.float32 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a float32 CUDA tensor with unit column stride")
    _need(wr, torch.float32, "wr")
    n_tok, k = x.shape
    e = wr.shape[0]
    if ids is None:
        ids = torch.empty((n_tok, top_k), dtype=torch.int32, device=x.device)
    if weights is None:
        weights = torch.empty((n_tok, top_k), dtype=torch.float32, device=x.device)
    if logits is None:
        logits = torch.empty((n_tok, e), dtype=torch.float32, device=x.device)
    _need(logits, torch.float32, "logits")
    ldx = x.stride(0) if n_tok > 1 else k
    if xq is not None:
        _need(xq, torch.uint8, "xq")
        if xq.numel() < act_bytes(n_tok, k):
            raise ValueError("activation buffer too small")
    _check(lib().qmv_router_topk(_ptr(x), ldx, n_tok, k, _ptr(wr), e, top_k, _ptr(ids), _ptr(weights),
                                 _ptr(logits), _ptr(xq), _stream(stream)), "qmv_router_topk")
    return ids, weights


def matvec_workspace_bytes(fmt: int, n_rows: int, k: int, n_tok: int) -> int:
    return int(lib().qmv_matvec_workspace_bytes(fmt, n_rows, k, n_tok))


def moe_workspace_bytes(fmt: int, n_experts: int, n_rows: int, k: int, n_tok: int,
                        top_k: int) -> int:
    return int(lib().qmv_moe_workspace_bytes(fmt, n_experts, n_rows, k, n_tok, top_k))


# --------------------------------------------------------------- entry points
def quantize_act(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x fp32 [T][K] (row stride >= K) -> Q8 activation buffer (uint8)."""
    if x.dim() == 1:
        x = x.view(1, -1)
    if x.dtype != torch.float32 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a float32 CUDA tensor with unit column stride")
    n_tok, k = x.shape
    nbytes = act_bytes(n_tok, k)
    if out is None:
        out = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    _need(out, torch.uint8, "out")
    if out.numel() < nbytes:
        raise ValueError("activation buffer too small")
    ldx = x.stride(0) if n_tok > 1 else k  # a single row's stride is arbitrary
    _check(lib().qmv_quantize_act(_ptr(x), ldx, n_tok, k, _ptr(out), _stream(stream)),
           "qmv_quantize_act")
    return out


def matvec(fmt: int, w: torch.Tensor, n_rows: int, k: int, xq: torch.Tensor, n_tok: int,
           y: torch.Tensor | None = None, ws: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """y fp32 [T][N] = W xq.  ``ws`` (uint8, zero-filled once) enables split-K."""
    _need(w, torch.uint8, "w")
    _need(xq, torch.uint8, "xq")
    if y is None:
        y = torch.empty((n_tok, n_rows), dtype=torch.float32, device=w.device)
    if y.dtype != torch.float32 or not y.is_cuda or y.dim() != 2 or y.stride(1) != 1:
        raise ValueError("y must be a float32 CUDA tensor [T][ldy] with unit column stride")
    if w.numel() < n_rows * row_bytes(fmt, k):
        raise ValueError("w holds fewer than n_rows rows")
    wsz = 0 if ws is None else ws.numel()
    if ws is not None:
        _need(ws, torch.uint8, "ws")
    ldy = y.stride(0) if y.shape[0] > 1 else y.shape[1]
    _check(lib().qmv_matvec(fmt, _ptr(w), n_rows, k, _ptr(xq), n_tok, _ptr(y), ldy,
                            _ptr(ws), wsz, _stream(stream)), "qmv_matvec")
    return y


def matvec_x(fmt: int, w: torch.Tensor, n_rows: int, k: int, x: torch.Tensor,
             xq: torch.Tensor | None = None, y: torch.Tensor | None = None, ws: torch.Tensor | None = None,
             stream=None):
    """The decode step from fp32 x [T][K]: (y [T][N] = W Q8(x), xq = Q8(x)).
    One launch for one or two tokens (the matvec quantizes x itself)."""
    _need(w, torch.uint8, "w")
    if x.dim() == 1:
        x = x.view(1, -1)
    if x.dtype != torch.float32 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a float32 CUDA tensor with unit column stride")
    n_tok = x.shape[0]
    if xq is None:
        xq = torch.empty(act_bytes(n_tok, k), dtype=torch.uint8, device=x.device)
    _need(xq, torch.uint8, "xq")
    if y is None:
        y = torch.empty((n_tok, n_rows), dtype=torch.float32, device=w.device)
    if y.dtype != torch.float32 or not y.is_cuda or y.dim() != 2 or y.stride(1) != 1:
        raise ValueError("y must be a float32 CUDA tensor [T][ldy] with unit column stride")
    if w.numel() < n_rows * row_bytes(fmt, k):
        raise ValueError("w holds fewer than n_rows rows")
    if ws is not None:
        _need(ws, torch.uint8, "ws")
    _check(lib().qmv_matvec_x(fmt, _ptr(w), n_rows, k, _ptr(x), _ld(x), n_tok, _ptr(y), _ld(y), _ptr(xq),
                              _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)), "qmv_matvec_x")
    return y, xq


def _ld(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]  # a single row's stride is arbitrary


def matvec_batch(fmt: int, items, k: int, xq: torch.Tensor, n_tok: int, stream=None) -> list:
    """Sibling matvecs over one activation buffer in one launch.  ``items`` is
    a sequence of (w, n_rows, y, residual): y (fp32 [T][>= n_rows], allocated
    when None) receives W xq, plus residual (fp32 [T][>= n_rows]) when it is
    not None; residual may be y itself.  Returns the list of y."""
    _need(xq, torch.uint8, "xq")
    arr = (_Item * max(1, len(items)))()
    outs = []
    for i, (w, n_rows, y, res) in enumerate(items):
        _need(w, torch.uint8, "w")
        if w.numel() < n_rows * row_bytes(fmt, k):
            raise ValueError("w holds fewer than n_rows rows")
        if y is None:
            y = torch.empty((n_tok, n_rows), dtype=torch.float32, device=w.device)
        for name, t in (("y", y), ("residual", res)):
            if t is not None and (t.dtype != torch.float32 or not t.is_cuda or t.dim() != 2
                                  or t.stride(1) != 1):
                raise ValueError(f"{name} must be a float32 CUDA tensor [T][ld] with unit column stride")
        arr[i] = _Item(w.data_ptr(), n_rows, y.data_ptr(), _ld(y),
                       None if res is None else res.data_ptr(), 0 if res is None else _ld(res))
        outs.append(y)
    _check(lib().qmv_matvec_batch(fmt, arr, len(items), k, _ptr(xq), n_tok, _stream(stream)),
           "qmv_matvec_batch")
    return outs


def moe_matvec(fmt: int, w: torch.Tensor, n_experts: int, n_rows: int, k: int,
               xq: torch.Tensor, x_per_slot: bool, ids: torch.Tensor,
               route_w: torch.Tensor | None, ws: torch.Tensor,
               y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Expert-grouped routed matvec.  route_w None -> y [T][top_k][N];
    else y [T][N] = sum_s route_w[t][s] * W[ids[t][s]] x."""
    _need(w, torch.uint8, "w")
    _need(xq, torch.uint8, "xq")
    _need(ids, torch.int32, "ids")
    _need(ws, torch.uint8, "ws")
    n_tok, top_k = ids.shape
    if route_w is not None:
        _need(route_w, torch.float32, "route_w")
        if tuple(route_w.shape) != (n_tok, top_k):
            raise ValueError("route_w must match ids")
    shape = (n_tok, n_rows) if route_w is not None else (n_tok, top_k, n_rows)
    if y is None:
        y = torch.empty(shape, dtype=torch.float32, device=w.device)
    _need(y, torch.float32, "y")
    if y.numel() < n_tok * n_rows * (1 if route_w is not None else top_k):
        raise ValueError("y too small")
    if w.numel() < n_experts * n_rows * row_bytes(fmt, k):
        raise ValueError("w holds fewer than n_experts * n_rows rows")
    _check(lib().qmv_moe_matvec(fmt, _ptr(w), n_experts, n_rows, k, _ptr(xq), int(bool(x_per_slot)),
                                _ptr(ids), _ptr(route_w), n_tok, top_k, _ptr(y), _ptr(ws),
                                ws.numel(), _stream(stream)), "qmv_moe_matvec")
    return y


def moe_gate_up_swiglu(fmt: int, w: torch.Tensor, n_experts: int, n_ff: int, k: int, xq: torch.Tensor,
                       ids: torch.Tensor, ws: torch.Tensor, hq: torch.Tensor | None = None,
                       gu: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Routed gate+up (2 n_ff rows per expert, gate first) with SwiGLU and
    Q8 folded in: returns hq, the Q8 activation buffer of the n_tok * top_k
    slot rows of h; gu (fp32 [T][top_k][2 n_ff]), if given, receives the
    gate+up outputs."""
    _need(w, torch.uint8, "w")
    _need(xq, torch.uint8, "xq")
    _need(ids, torch.int32, "ids")
    _need(ws, torch.uint8, "ws")
    n_tok, top_k = ids.shape
    if hq is None:
        hq = torch.empty(act_bytes(n_tok * top_k, n_ff), dtype=torch.uint8, device=w.device)
    _need(hq, torch.uint8, "hq")
    if hq.numel() < act_bytes(n_tok * top_k, n_ff):
        raise ValueError("hq too small")
    if gu is not None:
        _need(gu, torch.float32, "gu")
        if gu.numel() < n_tok * top_k * 2 * n_ff:
            raise ValueError("gu too small")
    if w.numel() < n_experts * 2 * n_ff * row_bytes(fmt, k):
        raise ValueError("w holds fewer than n_experts * 2 n_ff rows")
    _check(lib().qmv_moe_gate_up_swiglu(fmt, _ptr(w), n_experts, n_ff, k, _ptr(xq), _ptr(ids), n_tok, top_k,
                                        _ptr(hq), _ptr(gu), _ptr(ws), ws.numel(), _stream(stream)),
           "qmv_moe_gate_up_swiglu")
    return hq


def moe_matvec_noalloc(fmt: int, w: torch.Tensor, n_experts: int, n_rows: int, k: int,
                       xq: torch.Tensor, x_per_slot: bool, ids: torch.Tensor,
                       route_w: torch.Tensor | None, y: torch.Tensor, stream=None) -> torch.Tensor:
    """moe_matvec on the library's device-resident workspace (no caller
    workspace; y must be given, so that nothing is allocated)."""
    _need(w, torch.uint8, "w")
    _need(xq, torch.uint8, "xq")
    _need(ids, torch.int32, "ids")
    _need(y, torch.float32, "y")
    n_tok, top_k = ids.shape
    if route_w is not None:
        _need(route_w, torch.float32, "route_w")
        if tuple(route_w.shape) != (n_tok, top_k):
            raise ValueError("route_w must match ids")
    if y.numel() < n_tok * n_rows * (1 if route_w is not None else top_k):
        raise ValueError("y too small")
    if w.numel() < n_experts * n_rows * row_bytes(fmt, k):
        raise ValueError("w holds fewer than n_experts * n_rows rows")
    _check(lib().qmv_moe_matvec_noalloc(fmt, _ptr(w), n_experts, n_rows, k, _ptr(xq), int(bool(x_per_slot)),
                                        _ptr(ids), _ptr(route_w), n_tok, top_k, _ptr(y), _stream(stream)),
           "qmv_moe_matvec_noalloc")
    return y


# ------------------------------------- norm, cache append and attention
def _here(*tensors) -> int:
    """The current device, on which every tensor has to be: the call is
    enqueued on one of its streams."""
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() or torch.cuda.is_available() else -2
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("every tensor must be on the current CUDA device")
    return dev


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """A tensor for a call on `stream` to write, of that stream's memory."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _rows(t: torch.Tensor, shape, name: str) -> int:
    """Checks an fp32 row array and gives its row stride.  A single row may come without its dimension."""
    if t.dim() == 1 and len(shape) == 2 and shape[0] == 1:
        t = t.view(1, -1)
    st = t.stride()
    if t.dtype != torch.float32 or t.shape != shape or st[-1] != 1 \
            or (len(shape) == 3 and shape[1] > 1 and st[1] != shape[2]):
        raise ValueError(f"{name} must be a float32 tensor {list(shape)} whose rows lie in one piece")
    return st[0] if shape[0] > 1 else math.prod(shape[1:])  # a single row's stride is arbitrary


def _whole(t: torch.Tensor, dtype, name: str) -> int:
    """Checks a tensor that the call takes in one piece and gives its address."""
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor")
    return t.data_ptr()


def rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
                     residual: torch.Tensor | None = None, sum_out: torch.Tensor | None = None,
                     y_out: torch.Tensor | None = None, xq: torch.Tensor | None = None, stream=None):
    """x fp32 [T][K] (+ residual) -> (r, xq): r = x + residual (in sum_out,
    allocated when None; x itself without a residual and a sum_out) and the
    Q8 activation buffer of rmsnorm(r) * weight.  y_out fp32 [T][K], if given,
    receives the normed rows.  sum_out may be x or residual, and so may y_out
    if sum_out is not the same one (without a residual and a sum_out, a y_out
    that is x leaves the normed rows in what is returned as r).  A single row
    may be given as [K], the outputs and the residual too."""
    if x.dim() == 1:
        x = x.view(1, -1)
    if x.dim() != 2:
        raise ValueError("x must be a 1-D or 2-D tensor")
    _here(x, weight, residual, sum_out, y_out, xq)
    shape = x.shape
    n_tok, k = shape
    ldx = _rows(x, shape, "x")
    wp = _whole(weight, torch.float32, "weight")
    if weight.numel() != k:
        raise ValueError("weight must hold one value a column of x")
    rp = sp = yp = None
    ldr = lds = ldy = 0
    if residual is not None:
        ldr, rp = _rows(residual, shape, "residual"), residual.data_ptr()
        if sum_out is None:
            sum_out = _new(x, shape, torch.float32, stream)
    if sum_out is not None:
        lds, sp = _rows(sum_out, shape, "sum_out"), sum_out.data_ptr()
    if y_out is not None:
        ldy, yp = _rows(y_out, shape, "y_out"), y_out.data_ptr()
    nbytes = act_bytes(n_tok, k)
    if xq is None:
        xq = _new(x, (max(nbytes, 1),), torch.uint8, stream)
    qp = _whole(xq, torch.uint8, "xq")
    if xq.numel() < nbytes:
        raise ValueError("activation buffer too small")
    _check(lib().qmv_rmsnorm_quantize(x.data_ptr(), ldx, rp, ldr, n_tok, k, wp, eps, sp, lds, yp, ldy, qp,
                                      _stream(stream)), "qmv_rmsnorm_quantize")
    return (x if sum_out is None else sum_out), xq


def _kv(codes, scales, block_table, seq_lens, tok_start, n_tok, max_q, dim) -> _Kv:
    n_seqs = seq_lens.numel()
    cs = codes.shape
    if len(cs) != 4 or cs[1] != 2 or cs[3] != KV_BLOCK * dim:
        raise ValueError(f"codes must be [n_blocks][2][n_kv_heads][{KV_BLOCK} * head_dim]")
    if scales.shape != cs[:3]:
        raise ValueError("scales must be [n_blocks][2][n_kv_heads]")
    ts = block_table.shape
    if len(ts) != 2 or ts[0] != n_seqs:
        raise ValueError("block_table must be [n_seqs][blocks of a sequence]")
    start = None
    if tok_start is not None:
        start = _whole(tok_start, torch.int32, "tok_start")
        if tok_start.numel() != n_seqs + 1:
            raise ValueError("tok_start must hold n_seqs + 1 rows")
    return _Kv(_whole(codes, torch.int8, "codes"), _whole(scales, torch.float32, "scales"), cs[0], cs[2], dim,
               _whole(block_table, torch.int32, "block_table"), ts[1], _whole(seq_lens, torch.int32, "seq_lens"),
               start, n_seqs, n_tok, max_q)


def kv_append(k: torch.Tensor, v: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
              block_table: torch.Tensor, seq_lens: torch.Tensor, tok_start: torch.Tensor | None = None,
              max_q: int = 1, stream=None) -> None:
    """Writes keys and values fp32 [T][n_kv_heads][head_dim] (rows may be
    strided) at the end of their sequences in an 8-bit block cache: codes int8
    [n_blocks][2][n_kv_heads][64 * head_dim] and scales fp32
    [n_blocks][2][n_kv_heads], changed in place.  seq_lens (int32) counts the
    new tokens; block_table int32 [n_seqs][blocks]; tok_start int32
    [n_seqs + 1] the rows of each sequence, at most max_q (None: max_q each)."""
    shape = k.shape
    if len(shape) != 3:
        raise ValueError("k and v must be [T][n_kv_heads][head_dim]")
    _here(k, v, codes, scales, block_table, seq_lens, tok_start)
    kv = _kv(codes, scales, block_table, seq_lens, tok_start, shape[0], max_q, shape[2])
    if kv.n_kv_heads != shape[1]:
        raise ValueError("k has another number of heads than codes")
    _check(lib().qmv_kv_append(ctypes.byref(kv), k.data_ptr(), _rows(k, shape, "k"), v.data_ptr(),
                               _rows(v, shape, "v"), _stream(stream)), "qmv_kv_append")


def kv_attn_workspace_bytes(n_seqs: int, n_tok: int, max_q: int, n_heads: int, n_kv_heads: int, head_dim: int,
                            table_width: int) -> int:
    return int(lib().qmv_kv_attn_workspace_bytes(n_seqs, n_tok, max_q, n_heads, n_kv_heads, head_dim, table_width))


def kv_attn(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
            seq_lens: torch.Tensor, tok_start: torch.Tensor | None = None, max_q: int = 1,
            scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
            xq: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of q fp32 [T][n_heads][head_dim] over the cache that
    kv_append writes (see there), causal, over the last `window` positions if
    that is not 0; scale None: 1 / sqrt(head_dim).  Returns out fp32
    [T][n_heads][head_dim] (allocated when None); xq, if given, receives the
    Q8 blocks of its rows.  ``ws`` (uint8, zero-filled once, of
    kv_attn_workspace_bytes bytes) lets workgroups share a sequence; without
    it each kv head of a sequence has one workgroup for every tile of rows,
    which is slow for few sequences (131072 tokens: 8 of 256 compute units).
    Prompts and single tokens are better two calls than one (the call is
    planned for max_q new tokens of every sequence)."""
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [T][n_heads][head_dim]")
    n_tok, n_heads, dim = shape
    _here(q, codes, scales, block_table, seq_lens, tok_start, out, xq, ws)
    kv = _kv(codes, scales, block_table, seq_lens, tok_start, n_tok, max_q, dim)
    ldq = _rows(q, shape, "q")
    if out is None:
        out = _new(q, shape, torch.float32, stream)
    ldo = _rows(out, shape, "out")
    qp = wp = None
    ws_bytes = 0
    if xq is not None:
        qp = _whole(xq, torch.uint8, "xq")
        if xq.numel() < act_bytes(n_tok, n_heads * dim):
            raise ValueError("activation buffer too small")
    if ws is not None:
        wp, ws_bytes = _whole(ws, torch.uint8, "ws"), ws.numel()
    _check(lib().qmv_kv_attn(ctypes.byref(kv), q.data_ptr(), ldq, n_heads, dim ** -0.5 if scale is None else scale,
                             window, out.data_ptr(), ldo, qp, wp, ws_bytes, _stream(stream)), "qmv_kv_attn")
    return out


def block_dots(fmt: int, w: torch.Tensor, n_rows: int, k: int, xq: torch.Tensor, n_tok: int,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Exact integer partial of every 32-block: int32 [T][N][K/32][c]."""
    _need(w, torch.uint8, "w")
    _need(xq, torch.uint8, "xq")
    nc = 2 if fmt in (Q4_K, Q5_K) else 1
    if out is None:
        out = torch.empty((n_tok, n_rows, k // 32, nc), dtype=torch.int32, device=w.device)
    _need(out, torch.int32, "out")
    _check(lib().qmv_block_dots(fmt, _ptr(w), n_rows, k, _ptr(xq), n_tok, _ptr(out),
                                _stream(stream)), "qmv_block_dots")
    return out


def block_dots_mx(fmt: int, w: torch.Tensor, n_rows: int, k: int, xq: torch.Tensor, n_tok: int,
                  variant: int = -1, slices: int = 0, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """The block integers of block_dots, computed by the matrix-core kernel
    (variant -1: the one qmv_matvec runs; slices 0 unsplit, -1 automatic,
    n >= 2 forced): int32 [T][N][K/32][c]."""
    _need(w, torch.uint8, "w")
    _need(xq, torch.uint8, "xq")
    nc = 2 if fmt == Q4_K else 1
    if out is None:
        out = torch.empty((n_tok, n_rows, k // 32, nc), dtype=torch.int32, device=w.device)
    _need(out, torch.int32, "out")
    if out.numel() < n_tok * n_rows * (k // 32) * nc:
        raise ValueError("out too small")
    _check(lib().qmv_block_dots_mx(fmt, _ptr(w), n_rows, k, _ptr(xq), n_tok, variant, slices, _ptr(out),
                                   _stream(stream)), "qmv_block_dots_mx")
    return out


def moe_block_dots(fmt: int, w: torch.Tensor, n_experts: int, n_rows: int, k: int, xq: torch.Tensor,
                   x_per_slot: bool, ids: torch.Tensor, ws: torch.Tensor, slot_rows: int = 0,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The block integers of every routed slot from the matrix-core MoE
    kernel: int32 [T * top_k][N][K/32][c] (dropped slots' entries untouched)."""
    _need(w, torch.uint8, "w")
    _need(xq, torch.uint8, "xq")
    _need(ids, torch.int32, "ids")
    _need(ws, torch.uint8, "ws")
    n_tok, top_k = ids.shape
    nc = 2 if fmt == Q4_K else 1
    if out is None:
        out = torch.zeros((n_tok * top_k, n_rows, k // 32, nc), dtype=torch.int32, device=w.device)
    _need(out, torch.int32, "out")
    if out.numel() < n_tok * top_k * n_rows * (k // 32) * nc:
        raise ValueError("out too small")
    if w.numel() < n_experts * n_rows * row_bytes(fmt, k):
        raise ValueError("w holds fewer than n_experts * n_rows rows")
    _check(lib().qmv_moe_block_dots(fmt, _ptr(w), n_experts, n_rows, k, _ptr(xq), int(bool(x_per_slot)),
                                    _ptr(ids), n_tok, top_k, slot_rows, _ptr(out), _ptr(ws), ws.numel(),
                                    _stream(stream)), "qmv_moe_block_dots")
    return out


def stream_read(t: torch.Tensor, sink: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Read every byte of t once (the plain-read ceiling of a weight stream)."""
    _need(t, torch.uint8, "t")
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int32, device=t.device)
    _need(sink, torch.int32, "sink")
    _check(lib().qmv_stream_read(_ptr(t), t.numel(), _ptr(sink), _stream(stream)), "qmv_stream_read")
    return sink


# ------------------------------------------------------------------ tuning
def set_tuning(key: str, value: int) -> None:
    _check(lib().qmv_set_tuning(key.encode(), int(value)), f"qmv_set_tuning({key})")


def variant_name(index: int) -> str | None:
    r = lib().qmv_variant_name(index)
    return None if r is None else r.decode()


def variants() -> list[str]:
    out, i = [], 0
    while (n := variant_name(i)) is not None:
        out.append(n)
        i += 1
    return out


def pick_variant(fmt: int, n_rows: int, k: int, n_tok: int) -> int:
    return int(lib().qmv_pick_variant(fmt, n_rows, k, n_tok))


def matvec_plan(fmt: int, n_rows: int, k: int, n_tok: int, with_workspace: bool) -> tuple[int, int]:
    """(kernel variant, K slices over workgroups) qmv_matvec would run."""
    v, s = ctypes.c_int64(), ctypes.c_int()
    _check(lib().qmv_matvec_plan(fmt, n_rows, k, n_tok, int(with_workspace), ctypes.byref(v), ctypes.byref(s)),
           "qmv_matvec_plan")
    return int(v.value), int(s.value)
