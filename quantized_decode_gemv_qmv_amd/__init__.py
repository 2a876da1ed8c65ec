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
    "head_norm_rope", "lora", "lora_workspace_bytes", "router_gate", "router_gate_workspace_bytes",
    "token_logprobs", "token_logprobs_workspace_bytes",
    "set_tuning", "swiglu_quantize", "router_topk", "variant_name", "variants", "pick_variant", "matvec_plan", "MAX_TOKENS", "MAX_MOE_TOKENS",
    "MAX_SHARED_ROWS",
]

Q8_0, Q4_K, IQ4_XS, Q5_K, Q6_K, Q8G128 = 0, 1, 2, 3, 4, 5
MAX_TOKENS = 16
MAX_MOE_TOKENS = 64
MAX_SHARED_ROWS = 256  # of a token_logprobs call whose workgroups share rows
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


class _Rope(ctypes.Structure):
    """qmv_rope of include/qmv.h."""
    _fields_ = [("pos", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p), ("pair_axis", ctypes.c_void_p),
                ("n_axes", ctypes.c_int64), ("rot_dim", ctypes.c_int64), ("interleaved", ctypes.c_int64),
                ("scale", ctypes.c_float)]


class _LoraItem(ctypes.Structure):
    """qmv_lora_item of include/qmv.h."""
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("n_rows", ctypes.c_int64), ("base", ctypes.c_void_p),
                ("ldb", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


class _Gate(ctypes.Structure):
    """qmv_gate of include/qmv.h."""
    _fields_ = [("scoring", ctypes.c_int64), ("bias", ctypes.c_void_p), ("n_groups", ctypes.c_int64),
                ("top_groups", ctypes.c_int64), ("group_best", ctypes.c_int64), ("renorm", ctypes.c_int64),
                ("scale", ctypes.c_float)]


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
        "qmv_head_norm_rope": ([ctypes.POINTER(_Rope), P, I64, I64, P, P, I64, I64, P, I64, I64, ctypes.c_float, P,
                                I64, P, I64, P], I),
        "qmv_lora_workspace_bytes": ([I64, I64, I64], SZ),
        "qmv_lora": ([I, ctypes.POINTER(_LoraItem), I64, P, I64, I64, I64, P, I64, I64, P, P, P, SZ, P], I),
        "qmv_router_gate_workspace_bytes": ([I64, I64], SZ),
        "qmv_router_gate": ([P, I64, I64, I64, P, I64, I64, ctypes.POINTER(_Gate), P, P, P, P, P, SZ, P], I),
        "qmv_token_logprobs_workspace_bytes": ([I64, I64, I64], SZ),
        "qmv_token_logprobs": ([P, I64, I64, I64, ctypes.c_float, P, I64, P, P, I64, P, P, P, SZ, P], I),
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


def _stream_on(dev: int, stream):
    """The handle of `stream`, or of the current one of the current device `dev`, which `_here` gave."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


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


def _new_like(t: torch.Tensor, dtype, stream) -> torch.Tensor:
    """_new of the shape of t, which lies in one piece (0.3 us less than by its shape)."""
    if stream is None:
        return torch.empty_like(t, dtype=dtype)
    return _new(t, t.shape, dtype, stream)


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


# ------------------------------------- steps around a layer's matvecs
def head_norm_rope(q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor | None, inv_freq: torch.Tensor | None,
                   q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                   pair_axis: torch.Tensor | None = None, interleaved: bool = False, scale: float = 1.0,
                   q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Norm (where a weight fp32 [head_dim] is given) and rotation of the heads
    of q fp32 [T][n_heads][head_dim] and k fp32 [T][n_kv_heads][head_dim] or
    None (rows may be strided).  pos int32 [T] or [axes][T]: pair i of the first
    2 * len(inv_freq) dims turns by pos[pair_axis[i]] * inv_freq[i] (pair_axis
    int32, None: the first axis), its dims i and i + len(inv_freq), or 2i and
    2i + 1 if interleaved; rows with a negative first position are left as they
    are.  inv_freq fp32, None: no rotation (pos may be None then).  Returns
    (q_out, k_out): q and k themselves, changed in place, where None."""
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [T][n_heads][head_dim]")
    dev = _here(q, k, pos, inv_freq, q_weight, k_weight, pair_axis, q_out, k_out)
    n_tok, heads, dim = shape
    ldq = _rows(q, shape, "q")
    if q_out is None:
        q_out = q
    kp = kop = None
    kv = ldk = ldko = 0
    if k is not None:
        ks = k.shape
        if len(ks) != 3 or ks[0] != n_tok or ks[2] != dim:
            raise ValueError("k must be [T][n_kv_heads][head_dim] with the T and head_dim of q")
        if k_out is None:
            k_out = k
        kv, ldk, ldko, kp, kop = ks[1], _rows(k, ks, "k"), _rows(k_out, ks, "k_out"), k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    pp = fp = ap = qwp = kwp = None
    axes, n = 1, 0
    if pos is not None:
        ps = pos.shape
        if len(ps) not in (1, 2) or ps[-1] != n_tok:
            raise ValueError("pos must be [T] or [axes][T]")
        pp, axes = _whole(pos, torch.int32, "pos"), 1 if len(ps) == 1 else ps[0]
    if inv_freq is not None:
        fp, n = _whole(inv_freq, torch.float32, "inv_freq"), inv_freq.numel()
        if pair_axis is not None:
            ap = _whole(pair_axis, torch.int32, "pair_axis")
            if pair_axis.numel() != n:
                raise ValueError("pair_axis must hold one axis a pair")
    if q_weight is not None:
        qwp = _whole(q_weight, torch.float32, "q_weight")
        if q_weight.numel() != dim:
            raise ValueError("q_weight must hold one value a dim")
    if k_weight is not None:
        kwp = _whole(k_weight, torch.float32, "k_weight")
        if k_weight.numel() != dim:
            raise ValueError("k_weight must hold one value a dim")
    rope = _Rope(pp, fp, ap, axes, 2 * n, bool(interleaved), scale)
    _check(lib().qmv_head_norm_rope(ctypes.byref(rope), q.data_ptr(), ldq, heads, qwp, kp, ldk, kv, kwp,
                                    n_tok, dim, eps, q_out.data_ptr(), _rows(q_out, shape, "q_out"), kop, ldko,
                                    _stream_on(dev, stream)), "qmv_head_norm_rope")
    return q_out, k_out


def lora_workspace_bytes(n_items: int, max_rank: int, n_tok: int) -> int:
    """Bytes of lora's workspace, enough for every call of no more items, rank and rows."""
    return int(lib().qmv_lora_workspace_bytes(n_items, max_rank, n_tok))


_FLOATS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def lora(x: torch.Tensor, ids: torch.Tensor, items, ranks: torch.Tensor | None = None,
         scales: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> list:
    """Low-rank adapters beside projections that share x fp32 [T][K] (rows may
    be strided): for each (a, b, base, y) of ``items``, a [E][R][K] and b
    [E][N][R] of float16, bfloat16 or float32, row t of y becomes base[t] +
    scales[e] * b[e] (a[e] x[t]) with the adapter e = ids[t] (int32 [T]; outside
    0 .. E - 1: base alone), over the first ranks[e] (int32 [E], None: R) rows of
    a and columns of b.  base fp32 [T][N] (None: zeros) may be y itself; y None
    is allocated.  scales fp32 [E], None: 1.  ``ws`` (uint8, of
    lora_workspace_bytes bytes) is allocated when None.  Returns the list of y."""
    if x.dim() != 2 or not items:
        raise ValueError("x must be [T][K], and there must be an item")
    n_tok, k = x.shape
    first = items[0][0]
    kind = first.dtype
    if first.dim() != 3 or kind not in _FLOATS:
        raise ValueError("a must be [E][R][K] of float16, bfloat16 or float32")
    e, rank, _ = first.shape
    n_items = len(items)
    arr = (_LoraItem * n_items)()
    dev = _here(x, ids, ranks, scales, ws)
    outs = []
    for i, (a, b, base, y) in enumerate(items):
        bs = b.shape
        if a.shape != (e, rank, k) or len(bs) != 3 or bs[0] != e or bs[2] != rank:
            raise ValueError("a must be [E][R][K] and b [E][N][R], with the same E and R in every item")
        n = bs[1]
        if y is None:
            y = _new(x, (n_tok, n), torch.float32, stream)
        bp, ldb = None, 0
        if base is not None:
            bp, ldb = base.data_ptr(), _rows(base, (n_tok, n), "base")
        if not (a.get_device() == b.get_device() == y.get_device() == dev) \
                or (base is not None and base.get_device() != dev):
            raise ValueError("every tensor must be on the current CUDA device")
        arr[i] = (_whole(a, kind, "a"), _whole(b, kind, "b"), n, bp, ldb, y.data_ptr(), _rows(y, (n_tok, n), "y"))
        outs.append(y)
    if ws is None:
        ws = _new(x, (max(lora_workspace_bytes(n_items, rank, n_tok), 1),), torch.uint8, stream)
    if ids.numel() != n_tok or (ranks is not None and ranks.numel() != e) or (scales is not None and scales.numel() != e):
        raise ValueError("ids must hold one number a row of x, ranks and scales one an adapter")
    _check(lib().qmv_lora(_FLOATS[kind], arr, n_items, x.data_ptr(), _rows(x, (n_tok, k), "x"), n_tok, k,
                          _whole(ids, torch.int32, "ids"), e, rank,
                          None if ranks is None else _whole(ranks, torch.int32, "ranks"),
                          None if scales is None else _whole(scales, torch.float32, "scales"),
                          _whole(ws, torch.uint8, "ws"), ws.numel(), _stream_on(dev, stream)), "qmv_lora")
    return outs


def router_gate_workspace_bytes(n_tok: int, n_experts: int) -> int:
    """Bytes of router_gate's workspace, enough for every call of no more tokens and experts."""
    return int(lib().qmv_router_gate_workspace_bytes(n_tok, n_experts))


_SCORING = {"softmax": 0, "sigmoid": 1}


def router_gate(x: torch.Tensor, wr: torch.Tensor, top_k: int, scoring: str = "softmax",
                bias: torch.Tensor | None = None, n_groups: int = 1, top_groups: int = 1, group_best: int = 2,
                renorm: bool = True, scale: float = 1.0, ids: torch.Tensor | None = None,
                weights: torch.Tensor | None = None, logits: torch.Tensor | None = None,
                xq: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """x fp32 [T][K] (rows may be strided), router weights fp32 [E][K] -> (ids
    int32 [T][top_k], weights fp32 [T][top_k]): scores "softmax" (over all
    experts) or "sigmoid" of the router's logits; the choice goes by score +
    bias (fp32 [E]) within the top_groups of n_groups groups whose group_best
    largest choices sum highest; the weights are the scores, with renorm over
    their sum, times scale.  logits (fp32 [T][E]) and xq, if given, receive the
    logits and the Q8 blocks of x.  ``ws`` (uint8, zero-filled once, of
    router_gate_workspace_bytes bytes) is allocated when None."""
    if x.dim() == 1:
        x = x.view(1, -1)
    if x.dim() != 2 or wr.dim() != 2 or wr.shape[1] != x.shape[1]:
        raise ValueError("x must be [T][K] and wr [E][K]")
    if scoring not in _SCORING:
        raise ValueError("scoring must be 'softmax' or 'sigmoid'")
    n_tok, k = x.shape
    e = wr.shape[0]
    if ids is None:
        ids = _new(x, (n_tok, max(top_k, 1)), torch.int32, stream)
    if weights is None:
        weights = _new_like(ids, torch.float32, stream)
    if ids.shape != (n_tok, top_k) or weights.shape != (n_tok, top_k):
        raise ValueError("ids and weights must be [T][top_k]")
    if ws is None:
        ws = _new(x, (max(router_gate_workspace_bytes(n_tok, e), 1),), torch.uint8, stream)
        if stream is None:
            ws.zero_()
        else:
            with torch.cuda.stream(stream):
                ws.zero_()
    dev = _here(x, wr, bias, ids, weights, logits, xq, ws)
    if bias is not None and bias.numel() != e:
        raise ValueError("bias must hold one value an expert")
    if logits is not None and logits.shape != (n_tok, e):
        raise ValueError("logits must be [T][E]")
    if xq is not None and xq.numel() < act_bytes(n_tok, k):
        raise ValueError("activation buffer too small")
    gate = _Gate(_SCORING[scoring], None if bias is None else _whole(bias, torch.float32, "bias"), n_groups, top_groups,
                 group_best, bool(renorm), scale)
    _check(lib().qmv_router_gate(x.data_ptr(), _rows(x, (n_tok, k), "x"), n_tok, k, _whole(wr, torch.float32, "wr"), e,
                                 top_k, ctypes.byref(gate), _whole(ids, torch.int32, "ids"),
                                 _whole(weights, torch.float32, "weights"),
                                 None if logits is None else _whole(logits, torch.float32, "logits"),
                                 None if xq is None else _whole(xq, torch.uint8, "xq"), _whole(ws, torch.uint8, "ws"),
                                 ws.numel(), _stream_on(dev, stream)), "qmv_router_gate")
    return ids, weights


def token_logprobs_workspace_bytes(n_tok: int, n_vocab: int, top_n: int) -> int:
    """Bytes of token_logprobs' workspace, enough for every call of no more rows
    and tokens, whatever its alternatives; 0 where such calls use none, so also
    for more than MAX_SHARED_ROWS rows: a program of larger and smaller batches
    asks for min(rows, MAX_SHARED_ROWS)."""
    return int(lib().qmv_token_logprobs_workspace_bytes(n_tok, n_vocab, top_n))


def token_logprobs(logits: torch.Tensor, given: torch.Tensor | None = None, top_n: int = 0, scale: float = 1.0,
                   logprobs: torch.Tensor | None = None, entropy: torch.Tensor | None = None,
                   top_ids: torch.Tensor | None = None, top_logprobs: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None, stream=None):
    """logits fp32 [T][V] (rows may be strided) -> (logprobs, entropy, top_ids,
    top_logprobs) of softmax(scale * logits): the log probabilities of the
    tokens given (int32 [T] or [T][G]; None without them), the entropies [T],
    and the top_n likeliest tokens int32 [T][top_n] with theirs (None, None if
    top_n is 0).  Outputs are allocated when None.  ``ws`` (uint8, zero-filled
    once, of token_logprobs_workspace_bytes bytes) lets workgroups share a row;
    without it, or with an empty one, each row has one, which is slow for few
    rows."""
    if logits.dim() == 1:
        logits = logits.view(1, -1)
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError("logits must be [T][V]")
    t, v = shape
    ask = []  # the caller's own outputs
    n_given, gp, lp, ip, tp = 0, None, None, None, None
    if given is not None:
        gs = given.shape
        if gs[:1] != (t,) or len(gs) > 2:
            raise ValueError("given must be [T] or [T][G]")
        n_given, gp = 1 if len(gs) == 1 else gs[1], _whole(given, torch.int32, "given")
        if logprobs is None:
            logprobs = _new_like(given, torch.float32, stream)
        else:
            ask.append((logprobs, gs, torch.float32, "logprobs"))
        lp = logprobs.data_ptr()
    elif logprobs is not None:
        raise ValueError("logprobs without given")
    if entropy is None:
        entropy = _new(logits, (t,), torch.float32, stream)
    else:
        ask.append((entropy, (t,), torch.float32, "entropy"))
    if top_n > 0:
        if top_ids is None:
            top_ids = _new(logits, (t, top_n), torch.int32, stream)
        else:
            ask.append((top_ids, (t, top_n), torch.int32, "top_ids"))
        if top_logprobs is None:
            top_logprobs = _new_like(top_ids, torch.float32, stream)
        else:
            ask.append((top_logprobs, (t, top_n), torch.float32, "top_logprobs"))
        ip, tp = top_ids.data_ptr(), top_logprobs.data_ptr()
    elif top_ids is not None or top_logprobs is not None:
        raise ValueError("top_ids or top_logprobs without top_n")
    wp, ws_bytes = None, 0
    if ws is not None and ws.numel() > 0:
        wp, ws_bytes = _whole(ws, torch.uint8, "ws"), ws.numel()
    dev = _here(logits, given, ws, *[x[0] for x in ask])
    for x, want, dtype, name in ask:
        _whole(x, dtype, name)
        if x.shape != want:
            raise ValueError(f"{name} must be {list(want)}")
    _check(lib().qmv_token_logprobs(logits.data_ptr(), _rows(logits, shape, "logits"), t, v, scale, gp, n_given, lp,
                                    entropy.data_ptr(), top_n, ip, tp, wp, ws_bytes, _stream_on(dev, stream)),
           "qmv_token_logprobs")
    return logprobs, entropy, top_ids, top_logprobs


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
