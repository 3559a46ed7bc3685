"""ctypes binding of libmoe_gb300 (include/*.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. PyTorch provides device memory and the current stream. The library
must have been built (``python -m bit_moe_expert_route_gb300.build``); if it
is missing, the first call raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple

import numpy as np
import torch

from .synth import LayerShape

_PKG = os.path.dirname(os.path.abspath(__file__))
SO_PATH = os.path.join(_PKG, "libmoe_gb300.so")

EPI_NONE, EPI_SWIGLU, EPI_COMBINE = 0, 1, 2
OPERAND_BF16, OPERAND_F16 = 0, 1
DEV_OK, DEV_BAD_TILE, DEV_BAD_ROW, DEV_TIMEOUT, DEV_BAD_EXPERT = 0, 1, 2, 3, 4


class MoeError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {code} ({status_string(code)})")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "d_model", "n_experts", "top_k", "d_ff", "d_ff_shared", "group")]

    @classmethod
    def of(cls, shape: LayerShape, T: int):
        return cls(T, shape.d_model, shape.n_experts, shape.top_k, shape.d_ff,
                   shape.d_ff_shared, shape.group)


class W4(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class Weights(ctypes.Structure):
    _fields_ = [(n, W4) for n in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")] + [
        ("router", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
        ("shared_gate", ctypes.c_void_p)]


class ForwardViews(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "logits", "gate_logit", "topk_ids", "topk_w", "counts", "offsets", "perm", "inv_perm",
        "row_token", "row_weight", "block_map", "num_tiles", "x16", "h", "out_acc", "status")] + [
        ("max_tiles", ctypes.c_int32), ("block_n", ctypes.c_int32),
        ("down_block_map", ctypes.c_void_p), ("down_num_tiles", ctypes.c_void_p),
        ("down_max_tiles", ctypes.c_int32), ("down_block_n", ctypes.c_int32),
        ("y", ctypes.c_void_p), ("down_window", ctypes.c_int32)]


class DecodeViews(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("logits", "gate_logit", "topk_ids", "topk_w", "h", "status")]


_lib = None


def lib():
    """Load the CUDA library (no fallback: a missing library is an error)."""
    global _lib
    if _lib is None:
        if not os.path.exists(SO_PATH):
            raise RuntimeError(
                f"{SO_PATH} is missing; build it with `python -m bit_moe_expert_route_gb300.build`")
        L = ctypes.CDLL(SO_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [i32]
        L.moe_version.restype = i32
        L.moe_pick_block_n.argtypes = [i32, i32, i32]
        L.moe_max_tiles.argtypes = [i32, i32, i32, i32, i32]
        L.moe_route_workspace_bytes.restype = sz
        L.moe_route_workspace_bytes.argtypes = [i32, i32]
        L.moe_route.argtypes = [vp, vp, i32, i32, i32, i32, i32] + [vp] * 10 + [i32, vp, sz, vp]
        L.moe_gemm_workspace_bytes.restype = sz
        L.moe_grouped_gemm_w4a16.argtypes = [vp, i64, i32, vp, i64, vp, i32, i32, vp, vp, vp, i32,
                                             i32, i32, i32, vp, vp, vp, i64, i64, vp, sz, vp]
        L.moe_workspace_bytes.restype = sz
        L.moe_workspace_bytes.argtypes = [vp, i32]
        L.moe_forward_views.argtypes = [vp, sz, vp, i32, vp]
        L.moe_forward.argtypes = [vp, vp, vp, i32, vp, vp, sz, vp]
        L.moe_workspace_bytes_ex.restype = sz
        L.moe_workspace_bytes_ex.argtypes = [vp, i32, i32]
        L.moe_forward_views_ex.argtypes = [vp, sz, vp, i32, i32, vp]
        L.moe_forward_ex.argtypes = [vp, vp, vp, i32, i32, vp, vp, sz, vp]
        L.moe_gdn_scan.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
        L.moe_gdn_scan_ex.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, i32, vp]
        L.moe_decode_attention_workspace_bytes.restype = sz
        L.moe_decode_attention_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.moe_decode_attention.argtypes = [vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, vp, vp,
                                           sz, vp]
        L.moe_decode_workspace_bytes.restype = sz
        L.moe_decode_workspace_bytes.argtypes = [vp]
        L.moe_decode_views.argtypes = [vp, sz, vp, vp]
        L.moe_decode_gemv_w4.argtypes = [vp, vp, vp, vp, vp, sz, vp]
        L.moe_decode_gemv_w4_noalloc.argtypes = [vp, vp, vp, vp, vp]
        L.moe_decode_noalloc_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int32)]
        L.moe_decode_noalloc_reset.argtypes = [vp]
        L.moe_decode_batch_workspace_bytes.restype = sz
        L.moe_decode_batch_workspace_bytes.argtypes = [vp]
        L.moe_decode_batch_views.argtypes = [vp, sz, vp, vp]
        L.moe_decode_batch_w4.argtypes = [vp, vp, vp, vp, vp, sz, vp]
        L.moe_add_rmsnorm_q8.argtypes = [vp, i64, vp, vp, i32, i32, ctypes.c_float, i32, vp, vp, vp,
                                         vp, vp]
        L.moe_gemm_w8a8_workspace_bytes.restype = sz
        L.moe_gemm_w8a8_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_gemm_w8a8.argtypes = [vp, i64, vp, vp, vp, i32, i32, i32, i32, vp, i64, vp, sz, vp]
        L.moe_token_logprobs.argtypes = [vp, i32, i64, vp, i32, i32, i32, vp, vp, vp, vp, vp]
        L.moe_prefix_attention_workspace_bytes.restype = sz
        L.moe_prefix_attention_workspace_bytes.argtypes = [i32] * 6
        L.moe_prefix_attention.argtypes = [vp, vp, vp, i64, vp, vp, i64, i64, vp] + [i32] * 6 + [
            ctypes.c_float, vp, vp, sz, vp]
        L.moe_qk_norm_rope.argtypes = [vp, i64, vp, i64, i32, i32, i32, i32, vp, vp, ctypes.c_float,
                                       vp, vp, i64, vp, i64, vp]
        L.moe_append_paged.argtypes = [vp, i64, vp, i64, vp, i32, i32, vp, vp, vp, vp,
                                       ctypes.c_float, vp, vp]
        L.moe_tree_attention_workspace_bytes.restype = sz
        L.moe_tree_attention_workspace_bytes.argtypes = [i32, i32, vp]
        L.moe_tree_attention.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                         sz, vp]
        L.moe_get_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int32)]
        L.moe_debug_decode_fault.argtypes = [ctypes.c_uint64, i32]
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().moe_status_string(int(code)).decode()


def _check(fn, rc):
    if rc != 0:
        raise MoeError(fn, rc)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    """The stream's handle; by default the current device's current stream (asked for without
    making a Stream object, which costs more than a launch)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _tensors(x):
    if isinstance(x, torch.Tensor):
        return [x] if x.is_cuda else []
    if isinstance(x, dict):
        x = list(x.values())
    return [t for y in x for t in _tensors(y)] if isinstance(x, (tuple, list)) else []


def _on(stream, fn, *args):
    """fn(*args) with `stream` current: the tensors that it makes are that stream's, so no block
    that another stream is still using is handed to it. The arguments' memory is kept until
    `stream` is past them, the results' until the caller's stream is past what it has
    enqueued with them when they go."""
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        out = fn(*args)
    if stream != here:
        for t in _tensors(args):
            t.record_stream(stream)
        for t in _tensors(out):
            t.record_stream(here)
    return out


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Zero-filled device workspace (the decode call requires a zeroed one)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def device_status(ws: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int32(0)
    rc = lib().moe_get_device_status(_p(ws), _stream(stream), ctypes.byref(v))
    if rc not in (0, -6):
        raise MoeError("moe_get_device_status", rc)
    return int(v.value)


# ------------------------------------------------------------------ weights on the device
def to_device(a, device="cuda") -> torch.Tensor | None:
    """numpy -> device tensor with the same bytes (uint16 -> int16, uint32 -> int32)."""
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    elif a.dtype == np.uint32:
        a = a.view(np.int32)
    return torch.from_numpy(a).to(device)


class DeviceLayer:
    """One layer's weights resident on the GPU plus the moe_weights_t that points at them."""

    def __init__(self, host: dict, shape: LayerShape, device="cuda"):
        self.shape = shape
        self.t = {}
        for name in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down"):
            w = host.get(name)
            self.t[name] = None if w is None else tuple(to_device(a, device) for a in w)
        for name in ("router", "router_bias", "shared_gate"):
            self.t[name] = to_device(host.get(name), device)
        W = Weights()
        for name in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down"):
            w = self.t[name]
            if w is not None:
                setattr(W, name, W4(w[0].data_ptr(), w[1].data_ptr(), w[2].data_ptr()))
        W.router = self.t["router"].data_ptr()
        W.router_bias = None if self.t["router_bias"] is None else self.t["router_bias"].data_ptr()
        W.shared_gate = None if self.t["shared_gate"] is None else self.t["shared_gate"].data_ptr()
        self.weights = W

    @property
    def nbytes(self) -> int:
        n = 0
        for v in self.t.values():
            if v is None:
                continue
            for a in (v if isinstance(v, tuple) else (v,)):
                n += a.numel() * a.element_size()
        return n


# ------------------------------------------------------------------ entry points
def max_tiles(T, n_experts, top_k, block_n, with_shared=True) -> int:
    return lib().moe_max_tiles(T, n_experts, top_k, block_n, int(with_shared))


def pick_block_n(T, n_experts, top_k) -> int:
    return lib().moe_pick_block_n(T, n_experts, top_k)


def route(logits: torch.Tensor, top_k: int, block_n: int, with_shared: bool = True,
          bias: torch.Tensor | None = None, stream=None) -> dict:
    """moe_route on fp32 logits [T, E]; returns the routing arrays as device tensors."""
    if stream is not None:
        return _on(stream, route, logits, top_k, block_n, with_shared, bias)
    T, E = logits.shape
    dev = logits.device
    mt = max_tiles(T, E, top_k, block_n, with_shared)
    i32 = dict(dtype=torch.int32, device=dev)
    r = dict(
        topk_ids=torch.empty(T, top_k, **i32),
        topk_w=torch.empty(T, top_k, dtype=torch.float32, device=dev),
        counts=torch.empty(E, **i32),
        offsets=torch.empty(E + 1, **i32),
        perm=torch.empty(T * top_k, **i32),
        inv_perm=torch.empty(T * top_k, **i32),
        row_token=torch.empty(T * top_k + (T if with_shared else 0), **i32),
        row_weight=torch.empty(T * top_k, dtype=torch.float32, device=dev),
        block_map=torch.zeros(max(mt, 1), 4, **i32),
        num_tiles=torch.zeros(1, **i32),
    )
    ws = workspace(lib().moe_route_workspace_bytes(T, E), dev)
    rc = lib().moe_route(
        _p(logits), _p(bias), T, E, top_k, block_n, int(with_shared), _p(r["topk_ids"]),
        _p(r["topk_w"]), _p(r["counts"]), _p(r["offsets"]), _p(r["perm"]), _p(r["inv_perm"]),
        _p(r["row_token"]), _p(r["row_weight"]), _p(r["block_map"]), _p(r["num_tiles"]), mt,
        _p(ws), ws.numel(), _stream())
    _check("moe_route", rc)
    r["max_tiles"] = mt
    r["ws"] = ws
    return r


def grouped_gemm_w4a16(A, W, n_groups, N, block_map, num_tiles, max_tiles_, block_n, epilogue,
                       row_index=None, n_rows=None, W_extra=None, row_scale=None, out_row=None,
                       C=None, C_rows=None, operand=None, stream=None):
    """moe_grouped_gemm_w4a16. W / W_extra: list of (q, scale, bias) device tensors.
    operand: OPERAND_F16 / OPERAND_BF16; by default taken from A's dtype (float16 -> f16)."""
    if stream is not None:
        return _on(stream, grouped_gemm_w4a16, A, W, n_groups, N, block_map, num_tiles,
                   max_tiles_, block_n, epilogue, row_index, n_rows, W_extra, row_scale, out_row,
                   C, C_rows, operand)
    if operand is None:
        operand = OPERAND_F16 if A.dtype == torch.float16 else OPERAND_BF16
    A_rows, K = A.shape
    if n_rows is None:
        n_rows = row_index.numel() if row_index is not None else A_rows
    Ws = (W4 * len(W))(*[W4(q.data_ptr(), s.data_ptr(), b.data_ptr()) for q, s, b in W])
    Wx = None
    if W_extra is not None:
        Wx = (W4 * len(W_extra))(*[W4(q.data_ptr(), s.data_ptr(), b.data_ptr())
                                  for q, s, b in W_extra])
    if C is None:
        dt = torch.float32
        if epilogue == EPI_SWIGLU:
            dt = torch.float16 if operand == OPERAND_F16 else torch.bfloat16
        C = torch.zeros(C_rows if C_rows is not None else n_rows, N, dtype=dt, device=A.device)
    ws = workspace(lib().moe_gemm_workspace_bytes(), A.device)
    rc = lib().moe_grouped_gemm_w4a16(
        _p(A), A_rows, K, _p(row_index), n_rows, ctypes.cast(Ws, ctypes.c_void_p), n_groups, N,
        None if Wx is None else ctypes.cast(Wx, ctypes.c_void_p), _p(block_map), _p(num_tiles),
        max_tiles_, block_n, epilogue, operand, _p(row_scale), _p(out_row), _p(C), C.shape[0],
        C.stride(0), _p(ws), ws.numel(), _stream())
    _check("moe_grouped_gemm_w4a16", rc)
    return C, ws


GDN_STATE_EARLY = 1


def gdn_scan(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
             beta: torch.Tensor, state: torch.Tensor, out: torch.Tensor | None = None,
             stream=None, state_early: bool = False) -> torch.Tensor:
    """moe_gdn_scan_ex (include/gdn.h): q, k bf16 [T, Hk, dk]; v bf16 [T, Hv, dv]; alpha,
    beta fp32 [T, Hv]; state fp32 [Hv, dv, dk], advanced in place over the T tokens.
    state_early (MOE_GDN_STATE_EARLY): the previous launch on the stream does not write
    this state, so it is read before waiting for that launch. Returns out fp32 [T, Hv, dv]."""
    if stream is not None:
        return _on(stream, gdn_scan, q, k, v, alpha, beta, state, out, None, state_early)
    T, Hk, dk = k.shape
    Hv, dv = v.shape[1], v.shape[2]
    if out is None:
        out = torch.empty(T, Hv, dv, dtype=torch.float32, device=state.device)
    rc = lib().moe_gdn_scan_ex(_p(q), _p(k), _p(v), _p(alpha), _p(beta), T, Hk, Hv, dk, dv,
                               _p(state), _p(out), GDN_STATE_EARLY if state_early else 0,
                               _stream())
    _check("moe_gdn_scan_ex", rc)
    return out


def decode_attention(q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, scale: float = 0.0,
                     out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """moe_decode_attention (include/attn.h): q bf16 [Hq, d]; K, V bf16 [L, Hkv, d];
    scale <= 0 means 1/sqrt(d). Returns out fp32 [Hq, d]."""
    if stream is not None:
        return _on(stream, decode_attention, q, K, V, scale, out, ws)
    Hq, d = q.shape
    L, Hkv = K.shape[0], K.shape[1]
    nbytes = lib().moe_decode_attention_workspace_bytes(L, Hq, Hkv, d)
    if nbytes == 0:
        raise MoeError("moe_decode_attention_workspace_bytes", -3)
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(Hq, d, dtype=torch.float32, device=q.device)
    rc = lib().moe_decode_attention(_p(q), _p(K), _p(V), L, Hq, Hkv, d, float(scale), _p(out),
                                    _p(ws), ws.numel(), _stream())
    _check("moe_decode_attention", rc)
    return out


Q8_FORMATS = {"int8": (0, torch.int8), "e4m3": (1, torch.float8_e4m3fn)}
_FLOAT_TYPES = {torch.bfloat16: 0, torch.float32: 1}


class NormQ8(NamedTuple):
    """add_rmsnorm_q8's outputs: codes [T, d], scale fp32 [T], the new residual bf16 [T, d]
    and (where asked for) q * scale as bf16 [T, d]."""
    q: torch.Tensor
    scale: torch.Tensor
    residual: torch.Tensor
    values: torch.Tensor | None


def _want(fn, name, t, dtype, shape, rows=False):
    """The address of a tensor of the type, shape and layout that the call reads (rows: only
    each row has to be contiguous); refuses any other."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and (
            t.is_contiguous() or rows and t.stride(-1) == 1):
        return t.data_ptr()
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{fn}: {name} is {t.dtype} {tuple(t.shape)}, {dtype} {tuple(shape)} is wanted")
    if not t.is_cuda:
        raise ValueError(f"{fn}: {name} is not on the GPU")
    raise ValueError(f"{fn}: {name} is not contiguous")


def _want_cache(fn, name, k, v, shape):
    """The addresses of a K and a V cache whose heads are contiguous, and their strides (which
    have to be the same)."""
    bf, st, sv = torch.bfloat16, k.stride(), v.stride()
    if st != sv and k.shape == v.shape:  # the stride of an axis of one entry says nothing
        sv = tuple(a if n == 1 else b for n, a, b in zip(k.shape, st, sv))
    if (k.dtype is bf and v.dtype is bf and k.shape == shape and v.shape == shape and k.is_cuda
            and v.is_cuda and (k.numel() == 0 or st == sv and st[-1] == 1
                               and (st[-2] == shape[-1] or shape[-2] == 1))):
        return k.data_ptr(), v.data_ptr(), st
    for n, t in (("k_" + name, k), ("v_" + name, v)):
        if t.dtype != bf or t.shape != shape or not t.is_cuda:
            raise ValueError(f"{fn}: {n} is {t.dtype} {tuple(t.shape)} on {t.device}, "
                             f"{bf} {tuple(shape)} on the GPU is wanted")
    raise ValueError(f"{fn}: k_{name} and v_{name} have different strides or scattered heads")


def _want_ws(fn, ws):
    """The address and bytes of the caller's workspace."""
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError(f"{fn}: ws is not contiguous memory on the GPU")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _ld(t):
    """Elements from one row of a 2-D tensor to the next (its width where there is one row)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def add_rmsnorm_q8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                   eps: float = 1e-6, fmt: str = "int8", values: bool = False,
                   residual_out: torch.Tensor | None = None, stream=None) -> NormQ8:
    """moe_add_rmsnorm_q8 (include/step.h): x bf16 [T, d] (rows may be strided), weight bf16
    [d], residual bf16 [T, d] or None. fmt "int8" or "e4m3". residual_out may be `residual`
    (updated in place); without a residual and a residual_out, `.residual` is x itself."""
    if stream is not None:
        return _on(stream, add_rmsnorm_q8, x, weight, residual, eps, fmt, values, residual_out)
    T, d = x.shape
    fn, bf, dev = "add_rmsnorm_q8", torch.bfloat16, x.device
    if fmt not in Q8_FORMATS:
        raise ValueError(f"{fn}: fmt is {fmt!r}, 'int8' or 'e4m3' is wanted")
    code, dtype = Q8_FORMATS[fmt]
    shape = (T, d)
    px = _want(fn, "x", x, bf, shape, rows=True)
    pw = _want(fn, "weight", weight, bf, (d,))
    pr = po = pv = vals = None
    if residual is not None:
        pr = _want(fn, "residual", residual, bf, shape)
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=bf, device=dev)
            po = residual_out.data_ptr()
    if residual_out is not None and po is None:
        po = _want(fn, "residual_out", residual_out, bf, shape)
    q = torch.empty(shape, dtype=dtype, device=dev)
    scale = torch.empty(T, dtype=torch.float32, device=dev)
    if values:
        vals = torch.empty(shape, dtype=bf, device=dev)
        pv = vals.data_ptr()
    rc = lib().moe_add_rmsnorm_q8(px, _ld(x), pr, pw, T, d, eps, code, po, q.data_ptr(),
                                  scale.data_ptr(), pv, _stream())
    _check("moe_add_rmsnorm_q8", rc)
    return NormQ8(q, scale, x if residual_out is None else residual_out, vals)


W8A8_NO_WORKSPACE_T = 24


def gemm_w8a8(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
              ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """moe_gemm_w8a8 (include/step.h): a int8 [T, K] (rows may be strided) with a_scale fp32
    [T], w int8 [N, K] with w_scale fp32 [N]. Returns out [T, N], bf16 or fp32 (`dtype`, or
    `out`'s own type; out's rows may be strided)."""
    if stream is not None:
        return _on(stream, gemm_w8a8, a, a_scale, w, w_scale, dtype, out, ws)
    T, K = a.shape
    N = w.shape[0]
    fn, dev, f32 = "gemm_w8a8", a.device, torch.float32
    if out is not None:
        dtype = out.dtype
    if dtype not in _FLOAT_TYPES:
        raise ValueError(f"{fn}: the output is {dtype}, bfloat16 or float32 is wanted")
    pa = _want(fn, "a", a, torch.int8, (T, K), rows=True)
    ps = _want(fn, "a_scale", a_scale, f32, (T,))
    pw = _want(fn, "w", w, torch.int8, (N, K))
    pt = _want(fn, "w_scale", w_scale, f32, (N,))
    if out is None:
        out = torch.empty((T, N), dtype=dtype, device=dev)
        po = out.data_ptr()
    else:
        po = _want(fn, "out", out, dtype, (T, N), rows=True)
    pws, nbytes = None, 0
    if ws is not None:
        pws, nbytes = _want_ws(fn, ws)
    elif T > W8A8_NO_WORKSPACE_T:
        nbytes = lib().moe_gemm_w8a8_workspace_bytes(T, N, K)
        if nbytes == 0:
            raise MoeError("moe_gemm_w8a8_workspace_bytes", -3)
        if nbytes > 256:  # else the status word alone, of a call that cannot fail
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            pws = ws.data_ptr()
    rc = lib().moe_gemm_w8a8(pa, _ld(a), ps, pw, pt, T, N, K, _FLOAT_TYPES[dtype], po, _ld(out),
                             pws, nbytes, _stream())
    _check("moe_gemm_w8a8", rc)
    return out


PREFIX_NO_WORKSPACE_POSITIONS = 2048


def prefix_attention(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor,
                     k_suffix: torch.Tensor | None = None, v_suffix: torch.Tensor | None = None,
                     lens: torch.Tensor | None = None, scale: float = 0.0,
                     out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """moe_prefix_attention (include/attn.h): q bf16 [B, Hq, d]; the shared prefix K, V bf16
    [P, Hkv, d]; the sequences' own K, V bf16 [B, S, Hkv, d] (or None) of which lens int32 [B]
    positions count. Positions and sequences may be strided (K and V alike). scale <= 0 means
    1/sqrt(d). Returns out bf16 [B, Hq, d]."""
    if stream is not None:
        return _on(stream, prefix_attention, q, k_prefix, v_prefix, k_suffix, v_suffix, lens,
                   scale, out, ws)
    B, Hq, d = q.shape
    P, Hkv = k_prefix.shape[:2]
    fn, bf, dev = "prefix_attention", torch.bfloat16, q.device
    if k_suffix is None and v_suffix is not None:
        raise ValueError(f"{fn}: v_suffix without k_suffix")
    pq = _want(fn, "q", q, bf, (B, Hq, d))
    pk, pv, ld = _want_cache(fn, "prefix", k_prefix, v_prefix, (P, Hkv, d))
    S, pks, pvs, lds, pl = 0, None, None, (0, 0), None
    if k_suffix is not None:
        if v_suffix is None or lens is None:
            raise ValueError(f"{fn}: k_suffix without v_suffix or lens")
        S = k_suffix.shape[1]
        pks, pvs, lds = _want_cache(fn, "suffix", k_suffix, v_suffix, (B, S, Hkv, d))
        pl = _want(fn, "lens", lens, torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Hq, d), dtype=bf, device=dev)
        po = out.data_ptr()
    else:
        po = _want(fn, "out", out, bf, (B, Hq, d))
    width = Hkv * d  # the stride of an axis of one entry says nothing
    args = (pq, pk, pv, ld[0] if P > 1 else width, pks, pvs, lds[0] if B > 1 else 0,
            lds[1] if S > 1 else width, pl, B, P, S, Hq, Hkv, d, scale, po)
    rc, pws, nbytes = -4, None, 0
    if ws is not None:
        pws, nbytes = _want_ws(fn, ws)
    elif P + S <= PREFIX_NO_WORKSPACE_POSITIONS:  # little work needs none
        rc = lib().moe_prefix_attention(*args, None, 0, _stream())
    if rc == -4:
        if ws is None:
            nbytes = lib().moe_prefix_attention_workspace_bytes(B, P, S, Hq, Hkv, d)
            if nbytes == 0:
                raise MoeError("moe_prefix_attention_workspace_bytes", -3)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            pws = ws.data_ptr()
        rc = lib().moe_prefix_attention(*args, pws, nbytes, _stream())
    _check("moe_prefix_attention", rc)
    return out


class TokenLogprobs(NamedTuple):
    """token_logprobs' outputs: fp32 [N], fp32 [N], int32 [N, k], fp32 [N, k]."""
    logprob: torch.Tensor | None
    entropy: torch.Tensor
    top_ids: torch.Tensor
    top_logprobs: torch.Tensor


def token_logprobs(logits: torch.Tensor, ids: torch.Tensor | None = None, top_k: int = 0,
                   stream=None) -> TokenLogprobs:
    """moe_token_logprobs (include/step.h): logits bf16 or fp32 [N, V] (rows may be strided),
    ids int32 [N] or None. Returns the ids' log probabilities, each row's entropy (nats) and
    its top_k (at most 32) alternatives, largest first, ties to the lower id."""
    if stream is not None:
        return _on(stream, token_logprobs, logits, ids, top_k)
    N, V = logits.shape
    fn, dev = "token_logprobs", logits.device
    if logits.dtype not in _FLOAT_TYPES:
        raise ValueError(f"{fn}: logits are {logits.dtype}, bfloat16 or float32 is wanted")
    if not 0 <= top_k <= min(32, V):
        raise ValueError(f"{fn}: top_k is {top_k}, 0 .. min(32, {V}) is wanted")
    pz = _want(fn, "logits", logits, logits.dtype, (N, V), rows=True)
    pi = pl = pt = pp = logprob = None
    if ids is not None:
        pi = _want(fn, "ids", ids, torch.int32, (N,))
        logprob = torch.empty(N, dtype=torch.float32, device=dev)
        pl = logprob.data_ptr()
    entropy = torch.empty(N, dtype=torch.float32, device=dev)
    top_ids = torch.empty((N, top_k), dtype=torch.int32, device=dev)
    top_lp = torch.empty((N, top_k), dtype=torch.float32, device=dev)
    if top_k:
        pt, pp = top_ids.data_ptr(), top_lp.data_ptr()
    rc = lib().moe_token_logprobs(pz, _FLOAT_TYPES[logits.dtype], _ld(logits), pi, N, V, top_k, pl,
                                  entropy.data_ptr(), pt, pp, _stream())
    _check("moe_token_logprobs", rc)
    return TokenLogprobs(logprob, entropy, top_ids, top_lp)


# ------------------------------------------------------------------ the paged cache
class Rope(NamedTuple):
    """A rotation of heads by position (moe_rope, include/cache.h): freqs fp32 [pairs] on the GPU,
    radians a position; sections: pairs of each axis of the positions (None: one axis), in blocks or
    cyclic; adjacent: pairs are elements (2i, 2i + 1), else (i, i + pairs)."""
    freqs: torch.Tensor
    sections: tuple | None = None
    cyclic: bool = False
    adjacent: bool = False


class PagedCache(NamedTuple):
    """Keys and values in pages (moe_paged, include/cache.h): k_pages, v_pages bf16 [n_pages, page,
    Hkv, d] with the same strides (views of other orders too), table int32 [B, width]: position p of
    sequence b is place p % page of page table[b, p // page]."""
    k_pages: torch.Tensor
    v_pages: torch.Tensor
    table: torch.Tensor


# moe_rope and moe_paged as the C structures lie (packing bytes costs a small call a tenth of
# filling a ctypes.Structure)
_ROPE_ARGS = struct.Struct("@PPq8i")
_PAGED_ARGS = struct.Struct("@PP3qPq6i")


_MOST = 0x7fffffff  # what the C calls' sizes hold: ctypes would wrap larger ones


def rope_freqs(rotary: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """Frequencies theta^(-2i / rotary), i < rotary / 2, as Rope takes them (rounded to fp32 once)."""
    i = torch.arange(0, rotary, 2, dtype=torch.float64)
    return (float(theta) ** (-i / rotary)).to(torch.float32).to(device)


def tree_masks(parents) -> tuple[torch.Tensor, torch.Tensor]:
    """Masks and depths of a tree of drafted tokens: parents[i] is the index (below i) of the token
    that token i follows, or -1 where that is the last one before the draft. Returns int64 [n], a bit
    for each token on the path to i and i itself (tree_attention's `tree`), and int32 [n], how many
    drafted tokens come before i on it (a token's position is the cached ones' number plus that), on
    the CPU."""
    bits, depths = [], []
    for i, j in enumerate(parents):
        if not -1 <= j < i or i >= 64:
            raise ValueError(f"tree_masks: parents[{i}] is {j}, an earlier token or -1 (and 64 tokens) is wanted")
        bits.append((1 << i) | (bits[j] if j >= 0 else 0))
        depths.append(depths[j] + 1 if j >= 0 else 0)
    signed = [m - (1 << 64) if m >> 63 else m for m in bits]
    return torch.tensor(signed, dtype=torch.int64), torch.tensor(depths, dtype=torch.int32)


def _refuse(fn, name, t, dtype, shape, dev):
    """Why a tensor is not what a call on device `dev` reads."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_cuda:
        raise ValueError(f"{fn}: {name} is {t.dtype} {tuple(t.shape)} on {t.device}, {dtype} {tuple(shape)} on the GPU is wanted")
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} is on {t.device}, the call's other tensors on cuda:{dev}")
    raise ValueError(f"{fn}: {name} is not contiguous")


def _heads(fn, name, t, T, H, d, dev):
    """The address of bf16 [T, H, d] whose heads are contiguous, and its tokens' stride."""
    shape = (T, H, d)
    if t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != dev or dev < 0:
        _refuse(fn, name, t, torch.bfloat16, shape, dev)
    if T > _MOST or H > _MOST or d > _MOST:
        raise ValueError(f"{fn}: {name} {tuple(shape)} is too large")
    s0, s1, s2 = t.stride()
    if (s2 != 1 or s1 != d and H > 1) and T:
        raise ValueError(f"{fn}: {name} has scattered heads")
    return t.data_ptr(), s0 if T > 1 else H * d  # the stride of an axis of one entry says nothing


def _vector(fn, name, t, dtype, n, dev):
    """The address of a contiguous vector; None of None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        _refuse(fn, name, t, dtype, (n,), dev)
    if n > _MOST:
        raise ValueError(f"{fn}: {name} of {n} elements is too large")
    return t.data_ptr()


def _rows(fn, name, t, shape, dev):
    """The address of int32 rows, and their stride."""
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != dev or t.stride(1) != 1 and shape[1] > 1:
        _refuse(fn, name, t, torch.int32, shape, dev)
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]


def _current(fn, dev):
    """The stream for tensors on `dev`, which has to be the current device."""
    here = torch._C._cuda_getDevice()
    if dev != here:
        raise ValueError(f"{fn}: the tensors are on cuda:{dev}, cuda:{here} is the current device")
    return torch._C._cuda_getCurrentRawStream(here)


def _rope_args(fn, rope, positions, T, dev):
    """moe_rope of a rotation for T tokens (None: none)."""
    if rope is None:
        if positions is not None:
            raise ValueError(f"{fn}: positions without rope")
        return None
    freqs, sections, cyclic, adjacent = rope
    pairs = freqs.numel()
    A = 1 if sections is None else len(sections)
    if not 1 <= A <= 4:
        raise ValueError(f"{fn}: {A} sections, 1 to 4 are wanted")
    s = (pairs, 0, 0, 0) if sections is None else (*sections, 0, 0, 0)[:4]
    if min(s) < 0 or max(s) > pairs:
        raise ValueError(f"{fn}: sections {sections}, each of 0 to {pairs} pairs, are wanted")
    pp = ld = 0
    if positions is not None:
        if A == 1 and positions.dim() == 1:
            pp = _vector(fn, "positions", positions, torch.int32, T, dev)
        else:
            pp, ld = _rows(fn, "positions", positions, (A, T), dev)
    return _ROPE_ARGS.pack(_vector(fn, "rope.freqs", freqs, torch.float32, pairs, dev), pp, ld, pairs, A, *s,
                           bool(cyclic), bool(adjacent))


def _paged_args(fn, cache, Hkv, d, dev):
    """moe_paged of a cache with heads of the sizes that the call's other tensors have, and its
    sequences."""
    k, v, table = cache
    shape, size = k.shape, table.shape
    if len(shape) != 4 or len(size) != 2:
        raise ValueError(f"{fn}: k_pages {tuple(shape)} and table {tuple(size)}: "
                         "[n_pages, page, Hkv, d] and [B, width] are wanted")
    (n, page, heads, width), bf = shape, torch.bfloat16
    if heads != Hkv or width != d or k.dtype is not bf or k.get_device() != dev:
        _refuse(fn, "k_pages", k, bf, (n, page, Hkv, d), dev)
    if v.shape != shape or v.dtype is not bf or v.get_device() != dev:
        _refuse(fn, "v_pages", v, bf, shape, dev)
    st, sv = k.stride(), v.stride()
    if st[3] != 1 or st != sv and any(a != b and e > 1 for e, a, b in zip(shape, st, sv)):
        raise ValueError(f"{fn}: k_pages and v_pages have different strides or scattered elements")
    pt, ld = _rows(fn, "table", table, size, dev)
    B, width = size
    if max(n, page, width, B) > _MOST:
        raise ValueError(f"{fn}: a cache of {n} pages and {B} x {width} entries is too large")
    return _PAGED_ARGS.pack(k.data_ptr(), v.data_ptr(), st[0], st[1], st[2], pt, ld, n, page, width, B, Hkv, d), B


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None = None, rope: Rope | None = None,
                 positions: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """moe_qk_norm_rope (include/cache.h): q bf16 [T, Hq, d] and k bf16 [T, Hkv, d] (tokens may be
    strided), each head normed where its weight (bf16 [d]) is given and turned by positions
    (int32 [T], or [axes, T]). Returns (q, k), new or q_out, k_out (which may be q and k themselves);
    k may be None."""
    if stream is not None:
        return _on(stream, qk_norm_rope, q, k, rope, positions, q_weight, k_weight, eps, q_out, k_out)
    fn, bf = "qk_norm_rope", torch.bfloat16
    T, Hq, d = q.shape
    dev = q.get_device()
    if rope is not None and positions is None:
        raise ValueError(f"{fn}: rope without positions")
    if k is None and (k_weight is not None or k_out is not None):
        raise ValueError(f"{fn}: k_weight or k_out without k")
    pq, ldq = _heads(fn, "q", q, T, Hq, d, dev)
    pk = pko = None
    Hkv = ldk = ldko = 0
    if k is not None:
        Hkv = k.shape[1]
        pk, ldk = _heads(fn, "k", k, T, Hkv, d, dev)
        if k_out is None:
            k_out = torch.empty((T, Hkv, d), dtype=bf, device=q.device)
            pko, ldko = k_out.data_ptr(), Hkv * d
        else:
            pko, ldko = _heads(fn, "k_out", k_out, T, Hkv, d, dev)
    if q_out is None:
        q_out = torch.empty((T, Hq, d), dtype=bf, device=q.device)
        pqo, ldqo = q_out.data_ptr(), Hq * d
    else:
        pqo, ldqo = _heads(fn, "q_out", q_out, T, Hq, d, dev)
    rc = lib().moe_qk_norm_rope(pq, ldq, pk, ldk, T, Hq, Hkv, d, _vector(fn, "q_weight", q_weight, bf, d, dev),
                                _vector(fn, "k_weight", k_weight, bf, d, dev), eps,
                                _rope_args(fn, rope, positions, T, dev), pqo, ldqo, pko, ldko, _current(fn, dev))
    _check("moe_qk_norm_rope", rc)
    return q_out, k_out


def append_paged(k: torch.Tensor, v: torch.Tensor, cache: PagedCache, starts: torch.Tensor,
                 lens: torch.Tensor, rope: Rope | None = None, positions: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 rows: torch.Tensor | None = None, stream=None) -> None:
    """moe_append_paged (include/cache.h): writes new tokens' k, v bf16 [N, Hkv, d] (tokens may be
    strided) to the cache's pages, sequence b's (starts[b] .. starts[b + 1] - 1; starts int32 [B + 1])
    from position lens[b] on (int32 [B], not changed). Keys are normed (k_weight bf16 [d]) and turned on
    the way where asked, by positions (int32 [N] or [axes, N]) or, without, by their place in the cache.
    rows int32 [N]: token t's k and v are k[rows[t]], v[rows[t]]."""
    if stream is not None:
        return _on(stream, append_paged, k, v, cache, starts, lens, rope, positions, k_weight, eps, rows)
    fn, i32 = "append_paged", torch.int32
    M, Hkv, d = k.shape
    N = M if rows is None else rows.shape[0]
    dev = k.get_device()
    pk, ldk = _heads(fn, "k", k, M, Hkv, d, dev)
    pv, ldv = _heads(fn, "v", v, M, Hkv, d, dev)
    paged, B = _paged_args(fn, cache, Hkv, d, dev)
    rc = lib().moe_append_paged(pk, ldk, pv, ldv, _vector(fn, "rows", rows, i32, N, dev), M, N,
                                _vector(fn, "starts", starts, i32, B + 1, dev), _vector(fn, "lens", lens, i32, B, dev), paged,
                                _vector(fn, "k_weight", k_weight, torch.bfloat16, d, dev), eps,
                                _rope_args(fn, rope, positions, N, dev), _current(fn, dev))
    _check("moe_append_paged", rc)


def tree_attention(q: torch.Tensor, cache: PagedCache, starts: torch.Tensor, lens: torch.Tensor,
                   tree: torch.Tensor | None = None, scale: float = 0.0,
                   out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """moe_tree_attention (include/cache.h): q bf16 [N, Hq, d] (tokens may be strided) of sequences'
    new tokens (starts int32 [B + 1], at most 64 each), whose keys and values are in the cache already
    from position lens[b] on. A token attends to what was there before, and to the new tokens j of its
    sequence for which bit j of its word of tree (int64 [N]) is set; without, to those up to itself.
    scale <= 0 means 1/sqrt(d). Returns out bf16 [N, Hq, d]; tokens of no sequence are left as they were."""
    if stream is not None:
        return _on(stream, tree_attention, q, cache, starts, lens, tree, scale, out, ws)
    fn, bf, i32 = "tree_attention", torch.bfloat16, torch.int32
    N, Hq, d = q.shape
    dev, pages = q.get_device(), cache.k_pages
    pq, ldq = _heads(fn, "q", q, N, Hq, d, dev)
    paged, B = _paged_args(fn, cache, pages.shape[2] if pages.dim() == 4 else 0, d, dev)
    ps, pl = _vector(fn, "starts", starts, i32, B + 1, dev), _vector(fn, "lens", lens, i32, B, dev)
    pt = _vector(fn, "tree", tree, torch.int64, N, dev)
    if out is None:
        out = torch.empty((N, Hq, d), dtype=bf, device=q.device)
        po = out.data_ptr()
    else:
        po = _want(fn, "out", out, bf, (N, Hq, d))
    if ws is None:
        nbytes = lib().moe_tree_attention_workspace_bytes(N, Hq, paged)
        if nbytes == 0:
            raise MoeError("moe_tree_attention_workspace_bytes", -3)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        pws = ws.data_ptr()
    else:
        pws, nbytes = _want_ws(fn, ws)
    if out.get_device() != dev or ws.get_device() != dev:
        raise ValueError(f"{fn}: out or ws is on another device than q")
    rc = lib().moe_tree_attention(pq, ldq, N, Hq, ps, pl, pt, paged, scale, po, pws, nbytes, _current(fn, dev))
    _check("moe_tree_attention", rc)
    return out


FWD_DETERMINISTIC = 1
FWD_DOWN_WINDOWS = 2
FWD_FUSED = 4


class Forward:
    """moe_forward_ex with a reusable workspace for one (shape, T, block_n, flags);
    deterministic=True sets MOE_FWD_DETERMINISTIC (fixed-order combine),
    down_windows=True MOE_FWD_DOWN_WINDOWS (down tiles ordered by token window),
    fused=True MOE_FWD_FUSED (gate/up, SwiGLU and down per 64-row tile in one kernel)."""

    def __init__(self, layer: DeviceLayer, T: int, block_n: int = 0, device="cuda",
                 deterministic: bool = False, down_windows: bool = False, fused: bool = False):
        self.layer = layer
        self.T = T
        self.shape = Shape.of(layer.shape, T)
        self.flags = ((FWD_DETERMINISTIC if deterministic else 0) | (FWD_DOWN_WINDOWS if down_windows else 0)
                      | (FWD_FUSED if fused else 0))
        self.block_n = block_n or (64 if fused else pick_block_n(T, layer.shape.n_experts, layer.shape.top_k))
        nbytes = lib().moe_workspace_bytes_ex(ctypes.byref(self.shape), self.block_n, self.flags)
        if nbytes == 0:
            raise MoeError("moe_workspace_bytes_ex", -3)
        self.ws = workspace(nbytes, device)
        self.views = ForwardViews()
        _check("moe_forward_views_ex", lib().moe_forward_views_ex(
            _p(self.ws), self.ws.numel(), ctypes.byref(self.shape), self.block_n, self.flags,
            ctypes.byref(self.views)))

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None):
        if stream is not None:
            return _on(stream, self, x, out)
        if out is None:
            out = torch.empty(self.T, self.layer.shape.d_model, dtype=torch.bfloat16,
                              device=x.device)
        rc = lib().moe_forward_ex(_p(x), ctypes.byref(self.layer.weights),
                                  ctypes.byref(self.shape), self.block_n, self.flags, _p(out),
                                  _p(self.ws), self.ws.numel(), _stream())
        _check("moe_forward_ex", rc)
        return out

    def view(self, name: str, shape, dtype) -> torch.Tensor:
        """A device tensor aliasing one of the workspace intermediates."""
        base = self.ws.data_ptr()
        off = getattr(self.views, name) - base
        n = int(np.prod(shape))
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.ws[off:off + nbytes].view(dtype).view(*shape)


class DecodeBatch:
    """moe_decode_batch_w4 (1 <= T <= 8 tokens) with a reusable workspace."""

    def __init__(self, layer: DeviceLayer, T: int, device="cuda"):
        self.layer, self.T = layer, T
        self.shape = Shape.of(layer.shape, T)
        nbytes = lib().moe_decode_batch_workspace_bytes(ctypes.byref(self.shape))
        if nbytes == 0:
            raise MoeError("moe_decode_batch_workspace_bytes", -3)
        self.ws = workspace(nbytes, device)
        self.views = DecodeViews()
        _check("moe_decode_batch_views", lib().moe_decode_batch_views(
            _p(self.ws), self.ws.numel(), ctypes.byref(self.shape), ctypes.byref(self.views)))

    def view(self, name: str, shape, dtype) -> torch.Tensor:
        """A workspace array (logits [T][E], gate_logit [T], topk_ids [T][k],
        topk_w [T][k+1] with the shared gate last, h fp32 [T][k+1][d_ff])."""
        off = getattr(self.views, name) - self.ws.data_ptr()
        n = int(np.prod(shape))
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.ws[off:off + nbytes].view(dtype).view(*shape)

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None):
        if stream is not None:
            return _on(stream, self, x, out)
        if out is None:
            out = torch.empty(self.T, self.layer.shape.d_model, dtype=torch.bfloat16, device=x.device)
        rc = lib().moe_decode_batch_w4(_p(x), ctypes.byref(self.layer.weights),
                                       ctypes.byref(self.shape), _p(out), _p(self.ws),
                                       self.ws.numel(), _stream())
        _check("moe_decode_batch_w4", rc)
        return out


class Decode:
    """moe_decode_gemv_w4 (T = 1) with a reusable workspace."""

    def __init__(self, layer: DeviceLayer, device="cuda"):
        self.layer = layer
        self.shape = Shape.of(layer.shape, 1)
        nbytes = lib().moe_decode_workspace_bytes(ctypes.byref(self.shape))
        if nbytes == 0:
            raise MoeError("moe_decode_workspace_bytes", -3)
        self.ws = workspace(nbytes, device)
        self.views = DecodeViews()
        _check("moe_decode_views", lib().moe_decode_views(
            _p(self.ws), self.ws.numel(), ctypes.byref(self.shape), ctypes.byref(self.views)))

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None):
        if stream is not None:
            return _on(stream, self, x, out)
        if out is None:
            out = torch.empty(self.layer.shape.d_model, dtype=torch.bfloat16, device=x.device)
        rc = lib().moe_decode_gemv_w4(_p(x), ctypes.byref(self.layer.weights),
                                      ctypes.byref(self.shape), _p(out), _p(self.ws),
                                      self.ws.numel(), _stream())
        _check("moe_decode_gemv_w4", rc)
        return out

    def view(self, name: str, shape, dtype) -> torch.Tensor:
        off = getattr(self.views, name) - self.ws.data_ptr()
        n = int(np.prod(shape))
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.ws[off:off + nbytes].view(dtype).view(*shape)
