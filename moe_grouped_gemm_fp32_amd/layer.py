"""The operators around the FP8 GEMMs of a transformer layer: binding of include/fp8layer.h.

  rmsnorm_quantize_1x128   residual addition, RMS norm and 1x128 quantisation
  rmsnorm_backward         the norm's gradients
  rope_append_paged_kv     rotates queries and keys, appends keys and values to the cache
  paged_attention          causal attention over the cache

Like the GEMM bindings these only marshal tensors; they are exported by the package. The
paged cache of one layer is a PagedKVCache (make_paged_kv_cache); which pages hold a
sequence, and which rows of a call are its new tokens, is given by three int32 tensors:
block_table [B, max_pages], seq_lens [B] (new tokens included) and cu_q [B + 1] (row
offsets of the sequences' new tokens). They are read on the device only, so every call may
be captured into a graph.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _bytes_view, _check, _ld, _ptr, _require, _stream, lib, scale_ld, QUANT_BF16, QUANT_FP32

__all__ = ["PagedKVCache", "make_paged_kv_cache", "rmsnorm_quantize_1x128", "rmsnorm_backward", "rope_append_paged_kv",
           "paged_attention", "attention_workspace_size", "make_attention_workspace"]

_P, _I64, _INT, _SZ, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_SIGS = {
    "fp8_rmsnorm_quantize_1x128": (
        _INT, [_P, _I64, _P, _I64, _INT, _P, _INT, _F, _P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _INT, _INT, _P]),
    "fp8_rmsnorm_backward": (
        _INT, [_P, _I64, _P, _I64, _P, _I64, _INT, _P, _P, _INT, _P, _I64, _P, _INT, _INT, _P, _SZ, _P]),
    "fp8_rmsnorm_backward_workspace_size": (_SZ, [_INT, _INT]),
    "fp8_rope_append_paged_kv": (
        _INT, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _INT, _INT, _INT, _P, _P, _I64, _INT, _P, _P, _P, _I64,
               _P, _P, _P, _P, _INT, _INT, _INT, _INT, _INT, _INT, _INT, _P]),
    "fp8_paged_attention": (
        _INT, [_P, _I64, _P, _P, _P, _P, _INT, _INT, _P, _I64, _INT, _P, _P, _P, _I64, _P, _F, _INT, _INT, _INT, _INT,
               _INT, _INT, _P, _SZ, _P]),
    "fp8_paged_attention_workspace_size": (_SZ, []),
}
_fns: dict = {}


def _fn(name: str):
    fn = _fns.get(name)
    if fn is None:
        fn = getattr(lib(), name)
        fn.restype, fn.argtypes = _SIGS[name]
        _fns[name] = fn
    return fn


def _dtype_code(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return QUANT_BF16
    _require(t.dtype == torch.float32, f"{name} must be bfloat16 or float32")
    return QUANT_FP32


def _rows(t: torch.Tensor, name: str, M: int, K: int, dtype, dev):
    _require(t.shape == (M, K) and t.dtype == dtype and t.device == dev and t.stride(1) == 1,
             f"{name} must be {dtype} [{M}, {K}] on {dev} with a unit inner stride")


def rmsnorm_quantize_1x128(X: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, Q: Optional[torch.Tensor] = None, sa: Optional[torch.Tensor] = None,
                           H: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                           Y: Optional[torch.Tensor] = None, stream=None):
    """RMS norm of X [M, K] (bfloat16 or float32, unit inner stride), or of X + residual
    (rounded to X's type), quantised as by quantize_1x128 -> (Q, sa, H, rstd).

    Q: e4m3 bytes [M, K] uint8; sa: float32 [K/128, >=M], a GEMM's A operand. H: the sum
    that was normalised, the residual stream's next value (X itself without a residual; it
    may be given as X or residual, in place). rstd: float32 [M] = 1/sqrt(mean(H^2) + eps),
    for rmsnorm_backward. Y: optional bfloat16 [M, K], receives the norm unquantised.
    weight: [K], bfloat16 or float32. K: a multiple of 128, at most 65536. Outputs may be
    given (written in place)."""
    _require(X.device.type == "cuda" and X.dim() == 2 and X.stride(1) == 1,
             "X must be a 2-D GPU tensor with a unit inner stride")
    code, dev = _dtype_code(X, "X"), X.device
    M, K = X.shape
    _require(K % 128 == 0, "K must be a multiple of 128")
    wcode = _dtype_code(weight, "weight")
    _require(weight.shape == (K,) and weight.device == dev and weight.stride(0) == 1, "weight must be contiguous [K]")
    if residual is not None:
        _rows(residual, "residual", M, K, X.dtype, dev)
        if H is None:
            H = torch.empty_like(X, memory_format=torch.contiguous_format)
        _rows(H, "H", M, K, X.dtype, dev)
    else:
        _require(H is None or H is X, "H is written only with a residual")
    if Q is None:
        Q = torch.empty(M, K, dtype=torch.uint8, device=dev)
    if sa is None:
        sa = torch.empty(K // 128, scale_ld(M), dtype=torch.float32, device=dev)
    if rstd is None:
        rstd = torch.empty(M, dtype=torch.float32, device=dev)
    Q = _bytes_view(Q)
    _rows(Q, "Q", M, K, torch.uint8, dev)
    _require(sa.dtype == torch.float32 and sa.dim() == 2 and sa.shape[0] == K // 128 and sa.stride(1) == 1
             and sa.device == dev and sa.shape[1] >= M, "sa must be float32 [K/128, >=M]")
    _require(rstd.shape == (M,) and rstd.dtype == torch.float32 and rstd.is_contiguous() and rstd.device == dev,
             "rstd must be contiguous float32 [M]")
    if Y is not None:
        _rows(Y, "Y", M, K, torch.bfloat16, dev)
    st = _fn("fp8_rmsnorm_quantize_1x128")(
        _ptr(X), _ld(X), _ptr(residual), 0 if residual is None else _ld(residual), code, _ptr(weight), wcode, float(eps),
        _ptr(H if residual is not None else None), 0 if residual is None else _ld(H), _ptr(Y), 0 if Y is None else _ld(Y),
        _ptr(rstd), _ptr(Q), _ld(Q), _ptr(sa), _ld(sa), M, K, _stream(dev, stream))
    _check(st, "fp8_rmsnorm_quantize_1x128")
    return Q, sa, X if residual is None else H, rstd


def rmsnorm_backward(dY: torch.Tensor, H: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                     dH: Optional[torch.Tensor] = None, dX: Optional[torch.Tensor] = None,
                     dW: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of the norm for dY [M, K], the gradient of its (unquantised) output ->
    (dX, dW). H [M, K] and rstd [M] as rmsnorm_quantize_1x128 gave them; dH: optional
    gradient that arrives at H over the residual stream. dX [M, K] (dY's type) is the
    gradient of X and of the residual alike, and may be dY or dH itself; dW is float32 [K].
    workspace: optional uint8 buffer, fp8_rmsnorm_backward_workspace_size(M, K) bytes;
    allocated if not given."""
    _require(dY.device.type == "cuda" and dY.dim() == 2 and dY.stride(1) == 1,
             "dY must be a 2-D GPU tensor with a unit inner stride")
    code, dev = _dtype_code(dY, "dY"), dY.device
    M, K = dY.shape
    _require(K % 128 == 0, "K must be a multiple of 128")
    wcode = _dtype_code(weight, "weight")
    _require(weight.shape == (K,) and weight.device == dev and weight.stride(0) == 1, "weight must be contiguous [K]")
    _rows(H, "H", M, K, dY.dtype, dev)
    _require(rstd.shape == (M,) and rstd.dtype == torch.float32 and rstd.is_contiguous() and rstd.device == dev,
             "rstd must be contiguous float32 [M]")
    if dH is not None:
        _rows(dH, "dH", M, K, dY.dtype, dev)
    if dX is None:
        dX = torch.empty_like(dY, memory_format=torch.contiguous_format)
    _rows(dX, "dX", M, K, dY.dtype, dev)
    if dW is None:
        dW = torch.empty(K, dtype=torch.float32, device=dev)
    _require(dW.shape == (K,) and dW.dtype == torch.float32 and dW.is_contiguous() and dW.device == dev,
             "dW must be contiguous float32 [K]")
    if workspace is None:
        with torch.cuda.device(dev):
            workspace = torch.empty(_fn("fp8_rmsnorm_backward_workspace_size")(M, K), dtype=torch.uint8, device=dev)
        if stream is not None:  # used there after this function has let go of it
            workspace.record_stream(stream)
    _require(workspace.device == dev and workspace.is_contiguous(), "workspace must be contiguous on dY's device")
    st = _fn("fp8_rmsnorm_backward")(
        _ptr(dY), _ld(dY), _ptr(H), _ld(H), _ptr(dH), 0 if dH is None else _ld(dH), code, _ptr(rstd), _ptr(weight), wcode,
        _ptr(dX), _ld(dX), _ptr(dW), M, K, _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(dev, stream))
    _check(st, "fp8_rmsnorm_backward")
    return dX, dW


class PagedKVCache(NamedTuple):
    """Keys and values of one layer: codes, e4m3 bytes [num_pages, Hkv, page_size, D] (uint8
    or float8_e4m3fn), and scales, float32 [num_pages, Hkv], one power of two per page and
    head."""
    k: torch.Tensor
    k_scale: torch.Tensor
    v: torch.Tensor
    v_scale: torch.Tensor


def make_paged_kv_cache(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, device="cuda") -> PagedKVCache:
    """An empty cache (page_size 16, 32, 64, 128 or 256; head_dim 64, 128 or 256)."""
    _require(page_size in (16, 32, 64, 128, 256) and head_dim in (64, 128, 256),
             "page_size must be 16, 32, 64, 128 or 256 and head_dim 64, 128 or 256")
    shape = (num_pages, num_kv_heads, page_size, head_dim)
    codes = [torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
    return PagedKVCache(codes[0], scales[0], codes[1], scales[1])


def _check_cache(c: PagedKVCache, dev):
    k, v = _bytes_view(c.k), _bytes_view(c.v)
    _require(k.dim() == 4 and k.shape == v.shape and k.is_contiguous() and v.is_contiguous(),
             "cache codes must be contiguous [num_pages, Hkv, page_size, D], keys and values alike")
    for t in (c.k_scale, c.v_scale):
        _require(t.dtype == torch.float32 and t.shape == k.shape[:2] and t.is_contiguous(),
                 "cache scales must be contiguous float32 [num_pages, Hkv]")
    _require(k.device == dev and v.device == dev and c.k_scale.device == dev and c.v_scale.device == dev,
             "the cache is on another device")
    return k, v


def _heads(t: torch.Tensor, name: str, T: int, H: int, D: int, dev) -> int:
    """Row stride of a bfloat16 [T, H, D] tensor whose rows are contiguous."""
    _require(t.dtype == torch.bfloat16 and t.shape == (T, H, D) and t.device == dev
             and (D == 1 or t.stride(2) == 1) and (H == 1 or t.stride(1) == D),
             f"{name} must be bfloat16 [{T}, {H}, {D}] on {dev} with contiguous rows")
    return t.stride(0) if T > 1 else H * D


def _check_sequences(block_table, seq_lens, cu_q, dev):
    for t, d, name in ((block_table, 2, "block_table"), (seq_lens, 1, "seq_lens"), (cu_q, 1, "cu_q")):
        _require(t.dtype == torch.int32 and t.dim() == d and t.device == dev and (t.shape[-1] <= 1 or t.stride(-1) == 1),
                 f"{name} must be an int32 tensor on {dev} with a unit inner stride")
    B = seq_lens.shape[0]
    _require(block_table.shape[0] == B and cu_q.shape[0] == B + 1, "block_table must be [B, max_pages] and cu_q [B + 1]")
    return B


def rope_append_paged_kv(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, cos_sin: Optional[torch.Tensor],
                         cache: PagedKVCache, block_table: torch.Tensor, seq_lens: torch.Tensor, cu_q: torch.Tensor,
                         positions: Optional[torch.Tensor] = None, interleaved: bool = False,
                         q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Rotates the call's queries and keys by their positions and appends keys and values to
    the cache -> the rotated queries.

    q [T, Hq, D], k, v [T, Hkv, D]: bfloat16 with contiguous rows (views of one fused
    projection output will do); q None: only the cache is filled. cos_sin: float32
    [max_pos, rot_dim], the cosines of rot_dim / 2 angles, then their sines (None: no
    rotation); rot_dim a multiple of 16 up to D, later columns pass. interleaved: pairs are
    neighbouring columns instead of halves. positions: int32 [T] (default: the tokens'
    slots in their sequences, clamped to the table). q_out may be q itself.
    A page's scale is the smallest power of two by which what was appended fits e4m3; when
    it has to grow, the page's earlier codes are re-encoded. block_table, seq_lens, cu_q:
    see the module's text; seq_lens counts the new tokens."""
    dev = k.device
    _require(dev.type == "cuda" and k.dim() == 3, "k must be a 3-D GPU tensor")
    T, Hkv, D = k.shape
    kc, vc = _check_cache(cache, dev)
    num_pages, P = kc.shape[0], kc.shape[2]
    _require(kc.shape[1] == Hkv and kc.shape[3] == D, "the cache has other heads than k")
    ldk, ldv = _heads(k, "k", T, Hkv, D, dev), _heads(v, "v", T, Hkv, D, dev)
    Hq, ldq, ldqo = Hkv, 0, 0
    if q is not None:
        _require(q.dim() == 3, "q must be [T, Hq, D]")
        Hq = q.shape[1]
        ldq = _heads(q, "q", T, Hq, D, dev)
        if q_out is None:
            q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        ldqo = _heads(q_out, "q_out", T, Hq, D, dev)
    else:
        _require(q_out is None, "q_out without q")
    max_pos = rot_dim = ld_cs = 0
    if cos_sin is not None:
        _require(cos_sin.dtype == torch.float32 and cos_sin.dim() == 2 and cos_sin.device == dev and cos_sin.stride(1) == 1,
                 "cos_sin must be float32 [max_pos, rot_dim] with a unit inner stride")
        (max_pos, rot_dim), ld_cs = cos_sin.shape, _ld(cos_sin)
    B = _check_sequences(block_table, seq_lens, cu_q, dev)
    _require(positions is None or (positions.dtype == torch.int32 and positions.shape == (T,) and positions.device == dev
                                   and positions.is_contiguous()), "positions must be contiguous int32 [T]")
    st = _fn("fp8_rope_append_paged_kv")(
        _ptr(q), ldq, _ptr(k), ldk, _ptr(v), ldv, _ptr(cos_sin), ld_cs, max_pos, rot_dim, int(bool(interleaved)),
        _ptr(positions), _ptr(block_table), _ld(block_table), block_table.shape[1], _ptr(seq_lens), _ptr(cu_q), _ptr(q_out),
        ldqo, _ptr(kc), _ptr(cache.k_scale), _ptr(vc), _ptr(cache.v_scale), num_pages, P, B, T, Hq, Hkv, D,
        _stream(dev, stream))
    _check(st, "fp8_rope_append_paged_kv")
    return q_out


def attention_workspace_size() -> int:
    return int(_fn("fp8_paged_attention_workspace_size")())


def make_attention_workspace(device="cuda") -> torch.Tensor:
    """Zero-filled workspace for paged_attention calls of any shape, one after another."""
    return torch.zeros(attention_workspace_size(), dtype=torch.uint8, device=device)


def paged_attention(q: torch.Tensor, cache: PagedKVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    cu_q: torch.Tensor, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    softmax_scale: Optional[float] = None, window: int = 0, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Causal attention of q [T, Hq, D] (bfloat16, contiguous rows) over the cache, which
    holds the call's own tokens already -> out, bfloat16 [T, Hq, D].

    The new tokens of sequence b are the last of its seq_lens[b]; each sees its own slot and
    those before it (window > 0: the last `window` of these). Query head i reads key head
    i // (Hq // Hkv). softmax_scale: default D ** -0.5. lse: optional contiguous float32
    [T, Hq], receives log sum exp of each row's scaled logits. A row that sees nothing gives
    0 and -inf. workspace: optional (make_attention_workspace), lets sequences be split over
    workgroups; calls that may overlap in time must not share one."""
    dev = q.device
    _require(dev.type == "cuda" and q.dim() == 3, "q must be a 3-D GPU tensor")
    T, Hq, D = q.shape
    kc, vc = _check_cache(cache, dev)
    num_pages, Hkv, P = kc.shape[0], kc.shape[1], kc.shape[2]
    _require(kc.shape[3] == D and Hkv > 0 and Hq % Hkv == 0, "q's heads do not match the cache's")
    ldq = _heads(q, "q", T, Hq, D, dev)
    if out is None:
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    ldo = _heads(out, "out", T, Hq, D, dev)
    _require(lse is None or (lse.dtype == torch.float32 and lse.shape == (T, Hq) and lse.is_contiguous()
                             and lse.device == dev), "lse must be contiguous float32 [T, Hq]")
    B = _check_sequences(block_table, seq_lens, cu_q, dev)
    _require(workspace is None or (workspace.device == dev and workspace.is_contiguous()),
             "workspace must be contiguous on q's device")
    st = _fn("fp8_paged_attention")(
        _ptr(q), ldq, _ptr(kc), _ptr(cache.k_scale), _ptr(vc), _ptr(cache.v_scale), num_pages, P, _ptr(block_table),
        _ld(block_table), block_table.shape[1], _ptr(seq_lens), _ptr(cu_q), _ptr(out), ldo, _ptr(lse),
        D ** -0.5 if softmax_scale is None else float(softmax_scale), int(window), B, T, Hq, Hkv, D, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(dev, stream))
    _check(st, "fp8_paged_attention")
    return out
