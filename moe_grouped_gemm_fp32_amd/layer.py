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

from . import _check, _ld, _require, lib, scale_ld, QUANT_BF16, QUANT_FP32

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
_BF16, _FP32, _U8, _I32, _FP8 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.float8_e4m3fn
_DTYPES = {_BF16: QUANT_BF16, _FP32: QUANT_FP32}
_fns: dict = {}


# A decode step calls these operators for microseconds of GPU work each, so the checks below
# are plain comparisons: a message is only put together when one fails, and pointers go to
# the library as integers.
def _fn(name: str):
    fn = _fns.get(name)
    if fn is None:
        fn = getattr(lib(), name)
        fn.restype, fn.argtypes = _SIGS[name]
        _fns[name] = fn
    return fn


_current_stream = torch._C._cuda_getCurrentRawStream  # current_stream(dev).cuda_stream without a Stream object: 0.1 us, not 1.9


def _raw_stream(dev: torch.device, stream) -> int:
    return _current_stream(dev.index) if stream is None else stream.cuda_stream


def _refuse(msg: str):
    raise ValueError(msg)


def _matrix(t: torch.Tensor, name: str, shape, dtype, dev) -> int:
    """Row stride of a tensor that must be `dtype` of `shape` [M, K] with a unit inner stride."""
    if t.shape != shape or t.dtype is not dtype or t.device != dev or t.stride(1) != 1:
        _refuse(f"{name} must be {dtype} {list(shape)} on {dev} with a unit inner stride")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _vector(t: torch.Tensor, name: str, n: int, dtype, dev) -> int:
    """Address of a tensor that must be contiguous `dtype` [n]."""
    if t.dim() != 1 or t.shape[0] != n or t.dtype is not dtype or t.device != dev or (n > 1 and t.stride(0) != 1):
        _refuse(f"{name} must be contiguous {dtype} [{n}] on {dev}")
    return t.data_ptr()


def _rows_of(X: torch.Tensor, name: str):
    """(dtype code, M, K) of the 2-D GPU tensor that a norm call is about."""
    code = _DTYPES.get(X.dtype)
    if not X.is_cuda or X.dim() != 2 or X.stride(1) != 1 or code is None or X.shape[1] % 128 != 0:
        _refuse(f"{name} must be a 2-D bfloat16 or float32 GPU tensor with a unit inner stride and a multiple of 128 columns")
    return code, X.shape[0], X.shape[1]


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
    code, M, K = _rows_of(X, "X")
    dev, shape = X.device, (M, K)
    w = _vector(weight, "weight", K, weight.dtype if weight.dtype in _DTYPES else _FP32, dev)
    r = h = y = 0
    ldr = ldh = ldy = 0
    if residual is not None:
        ldr, r = _matrix(residual, "residual", shape, X.dtype, dev), residual.data_ptr()
        if H is None:
            H = torch.empty(shape, dtype=X.dtype, device=dev)
        ldh, h = _matrix(H, "H", shape, X.dtype, dev), H.data_ptr()
    else:
        if H is not None and H is not X:
            _refuse("H is written only with a residual")
        H = X
    if Q is None:
        Q = torch.empty(shape, dtype=_U8, device=dev)
    if sa is None:
        sa = torch.empty(K // 128, scale_ld(M), dtype=_FP32, device=dev)
    if rstd is None:
        rstd = torch.empty(M, dtype=_FP32, device=dev)
    ldq = _matrix(Q, "Q", shape, _FP8 if Q.dtype is _FP8 else _U8, dev)
    if sa.dtype is not _FP32 or sa.dim() != 2 or sa.shape[0] != K // 128 or sa.shape[1] < M or sa.stride(1) != 1 or sa.device != dev:
        _refuse(f"sa must be float32 [{K // 128}, >= {M}] on {dev} with a unit inner stride")
    if Y is not None:
        ldy, y = _matrix(Y, "Y", shape, _BF16, dev), Y.data_ptr()
    st = _fn("fp8_rmsnorm_quantize_1x128")(
        X.data_ptr(), _ld(X), r, ldr, code, w, _DTYPES[weight.dtype], eps, h, ldh, y, ldy, _vector(rstd, "rstd", M, _FP32, dev),
        Q.data_ptr(), ldq, sa.data_ptr(), _ld(sa), M, K, _raw_stream(dev, stream))
    if st:
        _check(st, "fp8_rmsnorm_quantize_1x128")
    return Q, sa, H, rstd


def rmsnorm_backward(dY: torch.Tensor, H: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                     dH: Optional[torch.Tensor] = None, dX: Optional[torch.Tensor] = None,
                     dW: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of the norm for dY [M, K], the gradient of its (unquantised) output ->
    (dX, dW). H [M, K] and rstd [M] as rmsnorm_quantize_1x128 gave them; dH: optional
    gradient that arrives at H over the residual stream. dX [M, K] (dY's type) is the
    gradient of X and of the residual alike, and may be dY or dH itself; dW is float32 [K].
    workspace: optional uint8 buffer, fp8_rmsnorm_backward_workspace_size(M, K) bytes;
    allocated if not given."""
    code, M, K = _rows_of(dY, "dY")
    dev, shape, dt = dY.device, (M, K), dY.dtype
    w = _vector(weight, "weight", K, weight.dtype if weight.dtype in _DTYPES else _FP32, dev)
    ldh = _matrix(H, "H", shape, dt, dev)
    d, ldd = 0, 0
    if dH is not None:
        ldd, d = _matrix(dH, "dH", shape, dt, dev), dH.data_ptr()
    if dX is None:
        dX = torch.empty(shape, dtype=dt, device=dev)
    if dW is None:
        dW = torch.empty(K, dtype=_FP32, device=dev)
    if workspace is None:
        with torch.cuda.device(dev):
            workspace = torch.empty(_fn("fp8_rmsnorm_backward_workspace_size")(M, K), dtype=_U8, device=dev)
        if stream is not None:  # used there after this function has let go of it
            workspace.record_stream(stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        _refuse("workspace must be contiguous on dY's device")
    st = _fn("fp8_rmsnorm_backward")(
        dY.data_ptr(), _ld(dY), H.data_ptr(), ldh, d, ldd, code, _vector(rstd, "rstd", M, _FP32, dev), w, _DTYPES[weight.dtype],
        dX.data_ptr(), _matrix(dX, "dX", shape, dt, dev), _vector(dW, "dW", K, _FP32, dev), M, K, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _raw_stream(dev, stream))
    if st:
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


def _cache_shape(c: PagedKVCache, dev):
    """(num_pages, Hkv, page_size, D) of a cache that must be whole."""
    k, ks, v, vs = c
    shape = k.shape
    if (len(shape) != 4 or v.shape != shape or k.dtype not in (_U8, _FP8) or v.dtype not in (_U8, _FP8) or not k.is_contiguous()
            or not v.is_contiguous() or k.device != dev or v.device != dev):
        _refuse(f"cache codes must be contiguous uint8 or float8_e4m3fn [num_pages, Hkv, page_size, D] on {dev}, keys and values alike")
    if (ks.shape != shape[:2] or vs.shape != shape[:2] or ks.dtype is not _FP32 or vs.dtype is not _FP32 or not ks.is_contiguous()
            or not vs.is_contiguous() or ks.device != dev or vs.device != dev):
        _refuse(f"cache scales must be contiguous float32 [num_pages, Hkv] on {dev}")
    return shape


def _heads(t: torch.Tensor, name: str, T: int, H: int, D: int, dev) -> int:
    """Row stride of a tensor that must be bfloat16 [T, H, D] with contiguous rows."""
    if t.shape != (T, H, D) or t.dtype is not _BF16 or t.device != dev or t.stride(2) != 1 or (H > 1 and t.stride(1) != D):
        _refuse(f"{name} must be bfloat16 [{T}, {H}, {D}] on {dev} with contiguous rows")
    return t.stride(0) if T > 1 else H * D


def _sequences(block_table, seq_lens, cu_q, dev):
    """(B, max_pages, row stride of the table)."""
    B = seq_lens.shape[0]
    if (block_table.dim() != 2 or block_table.shape[0] != B or block_table.dtype is not _I32 or block_table.device != dev
            or (block_table.shape[1] > 1 and block_table.stride(1) != 1)):
        _refuse(f"block_table must be int32 [{B}, max_pages] on {dev} with a unit inner stride")
    _vector(seq_lens, "seq_lens", B, _I32, dev)
    _vector(cu_q, "cu_q", B + 1, _I32, dev)
    pages = block_table.shape[1]
    return B, pages, block_table.stride(0) if B > 1 else pages


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
    if not k.is_cuda or k.dim() != 3:
        _refuse("k must be a 3-D GPU tensor")
    T, Hkv, D = k.shape
    num_pages, heads, P, dim = _cache_shape(cache, dev)
    if heads != Hkv or dim != D:
        _refuse("the cache has other heads than k")
    ldk, ldv = _heads(k, "k", T, Hkv, D, dev), _heads(v, "v", T, Hkv, D, dev)
    Hq, ldq, ldqo, qp, qop = Hkv, 0, 0, 0, 0
    if q is not None:
        if q.dim() != 3:
            _refuse("q must be [T, Hq, D]")
        Hq = q.shape[1]
        ldq, qp = _heads(q, "q", T, Hq, D, dev), q.data_ptr()
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=_BF16, device=dev)
        ldqo, qop = _heads(q_out, "q_out", T, Hq, D, dev), q_out.data_ptr()
    elif q_out is not None:
        _refuse("q_out without q")
    max_pos = rot_dim = ld_cs = table = 0
    if cos_sin is not None:
        if cos_sin.dtype is not _FP32 or cos_sin.dim() != 2 or cos_sin.device != dev or cos_sin.stride(1) != 1:
            _refuse(f"cos_sin must be float32 [max_pos, rot_dim] on {dev} with a unit inner stride")
        (max_pos, rot_dim), ld_cs, table = cos_sin.shape, _ld(cos_sin), cos_sin.data_ptr()
    B, pages, ld_bt = _sequences(block_table, seq_lens, cu_q, dev)
    st = _fn("fp8_rope_append_paged_kv")(
        qp, ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, table, ld_cs, max_pos, rot_dim, 1 if interleaved else 0,
        0 if positions is None else _vector(positions, "positions", T, _I32, dev), block_table.data_ptr(), ld_bt, pages,
        seq_lens.data_ptr(), cu_q.data_ptr(), qop, ldqo, cache[0].data_ptr(), cache[1].data_ptr(), cache[2].data_ptr(),
        cache[3].data_ptr(), num_pages, P, B, T, Hq, Hkv, D, _raw_stream(dev, stream))
    if st:
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
    if not q.is_cuda or q.dim() != 3:
        _refuse("q must be a 3-D GPU tensor")
    T, Hq, D = q.shape
    num_pages, Hkv, P, dim = _cache_shape(cache, dev)
    if dim != D or Hkv == 0 or Hq % Hkv != 0:
        _refuse("q's heads do not match the cache's")
    ldq = _heads(q, "q", T, Hq, D, dev)
    if out is None:
        out = torch.empty((T, Hq, D), dtype=_BF16, device=dev)
    ldo = _heads(out, "out", T, Hq, D, dev)
    lp = wp = wbytes = 0
    if lse is not None:
        if lse.dtype is not _FP32 or lse.shape != (T, Hq) or not lse.is_contiguous() or lse.device != dev:
            _refuse(f"lse must be contiguous float32 [{T}, {Hq}] on {dev}")
        lp = lse.data_ptr()
    B, pages, ld_bt = _sequences(block_table, seq_lens, cu_q, dev)
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            _refuse("workspace must be contiguous on q's device")
        wp, wbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = _fn("fp8_paged_attention")(
        q.data_ptr(), ldq, cache[0].data_ptr(), cache[1].data_ptr(), cache[2].data_ptr(), cache[3].data_ptr(), num_pages, P,
        block_table.data_ptr(), ld_bt, pages, seq_lens.data_ptr(), cu_q.data_ptr(), out.data_ptr(), ldo, lp,
        D ** -0.5 if softmax_scale is None else softmax_scale, window, B, T, Hq, Hkv, D, wp, wbytes, _raw_stream(dev, stream))
    if st:
        _check(st, "fp8_paged_attention")
    return out
