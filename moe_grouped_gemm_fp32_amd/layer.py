"""The operators around the FP8 GEMMs of a transformer layer: binding of include/fp8layer.h.

  rmsnorm_quantize_1x128   residual addition, RMS norm and 1x128 quantisation
  rmsnorm_backward         the norm's gradients
  rope_append_paged_kv     rotates queries and keys, appends keys and values to the cache
  paged_attention          causal attention over the cache

Like the GEMM bindings these only marshal tensors; they are exported by the package. The
checks and conversions are native (csrc_layer/binding.cpp), since a decode step makes these
calls for a few microseconds of GPU work each.

The paged cache of one layer is a PagedKVCache (make_paged_kv_cache); which pages hold a
sequence, and which rows of a call are its new tokens, is given by three int32 tensors:
block_table [B, max_pages], seq_lens [B] (new tokens included) and cu_q [B + 1] (row
offsets of the sequences' new tokens). They are read on the device only, so every call may
be captured into a graph.

Calls take a `stream`, the current one by default. What a call allocates belongs to the stream
it runs on, as under torch.cuda.stream(), and stays allocated until the work that the current
stream had when it was let go of is done.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple, Optional

import torch

from . import _check, _require, lib

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


CALL_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_layer_call.so")
_native = None


def _calls():
    """The native half of this binding (raises if it has not been built)."""
    global _native
    if _native is None:
        if not os.path.exists(CALL_PATH):
            raise ImportError(f"{CALL_PATH} is missing: build it with moe_grouped_gemm_fp32_amd/build.py "
                              "(or __graft_entry__.build())")
        loader = importlib.machinery.ExtensionFileLoader("_layer_call", CALL_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_layer_call", loader))
        loader.exec_module(module)
        names = [*_SIGS, "fp8_gemm_scale_ld"]
        address = {n: ctypes.cast(getattr(lib(), n), ctypes.c_void_p).value for n in names}
        module.bind(address, _check, torch._C._cuda_getCurrentRawStream, torch.cuda.ExternalStream)
        _native = module
    return _native


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
    return (_native or _calls()).rmsnorm_quantize(X, weight, residual, eps, Q, sa, H, rstd, Y, stream)


def rmsnorm_backward(dY: torch.Tensor, H: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                     dH: Optional[torch.Tensor] = None, dX: Optional[torch.Tensor] = None,
                     dW: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of the norm for dY [M, K], the gradient of its (unquantised) output ->
    (dX, dW). H [M, K] and rstd [M] as rmsnorm_quantize_1x128 gave them; dH: optional
    gradient that arrives at H over the residual stream. dX [M, K] (dY's type) is the
    gradient of X and of the residual alike, and may be dY or dH itself; dW is float32 [K].
    workspace: optional uint8 buffer, fp8_rmsnorm_backward_workspace_size(M, K) bytes;
    allocated if not given."""
    return (_native or _calls()).rmsnorm_backward(dY, H, rstd, weight, dH, dX, dW, workspace, stream)


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
    see the module's text; seq_lens counts the new tokens. Tokens past the table's slots are
    not stored."""
    return (_native or _calls()).rope_append(q, k, v, cos_sin, cache, block_table, seq_lens, cu_q, positions, interleaved,
                                             q_out, stream)


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
    return (_native or _calls()).attend(q, cache, block_table, seq_lens, cu_q, out, lse, softmax_scale, window, workspace, stream)
