"""The operators that a mixture-of-experts decoder layer needs around the grouped GEMMs: binding
of include/fp8moe.h.

  moe_route                 scores of experts, the choice among them, the weights of the chosen
  moe_route_backward        the gradient of the logits
  moe_dispatch              lays tokens' 8-bit rows out by expert, as the grouped GEMMs read them
  moe_gather                the same rows again, for a layout that is there
  moe_combine               weighted sum of the experts' rows of each token
  moe_combine_backward      its gradients
  qk_norm_rope              norm of queries and keys for each head, and their rotation
  qk_norm_rope_backward     its gradients

Like the layer operators' calls these only marshal tensors, in native code, read numbers of
experts and rows on the device only (every call may be captured into a graph), take a `stream`,
and are exported by the package. Equal calls give equal bits; scores, routing weights and the heads' weight
gradients may differ in their last bits between calls of other numbers of tokens or compute
units, chosen experts do not.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from . import _require, layer, lib

__all__ = ["MoeLayout", "make_moe_layout", "moe_rows", "moe_route", "moe_route_backward", "moe_dispatch", "moe_gather",
           "moe_combine", "moe_combine_backward", "qk_norm_rope", "qk_norm_rope_backward"]

_P, _I64, _INT, _SZ, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_SIGS = {
    "fp8_moe_route": (_INT, [_P, _I64, _INT, _P, _INT, _INT, _INT, _INT, _INT, _F, _P, _P, _P, _I64, _INT, _INT, _INT, _P]),
    "fp8_moe_route_backward": (
        _INT, [_P, _P, _I64, _INT, _P, _INT, _INT, _F, _P, _I64, _P, _I64, _INT, _INT, _INT, _P]),
    "fp8_moe_rows": (_I64, [_INT, _INT, _INT]),
    "fp8_moe_dispatch": (
        _INT, [_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _INT, _INT, _INT, _INT, _INT, _P, _SZ, _P]),
    "fp8_moe_dispatch_workspace_size": (_SZ, [_INT, _INT, _INT]),
    "fp8_moe_gather": (
        _INT, [_P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _P, _I64, _INT, _INT, _INT, _INT, _INT, _P]),
    "fp8_moe_combine": (_INT, [_P, _I64, _INT, _P, _P, _P, _I64, _P, _I64, _I64, _INT, _INT, _INT, _P]),
    "fp8_moe_combine_backward": (
        _INT, [_P, _I64, _P, _I64, _INT, _P, _P, _P, _I64, _P, _I64, _INT, _INT, _INT, _P]),
    "fp8_qk_norm_rope": (
        _INT, [_P, _I64, _P, _I64, _INT, _P, _P, _INT, _P, _I64, _INT, _INT, _INT, _P, _F, _P, _I64, _P, _I64, _INT, _INT, _INT,
               _INT, _P]),
    "fp8_qk_norm_rope_backward": (
        _INT, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _INT, _P, _P, _INT, _P, _I64, _INT, _INT, _INT, _P, _F, _P, _I64, _P, _I64,
               _P, _P, _INT, _INT, _INT, _INT, _P, _SZ, _P]),
    "fp8_qk_norm_rope_backward_workspace_size": (_SZ, [_INT]),
}
_fns: dict = {}


def _fn(name: str):
    fn = _fns.get(name)
    if fn is None:
        fn = getattr(lib(), name)
        fn.restype, fn.argtypes = _SIGS[name]
        _fns[name] = fn
    return fn


_native = None


def _calls():
    """The native half of this binding (raises if it has not been built)."""
    global _native
    if _native is None:
        module = layer._calls()
        module.bind_moe({n: ctypes.cast(getattr(lib(), n), ctypes.c_void_p).value for n in _SIGS})
        _native = module
    return _native


def moe_route(logits: torch.Tensor, top_k: int, bias: Optional[torch.Tensor] = None, scoring: str = "softmax", groups: int = 1,
              top_groups: int = 1, group_best: int = 1, renormalize: bool = True, scale: float = 1.0,
              ids: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
              stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Chooses top_k experts for each row of logits [T, E] (bfloat16 or float32, unit inner
    stride) -> (ids, weights): int32 and float32 [T, top_k], best first.

    The scores s are the softmax or the sigmoid (`scoring`) of the logits; experts are chosen
    by s + bias (float32 [E], for balance), ties by the lower index, and exactly: keys that
    float32 cannot tell apart are computed in float64. groups > 1: the experts are that many
    runs of equal length, and only those of the top_groups runs with the largest sums of
    their group_best (1 or 2) best keys take part. weights = scale * s / (sum of the chosen s
    + 1e-20), or scale * s without renormalize. A logit or key of -inf is never chosen; where
    fewer than top_k are left, ids end with -1 and weights with 0. scores: optional float32
    [T, E], receives s. E at most 1024, top_k at most 64, groups at most 64, scale
    at most 2^60 either way."""
    return (_native or _calls()).moe_route(logits, top_k, bias, scoring, groups, top_groups, group_best, renormalize, scale, ids,
                                           weights, scores, stream)


def moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, scoring: str = "softmax",
                       renormalize: bool = True, scale: float = 1.0, dscores: Optional[torch.Tensor] = None,
                       dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of the logits (of their type) for dweights, float32 [T, top_k], the gradient of
    moe_route's weights, and optionally dscores, float32 [T, E], that of its scores (a loss on
    balance). The choice counts as given; ids -1 have no part in it. dlogits may be the
    logits themselves. The bias, which only chooses, has no gradient."""
    return (_native or _calls()).moe_route_backward(dweights, logits, ids, scoring, renormalize, scale, dscores, dlogits, stream)


class MoeLayout(NamedTuple):
    """Where the choices of a batch lie among the experts' rows; int32 tensors.

    positions [T, top_k]: the row of each choice (-1: none); sources [rows]: the choice
    t * top_k + j in each row (-1: none); m_indices [rows]: the expert of each row (-1:
    none), as fp8_grouped_gemm_nt_contiguous takes it, None in the masked layout; counts
    [E]: rows of each expert that hold a choice, the masked GEMM's masked_m."""
    positions: torch.Tensor
    sources: torch.Tensor
    m_indices: Optional[torch.Tensor]
    counts: torch.Tensor


def moe_rows(tokens: int, top_k: int, num_experts: int) -> int:
    """Rows that the contiguous layout can need: every expert's segment rounded up to 128."""
    rows = _fn("fp8_moe_rows")
    # 0 is also what a call out of range gets: no tokens are in range where one is
    _require(rows(tokens or 1, top_k, num_experts) > 0, "tokens, top_k or num_experts out of range")
    return int(rows(tokens, top_k, num_experts))


def make_moe_layout(tokens: int, top_k: int, num_experts: int, max_m: Optional[int] = None, rows: Optional[int] = None,
                    device="cuda") -> MoeLayout:
    """Tensors for moe_dispatch to write a layout into: the contiguous one of `rows` rows
    (default moe_rows(...), a multiple of 128), or the masked one with max_m rows an expert."""
    _require(max_m is None or (max_m >= 1 and rows is None), "max_m must be at least 1, and the masked layout has max_m rows an expert")
    if max_m is not None:
        rows = num_experts * max_m
    elif rows is None:
        rows = moe_rows(tokens, top_k, num_experts)
    _require(max_m is not None or rows % 128 == 0, "rows must be a multiple of 128")

    def empty(*shape):
        return torch.empty(shape, dtype=torch.int32, device=device)

    return MoeLayout(empty(tokens, top_k), empty(rows), empty(rows) if max_m is None else None, empty(num_experts))


def moe_dispatch(Q: torch.Tensor, sa: torch.Tensor, ids: torch.Tensor, num_experts: int, max_m: Optional[int] = None,
                 weights: Optional[torch.Tensor] = None, Qx: Optional[torch.Tensor] = None, sax: Optional[torch.Tensor] = None,
                 layout: Optional[MoeLayout] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, MoeLayout]:
    """Lays the tokens' rows out by expert -> (Qx, sax, layout).

    Q [T, K], sa [K/128, >=T]: rows and scales as quantize_1x128 and rmsnorm_quantize_1x128
    give them; ids: int32 [T, top_k], those outside [0, num_experts) are no choice. Without
    max_m the contiguous layout: Qx [rows, K] uint8, sax [K/128, >=rows], expert segments
    beginning at multiples of 128 rows, layout.m_indices. With it the masked one: Qx
    [num_experts, max_m, K], sax [num_experts, K/128, >=max_m], masked_m = layout.counts;
    choices past an expert's max_m rows have no row. Within an expert rows are in the order
    of tokens. Rows without a choice are not written (in Qx, sax; the layout is whole).
    weights: optional float32 [T, top_k], multiplied into the rows' scales. A layout given
    (make_moe_layout) is written in place; its number of rows is the contiguous layout's,
    and choices past it have no row. workspace: optional uint8 buffer,
    fp8_moe_dispatch_workspace_size(T, top_k, E) bytes; allocated if not given."""
    Qx, sax, made = (_native or _calls()).moe_dispatch(Q, sa, ids, num_experts, max_m, weights, Qx, sax, layout, workspace, stream)
    return Qx, sax, MoeLayout(*made)


def moe_gather(Q: torch.Tensor, sa: torch.Tensor, layout: MoeLayout, weights: Optional[torch.Tensor] = None,
               Qx: Optional[torch.Tensor] = None, sax: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The rows of a layout that moe_dispatch made, for other Q and sa of its tokens -> (Qx,
    sax). With weights this is the combination's backward pass in 8 bits: the rows of
    quantize_1x128(dO), each standing for weight * dO."""
    return (_native or _calls()).moe_gather(Q, sa, layout, weights, Qx, sax, stream)


def moe_combine(Y: torch.Tensor, positions: torch.Tensor, weights: Optional[torch.Tensor] = None, C: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = C[t] + sum_j weights[t, j] * Y[positions[t, j]] -> out [T, N] of Y's type, summed
    in float32 in the order of j and rounded once.

    Y: the experts' rows, bfloat16 or float32 [rows, N] or [E, max_m, N]; positions: int32 [T,
    top_k] (layout.positions), -1 adds nothing; weights: float32 [T, top_k] (None: ones, the
    backward pass of a dispatch); C: optional [T, N] of Y's type, may be out. N a multiple
    of 8."""
    return (_native or _calls()).moe_combine(Y, positions, weights, C, out, stream)


def moe_combine_backward(dO: torch.Tensor, Y: torch.Tensor, positions: torch.Tensor, weights: torch.Tensor,
                         dY: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None, rows: bool = True,
                         stream=None) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """Gradients of moe_combine for dO [T, N] -> (dY, dweights): dY[positions[t, j]] =
    weights[t, j] * dO[t] in Y's shape and type, dweights[t, j] = dO[t] . Y[positions[t, j]]
    in float32 (0 without a row). Rows of dY that no position names are not written; dY may
    be Y. Without `rows`, dY is None and only dweights is computed (moe_gather has the rows'
    gradients in 8 bits). C's gradient is dO."""
    return (_native or _calls()).moe_combine_backward(dO, Y, positions, weights, dY, dweights, rows, stream)


def qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                 k_weight: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """RMS norm of each head of q [T, Hq, D] and k [T, Hk, D], then its rotation, in one pass ->
    (q_out, k_out). What comes out is appended by rope_append_paged_kv with cos_sin None.

    q, k: bfloat16 or float32 with contiguous rows (views of one fused projection output will
    do); either may be None. q_weight, k_weight: [D], bfloat16 or float32, alike. cos_sin,
    interleaved: as for rope_append_paged_kv, so that the first rot_dim columns turn.
    positions: int32 [T], clamped to the table (default: 0, 1, ...). D 64, 128 or 256.
    Outputs may be q and k themselves."""
    return (_native or _calls()).qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, q_out, k_out, stream)


def qk_norm_rope_backward(dq: Optional[torch.Tensor], dk: Optional[torch.Tensor], q: Optional[torch.Tensor],
                          k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                          cos_sin: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          interleaved: bool = False, dq_out: Optional[torch.Tensor] = None, dk_out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of qk_norm_rope for dq and dk, those of its outputs -> (dq_out, dk_out, dq_weight,
    dk_weight). q and k are its inputs; the weights' gradients are float32 [D], summed over
    tokens and heads in a fixed order. dq or dk may be None, with None for its results.
    dq_out may be dq or q, dk_out dk or k. workspace: optional uint8 buffer,
    fp8_qk_norm_rope_backward_workspace_size(D) bytes; allocated if not given."""
    return (_native or _calls()).qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, dq_out,
                                                       dk_out, workspace, stream)
