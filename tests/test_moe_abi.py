"""Host-side checks of the expert and head operators that need no GPU: the header's symbols are
exported and bound, and invalid arguments are refused with the documented codes before anything
is launched."""
import ctypes
import os
import re

import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
from moe_grouped_gemm_fp32_amd import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8moe.h")
NULL, SHAPE, LAYOUT, WORKSPACE, DEVICE = -1, -2, -3, -4, -5
A = 1 << 20  # an aligned address; never followed


def test_every_declared_symbol_is_exported_and_bound():
    names = re.findall(r"^\s*(?:size_t|int|int64_t)\s+(fp8_\w+)\s*\(", open(HEADER).read(), re.M)
    lib = ctypes.CDLL(fg.LIB_PATH)
    assert len(names) == 11 and set(names) == set(moe._SIGS)
    for n in names:
        assert hasattr(lib, n), n
    for n in moe.__all__:
        assert getattr(fg, n) is getattr(moe, n) and n in fg.__all__


def call(name, defaults, **kw):
    bad = set(kw) - set(defaults)
    assert not bad, bad
    return moe._fn(name)(*{**defaults, **kw}.values())


ROUTE = dict(logits=A, ldl=64, dtype=1, bias=A, scoring=1, groups=8, top_groups=4, group_best=2, renormalize=1, scale=1.0, ids=A,
             weights=A, scores=A, lds=64, T=5, E=64, top_k=6, stream=None)
ROUTE_GRAD = dict(dweights=A, logits=A, ldl=64, dtype=0, ids=A, scoring=0, renormalize=1, scale=1.0, dscores=A, ldds=64, dlogits=A,
                  lddl=64, T=5, E=64, top_k=6, stream=None)
DISPATCH = dict(Q=A, ldq=256, sa=A, ld_sa=8, ids=A, weights=A, Qx=A, ldqx=256, sax=A, ld_sax=1024, positions=A, sources=A, m_indices=A,
                counts=A, rows=1024, max_m=0, T=5, top_k=2, E=8, K=256, workspace=A, workspace_bytes=1 << 20, stream=None)
GATHER = dict(Q=A, ldq=256, sa=A, ld_sa=8, weights=A, Qx=A, ldqx=256, sax=A, ld_sax=1024, positions=A, sources=A, rows=1024, max_m=0,
              T=5, top_k=2, E=8, K=256, stream=None)
COMBINE = dict(Y=A, ldy=256, dtype=0, positions=A, weights=A, C=A, ldc=256, out=A, ldo=256, rows=1024, T=5, top_k=2, N=256, stream=None)
COMBINE_GRAD = dict(dO=A, lddo=256, Y=A, ldy=256, dtype=0, positions=A, weights=A, dY=A, lddy=256, dweights=A, rows=1024, T=5, top_k=2,
                    N=256, stream=None)
HEADS = dict(q=A, ldq=512, k=A, ldk=256, dtype=0, qw=A, kw=A, w_dtype=0, cos_sin=A, ld_cs=128, max_pos=9, rot_dim=128, interleaved=0,
             positions=A, eps=1e-6, q_out=A, ldqo=512, k_out=A, ldko=256, T=5, Hq=4, Hk=2, D=128, stream=None)
HEADS_GRAD = dict(dq=A, lddq=512, dk=A, lddk=256, q=A, ldq=512, k=A, ldk=256, dtype=0, qw=A, kw=A, w_dtype=0, cos_sin=A, ld_cs=128,
                  max_pos=9, rot_dim=128, interleaved=0, positions=A, eps=1e-6, dq_out=A, lddqo=512, dk_out=A, lddko=256, dqw=A, dkw=A,
                  T=5, Hq=4, Hk=2, D=128, workspace=A, workspace_bytes=1 << 24, stream=None)


def each(*names, value=None):
    return [{n: value} for n in names]


REFUSED = [
    ("fp8_moe_route", ROUTE, NULL, each("logits", "ids", "weights")),
    ("fp8_moe_route", ROUTE, SHAPE,
     [dict(T=-1), dict(E=0), dict(E=1025), dict(top_k=0), dict(top_k=65), dict(top_k=7, E=6, groups=1, top_groups=1), dict(groups=0),
      dict(groups=5), dict(groups=128, E=256), dict(top_groups=0), dict(top_groups=9), dict(group_best=0), dict(group_best=3),
      dict(scale=float("nan")), dict(scale=float("inf"))]),
    ("fp8_moe_route", ROUTE, LAYOUT,
     [dict(dtype=2), dict(scoring=2), dict(scoring=-1), dict(ldl=63), dict(lds=63), dict(logits=A + 2), dict(bias=A + 2), dict(ids=A + 2),
      dict(weights=A + 1), dict(scores=A + 2), dict(dtype=0, logits=A + 1)]),
    ("fp8_moe_route_backward", ROUTE_GRAD, NULL, each("dweights", "logits", "ids", "dlogits")),
    ("fp8_moe_route_backward", ROUTE_GRAD, SHAPE, [dict(T=-1), dict(E=0), dict(E=2000), dict(top_k=0), dict(top_k=65), dict(scale=float("inf"))]),
    ("fp8_moe_route_backward", ROUTE_GRAD, LAYOUT,
     [dict(dtype=3), dict(scoring=5), dict(ldl=60), dict(lddl=60), dict(ldds=60), dict(logits=A + 1), dict(dlogits=A + 1), dict(ids=A + 2),
      dict(dweights=A + 2), dict(dscores=A + 2)]),
    ("fp8_moe_dispatch", DISPATCH, NULL, each("sa", "ids", "Qx", "sax", "positions", "sources", "m_indices", "counts")),
    ("fp8_moe_dispatch", DISPATCH, SHAPE,
     [dict(T=-1), dict(top_k=0), dict(top_k=65), dict(E=0), dict(E=1025), dict(K=0), dict(K=200), dict(K=65536 + 128), dict(rows=-128),
      dict(rows=1000), dict(max_m=-1), dict(max_m=100), dict(T=1 << 30, top_k=2), dict(rows=1 << 31)]),
    ("fp8_moe_dispatch", DISPATCH, LAYOUT,
     [dict(Q=A + 8), dict(ldq=240), dict(ldq=264), dict(sa=A + 2), dict(ld_sa=4), dict(ld_sa=10), dict(Qx=A + 8), dict(ldqx=128),
      dict(ldqx=260), dict(sax=A + 1), dict(ld_sax=1020), dict(ld_sax=1026), dict(ids=A + 2), dict(weights=A + 2), dict(positions=A + 2),
      dict(sources=A + 2), dict(m_indices=A + 1), dict(counts=A + 2), dict(workspace=A + 8)]),
    ("fp8_moe_gather", GATHER, NULL, each("Q", "sa", "Qx", "sax", "positions", "sources")),
    ("fp8_moe_gather", GATHER, SHAPE, [dict(T=-1), dict(top_k=0), dict(K=64), dict(rows=100), dict(max_m=7), dict(max_m=128, E=0)]),
    ("fp8_moe_gather", GATHER, LAYOUT, [dict(Q=A + 4), dict(ldq=255), dict(ld_sa=4), dict(Qx=A + 4), dict(ld_sax=1000), dict(positions=A + 2),
                                        dict(sources=A + 3), dict(weights=A + 2)]),
    ("fp8_moe_combine", COMBINE, NULL, each("Y", "positions", "out")),
    ("fp8_moe_combine", COMBINE, SHAPE,
     [dict(T=-1), dict(top_k=0), dict(top_k=65), dict(N=0), dict(N=12), dict(rows=-1), dict(rows=1 << 31)]),
    ("fp8_moe_combine", COMBINE, LAYOUT,
     [dict(dtype=2), dict(Y=A + 8), dict(ldy=248), dict(ldy=260), dict(dtype=1, ldy=258), dict(C=A + 2), dict(ldc=128), dict(out=A + 8),
      dict(ldo=252), dict(positions=A + 2), dict(weights=A + 2)]),
    ("fp8_moe_combine_backward", COMBINE_GRAD, NULL, each("dO", "Y", "positions", "weights", "dweights")),
    ("fp8_moe_combine_backward", COMBINE_GRAD, SHAPE, [dict(T=-1), dict(top_k=65), dict(N=4), dict(rows=-1)]),
    ("fp8_moe_combine_backward", COMBINE_GRAD, LAYOUT,
     [dict(dtype=2), dict(dO=A + 8), dict(lddo=250), dict(Y=A + 8), dict(ldy=128), dict(dY=A + 8), dict(lddy=252), dict(positions=A + 2),
      dict(weights=A + 2), dict(dweights=A + 2)]),
    ("fp8_qk_norm_rope", HEADS, NULL, each("q_out", "k_out", "q", "k", "qw", "kw", "cos_sin")),
    ("fp8_qk_norm_rope", HEADS, SHAPE,
     [dict(T=-1), dict(D=96), dict(D=32), dict(rot_dim=8), dict(rot_dim=144), dict(rot_dim=-16), dict(max_pos=0), dict(eps=-1.0),
      dict(eps=float("nan")), dict(Hq=-1), dict(T=1 << 30), dict(Hq=1 << 24, T=1)]),
    ("fp8_qk_norm_rope", HEADS, LAYOUT,
     [dict(dtype=2), dict(w_dtype=4), dict(q=A + 8), dict(ldq=504), dict(ldq=516), dict(ldk=128), dict(k=A + 2), dict(q_out=A + 8),
      dict(ldqo=256), dict(ldko=260), dict(qw=A + 8), dict(kw=A + 4), dict(cos_sin=A + 8), dict(ld_cs=64), dict(ld_cs=130),
      dict(positions=A + 2)]),
    ("fp8_qk_norm_rope_backward", HEADS_GRAD, NULL,
     [*each("dq", "dk", "q", "k", "qw", "kw", "dq_out", "dk_out", "cos_sin"), dict(dqw=None, dkw=None)]),
    ("fp8_qk_norm_rope_backward", HEADS_GRAD, SHAPE, [dict(T=-1), dict(D=48), dict(rot_dim=24), dict(max_pos=0), dict(eps=-1.0), dict(T=1 << 30)]),
    ("fp8_qk_norm_rope_backward", HEADS_GRAD, LAYOUT,
     [dict(dtype=2), dict(w_dtype=4), dict(dq=A + 8), dict(lddq=500), dict(lddk=128), dict(q=A + 8), dict(ldk=260), dict(dq_out=A + 4),
      dict(lddko=252), dict(dqw=A + 2), dict(dkw=A + 2), dict(workspace=A + 8), dict(cos_sin=A + 4), dict(ld_cs=120), dict(positions=A + 1)]),
]


@pytest.mark.parametrize("name,defaults,code,changes", REFUSED, ids=["%s%d" % (r[0][4:], r[2]) for r in REFUSED])
def test_refusals(name, defaults, code, changes):
    for kw in changes:
        assert call(name, defaults, **kw) == code, kw


ALL = [("fp8_moe_route", ROUTE), ("fp8_moe_route_backward", ROUTE_GRAD), ("fp8_moe_dispatch", DISPATCH), ("fp8_moe_gather", GATHER),
       ("fp8_moe_combine", COMBINE), ("fp8_moe_combine_backward", COMBINE_GRAD), ("fp8_qk_norm_rope", HEADS),
       ("fp8_qk_norm_rope_backward", HEADS_GRAD)]


def test_valid_calls_without_a_gpu_report_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for name, defaults in ALL:
        assert call(name, defaults) == DEVICE
    assert call("fp8_moe_dispatch", DISPATCH, Q=None, sa=None, Qx=None, sax=None, K=0) == DEVICE
    assert call("fp8_moe_dispatch", DISPATCH, max_m=128, rows=1024, m_indices=None, ld_sax=128) == DEVICE
    assert call("fp8_moe_route", ROUTE, bias=None, scores=None, groups=1, top_groups=1, dtype=0) == DEVICE
    assert call("fp8_moe_combine_backward", COMBINE_GRAD, dY=None) == DEVICE
    assert call("fp8_qk_norm_rope", HEADS, q=None, q_out=None, qw=None, ldq=0, ldqo=0) == DEVICE
    assert call("fp8_qk_norm_rope", HEADS, cos_sin=None, rot_dim=0, max_pos=0) == DEVICE


def test_calls_without_tokens_look_at_no_tokens():
    assert call("fp8_moe_route", ROUTE, T=0, logits=None, ids=None, weights=None) == 0
    assert call("fp8_moe_route_backward", ROUTE_GRAD, T=0, dweights=None, logits=None, ids=None, dlogits=None) == 0
    assert call("fp8_moe_gather", GATHER, T=0, Q=None, sa=None) == 0
    assert call("fp8_moe_combine", COMBINE, T=0, Y=None, positions=None, out=None) == 0
    assert call("fp8_moe_combine_backward", COMBINE_GRAD, T=0, dO=None, positions=None) == 0
    assert call("fp8_qk_norm_rope", HEADS, T=0, cos_sin=None) == 0
    assert call("fp8_qk_norm_rope", HEADS, q=None, k=None, q_out=None, k_out=None) == 0  # nor calls without heads at heads
    assert call("fp8_qk_norm_rope", HEADS, Hq=0, q=None, q_out=A, Hk=0, k_out=None) == 0


def test_sizes():
    rows = fg.moe_rows
    assert rows(0, 8, 256) == 0 and rows(1, 1, 1) == 128 and rows(1, 8, 256) == 1024 and rows(4096, 8, 256) == 65280
    assert rows(128, 1, 4) == (128 + 4 * 127) // 128 * 128
    for bad in ((5, 0, 8), (5, 65, 8), (-1, 2, 8), (5, 2, 0), (5, 2, 1025)):
        with pytest.raises(ValueError):
            rows(*bad)
    size = moe._fn("fp8_moe_dispatch_workspace_size")
    assert size(8, 8, 256) == 0 and size(-1, 2, 3) == 0 and size(5, 0, 8) == 0 and size(1 << 30, 2, 8) == 0
    assert size(65536, 8, 1000) == 513 * 1000 * 4
    if not torch.cuda.is_available():
        assert call("fp8_moe_dispatch", DISPATCH, T=4096, top_k=8, ld_sa=4096, rows=65280, ld_sax=65280, workspace_bytes=0) == DEVICE
    size = moe._fn("fp8_qk_norm_rope_backward_workspace_size")
    assert size(96) == 0 and size(128) == 2 * size(64) > 0


def test_bindings_refuse_host_tensors_and_wrong_types():
    x, i = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for f in (lambda: fg.moe_route(x, 2), lambda: fg.moe_route_backward(x[:, :2], x, i), lambda: fg.moe_dispatch(x, x, i, 8),
              lambda: fg.moe_gather(x, x, fg.make_moe_layout(4, 2, 8, device="cpu")), lambda: fg.moe_combine(x, i),
              lambda: fg.moe_combine_backward(x, x, i, x[:, :2]), lambda: fg.qk_norm_rope(q, q, x[0], x[0]),
              lambda: fg.qk_norm_rope_backward(q, q, q, q, x[0], x[0]), lambda: fg.qk_norm_rope(None, None, None, None)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: fg.moe_route(7, 2), lambda: fg.moe_combine([1.0], i), lambda: fg.qk_norm_rope(7, None, None, None)):
        with pytest.raises(TypeError):
            f()


def test_layout_tensors():
    at = fg.make_moe_layout(5, 2, 8, device="cpu")
    assert [tuple(t.shape) for t in at] == [(5, 2), (1024,), (1024,), (8,)] and all(t.dtype == torch.int32 for t in at)
    at = fg.make_moe_layout(5, 2, 8, max_m=3, device="cpu")
    assert at.m_indices is None and at.sources.shape == (24,)
    assert fg.make_moe_layout(5, 2, 8, rows=256, device="cpu").m_indices.shape == (256,)
    for bad in (dict(rows=100), dict(max_m=0), dict(max_m=4, rows=128)):
        with pytest.raises(ValueError):
            fg.make_moe_layout(5, 2, 8, device="cpu", **bad)
