"""Host-side checks of the layer operators that need no GPU: the header's symbols are
exported and bound, and invalid arguments are refused with the documented codes before
anything is launched."""
import ctypes
import os
import re

import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
from moe_grouped_gemm_fp32_amd import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8layer.h")
NULL, SHAPE, LAYOUT, WORKSPACE, DEVICE = -1, -2, -3, -4, -5
A = 1 << 20  # an aligned address; never followed


def test_every_declared_symbol_is_exported_and_bound():
    names = re.findall(r"^\s*(?:size_t|int)\s+(fp8_\w+)\s*\(", open(HEADER).read(), re.M)
    lib = ctypes.CDLL(fg.LIB_PATH)
    assert len(names) == 6 and set(names) == set(layer._SIGS)
    for n in names:
        assert hasattr(lib, n), n
    for n in layer.__all__:
        assert getattr(fg, n) is getattr(layer, n) and n in fg.__all__


def call(name, defaults, **kw):
    bad = set(kw) - set(defaults)
    assert not bad, bad
    args = {**defaults, **kw}
    return layer._fn(name)(*args.values())


NORM = dict(X=A, ldx=256, R=A, ldr=256, x_dtype=0, w=A, w_dtype=0, eps=1e-6, H=A, ldh=256, Y=A, ldy=256, rstd=A, Q=A, ldq=256,
            sa=A, ld_sa=8, M=5, K=256, stream=None)
GRAD = dict(dY=A, lddy=256, H=A, ldh=256, dH=A, lddh=256, dtype=0, rstd=A, w=A, w_dtype=0, dX=A, lddx=256, dW=A, M=5, K=256,
            workspace=A, workspace_bytes=1 << 30, stream=None)
APPEND = dict(q=A, ldq=1024, k=A, ldk=256, v=A, ldv=256, cos_sin=A, ld_cs=128, max_pos=100, rot_dim=128, interleaved=0, positions=A,
              block_table=A, ld_bt=7, max_pages=7, seq_lens=A, cu_q=A, q_out=A, ldqo=1024, k_cache=A, k_scale=A, v_cache=A,
              v_scale=A, num_pages=9, P=64, B=3, T=5, Hq=8, Hkv=2, D=128, stream=None)
ATTEND = dict(q=A, ldq=1024, k_cache=A, k_scale=A, v_cache=A, v_scale=A, num_pages=9, P=64, block_table=A, ld_bt=7, max_pages=7,
              seq_lens=A, cu_q=A, O=A, ldo=1024, lse=A, scale=0.1, window=0, B=3, T=5, Hq=8, Hkv=2, D=128, workspace=A,
              workspace_bytes=1 << 26, stream=None)

REFUSED = [
    ("fp8_rmsnorm_quantize_1x128", NORM, NULL, [dict(X=None), dict(w=None), dict(Q=None), dict(sa=None), dict(H=None)]),
    ("fp8_rmsnorm_quantize_1x128", NORM, SHAPE, [dict(M=-1), dict(K=0), dict(K=200), dict(K=65536 + 128), dict(eps=-1.0),
                                                 dict(eps=float("nan"))]),
    ("fp8_rmsnorm_quantize_1x128", NORM, LAYOUT,
     [dict(x_dtype=2), dict(w_dtype=-1), dict(X=A + 8), dict(ldx=255), dict(ldx=260), dict(x_dtype=1, ldx=258), dict(w=A + 4),
      dict(R=A + 2), dict(ldr=128), dict(H=A + 8), dict(ldh=252), dict(Y=A + 8), dict(ldy=248), dict(Q=A + 4), dict(ldq=260),
      dict(sa=A + 2), dict(ld_sa=4), dict(ld_sa=10), dict(rstd=A + 1)]),
    ("fp8_rmsnorm_backward", GRAD, NULL, [dict(dY=None), dict(H=None), dict(rstd=None), dict(w=None), dict(dX=None), dict(dW=None)]),
    ("fp8_rmsnorm_backward", GRAD, SHAPE, [dict(M=-1), dict(K=0), dict(K=130), dict(K=1 << 17)]),
    ("fp8_rmsnorm_backward", GRAD, LAYOUT,
     [dict(dtype=7), dict(w_dtype=2), dict(dY=A + 8), dict(lddy=250), dict(ldh=128), dict(dH=A + 4), dict(lddh=260), dict(dX=A + 8),
      dict(dW=A + 2), dict(w=A + 8), dict(workspace=A + 8), dict(rstd=A + 2)]),
    ("fp8_rope_append_paged_kv", APPEND, NULL,
     [dict([(n, None)]) for n in ("k", "v", "cos_sin", "block_table", "seq_lens", "cu_q", "q", "q_out", "k_cache", "k_scale",
                                  "v_cache", "v_scale")]),
    ("fp8_rope_append_paged_kv", APPEND, SHAPE,
     [dict(num_pages=0), dict(P=48), dict(P=8), dict(D=96), dict(D=512), dict(Hkv=0), dict(Hq=0), dict(B=-1), dict(T=-1),
      dict(max_pages=-1), dict(rot_dim=8), dict(rot_dim=144), dict(rot_dim=-16), dict(max_pos=0), dict(T=1 << 28),
      dict(max_pages=1 << 26, ld_bt=1 << 26)]),
    ("fp8_rope_append_paged_kv", APPEND, LAYOUT,
     [dict(ldk=128), dict(ldk=260), dict(ldv=255), dict(ldq=1016), dict(ldq=1028), dict(ldqo=512), dict(ld_bt=6), dict(ld_cs=64),
      dict(ld_cs=130), dict(q=A + 8), dict(k=A + 2), dict(v=A + 8), dict(q_out=A + 4), dict(k_cache=A + 8), dict(v_cache=A + 4),
      dict(cos_sin=A + 8), dict(k_scale=A + 2), dict(v_scale=A + 1), dict(positions=A + 2), dict(block_table=A + 2),
      dict(seq_lens=A + 1), dict(cu_q=A + 2)]),
    ("fp8_paged_attention", ATTEND, NULL,
     [dict([(n, None)]) for n in ("q", "k_cache", "k_scale", "v_cache", "v_scale", "block_table", "seq_lens", "cu_q", "O")]),
    ("fp8_paged_attention", ATTEND, SHAPE,
     [dict(num_pages=0), dict(P=100), dict(D=192), dict(Hkv=3), dict(Hkv=0), dict(Hq=0), dict(B=-1), dict(T=-2), dict(max_pages=-1),
      dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan")), dict(T=1 << 28), dict(max_pages=1 << 26, ld_bt=1 << 26)]),
    ("fp8_paged_attention", ATTEND, LAYOUT,
     [dict(ldq=1016), dict(ldq=1028), dict(ldo=512), dict(ldo=1026), dict(ld_bt=6), dict(q=A + 8), dict(O=A + 2), dict(k_cache=A + 8),
      dict(v_cache=A + 8), dict(k_scale=A + 2), dict(v_scale=A + 2), dict(block_table=A + 2), dict(seq_lens=A + 2), dict(cu_q=A + 2),
      dict(lse=A + 2), dict(workspace=A + 8)]),
]


@pytest.mark.parametrize("name,defaults,code,changes", REFUSED, ids=["%s%d" % (r[0][4:], r[2]) for r in REFUSED])
def test_refusals(name, defaults, code, changes):
    for kw in changes:
        assert call(name, defaults, **kw) == code, kw


def test_valid_calls_without_a_gpu_report_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for name, defaults in (("fp8_rmsnorm_quantize_1x128", NORM), ("fp8_rmsnorm_backward", GRAD), ("fp8_rope_append_paged_kv", APPEND),
                           ("fp8_paged_attention", ATTEND)):
        assert call(name, defaults) == DEVICE


def test_workspace_sizes():
    assert fg.attention_workspace_size() == (64 << 20) + (64 << 10)
    size = layer._fn("fp8_rmsnorm_backward_workspace_size")
    assert size(0, 256) == 0 and size(5, 200) == 0 and size(5, -128) == 0 and size(5, 1 << 17) == 0
    for M, K in ((1, 128), (5, 7168), (10000, 65536)):
        assert size(M, K) >= K * 4 and size(M, K) % (K * 4) == 0
    assert size(10 ** 9, 7168) == size(10 ** 6, 7168)  # one part for each workgroup, however many rows


def test_bindings_refuse_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fg.rmsnorm_quantize_1x128(x, torch.ones(256))
    with pytest.raises(ValueError):
        fg.rmsnorm_backward(x, x, torch.ones(4), torch.ones(256))
    cache = fg.make_paged_kv_cache(2, 1, 16, 64, device="cpu")
    assert cache.k.shape == (2, 1, 16, 64) and cache.v_scale.shape == (2, 1)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fg.paged_attention(torch.zeros(1, 1, 64, dtype=torch.bfloat16), cache, i[None], i[:1], i)
    with pytest.raises(ValueError):
        fg.rope_append_paged_kv(None, torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 64, dtype=torch.bfloat16), None,
                                cache, i[None], i[:1], i)
    with pytest.raises(ValueError):
        fg.make_paged_kv_cache(2, 1, 24, 64, device="cpu")
