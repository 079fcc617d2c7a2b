"""The dispatch of tokens to experts on the GPU: positions, sources, numbers of experts and codes
are those of the oracle, scales too but for one rounding where weights are multiplied in."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from moe_grouped_gemm_fp32_amd import moe
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu

FP32, I32, U8 = torch.float32, torch.int32, torch.uint8


def tokens_of(T, K, seed, dev, pad=0):
    g = synth.make_generator(seed, dev)
    Q = torch.randint(0, 256, (T, K + pad), generator=g, device=dev, dtype=U8)[:, :K]
    sa = torch.rand(K // 128, fg.scale_ld(T) + pad // 4, generator=g, device=dev) + 0.25
    return Q, sa


def choices_of(T, k, E, seed, dev, bad=0.0):
    g = synth.make_generator(seed, dev)
    ids = torch.rand(T, E, generator=g, device=dev).pow(torch.linspace(0.2, 3, E, device=dev)).topk(k, dim=1).indices.to(I32)
    if bad:
        worse = torch.tensor([-1, E, 1 << 30, -(1 << 31)], dtype=I32, device=dev)[torch.randint(0, 4, (T, k), generator=g, device=dev)]
        ids = torch.where(torch.rand(T, k, generator=g, device=dev) < bad, worse, ids)
    return ids


def check(Q, sa, ids, E, max_m=None, rows=None, weights=None, **kw):
    T, K = Q.shape
    k, dev = ids.shape[1], Q.device
    p, s, m, c = mo.layout(ids.cpu().numpy(), E, max_m or 0, rows)
    n = len(s)
    shape = (E, max_m) if max_m else (n,)
    ld = fg.scale_ld(max_m or n) + 4
    Qx = torch.full((*shape, K + 16), 0xA5, dtype=U8, device=dev)[..., :K]
    sax = torch.full((*shape[:-1], K // 128, ld), -7.0, device=dev)
    given = fg.make_moe_layout(T, k, E, max_m, rows) if rows is not None else None
    gx, gs, at = fg.moe_dispatch(Q, sa, ids, E, max_m=max_m, weights=weights, Qx=Qx, sax=sax, layout=given, **kw)
    torch.cuda.synchronize()
    assert gx is Qx and gs is sax and isinstance(at, fg.MoeLayout)
    assert np.array_equal(at.positions.cpu().numpy(), p) and np.array_equal(at.sources.cpu().numpy(), s)
    assert np.array_equal(at.counts.cpu().numpy(), c)
    if max_m:
        assert at.m_indices is None
    else:
        assert np.array_equal(at.m_indices.cpu().numpy(), m)
    q, a, w = Q.cpu().numpy(), sa.cpu().numpy(), None if weights is None else weights.cpu().numpy().reshape(-1)
    want = np.full((n, K), 0xA5, np.uint8)
    scale = np.full((n, K // 128), -7.0, np.float32)
    live = s >= 0
    want[live] = q[s[live] // k]
    scale[live] = a[:, s[live] // k].T if w is None else (a[:, s[live] // k] * w[s[live]]).T
    whole = Qx.as_strided((n, K + 16), (K + 16, 1)).cpu().numpy()
    assert np.array_equal(whole[:, :K], want) and (whole[:, K:] == 0xA5).all()
    got = sax.cpu().numpy()
    if max_m:
        assert np.array_equal(got[:, :, :max_m].transpose(0, 2, 1).reshape(n, -1), scale) and (got[:, :, max_m:] == -7).all()
    else:
        assert np.array_equal(got[:, :n].T, scale) and (got[:, n:] == -7).all()
    # the same again into other buffers, from the layout
    Q2, s2 = torch.full_like(Qx, 0x11), torch.zeros_like(sax)
    fg.moe_gather(Q, sa, at, weights=weights, Qx=Q2, sax=s2)
    torch.cuda.synchronize()
    assert np.array_equal(Q2.reshape(n, K).cpu().numpy()[live], want[live]) and (Q2.reshape(n, K).cpu().numpy()[~live] == 0x11).all()
    back = s2.cpu().numpy()
    back = back[:, :, :max_m].transpose(0, 2, 1).reshape(n, -1) if max_m else back[:, :n].T
    assert np.array_equal(back[live], scale[live]) and (back[~live] == 0).all()
    return at


@pytest.mark.parametrize("T,k,E,K", [(1, 1, 1, 128), (1, 8, 256, 7168), (5, 3, 4, 384), (64, 8, 256, 1024), (127, 1, 3, 128), (333, 5, 17, 640),
                                     (700, 6, 64, 256), (900, 7, 1024, 128), (2000, 8, 100, 128), (129, 64, 70, 128), (3, 2, 2, 8320)])
def test_contiguous(cuda_device, T, k, E, K):
    Q, sa = tokens_of(T, K, 1, cuda_device, pad=32)
    ids = choices_of(T, k, E, 2, cuda_device)
    w = torch.randn(T, k, device=cuda_device)
    check(Q, sa, ids, E)
    check(Q, sa, ids, E, weights=w)
    check(Q, sa, choices_of(T, k, E, 3, cuda_device, bad=0.3), E, weights=w)
    if T * k > 200:
        check(Q, sa, ids, E, rows=256)  # what does not fit has no row
    check(Q, sa, ids, E, rows=0)


@pytest.mark.parametrize("T,k,E,K,max_m", [(1, 1, 1, 128, 1), (64, 8, 256, 7168, 64), (64, 8, 32, 256, 7), (333, 5, 17, 640, 333), (700, 6, 64, 256, 65),
                                           (900, 7, 1024, 128, 3), (2000, 8, 100, 128, 130)])
def test_masked(cuda_device, T, k, E, K, max_m):
    Q, sa = tokens_of(T, K, 4, cuda_device, pad=16)
    w = torch.rand(T, k, device=cuda_device)
    check(Q, sa, choices_of(T, k, E, 5, cuda_device), E, max_m=max_m)
    check(Q, sa, choices_of(T, k, E, 6, cuda_device, bad=0.4), E, max_m=max_m, weights=w)


@pytest.mark.parametrize("T", [1, 100, 1500])
def test_one_expert_takes_all_and_the_same_expert_twice(cuda_device, T):
    Q, sa = tokens_of(T, 256, 7, cuda_device)
    for E in (1, 5):
        ids = torch.full((T, 4), E - 1, dtype=I32, device=cuda_device)
        at = check(Q, sa, ids, E)
        assert at.counts.tolist() == [0] * (E - 1) + [4 * T]
        check(Q, sa, ids, E, max_m=2 * T + 1)
        check(Q, sa, torch.full_like(ids, -1), E)  # none at all


def test_outputs_of_its_own_and_many_choices(cuda_device):
    T, k, E, K = 40000, 2, 300, 128
    Q, sa = tokens_of(T, K, 8, cuda_device)
    ids = choices_of(T, k, E, 9, cuda_device)
    Qx, sax, at = fg.moe_dispatch(Q, sa, ids, E)
    torch.cuda.synchronize()
    p, s, m, c = mo.layout(ids.cpu().numpy(), E)
    assert Qx.shape == (fg.moe_rows(T, k, E), K) and sax.shape == (1, fg.scale_ld(Qx.shape[0]))
    assert np.array_equal(at.positions.cpu().numpy(), p) and np.array_equal(at.sources.cpu().numpy(), s)
    assert np.array_equal(at.m_indices.cpu().numpy(), m) and np.array_equal(at.counts.cpu().numpy(), c)
    live = at.positions.flatten().long()
    assert torch.equal(Qx[live], Q.repeat_interleave(k, 0)) and torch.equal(sax[0, live], sa[0, :T].repeat_interleave(k))
    need = moe._fn("fp8_moe_dispatch_workspace_size")(T, k, E)
    guard = torch.full((need + 64,), 0x5A, dtype=U8, device=cuda_device)
    again = fg.moe_dispatch(Q, sa, ids, E, workspace=guard[:need])
    torch.cuda.synchronize()
    assert bool((guard[need:] == 0x5A).all()) and torch.equal(again[2].positions, at.positions)
    with pytest.raises(fg.Fp8GemmError):
        fg.moe_dispatch(Q, sa, ids, E, workspace=guard[:need - 16])


def test_no_tokens(cuda_device):
    Q, sa = tokens_of(4, 256, 1, cuda_device)
    ids = choices_of(4, 2, 8, 1, cuda_device)
    Qx, sax, at = fg.moe_dispatch(Q[:0], sa, ids[:0], 8)
    torch.cuda.synchronize()
    assert Qx.shape == (0, 256) and at.counts.tolist() == [0] * 8
    at = fg.make_moe_layout(0, 2, 8, rows=256)
    fg.moe_dispatch(Q[:0], sa, ids[:0], 8, layout=at)
    assert at.counts.tolist() == [0] * 8 and bool((at.sources == -1).all()) and bool((at.m_indices == -1).all())
    at = fg.make_moe_layout(0, 2, 8, max_m=5)
    fg.moe_dispatch(Q[:0], sa, ids[:0], 8, max_m=5, layout=at)
    assert at.counts.tolist() == [0] * 8 and bool((at.sources == -1).all())


def test_a_layout_of_nonsense_is_not_followed(cuda_device):
    """Positions and sources outside the rows and choices are left out."""
    T, k, K = 6, 2, 256
    Q, sa = tokens_of(T, K, 2, cuda_device)
    at = fg.make_moe_layout(T, k, 4)
    for t in at:
        t.fill_(1 << 30)
    at.positions[0], at.sources[5] = 5, 1
    at.positions[1], at.sources[7] = -(1 << 31), -(1 << 31)
    Qx, sax = torch.full((512, K), 3, dtype=U8, device=cuda_device), torch.zeros(2, 512, device=cuda_device)
    fg.moe_gather(Q, sa, at, Qx=Qx, sax=sax)
    torch.cuda.synchronize()
    assert torch.equal(Qx[5], Q[0]) and bool((Qx[6:] == 3).all()) and bool((Qx[:5] == 3).all())
    assert torch.equal(sax[:, 5], sa[:, 0]) and int((sax != 0).sum()) == 2


def test_refusals(cuda_device):
    T, k, E, K = 6, 2, 4, 256
    Q, sa = tokens_of(T, K, 3, cuda_device)
    ids = choices_of(T, k, E, 3, cuda_device)
    Qx, sax, at = fg.moe_dispatch(Q, sa, ids, E)
    masked = fg.make_moe_layout(T, k, E, max_m=8)
    for bad in (dict(Q=Q[:, :200]), dict(Q=Q.t()), dict(Q=Q.float()), dict(sa=sa[:1]), dict(sa=sa[:, :5]), dict(ids=ids[:5]), dict(ids=ids.long()),
                dict(num_experts=0), dict(max_m=0), dict(max_m=-1), dict(weights=ids), dict(weights=sa[:1, :1]), dict(Qx=Qx[:-1]), dict(Qx=Qx.float()),
                dict(sax=sax[:, :100]), dict(layout=masked), dict(layout=at, max_m=8), dict(layout=at._replace(positions=ids[:5])),
                dict(layout=at._replace(counts=at.counts[:3])), dict(layout=at._replace(m_indices=at.m_indices[:128]))):
        with pytest.raises(ValueError):
            fg.moe_dispatch(**{"Q": Q, "sa": sa, "ids": ids, "num_experts": E, **bad})
    with pytest.raises(TypeError):
        fg.moe_dispatch(Q, sa, ids, E, layout=at[:3])
    with pytest.raises(fg.Fp8GemmError):
        fg.moe_dispatch(Q, sa, ids, 1025)
    for bad in (dict(Q=Q[:5]), dict(weights=ids), dict(Qx=Qx[:3]), dict(layout=masked, Qx=Qx)):
        with pytest.raises(ValueError):
            fg.moe_gather(**{"Q": Q, "sa": sa, "layout": at, **bad})


def test_masked_rows_of_one_stride(cuda_device):
    """One row an expert of a larger buffer, and one K block, lie at one stride as well."""
    T, E, K = 5, 4, 128
    Q, sa = tokens_of(T, K, 9, cuda_device)
    ids = torch.tensor([[2], [0], [2], [3], [0]], dtype=I32, device=cuda_device)
    base, scales = torch.zeros(E, 3, K, dtype=U8, device=cuda_device), torch.zeros(E, 2, 8, device=cuda_device)
    _, _, at = fg.moe_dispatch(Q, sa, ids, E, max_m=1, Qx=base[:, :1], sax=scales[:, :1])
    torch.cuda.synchronize()
    assert at.positions.flatten().tolist() == [2, 0, -1, 3, -1] and at.counts.tolist() == [1, 0, 1, 1]
    for e, t in ((2, 0), (0, 1), (3, 3)):
        assert torch.equal(base[e, 0], Q[t]) and float(scales[e, 0, 0]) == float(sa[0, t])
    assert int(base[:, 1:].max()) == 0 and int((scales != 0).sum()) == 3
    y = torch.randn(E, 3, 16, device=cuda_device)[:, 1:2]
    out = fg.moe_combine(y, at.positions)
    assert torch.equal(out, torch.where(at.positions >= 0, y[:, 0][at.positions[:, 0].clamp(min=0).long()], 0.0))
    with pytest.raises(ValueError):
        fg.moe_combine(torch.randn(E, 3, 16, device=cuda_device)[:, :2], at.positions)
