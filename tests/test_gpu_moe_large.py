"""The expert and head operators where offsets pass 32 bits, and where tokens are very many."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg

pytestmark = pytest.mark.gpu
BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def test_rows_past_2_to_the_32_bytes(cuda_device):
    """Expanded rows of 8192 columns on both sides of 2^32 bytes and elements: dispatched, gathered, summed
    and differentiated."""
    K, rows = 8192, 640 * 1024
    Qx = torch.zeros(rows, K, dtype=U8, device=cuda_device)
    sax = torch.zeros(K // 128, rows, device=cuda_device)
    T, E = 64, 1000
    Q = torch.randint(1, 100, (T, K), device=cuda_device, dtype=U8)
    sa = torch.rand(K // 128, T, device=cuda_device)
    per = rows // E // 128 * 128  # rows of an expert in the masked layout
    ids = torch.tensor([0, 1, 500, 999, 998, 820], dtype=I32, device=cuda_device).repeat(T, 1)
    Qm, sm = Qx[:E * per].view(E, per, K), torch.zeros(E, K // 128, per, device=cuda_device)
    _, _, at = fg.moe_dispatch(Q, sa, ids, E, max_m=per, Qx=Qm, sax=sm)
    torch.cuda.synchronize()
    assert int(at.positions.max()) * K > 1 << 32
    for e in (0, 1, 500, 820, 998, 999):
        assert torch.equal(Qm[e, :T], Q) and torch.equal(sm[e, :, :T], sa) and int(Qm[e, T:].max()) == 0
    # the contiguous layout with most rows in one expert
    many = 600 * 1024
    ids = torch.zeros(many, 1, dtype=I32, device=cuda_device)
    ids[-3:] = torch.tensor([[1], [2], [1]], dtype=I32, device=cuda_device)
    Q = torch.randint(1, 100, (1, K), device=cuda_device, dtype=U8)
    big = torch.zeros(many, 128, dtype=U8, device=cuda_device)
    at = fg.moe_dispatch(big, torch.ones(1, many, device=cuda_device), ids, 3, layout=fg.make_moe_layout(many, 1, 3, rows=rows))[2]
    assert at.counts.tolist() == [many - 3, 2, 1] and at.positions[-3:, 0].tolist() == [many, many + 128, many + 1]
    tail = fg.MoeLayout(at.positions[-64:].contiguous(), torch.where(at.sources >= 0, at.sources - (many - 64), -1), at.m_indices, at.counts)
    Q = Q.repeat(64, 1)
    Qx.zero_()
    fg.moe_gather(Q, torch.ones(K // 128, 64, device=cuda_device), tail, Qx=Qx, sax=sax)
    torch.cuda.synchronize()
    live = tail.positions[:, 0].long()
    assert torch.equal(Qx[live], Q) and int(Qx[:many - 64].max()) == 0 and bool((sax[:, live] == 1).all())
    del Qx, sax, Qm
    Y = torch.zeros(rows, K, dtype=BF16, device=cuda_device)
    Y[live] = torch.randn(64, K, device=cuda_device).to(BF16)
    w = torch.rand(64, 1, device=cuda_device)
    out = fg.moe_combine(Y, tail.positions, w)
    assert torch.equal(out, (Y[live].float() * w).to(BF16))
    dO = torch.randn(64, K, device=cuda_device).to(BF16)
    want = (dO.double() * Y[live].double()).sum(1)
    mag = (dO.double() * Y[live].double()).abs().sum(1)
    dY, dw = fg.moe_combine_backward(dO, Y, tail.positions, w, dY=Y)
    assert torch.equal(dY[live], (dO.float() * w).to(BF16))
    assert bool(((dw[:, 0].double() - want).abs() <= (K / 64 + 16) * 2.0 ** -24 * mag).all())


def test_heads_past_2_to_the_32_elements(cuda_device):
    T, H, D = 9000, 4, 128
    ld = 1 << 19  # rows far apart: 4.7 G elements from the first to the last
    x = torch.empty((T - 1) * ld + H * D, dtype=BF16, device=cuda_device)
    q = x.as_strided((T, H, D), (ld, D, 1))
    assert (T - 1) * ld > 1 << 32
    q.copy_(torch.randn(T, H, D, device=cuda_device))
    dense = q.contiguous()
    w, table = torch.rand(D, device=cuda_device) + 0.5, torch.rand(T, 64, device=cuda_device)
    want = fg.qk_norm_rope(dense, dense[:, :1], w, w, table)
    got = fg.qk_norm_rope(q, q[:, :1], w, w, table, q_out=q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q.copy_(dense)
    dy = torch.randn(T, H, D, device=cuda_device).to(BF16)
    a = fg.qk_norm_rope_backward(dy, None, dense, None, w, None, table)
    b = fg.qk_norm_rope_backward(dy, None, q, None, w, None, table, dq_out=q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_routing_of_very_many_tokens(cuda_device):
    """More rows than 2^32 bytes of logits hold; the ends against the same rows alone."""
    T, E, k = 5_000_000, 256, 4
    x = torch.empty(T, E, device=cuda_device)
    x.normal_(generator=torch.Generator(cuda_device).manual_seed(1))
    bias = torch.rand(E, device=cuda_device) * 0.1
    ids, w = fg.moe_route(x, k, bias=bias, scoring="sigmoid", groups=4, top_groups=2, group_best=2)
    for part in (slice(0, 1000), slice(T - 1000, T)):
        i2, w2 = fg.moe_route(x[part], k, bias=bias, scoring="sigmoid", groups=4, top_groups=2, group_best=2)
        assert torch.equal(ids[part], i2) and torch.equal(w[part], w2)
    dx = fg.moe_route_backward(w, x, ids)
    assert torch.equal(dx[-1000:], fg.moe_route_backward(w[-1000:], x[-1000:], ids[-1000:]))
    # and the layout of their choices: 20 million, in expert order
    at = fg.moe_dispatch(torch.zeros(T, 128, dtype=U8, device=cuda_device), torch.ones(1, T, device=cuda_device), ids, E)[2]
    counts = torch.bincount(ids.flatten().long(), minlength=E)
    assert torch.equal(at.counts.long(), counts)
    start = ((counts + 127) // 128 * 128).cumsum(0) - (counts + 127) // 128 * 128
    order = torch.sort(ids.flatten(), stable=True).indices
    rank = torch.arange(T * k, device=cuda_device) - (counts.cumsum(0) - counts).repeat_interleave(counts)
    rows = start.repeat_interleave(counts) + rank
    assert torch.equal(at.positions.flatten()[order].long(), rows) and torch.equal(at.sources[rows].long(), order)
