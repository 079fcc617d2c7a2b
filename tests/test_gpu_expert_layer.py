"""The example's expert layer: routing, dispatch, the grouped products, the return, and the heads'
norm and rotation together with the GEMMs, the cache and attention, against plain layers in FP64.

Bounds. Every tensor that enters a product or the cache is rounded to e4m3: 2.6% in the root mean
square (test_gpu_decoder_layer.py). The layer's increment passes through nine such roundings; as if
independent and each at full size, sqrt(6) 2.6% = 6.4%, and 0.13 is twice that. The routing is
taken from the layer itself, since a choice may turn on a rounding of its input; that it is the
right one for its logits is tested by itself. The routed product has two (weights count as
given): twice sqrt(2) 2.6%."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from examples import decoder_layer as dec
from examples import expert_layer as ex
from oracle import moe_oracle as mo
from test_gpu_decoder_layer import dequantised, error, norm

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def head_norm(x, w):
    return x / torch.sqrt((x * x).mean(dim=2, keepdim=True) + 1e-6) * w.double().cpu()


def experts_of(weight):
    return [dequantised((weight[0][e], weight[1][e])) for e in range(weight[0].shape[0])]


def plain_layer(layer, x, routing):
    """One sequence from its first token, [n, hidden] in FP64 on the CPU; routing: ids and weights."""
    H, Hkv, D, n = layer.heads, layer.kv_heads, layer.dim, x.shape[0]
    qkv = (norm(x, layer.norm_in) @ dequantised(layer.qkv).T).view(n, H + 2 * Hkv, D)
    table = layer.cos_sin.double().cpu()[:n]
    cos, sin = table[:, None, : D // 2], table[:, None, D // 2:]
    turned = []
    for part, w in ((qkv[:, :H], layer.norm_q), (qkv[:, H:H + Hkv], layer.norm_k)):
        part = head_norm(part, w)
        a, b = part[..., : D // 2], part[..., D // 2:]
        turned.append(torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2))
    q, k, v = *turned, qkv[:, H + Hkv:]
    i = torch.arange(n)
    o = torch.empty(n, H, D, dtype=torch.float64)
    for h in range(H):
        s = (q[:, h] @ k[:, h // (H // Hkv)].T * D ** -0.5).masked_fill(i[None, :] > i[:, None], -torch.inf)
        o[:, h] = torch.softmax(s, dim=1) @ v[:, h // (H // Hkv)]
    h1 = x + o.reshape(n, H * D) @ dequantised(layer.out).T
    y, m = h1.clone(), norm(h1, layer.norm_ffn)
    up, down = experts_of(layer.gate_up), experts_of(layer.down)
    F = down[0].shape[1]
    for t in range(n):
        for e, w in zip(*(r[t].tolist() for r in routing)):
            gu = up[e] @ m[t]
            y[t] += w * (down[e] @ (torch.nn.functional.silu(gu[:F]) * gu[F:]))
    return y


class Recorded(ex.ExpertLayer):
    """Keeps what it routed."""
    def route(self, n):
        logits = n.float() @ self.router.t()
        ids, w = super().route(n)
        self.routed.append((logits, ids, w))
        return ids, w


@pytest.mark.parametrize("heads,kv_heads,dim,page,experts,top_k,groups", [(4, 2, 128, 64, 16, 4, 4), (8, 8, 64, 16, 6, 2, 1), (4, 1, 256, 32, 40, 8, 8)])
def test_prompts_and_decoding_follow_the_plain_layer(cuda_device, heads, kv_heads, dim, page, experts, top_k, groups):
    hidden, ffn, lens, steps = 512, 256, [40, 1, 70], 2
    table, pages = dec.paged_batch([n + steps for n in lens], page, cuda_device)
    layer = Recorded(hidden, heads, kv_heads, dim, ffn, pages, experts, top_k, groups, max(1, groups // 2), page, max_pos=128, device=cuda_device)
    gen = synth.make_generator(3, cuda_device)
    xs = [torch.randn(n + steps, hidden, generator=gen, device=cuda_device).to(BF16) for n in lens]
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    cu = torch.tensor([0] + lens, device=cuda_device).cumsum(0).to(torch.int32)
    layer.routed = []
    ys = [layer(torch.cat([x[:n] for x, n in zip(xs, lens)]), table, seq_lens, cu, ex.new_positions(seq_lens, cu))]
    one_each = torch.arange(len(lens) + 1, dtype=torch.int32, device=cuda_device)
    for s in range(steps):
        seq_lens += 1
        ys.append(layer(torch.stack([x[n + s] for x, n in zip(xs, lens)]), table, seq_lens, one_each, (seq_lens - 1).contiguous()))
    torch.cuda.synchronize()
    for logits, ids, w in layer.routed:  # what was chosen is what the logits say
        ri, rw, _ = mo.route(logits.double().cpu().numpy(), top_k, layer.bias.double().cpu().numpy(), "sigmoid", groups, max(1, groups // 2), 2, True, 2.5)
        assert np.array_equal(ids.cpu().numpy(), ri) and np.allclose(w.double().cpu().numpy(), rw, rtol=2.0 ** -16)
    at = 0
    for b, (x, n) in enumerate(zip(xs, lens)):
        rows = lambda part: torch.cat([part(0)[at:at + n]] + [part(1 + s)[b:b + 1] for s in range(steps)]).cpu()  # noqa: E731
        routing = rows(lambda i: layer.routed[i][1]), rows(lambda i: layer.routed[i][2]).double()
        ref = plain_layer(layer, x.double().cpu(), routing)
        assert error(rows(lambda i: ys[i]), ref, x) < 0.13
        at += n


def test_a_captured_step_repeats_the_eager_one(cuda_device):
    hidden, users = 256, 5
    table, pages = dec.paged_batch([100] * users, 64, cuda_device)
    layer = ex.ExpertLayer(hidden, 4, 2, 64, 128, pages, 12, 3, max_pos=100, device=cuda_device)
    gen = synth.make_generator(4, cuda_device)
    lens = [60, 7, 64, 33, 1]
    cu = torch.tensor([0] + lens, device=cuda_device).cumsum(0).to(torch.int32)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    layer(torch.randn(sum(lens), hidden, generator=gen, device=cuda_device).to(BF16), table, seq_lens, cu, ex.new_positions(seq_lens, cu))
    one_each = torch.arange(users + 1, dtype=torch.int32, device=cuda_device)
    positions = seq_lens.clone()
    seq_lens += 1
    token = torch.randn(users, hidden, generator=gen, device=cuda_device).to(BF16)
    layer(token, table, seq_lens, one_each, positions)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(token, table, seq_lens, one_each, positions)
    for _ in range(4):
        seq_lens += 1
        positions += 1
        token.copy_(torch.randn(users, hidden, generator=gen, device=cuda_device))
        before = [t.clone() for t in layer.cache]
        graph.replay()
        torch.cuda.synchronize()
        after = [t.clone() for t in layer.cache]
        for t, b in zip(layer.cache, before):
            t.copy_(b)
        eager = layer(token, table, seq_lens, one_each, positions)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
        for t, a in zip(layer.cache, after):
            assert torch.equal(t, a)


def test_routed_product_and_its_gradients_follow_the_formula(cuda_device):
    """Against autograd of the unrounded layer in FP64 with the same choice."""
    T, E, N, K, k = 150, 10, 384, 512, 3
    layer = ex.RoutedLinear(E, N, K, k, device=cuda_device)
    gen = synth.make_generator(5, cuda_device)
    x, dy = (torch.randn(T, n, generator=gen, device=cuda_device).to(BF16) for n in (K, N))
    y = layer.forward(x)
    dx, dlogits = layer.backward(dy)
    torch.cuda.synchronize()
    W = torch.stack(experts_of(layer.weight))
    ids = layer.ids.long().cpu()
    xd = x.double().cpu().requires_grad_()
    logits = layer.logits.double().cpu().requires_grad_()
    s = torch.softmax(logits, 1).gather(1, ids)
    w = s / s.sum(1, keepdim=True)
    yd = (w[:, :, None] * torch.stack([torch.stack([W[e] @ xd[t] for e in ids[t].tolist()]) for t in range(T)])).sum(1)
    (yd * dy.double().cpu()).sum().backward()
    for got, ref in ((y, yd.detach()), (dx, xd.grad), (dlogits, logits.grad)):
        d = got.double().cpu() - ref
        assert float(d.norm() / ref.norm()) < 2 * np.hypot(0.026, 0.026)
