"""The example's decoder layer: the operators and the GEMMs together, against a plain layer
in FP64 that rounds nothing.

Bound. Every tensor that enters a product or the cache is rounded to e4m3: at most 2^-4
relative, 2^-4 / sqrt(3) / sqrt(2) = 2.6% in the root mean square (the step is 2^-3 to 2^-4
of a value, uniformly). The layer's increment passes through nine such roundings (norm
output, keys, values, attention output, norm output, SwiGLU output, and three of BF16 that
are far smaller), most of them partly averaged out; as if independent and each at full size,
sqrt(6) 2.6% = 6.4%. 0.13 is twice that."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from examples import decoder_layer as ex

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = 1e-6


def dequantised(weight):
    codes, scales = weight
    n, k = codes.shape
    s = scales.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return codes.cpu().view(torch.float8_e4m3fn).double() * s.cpu()


def norm(x, w):
    return x / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS) * w.double().cpu()


def plain_layer(layer, x):
    """One sequence from its first token, [n, hidden] in FP64 on the CPU."""
    H, Hkv, D, n = layer.heads, layer.kv_heads, layer.dim, x.shape[0]
    qkv = (norm(x, layer.norm_in) @ dequantised(layer.qkv).T).view(n, H + 2 * Hkv, D)
    table = layer.cos_sin.double().cpu()[:n]
    cos, sin = table[:, None, : D // 2], table[:, None, D // 2:]
    a, b = qkv[:, : H + Hkv, : D // 2], qkv[:, : H + Hkv, D // 2:]
    turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2)
    q, k, v = turned[:, :H], turned[:, H:], qkv[:, H + Hkv:]
    i = torch.arange(n)
    seen = i[None, :] <= i[:, None]
    if layer.window:
        seen &= i[None, :] > i[:, None] - layer.window
    o = torch.empty(n, H, D, dtype=torch.float64)
    for h in range(H):
        s = q[:, h] @ k[:, h // (H // Hkv)].T * D ** -0.5
        o[:, h] = torch.softmax(s.masked_fill(~seen, -torch.inf), dim=1) @ v[:, h // (H // Hkv)]
    h1 = x + o.reshape(n, H * D) @ dequantised(layer.out).T
    gu = norm(h1, layer.norm_ffn) @ dequantised(layer.gate_up).T
    F = gu.shape[1] // 2
    return h1 + (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) @ dequantised(layer.down).T


def error(got, ref, x):
    """Of the layer's increment, in the root mean square."""
    d = got.double().cpu() - ref
    return float(d.norm() / (ref - x.double().cpu()).norm())


@pytest.mark.parametrize("heads,kv_heads,dim,page,window", [(4, 2, 128, 64, 0), (8, 8, 64, 16, 40), (4, 1, 256, 32, 0)])
def test_prompts_and_decoding_follow_the_plain_layer(cuda_device, heads, kv_heads, dim, page, window):
    hidden, ffn, lens, steps = 512, 384, [70, 1, 129], 3
    table, pages = ex.paged_batch([n + steps for n in lens], page, cuda_device)
    layer = ex.DecoderLayer(hidden, heads, kv_heads, dim, ffn, pages, page, max_pos=256, window=window, device=cuda_device)
    gen = synth.make_generator(3, cuda_device)
    xs = [torch.randn(n + steps, hidden, generator=gen, device=cuda_device).to(BF16) for n in lens]
    refs = [plain_layer(layer, x.double().cpu()) for x in xs]
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    cu = torch.tensor([0] + lens, device=cuda_device).cumsum(0).to(torch.int32)
    y = layer(torch.cat([x[:n] for x, n in zip(xs, lens)]), table, seq_lens, cu)
    at = 0
    for x, ref, n in zip(xs, refs, lens):
        assert error(y[at:at + n], ref[:n], x[:n]) < 0.13
        at += n
    one_each = torch.arange(len(lens) + 1, dtype=torch.int32, device=cuda_device)
    for s in range(steps):
        seq_lens += 1
        new = torch.stack([x[n + s] for x, n in zip(xs, lens)])
        y = layer(new, table, seq_lens, one_each)
        ref = torch.stack([r[n + s] for r, n in zip(refs, lens)])
        assert error(y, ref, new) < 0.13


def test_a_captured_step_repeats_the_eager_one(cuda_device):
    hidden, users = 256, 5
    table, pages = ex.paged_batch([300] * users, 64, cuda_device)
    layer = ex.DecoderLayer(hidden, 4, 2, 64, 256, pages, 64, max_pos=300, device=cuda_device)
    gen = synth.make_generator(4, cuda_device)
    lens = [130, 7, 64, 255, 1]
    cu = torch.tensor([0] + lens, device=cuda_device).cumsum(0).to(torch.int32)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    layer(torch.randn(sum(lens), hidden, generator=gen, device=cuda_device).to(BF16), table, seq_lens, cu)
    one_each = torch.arange(users + 1, dtype=torch.int32, device=cuda_device)
    seq_lens += 1
    token = torch.randn(users, hidden, generator=gen, device=cuda_device).to(BF16)
    layer(token, table, seq_lens, one_each)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(token, table, seq_lens, one_each)
    for _ in range(4):
        seq_lens += 1
        token.copy_(torch.randn(users, hidden, generator=gen, device=cuda_device))
        before = [t.clone() for t in layer.cache]
        graph.replay()
        torch.cuda.synchronize()
        after = [t.clone() for t in layer.cache]
        for t, b in zip(layer.cache, before):
            t.copy_(b)
        eager = layer(token, table, seq_lens, one_each)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
        for t, a in zip(layer.cache, after):
            assert torch.equal(t, a)


def test_norm_product_gradient_follows_the_formula(cuda_device):
    """Against autograd of the unrounded product in FP64; two roundings to e4m3 on dx's way
    (dy, and h in BF16, far smaller): 2.6% each as above, twice that allowed."""
    M, K, N = 200, 512, 640
    gen = synth.make_generator(5, cuda_device)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=cuda_device)

    weight = synth.quantize_weight(randn(N, K) * K ** -0.5)
    x, r, dy, dh = randn(M, K).to(BF16), randn(M, K).to(BF16), randn(M, N).to(BF16), randn(M, K).to(BF16)
    w = (1 + 0.1 * randn(K)).to(BF16)
    y, h, dx, dw = ex.norm_product_gradient(x, r, w, weight, dy, dh)
    hd = (x.float() + r.float()).to(BF16).double().cpu().requires_grad_()
    wd = w.double().cpu().requires_grad_()
    yd = (hd / torch.sqrt((hd * hd).mean(dim=1, keepdim=True) + EPS) * wd) @ dequantised(weight).T
    (yd * dy.double().cpu()).sum().add((hd * dh.double().cpu()).sum()).backward()
    assert torch.equal(h.double().cpu(), hd.detach())
    for got, ref in ((y, yd.detach()), (dx, hd.grad), (dw, wd.grad)):
        d = got.double().cpu() - ref
        assert float(d.norm() / ref.norm()) < 2 * np.hypot(0.026, 0.026)
