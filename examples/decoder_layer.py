"""One decoder layer, served and trained through, from the package's public calls.

    python examples/decoder_layer.py [--users 64] [--prompt 512] [--steps 32]

Serving: prompts of ragged lengths enter together, then one token a user and step, the step
captured into a graph. A layer is

    norm + quantise -> QKV product -> rotate, append to the paged cache -> attention
    -> quantise -> output product -> residual, norm + quantise -> gate and up product
    -> SwiGLU + quantise -> down product

Training: the gradient of the norm that feeds a product (norm_product_gradient).
Synthetic inputs, weights drawn at random.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_grouped_gemm_fp32_amd as fg  # noqa: E402
import synth  # noqa: E402

BF16 = torch.bfloat16


def rotation_table(positions, dim, device, base=10000.0):
    """Cosines, then sines, of dim / 2 angles at each position."""
    freq = base ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim)
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


class DecoderLayer:
    """Weights, cache and workspaces of a layer. Tokens: rows of a BF16 [T, hidden] tensor."""

    def __init__(self, hidden, heads, kv_heads, dim, ffn, pages, page_size=64, max_pos=4096, window=0, seed=0, device="cuda"):
        gen = synth.make_generator(seed, device)

        def weight(n, k):
            return synth.quantize_weight(torch.randn(n, k, generator=gen, device=device) * k ** -0.5)

        self.heads, self.kv_heads, self.dim, self.window = heads, kv_heads, dim, window
        self.qkv = weight((heads + 2 * kv_heads) * dim, hidden)
        self.out = weight(hidden, heads * dim)
        self.gate_up = weight(2 * ffn, hidden)
        self.down = weight(hidden, ffn)
        self.norm_in = (1 + 0.1 * torch.randn(hidden, generator=gen, device=device)).to(BF16)
        self.norm_ffn = (1 + 0.1 * torch.randn(hidden, generator=gen, device=device)).to(BF16)
        self.cos_sin = rotation_table(max_pos, dim, device)
        self.cache = fg.make_paged_kv_cache(pages, kv_heads, page_size, dim, device=device)
        self.workspace = fg.make_attention_workspace(device)

    @staticmethod
    def _product(q, sa, weight, rows):
        D = torch.empty(rows, weight[0].shape[0], dtype=BF16, device=q.device)
        return fg.fp8_gemm_nt(q, sa, weight[0], weight[1], D)

    def __call__(self, x, block_table, seq_lens, cu_q):
        """x [T, hidden]: the new tokens' residual stream -> the layer's. seq_lens [B] counts
        the new tokens; cu_q [B + 1] says which rows are whose."""
        T, H, Hkv, D = x.shape[0], self.heads, self.kv_heads, self.dim
        q8, sa, _, _ = fg.rmsnorm_quantize_1x128(x, self.norm_in)
        qkv = self._product(q8, sa, self.qkv, T).view(T, H + 2 * Hkv, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        fg.rope_append_paged_kv(q, k, v, self.cos_sin, self.cache, block_table, seq_lens, cu_q, q_out=q)
        o = fg.paged_attention(q, self.cache, block_table, seq_lens, cu_q, window=self.window, workspace=self.workspace)
        q8, sa = fg.quantize_1x128(o.view(T, H * D))
        o = self._product(q8, sa, self.out, T)
        q8, sa, h, _ = fg.rmsnorm_quantize_1x128(o, self.norm_ffn, residual=x, H=o)
        q8, sa = fg.swiglu_quantize_1x128(self._product(q8, sa, self.gate_up, T))
        return fg.fp8_gemm_nt(q8, sa, self.down[0], self.down[1], torch.empty_like(h), C=h)


def norm_product_gradient(x, residual, norm_weight, weight, dy, dh=None):
    """y = W norm(x + residual) with an 8-bit product, and from dy = dL/dy (and dh, what
    arrives at the sum over the residual stream) -> (y, h, dL/dx, dL/dnorm_weight). weight:
    synth.quantize_weight's codes and scales."""
    codes, scales = weight
    M, K = x.shape
    q8, sa, h, rstd = fg.rmsnorm_quantize_1x128(x, norm_weight, residual=residual)
    y = fg.fp8_gemm_nt(q8, sa, codes, scales, torch.empty(M, codes.shape[0], dtype=BF16, device=x.device))
    q8, sa = fg.quantize_1x128(dy)
    # the product's gradient is dy W: W's rows are the sum, as they lie
    dn = fg.fp8_gemm_nn(q8, sa, codes, scales.t().contiguous(), torch.empty(M, K, dtype=BF16, device=x.device))
    dx, dw = fg.rmsnorm_backward(dn, h, rstd, norm_weight, dH=dh)
    return y, h, dx, dw


def paged_batch(capacity, page_size, device):
    """Block table for sequences of at most capacity[b] tokens, pages in a scattered order ->
    (table, number of pages)."""
    counts = [-(-n // page_size) for n in capacity]
    order = torch.randperm(sum(counts), generator=torch.Generator().manual_seed(1)).tolist()
    table = torch.full((len(capacity), max(counts)), -1, dtype=torch.int32)
    for b, n in enumerate(counts):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    return table.to(device), sum(counts)


def serve(users, prompt, steps, hidden=4096, heads=32, kv_heads=8, dim=128, ffn=11008, page_size=64, device="cuda"):
    lens = [max(1, prompt - (37 * b) % prompt) for b in range(users)]
    table, pages = paged_batch([n + steps for n in lens], page_size, device)
    layer = DecoderLayer(hidden, heads, kv_heads, dim, ffn, pages, page_size, max_pos=prompt + steps, device=device)
    gen = synth.make_generator(7, device)
    cu = torch.tensor([0] + lens, device=device).cumsum(0).to(torch.int32)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=device)
    x = torch.randn(sum(lens), hidden, generator=gen, device=device).to(BF16)

    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    y = layer(x, table, seq_lens, cu)
    end.record()
    end.synchronize()
    print(f"prompts: {sum(lens)} tokens of {users} users, {start.elapsed_time(end):.2f} ms (first call)", flush=True)

    token = y[cu[1:].long() - 1].clone()  # the step's input: here the last token's output again
    one_each = torch.arange(users + 1, dtype=torch.int32, device=device)
    seq_lens += 1
    result = layer(token, table, seq_lens, one_each)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = layer(token, table, seq_lens, one_each)
    start.record()
    for _ in range(steps - 1):
        seq_lens += 1
        graph.replay()
        token.copy_(result)
    end.record()
    end.synchronize()
    print(f"decoding: {users} users, {start.elapsed_time(end) / max(1, steps - 1) * 1e3:.1f} us a step", flush=True)
    return result


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--users", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=512, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=32, help="tokens each user decodes")
    args = ap.parse_args()
    with torch.no_grad():
        serve(args.users, args.prompt, args.steps)
