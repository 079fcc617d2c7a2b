"""A decoder layer whose feed-forward part is a mixture of experts, served, and a routed product
trained through, from the package's public calls.

    python examples/expert_layer.py [--users 64] [--prompt 256] [--steps 16] [--experts 64]

Serving: prompts, then one token a user and step, the step captured into a graph. A layer is

    norm + quantise -> QKV product -> norm and rotation of heads -> append to the paged cache
    -> attention -> quantise -> output product -> residual, norm + quantise -> router product
    -> routing -> dispatch -> experts' gate and up product -> SwiGLU + quantise -> experts' down
    product -> weighted return to the residual stream

Training: a routed linear layer, its gradients of the logits and of the input by way of the experts
(RoutedLinear). The router's part of the input's gradient is a plain product of the logits'; the experts'
weight gradients need rows scaled by columns, which the package's calls do not lay out.
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
from examples.decoder_layer import DecoderLayer, paged_batch  # noqa: E402

BF16 = torch.bfloat16


def expert_weights(experts, n, k, gen, device):
    """[experts, n, k] codes and their scales."""
    parts = [synth.quantize_weight(torch.randn(n, k, generator=gen, device=device) * k ** -0.5) for _ in range(experts)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def experts_product(q8, sa, weight, layout):
    """Each row times its expert's weight, [rows, N]; rows without a choice are not written."""
    codes, scales = weight
    D = torch.empty(q8.shape[0], codes.shape[1], dtype=BF16, device=q8.device)
    return fg.fp8_grouped_gemm_nt_contiguous(q8, sa, codes, scales, D, layout.m_indices)


class ExpertLayer(DecoderLayer):
    """A decoder layer with norms of heads and `experts` experts, of which `top_k` take a token,
    from `top_groups` of `groups`."""

    def __init__(self, hidden, heads, kv_heads, dim, ffn, pages, experts, top_k, groups=1, top_groups=1, page_size=64, max_pos=4096,
                 seed=0, device="cuda"):
        super().__init__(hidden, heads, kv_heads, dim, 128, pages, page_size, max_pos=max_pos, seed=seed, device=device)
        gen = synth.make_generator(seed + 1, device)
        self.top_k, self.groups, self.top_groups = top_k, groups, top_groups
        self.norm_q, self.norm_k = ((1 + 0.1 * torch.randn(dim, generator=gen, device=device)).to(BF16) for _ in range(2))
        self.router = torch.randn(experts, hidden, generator=gen, device=device) * hidden ** -0.5
        self.bias = torch.randn(experts, generator=gen, device=device) * 0.05
        self.gate_up = expert_weights(experts, 2 * ffn, hidden, gen, device)
        self.down = expert_weights(experts, hidden, ffn, gen, device)

    def route(self, n):
        """Experts and weights of rows n [T, hidden], the norm's output."""
        logits = n.float() @ self.router.t()
        return fg.moe_route(logits, self.top_k, bias=self.bias, scoring="sigmoid", groups=self.groups, top_groups=self.top_groups,
                            group_best=2, scale=2.5)

    def __call__(self, x, block_table, seq_lens, cu_q, positions):
        """x [T, hidden]: the new tokens' residual stream -> the layer's; positions int32 [T]."""
        T, H, Hkv, D = x.shape[0], self.heads, self.kv_heads, self.dim
        q8, sa, _, _ = fg.rmsnorm_quantize_1x128(x, self.norm_in)
        qkv = self._product(q8, sa, self.qkv, T).view(T, H + 2 * Hkv, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        fg.qk_norm_rope(q, k, self.norm_q, self.norm_k, self.cos_sin, positions, q_out=q, k_out=k)
        fg.rope_append_paged_kv(None, k, v, None, self.cache, block_table, seq_lens, cu_q)
        o = fg.paged_attention(q, self.cache, block_table, seq_lens, cu_q, workspace=self.workspace)
        q8, sa = fg.quantize_1x128(o.view(T, H * D))
        o = self._product(q8, sa, self.out, T)
        n = torch.empty_like(o)
        q8, sa, h, _ = fg.rmsnorm_quantize_1x128(o, self.norm_ffn, residual=x, H=o, Y=n)
        ids, weights = self.route(n)
        q8, sa, layout = fg.moe_dispatch(q8, sa, ids, self.router.shape[0])
        q8, sa = fg.swiglu_quantize_1x128(experts_product(q8, sa, self.gate_up, layout), m_indices=layout.m_indices)
        y = experts_product(q8, sa, self.down, layout)
        return fg.moe_combine(y, layout.positions, weights, C=h, out=h)


class RoutedLinear:
    """y[t] = sum_j w[t, j] W[e(t, j)] x[t], with 8-bit products, and gradients of x and of the logits."""

    def __init__(self, experts, n, k, top_k, seed=0, device="cuda"):
        gen = synth.make_generator(seed, device)
        self.top_k = top_k
        self.router = torch.randn(experts, k, generator=gen, device=device) * k ** -0.5
        self.weight = expert_weights(experts, n, k, gen, device)
        # the gradient's products read the weights transposed: laid out once
        self.transposed = tuple(t.transpose(1, 2).contiguous() for t in self.weight)

    def forward(self, x):
        q8, sa = fg.quantize_1x128(x)
        self.logits = x.float() @ self.router.t()
        self.ids, self.w = fg.moe_route(self.logits, self.top_k)
        q8, sa, self.layout = fg.moe_dispatch(q8, sa, self.ids, self.router.shape[0])
        self.y = experts_product(q8, sa, self.weight, self.layout)
        return fg.moe_combine(self.y, self.layout.positions, self.w)

    def backward(self, dy):
        """dL/dy -> (dL/dx by way of the experts, dL/dlogits)."""
        _, dw = fg.moe_combine_backward(dy, self.y, self.layout.positions, self.w, rows=False)
        dlogits = fg.moe_route_backward(dw, self.logits, self.ids)
        q8, sa = fg.moe_gather(*fg.quantize_1x128(dy), self.layout, weights=self.w)
        return fg.moe_combine(experts_product(q8, sa, self.transposed, self.layout), self.layout.positions), dlogits


def new_positions(seq_lens, cu_q):
    """Each row's position in its sequence."""
    T, B = int(cu_q[-1]), len(seq_lens)
    of = torch.repeat_interleave(torch.arange(B, device=cu_q.device), cu_q.diff().long(), output_size=T)
    return (seq_lens[of] - cu_q[of + 1] + torch.arange(T, device=cu_q.device)).to(torch.int32)


def serve(users, prompt, steps, hidden=2048, heads=16, kv_heads=4, dim=128, ffn=1024, experts=64, top_k=8, page_size=64, device="cuda"):
    lens = [max(1, prompt - (37 * b) % prompt) for b in range(users)]
    table, pages = paged_batch([n + steps for n in lens], page_size, device)
    groups = next(g for g in (8, 4, 2, 1) if experts % g == 0)
    layer = ExpertLayer(hidden, heads, kv_heads, dim, ffn, pages, experts, min(top_k, experts), groups, max(1, groups // 2), page_size,
                        max_pos=prompt + steps, device=device)
    gen = synth.make_generator(7, device)
    cu = torch.tensor([0] + lens, device=device).cumsum(0).to(torch.int32)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=device)
    x = torch.randn(sum(lens), hidden, generator=gen, device=device).to(BF16)

    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    y = layer(x, table, seq_lens, cu, new_positions(seq_lens, cu))
    end.record()
    end.synchronize()
    print(f"prompts: {sum(lens)} tokens of {users} users, {start.elapsed_time(end):.2f} ms (first call)", flush=True)

    token = y[cu[1:].long() - 1].clone()  # the step's input: here the last token's output again
    one_each = torch.arange(users + 1, dtype=torch.int32, device=device)
    positions = seq_lens.clone()
    seq_lens += 1
    result = layer(token, table, seq_lens, one_each, positions)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = layer(token, table, seq_lens, one_each, positions)
    start.record()
    for _ in range(steps - 1):
        seq_lens += 1
        positions += 1
        graph.replay()
        token.copy_(result)
    end.record()
    end.synchronize()
    print(f"decoding: {users} users, {start.elapsed_time(end) / max(1, steps - 1) * 1e3:.1f} us a step", flush=True)
    return result


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--users", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=256, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=16, help="tokens each user decodes")
    ap.add_argument("--experts", type=int, default=64)
    args = ap.parse_args()
    with torch.no_grad():
        serve(args.users, args.prompt, args.steps, experts=args.experts)
