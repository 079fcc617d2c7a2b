"""GPU parity of attention over the paged 8-bit cache against the FP64 oracle.

Bounds, u = 2^-24. A logit is a sum of D exact products in FP32 (off by at most D u times
the sum of their magnitudes), times a rounded scale, and the exponent's argument is rounded
once more: delta = (D + 8) u * depth with depth the largest sum of magnitudes of a row,
natural units. A probability is then off by 2 delta relative (numerator and sum), rounded
to 11 bits (2^-11) for the second product, summed in FP32 over n keys (n u at most, in
practice far less: 2^-14 is allowed). Over |v| that makes
    |out - ref| <= 2^-8 |ref| + (2^-11 + 2^-14 + 2 delta) sum_j p_j |v_j|
and |lse - ref| <= 2 delta + 2^-20 + 2^-22 |ref|."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.fixture(scope="module")
def workspace():
    return fg.make_attention_workspace()


class Setup:
    def __init__(self, dev, new, lens, Hq, Hkv, D, P, seed=0, q_std=1.0, spread=2, poison=True):
        g = synth.make_generator(seed, dev)
        self.new, self.lens = new, lens
        npages = [-(-m // P) for m in lens]
        N = sum(npages) + 2
        order = torch.randperm(N, generator=synth.make_generator(seed + 1)).tolist()
        width, at, self.pages = max(npages + [1]) + 1, 0, []
        for n in npages:
            self.pages.append(order[at:at + n] + [N + 5, -1][: width - n] + [-7] * max(0, width - n - 2))
            at += n
        self.cache = fg.make_paged_kv_cache(N, Hkv, P, D, device=dev)
        for codes, scale in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            x = torch.randn(codes.shape, generator=g, device=dev) * 60
            codes.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
            scale.copy_(2.0 ** (torch.randint(0, spread + 1, scale.shape, generator=g, device=dev).float() - 6 - spread))
        if poison:  # what no sequence holds is NaN: whole pages, the ends of last pages, their scales
            held = torch.zeros(N, P, dtype=torch.bool)
            for row, m in zip(self.pages, lens):
                for j in range(-(-m // P)):
                    held[row[j], : min(P, m - j * P)] = True
            held = held.to(dev)
            for codes, scale in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
                codes.masked_fill_(~held[:, None, :, None], 0x7F)
                scale.masked_fill_(~held.any(dim=1)[:, None], float("nan"))
        self.table = torch.tensor(self.pages, dtype=torch.int32, device=dev).reshape(len(lens), width)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.cu_q = torch.tensor(self.cu, dtype=torch.int32, device=dev)
        self.T, self.Hq, self.Hkv, self.D = self.cu[-1], Hq, Hkv, D
        self.q = (torch.randn(self.T, Hq, D, generator=g, device=dev) * q_std).to(BF16)
        self.scale = D ** -0.5

    def run(self, **kw):
        lse = torch.full((self.T, self.Hq), float("nan"), device=self.q.device)
        kw = {"softmax_scale": self.scale, "lse": lse, **kw}
        out = fg.paged_attention(kw.pop("q", self.q), self.cache, self.table, self.seq_lens, self.cu_q, **kw)
        torch.cuda.synchronize()
        return out, lse

    def reference(self, window=0):
        c = [t.cpu().numpy() for t in self.cache]
        return lo.attention(f64(self.q), *c, self.pages, self.lens, self.cu, self.scale, window)

    def check(self, out, lse, window=0, ref=None):
        o, s, spread, depth = ref or self.reference(window)
        delta = (self.D + 8) * U * depth
        bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -14 + 2 * delta)[..., None] * spread
        got = f64(out)
        bad = np.argwhere(~(np.abs(got - o) <= bound))
        assert not len(bad), (len(bad), tuple(bad[0]), got[tuple(bad[0])], o[tuple(bad[0])], bound[tuple(bad[0])])
        g = f64(lse)
        none = np.isneginf(s)
        assert np.array_equal(np.isneginf(g), none) and np.all(got[none] == 0)
        assert np.all(np.abs(g[~none] - s[~none]) <= (2 * delta + 2.0 ** -20)[~none] + 2.0 ** -22 * np.abs(s[~none]))


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 300]
CASES = [
    # new tokens, lengths, Hq, Hkv, D, P
    ([1] * len(LENS), LENS, 8, 2, 128, 64),
    ([1] * len(LENS), LENS, 3, 3, 64, 16),
    ([1] * 5, [700, 0, 1, 513, 90], 16, 1, 256, 32),
    ([1, 0, 1, 2], [9, 40, 0, 1], 4, 4, 128, 128),           # none new; no keys at all; more new than keys
    ([3, 1, 8, 0, 2], [70, 1, 8, 5, 260], 20, 4, 128, 16),    # drafts; 15, 5, 40, 10 rows a key head
    ([40, 7, 129], [40, 300, 200], 6, 2, 64, 256),
    ([65], [65], 32, 1, 128, 16),                             # 32 rows a token
    ([200, 1], [333, 1500], 4, 1, 128, 64),
    ([17, 33], [17, 100], 48, 2, 64, 32),                     # 24 heads a key head
    ([300], [900], 2, 2, 256, 64),
    ([1] * 67, [13 * i % 97 for i in range(67)], 2, 1, 64, 16),  # over a wave of sequences
]


@pytest.mark.parametrize("window", [0, 1, 37, 256])
@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,P", CASES)
def test_attention(cuda_device, workspace, new, lens, Hq, Hkv, D, P, split, window):
    s = Setup(cuda_device, new, lens, Hq, Hkv, D, P)
    s.check(*s.run(window=window, workspace=workspace if split else None), window)


@pytest.mark.parametrize("new,lens,Hkv,P,window", [([1], [9000], 1, 64, 0), ([4, 1], [5000, 77], 2, 16, 0), ([1, 1], [7000, 6999], 1, 128, 4000),
                                                  ([150], [3500], 1, 64, 0)])
def test_long_sequences_are_split_and_joined_alike(cuda_device, workspace, new, lens, Hkv, P, window):
    s = Setup(cuda_device, new, lens, 4 * Hkv, Hkv, 128, P, seed=5, q_std=2.0)
    ref = s.reference(window)
    out, lse = s.run(window=window, workspace=workspace)
    s.check(out, lse, window, ref)
    for _ in range(3):  # the parts are joined in their order, whoever comes last
        again, l2 = s.run(window=window, workspace=workspace)
        assert torch.equal(again, out) and torch.equal(l2, lse)
    whole = s.run(window=window)
    s.check(*whole, window, ref)
    assert int(workspace[: 64 << 10].count_nonzero()) == 0  # the counters are zero again
    small = torch.zeros((64 << 10) + 9 * 16 * 129 * 4 + 4, dtype=torch.uint8, device=cuda_device)  # few parts
    guard = torch.full((small.numel() + 4096,), 0x5A, dtype=torch.uint8, device=cuda_device)
    guard[: small.numel()] = 0
    s.check(*s.run(window=window, workspace=guard[: small.numel()]), window, ref)
    assert bool((guard[small.numel():] == 0x5A).all())


@pytest.mark.parametrize("new", [1, 5, 90])
def test_strides_of_queries_and_output(cuda_device, workspace, new):
    s = Setup(cuda_device, [new, new], [100, 260], 4, 2, 128, 32, seed=6)
    qkv = torch.full((s.T, 8 * 128 + 8), float("nan"), dtype=BF16, device=cuda_device)
    q = qkv[:, : 4 * 128].view(s.T, 4, 128)
    q.copy_(s.q)
    o = torch.full((s.T, 6 * 128), 7.0, dtype=BF16, device=cuda_device)
    out, lse = s.run(q=q, out=o[:, 128: 5 * 128].view(s.T, 4, 128), workspace=workspace)
    s.check(out, lse)
    assert bool((o[:, :128] == 7).all()) and bool((o[:, 5 * 128:] == 7).all())


def test_peaked_and_flat_rows(cuda_device, workspace):
    """Logits from nearly equal to hundreds apart, growing along the keys (the running
    maximum moves at every step) and falling."""
    for sign in (1.0, -1.0):
        s = Setup(cuda_device, [1, 3], [600, 500], 4, 1, 64, 16, seed=7)
        ramp = torch.linspace(0.02, 1.0, 38, device=cuda_device)
        for row in range(2):
            for j, page in enumerate(s.pages[row][: -(-s.lens[row] // 16)]):
                s.cache.k[page].copy_((torch.ones(16, 64, device=cuda_device) * sign * ramp[j] * 16).to(torch.float8_e4m3fn).view(torch.uint8)[None])
                s.cache.k_scale[page] = 1.0
        s.q.copy_(torch.tensor([0.0, 0.01, 1.0, 4.0], device=cuda_device)[None, :, None].expand(s.T, 4, 64).to(BF16))
        s.scale = 1.0
        s.check(*s.run(workspace=workspace))


@pytest.mark.parametrize("new,P", [([1], 16), ([2, 33], 64)])
def test_value_scales_far_apart(cuda_device, workspace, new, P):
    """Pages whose value scales differ by up to 2^200, in any order; keys' scales as well."""
    s = Setup(cuda_device, new, [400] * len(new), 4, 1, 128, P, seed=8)
    g = synth.make_generator(1, cuda_device)
    s.cache.v_scale.copy_(2.0 ** torch.randint(-100, 101, s.cache.v_scale.shape, generator=g, device=cuda_device).float())
    s.check(*s.run(workspace=workspace))
    s.cache.v_scale.fill_(2.0 ** -126)
    s.cache.k_scale.copy_(2.0 ** torch.randint(-126, -6, s.cache.k_scale.shape, generator=g, device=cuda_device).float())
    out, lse = s.run(workspace=workspace)
    assert bool(torch.isfinite(out).all())
    s.check(out, lse)


def test_pages_of_no_number_are_left_out(cuda_device, workspace):
    s = Setup(cuda_device, [1, 40, 1], [100, 100, 50], 4, 2, 128, 16, seed=9)
    s.pages[0][2], s.pages[0][3], s.pages[1][5] = -1, s.cache.k.shape[0], 1 << 30
    s.pages[2][:4] = [-1] * 4
    s.table = torch.tensor(s.pages, dtype=torch.int32, device=cuda_device)
    s.check(*s.run(workspace=workspace))


@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("new", [6, 200])
def test_a_bad_key_or_value_spoils_only_the_rows_that_see_it(cuda_device, workspace, new, group):
    """A NaN code among the call's own tokens: earlier rows are as if it were not there,
    later ones give NaN; with a window, rows past it are sound again."""
    for window in (0, 3):
        for which in (0, 2):
            clean = Setup(cuda_device, [new], [new + 50], group, 1, 128, 32, seed=10)
            want, wl = clean.run(window=window, workspace=workspace)
            bad = Setup(cuda_device, [new], [new + 50], group, 1, 128, 32, seed=10)
            slot = 50 + new // 2
            bad.cache[which][bad.pages[0][slot // 32], 0, slot % 32, 77] = 0xFF
            got, gl = bad.run(window=window, workspace=workspace)
            first, last = new // 2, min(new, new // 2 + (window or new))
            sound = torch.ones(new, dtype=torch.bool)
            sound[first:last] = False
            assert torch.equal(got[sound], want[sound]) and torch.equal(gl[sound], wl[sound])
            assert bool(got[~sound][:, :, 77].isnan().all())


def test_rows_past_the_last_sequence_and_empty_calls(cuda_device, workspace):
    s = Setup(cuda_device, [2, 1], [40, 3], 2, 1, 64, 16, seed=11)
    q = torch.cat([s.q, torch.full((4, 2, 64), float("nan"), dtype=BF16, device=cuda_device)])
    out = torch.full_like(q, 5.0)
    lse = torch.full((7, 2), 6.0, device=cuda_device)
    fg.paged_attention(q, s.cache, s.table, s.seq_lens, s.cu_q, out=out, lse=lse, workspace=workspace)
    torch.cuda.synchronize()
    s.check(out[:3], lse[:3])
    assert bool((out[3:] == 5).all()) and bool((lse[3:] == 6).all())
    e = torch.empty(0, 2, 64, dtype=BF16, device=cuda_device)
    assert fg.paged_attention(e, s.cache, s.table, s.seq_lens, torch.zeros_like(s.cu_q)).shape == (0, 2, 64)
    none = fg.paged_attention(e, s.cache, s.table[:0], s.seq_lens[:0], s.cu_q[:1])
    assert none.shape == (0, 2, 64)


def test_lengths_past_the_table_are_clamped(cuda_device):
    """A length that the table cannot hold counts as the table's slots; row numbers past the
    call's rows as its rows."""
    s = Setup(cuda_device, [1], [48], 2, 1, 64, 16, seed=12, poison=False)
    want = s.run()[0]
    lens, cu = (torch.tensor(x, dtype=torch.int32, device=cuda_device) for x in ([1 << 30], [0, 99]))
    got = fg.paged_attention(s.q, s.cache, s.table[:, :3], lens, cu)
    assert torch.equal(got, want)


def test_offsets_past_32_bits(cuda_device, workspace):
    """A cache of over 4 GiB of codes, a sequence in its first and last pages."""
    Hkv, P, D = 8, 128, 128
    N = (1 << 32) // (Hkv * P * D) + 40
    small = Setup(cuda_device, [1, 150], [300, 150], 16, Hkv, D, P, seed=13, poison=False)
    big = fg.make_paged_kv_cache(N, Hkv, P, D, device=cuda_device)
    n = small.cache.k.shape[0]
    place = torch.tensor([N - 1 - 3 * i if i % 2 else i for i in range(n)], device=cuda_device)
    for a, b in zip(big, small.cache):
        a[place] = b
    table = torch.tensor([[int(place[j]) if 0 <= j < n else j for j in row] for row in small.pages], dtype=torch.int32, device=cuda_device)
    want = small.run(workspace=workspace)[0]
    got = fg.paged_attention(small.q, big, table, small.seq_lens, small.cu_q, softmax_scale=small.scale, workspace=workspace)
    assert torch.equal(got, want)


def test_another_stream_and_a_graph(cuda_device, workspace):
    s = Setup(cuda_device, [1, 1, 1], [33, 900, 2500], 8, 2, 128, 32, seed=14)
    want, wl = s.run(workspace=workspace)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.paged_attention(s.q, s.cache, s.table, s.seq_lens, s.cu_q, out=out, lse=lse, softmax_scale=s.scale, workspace=workspace)
    lens = s.seq_lens.clone()
    for i in range(4):  # the lengths are read on the device: a replay follows them
        s.seq_lens.copy_(lens - i)
        eager, _ = s.run(workspace=workspace)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    s.seq_lens.copy_(lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = fg.make_attention_workspace()
    torch.cuda.synchronize()
    got = fg.paged_attention(s.q, s.cache, s.table, s.seq_lens, s.cu_q, out=out, softmax_scale=s.scale, workspace=other, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_append_then_attend_matches_attention_over_what_was_given(cuda_device, workspace):
    """The two operators together: prompts, then single tokens, against FP64 attention over
    the unquantised keys and values (8-bit storage moves each by at most 2^-4 relative; the
    attention's result by that order)."""
    from test_gpu_paged_append import table_of
    Hq, Hkv, D, P, B, steps = 4, 2, 64, 16, 3, 5
    g = synth.make_generator(15, cuda_device)
    prompts = [19, 40, 1]
    rot = table_of(64, D // 2, cuda_device)
    cache = fg.make_paged_kv_cache(16, Hkv, P, D, device=cuda_device)
    table = torch.arange(12, dtype=torch.int32, device=cuda_device).view(3, 4)
    ks = [[] for _ in range(B)]
    vs = [[] for _ in range(B)]
    lens = [0] * B
    for step in range(steps):
        new = prompts if step == 0 else [1] * B
        T = sum(new)
        q, k, v = (torch.randn(T, h, D, generator=g, device=cuda_device).to(BF16) for h in (Hq, Hkv, Hkv))
        lens = [a + b for a, b in zip(lens, new)]
        cu = np.cumsum([0] + new).tolist()
        dl, dc = (torch.tensor(x, dtype=torch.int32, device=cuda_device) for x in (lens, cu))
        qr = fg.rope_append_paged_kv(q, k, v, rot, cache, table, dl, dc)
        out = f64(fg.paged_attention(qr, cache, table, dl, dc, workspace=workspace))
        for b in range(B):
            pos = np.arange(lens[b] - new[b], lens[b])
            t = f64(rot)[pos][:, None]
            ks[b].append(lo.rotate(f64(k[cu[b]:cu[b + 1]]), t[..., : D // 2], t[..., D // 2:])[0])
            vs[b].append(f64(v[cu[b]:cu[b + 1]]))
            kk, vv = np.concatenate(ks[b]), np.concatenate(vs[b])
            qq = lo.rotate(f64(q[cu[b]:cu[b + 1]]), t[..., : D // 2], t[..., D // 2:])[0]
            for h in range(Hq):
                s = qq[:, h] @ kk[:, h // 2].T * D ** -0.5
                s = np.where(np.arange(lens[b])[None] <= pos[:, None], s, -np.inf)
                p = np.exp(s - s.max(axis=1, keepdims=True))
                ref = p / p.sum(axis=1, keepdims=True) @ vv[:, h // 2]
                got = out[cu[b]:cu[b + 1], h]
                assert np.sqrt(((got - ref) ** 2).mean()) <= 2.0 ** -4 * np.sqrt((vv ** 2).mean())
