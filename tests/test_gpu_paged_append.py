"""GPU parity of the rotation and append to the paged 8-bit cache against the FP64 oracle.

Bounds, u = 2^-24: a turned column is two rounded products and their rounded sum, off by at
most 3 u (|x1 cos| + |x2 sin|) =: r; a query is then rounded to BF16 (2^-8 relative). A code
is the nearest to the value over a power of two, so it is within half a step of its binade
of the true quotient, plus r over the scale. Scales are exact: the tests' largest values
are not within r of a power's border (checked). Bytes that no new token touches, and whose
page's scale stays, are unchanged."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import oracle
import synth
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
POS = oracle.E4M3_TABLE[:0x7F]


def half_step(a):
    hi = np.clip(np.searchsorted(POS, a, side="right"), 1, 0x7E)
    return 0.5 * (POS[hi] - POS[hi - 1])


def f64(t):
    return t.detach().double().cpu().numpy()


def table_of(positions, half, dev):
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * 1000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().to(dev)


class Setup:
    """A cache part-filled by random codes, sequences on shuffled pages, and new tokens."""

    def __init__(self, dev, new, lens, Hq, Hkv, D, P, seed=0, spare=3, scale_exp=(-8, -5), std=1.0):
        g = synth.make_generator(seed, dev)
        self.new, self.lens, self.T = new, lens, sum(new)
        npages = [-(-max(m, 1) // P) for m in lens]
        N = sum(npages) + spare
        order = torch.randperm(N, generator=synth.make_generator(seed + 1)).tolist()
        self.pages, at = [], 0
        width = max(npages) + 1
        for n in npages:
            self.pages.append(order[at:at + n] + [-1] * (width - n))
            at += n
        self.cache = fg.make_paged_kv_cache(N, Hkv, P, D, device=dev)
        for codes, scale in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device=dev, dtype=torch.uint8))
            codes[(codes & 0x7F) == 0x7F] = 0x11
            scale.copy_(2.0 ** torch.randint(*scale_exp, scale.shape, generator=g, device=dev).float())
        self.table = torch.tensor(self.pages, dtype=torch.int32, device=dev)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.cu_q = torch.tensor(self.cu, dtype=torch.int32, device=dev)
        qkv = (torch.randn(self.T, (Hq + 2 * Hkv) * D, generator=g, device=dev) * std
               * torch.exp(torch.randn(self.T, 1, generator=g, device=dev))).to(BF16)
        self.q = qkv[:, :Hq * D].view(self.T, Hq, D)
        self.k = qkv[:, Hq * D:(Hq + Hkv) * D].view(self.T, Hkv, D)
        self.v = qkv[:, (Hq + Hkv) * D:].view(self.T, Hkv, D)

    def positions(self):
        return np.concatenate([np.arange(m - n, m) for n, m in zip(self.new, self.lens)] + [np.zeros(0, int)]).astype(int)

    def run(self, rot, interleaved=False, positions=None, **kw):
        self.before = [t.clone() for t in self.cache]
        out = fg.rope_append_paged_kv(kw.pop("q", self.q), self.k, self.v, rot, self.cache, self.table, self.seq_lens, self.cu_q,
                                      positions=positions, interleaved=interleaved, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, rot, interleaved=False, positions=None):
        pos = self.positions() if positions is None else f64(positions).astype(int)
        half = 0 if rot is None else rot.shape[1] // 2
        t = np.zeros((self.T, 0)) if rot is None else f64(rot)[np.clip(pos, 0, rot.shape[0] - 1)]
        cos, sin = t[:, None, :half], t[:, None, half:]
        if out is not None:
            y, mag = lo.rotate(f64(self.q), cos, sin, interleaved)
            assert np.all(np.abs(f64(out) - y) <= 2.0 ** -8 * np.abs(y) + 4 * 2.0 ** -24 * mag)
        k, kmag = lo.rotate(f64(self.k), cos, sin, interleaved)
        v = f64(self.v)
        for x, mag, codes, scale, c0, s0 in ((k, kmag, self.cache.k, self.cache.k_scale, self.before[0], self.before[1]),
                                             (v, np.zeros_like(v), self.cache.v, self.cache.v_scale, self.before[2], self.before[3])):
            P = codes.shape[2]
            c0, s0 = c0.cpu().numpy(), f64(s0)
            value, want, written = lo.append(c0, s0, x, self.pages, self.lens, self.cu, P)
            r, _, _ = lo.append(np.zeros_like(c0), want, 3 * 2.0 ** -24 * mag, self.pages, self.lens, self.cu, P)
            got, c1 = f64(scale), codes.cpu().numpy()
            assert np.array_equal(got, want)
            r *= (lo.append(np.zeros_like(c0), want, 3 * 2.0 ** -24 * mag, self.pages, self.lens, self.cu, P)[1] / want)[:, :, None, None]
            deq = oracle.decode_e4m3(c1)
            err = np.abs(deq - value)
            moved = written | np.broadcast_to((want != s0)[:, :, None], written.shape)
            assert np.array_equal(c1[~moved], c0[~moved])
            bound = half_step(np.minimum(np.abs(value) + r, 448.0)) + r
            bad = np.argwhere((err > bound) & moved[..., None])
            assert not len(bad), (len(bad), bad[0], deq[tuple(bad[0])], value[tuple(bad[0])])


CASES = [
    # new tokens, lengths, Hq, Hkv, D, P, rot_dim
    ([1], [1], 1, 1, 128, 16, 128),
    ([1, 1, 1, 1, 1], [1, 16, 17, 64, 333], 8, 2, 128, 64, 128),
    ([1] * 70, list(range(1, 71)), 4, 4, 64, 32, 64),
    ([40], [40], 2, 1, 256, 16, 256),
    ([3, 0, 130, 1], [100, 7, 130, 1], 6, 2, 128, 128, 64),
    ([257, 5], [300, 261], 3, 3, 64, 256, 32),
    ([33, 17, 64], [65, 17, 128], 16, 1, 128, 16, 0),
    ([2, 3, 1], [34, 515, 48], 4, 2, 256, 64, 96),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,P,rot_dim", CASES)
def test_append(cuda_device, new, lens, Hq, Hkv, D, P, rot_dim, interleaved):
    s = Setup(cuda_device, new, lens, Hq, Hkv, D, P)
    rot = table_of(max(lens), rot_dim // 2, cuda_device) if rot_dim else None
    s.check(s.run(rot, interleaved), rot, interleaved)


@pytest.mark.parametrize("std", [1e-6, 3e4])
def test_scales_grow_and_stay(cuda_device, std):
    """Earlier codes stay at a scale that is large enough and move to one that is not,
    whether a wave or a workgroup holds the page."""
    for new in ([1, 1], [20, 9]):
        s = Setup(cuda_device, new, [60, 41], 2, 2, 128, 64, seed=3, std=std)
        rot = table_of(64, 64, cuda_device)
        s.check(s.run(rot), rot)
        grew = (s.cache.k_scale != s.before[1])
        assert bool(grew.any()) == (std > 1)


def test_a_page_begun_anew_forgets_its_scale_and_zeros_take_the_least(cuda_device):
    s = Setup(cuda_device, [1, 16], [17, 16], 1, 1, 64, 16, seed=4, scale_exp=(90, 100))
    s.k.zero_()
    s.check(s.run(None), None)
    assert float(s.cache.k_scale[s.pages[0][1], 0]) == 2.0 ** -126
    # the second append to that page starts from the least scale
    s.k.fill_(2.0)
    s.new, s.lens, s.cu = [1, 0], [18, 16], [0, 1, 1]
    s.k, s.v, s.q, s.T = s.k[:1], s.v[:1], s.q[:1], 1
    s.seq_lens = torch.tensor(s.lens, dtype=torch.int32, device=cuda_device)
    s.cu_q = torch.tensor(s.cu, dtype=torch.int32, device=cuda_device)
    s.check(s.run(None), None)
    assert float(s.cache.k_scale[s.pages[0][1], 0]) == 2.0 ** -7


def test_not_a_number_and_infinities(cuda_device):
    s = Setup(cuda_device, [3], [20], 1, 1, 64, 32, seed=5)
    for x in (s.k, s.v):
        x[0, 0, 3], x[1, 0, 4], x[2, 0, 5] = float("nan"), float("inf"), float("-inf")
    s.run(None)
    for codes, scale, x in ((s.cache.k, s.cache.k_scale, s.k), (s.cache.v, s.cache.v_scale, s.v)):
        page = s.pages[0][0]
        got = codes[page, 0, 17:20].cpu().numpy()
        bad = ~np.isfinite(f64(x)[:, 0])
        assert bad.sum() == 3 and np.array_equal((got & 0x7F) == 0x7F, bad)
        finite = np.where(bad, 0.0, f64(x)[:, 0])
        assert float(scale[page, 0]) >= lo.fit_scale(np.abs(finite).max())
        want = finite / float(scale[page, 0])
        assert np.all(np.abs(np.where(bad, 0, oracle.decode_e4m3(np.where(bad, 0, got))) - want) <= half_step(np.abs(want)))


def test_positions_strides_and_in_place_queries(cuda_device):
    """Given positions beyond the table are clamped; queries turn in place."""
    s = Setup(cuda_device, [2, 30], [5, 77], 4, 2, 128, 32, seed=6)
    rot = table_of(50, 64, cuda_device)[:, :96].contiguous()
    rot = torch.cat([rot[:, :48], rot[:, :48]], dim=1)
    wide = torch.full((50, 104), float("nan"), device=cuda_device)
    wide[:, :96] = rot
    positions = torch.tensor([-4, 3] + list(range(30, 60)), dtype=torch.int32, device=cuda_device)
    s.check(s.run(wide[:, :96], positions=positions), rot, positions=positions)
    again = Setup(cuda_device, [2, 30], [5, 77], 4, 2, 128, 32, seed=6)
    want = again.q.clone()
    out = again.run(wide[:, :96], positions=positions, q_out=again.q)
    again.q = want
    again.check(out, rot, positions=positions)


def test_only_the_cache(cuda_device):
    s = Setup(cuda_device, [4, 1], [4, 50], 4, 2, 64, 16, seed=7)
    rot = table_of(64, 32, cuda_device)
    assert s.run(rot, q=None) is None
    s.check(None, rot)


def test_what_has_no_place_is_dropped(cuda_device):
    """Pages of no number, slots past the table or below zero, rows past the last sequence."""
    s = Setup(cuda_device, [20, 6, 4], [20, 70, 2], 1, 1, 64, 16, seed=8)
    s.pages[0][1] = -1
    s.pages[1][4] = s.cache.k.shape[0]
    s.table = torch.tensor(s.pages, dtype=torch.int32, device=cuda_device)
    rows = torch.zeros(s.T + 3, 1, 64, dtype=BF16, device=cuda_device)
    k, v, q = (torch.cat([x, rows[:3]]) for x in (s.k, s.v, s.q))
    q_out = torch.full_like(q, 9.0)
    before = [t.clone() for t in s.cache]
    fg.rope_append_paged_kv(q, k, v, None, s.cache, s.table, s.seq_lens, s.cu_q, q_out=q_out)
    torch.cuda.synchronize()
    assert torch.equal(q_out[:s.T], s.q) and bool((q_out[s.T:] == 9).all())
    s.before = before
    s.check(None, None)
    # a table narrower than the lengths say: slots past it are dropped
    t = Setup(cuda_device, [20], [20], 1, 1, 64, 16, seed=9)
    keep = [x.clone() for x in t.cache]
    fg.rope_append_paged_kv(None, t.k, t.v, None, t.cache, t.table[:, :1], t.seq_lens, t.cu_q)
    torch.cuda.synchronize()
    assert torch.equal(t.cache.k[t.pages[0][1]], keep[0][t.pages[0][1]])


def test_no_tokens(cuda_device):
    s = Setup(cuda_device, [0, 0], [5, 0], 1, 1, 64, 16, seed=10)
    before = [t.clone() for t in s.cache]
    out = s.run(None)
    assert out.shape == (0, 1, 64) and all(torch.equal(a, b) for a, b in zip(before, s.cache))


def test_wave_and_workgroup_units_agree(cuda_device):
    """The same tokens appended one call at a time and all at once: the same cache, where
    the largest value comes first (so that no re-encoding rounds twice)."""
    one, all_ = (Setup(cuda_device, [40], [45], 2, 2, 128, 64, seed=11) for _ in range(2))
    for s in (one, all_):
        s.k[0] = 500.0
        s.v[0] = -300.0
    rot = table_of(64, 64, cuda_device)
    want = all_.run(rot)
    got = []
    for i in range(40):
        step = [torch.tensor(x, dtype=torch.int32, device=cuda_device) for x in ([6 + i], [0, 1])]
        got.append(fg.rope_append_paged_kv(one.q[i:i + 1], one.k[i:i + 1], one.v[i:i + 1], rot, one.cache, one.table, *step))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(got), want) and all(torch.equal(a, b) for a, b in zip(one.cache, all_.cache))


def test_offsets_past_32_bits(cuda_device):
    """A cache of over 4 GiB of codes, tokens in its last pages."""
    Hkv, P, D = 8, 128, 128
    N = (1 << 32) // (Hkv * P * D) + 40
    cache = fg.make_paged_kv_cache(N, Hkv, P, D, device=cuda_device)
    g = synth.make_generator(12, cuda_device)
    k, v = (torch.randn(130, Hkv, D, generator=g, device=cuda_device).to(BF16) for _ in range(2))
    table = torch.tensor([[N - 1, N - 7]], dtype=torch.int32, device=cuda_device)
    lens, cu = (torch.tensor(x, dtype=torch.int32, device=cuda_device) for x in ([130], [0, 130]))
    fg.rope_append_paged_kv(None, k, v, None, cache, table, lens, cu)
    torch.cuda.synchronize()
    for codes, scale, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        for page, rows in ((N - 1, x[:128]), (N - 7, x[128:])):
            deq = codes[page, :, :rows.shape[0]].view(torch.float8_e4m3fn).double() * scale[page].double()[:, None, None]
            want = rows.double().transpose(0, 1)
            assert bool(((deq - want).abs() <= want.abs() * 2.0 ** -4 + 2.0 ** -10 * scale[page].double()[:, None, None]).all())
        assert int((codes[:N - 8] != 0).sum()) == 0


def test_another_stream_and_a_graph(cuda_device):
    s = Setup(cuda_device, [1, 1], [33, 90], 2, 1, 128, 32, seed=13)
    rot = table_of(128, 64, cuda_device)
    ref = Setup(cuda_device, [1, 1], [33, 90], 2, 1, 128, 32, seed=13)
    want = ref.run(rot)
    q_out = torch.empty_like(s.q, memory_format=torch.contiguous_format)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = [t.clone() for t in s.cache]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fg.rope_append_paged_kv(s.q, s.k, s.v, rot, s.cache, s.table, s.seq_lens, s.cu_q, q_out=q_out)
    for _ in range(3):
        for t, b in zip(s.cache, keep):
            t.copy_(b)
        q_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, want) and all(torch.equal(a, b) for a, b in zip(s.cache, ref.cache))
    side = torch.cuda.Stream()
    for t, b in zip(s.cache, keep):
        t.copy_(b)
    torch.cuda.synchronize()
    out = fg.rope_append_paged_kv(s.q, s.k, s.v, rot, s.cache, s.table, s.seq_lens, s.cu_q, q_out=q_out.zero_(), stream=torch.cuda.current_stream())
    side.wait_stream(torch.cuda.current_stream())
    out = fg.rope_append_paged_kv(s.q, s.k, s.v, rot, s.cache, s.table, s.seq_lens, s.cu_q, q_out=q_out, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(s.cache, ref.cache))
