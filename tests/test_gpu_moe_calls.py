"""The expert and head operators' calls on other streams than the current one, in captured graphs,
and on one compute unit: what a call allocates is free of earlier work, stays the call's until it
has run, is not given away while the current stream reads it, and belongs to the graph that
captures it; replays follow their inputs."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
from moe_grouped_gemm_fp32_amd import moe
from test_gpu_layer_other_stream import blocks_like, busy

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def route(dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    x, b = torch.randn(6000, 192, generator=g, device=dev), torch.randn(192, generator=g, device=dev) * 0.1
    return [x], lambda **kw: fg.moe_route(x, 6, bias=b, scoring="sigmoid", groups=6, top_groups=3, group_best=2, **kw)


def route_grad(dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    x, w = torch.randn(6000, 192, generator=g, device=dev).to(BF16), torch.randn(6000, 6, generator=g, device=dev)
    ids = torch.rand(6000, 192, generator=g, device=dev).topk(6, 1).indices.to(I32)
    return [x, w], lambda **kw: (fg.moe_route_backward(w, x, ids, **kw),)


def layout(dev, seed, T=20000):
    """Of many choices: with the workspace that a call allocates."""
    g = torch.Generator(dev).manual_seed(seed)
    Q, sa = torch.zeros(T, 128, dtype=torch.uint8, device=dev), torch.ones(1, T, device=dev)
    ids = torch.rand(T, 50, generator=g, device=dev).topk(4, 1).indices.to(I32)
    return [ids], lambda **kw: tuple(fg.moe_dispatch(Q, sa, ids, 50, **kw)[2])


def layout_by_all(dev, seed):
    return layout(dev, seed, 5000)


def dispatch(dev, seed, T=2048):
    g = torch.Generator(dev).manual_seed(seed)
    Q = torch.randint(0, 100, (T, 512), generator=g, device=dev, dtype=torch.uint8)
    sa, w = torch.rand(4, T, generator=g, device=dev), torch.rand(T, 4, generator=g, device=dev)
    ids = (torch.arange(T * 4, dtype=I32, device=dev) % (T // 32)).view(T, 4)  # 128 choices for each expert
    at = fg.make_moe_layout(T, 4, T // 32, rows=4 * T)
    return [Q, sa, w], lambda **kw: fg.moe_dispatch(Q, sa, ids, T // 32, weights=w, layout=at, **kw)[:2]


def dispatch_few(dev, seed):
    return dispatch(dev, seed, 512)


def gather(dev, seed):
    inputs, call = dispatch(dev, seed)
    Q, sa, w = inputs
    ids = (torch.arange(8192, dtype=I32, device=dev) % 64).view(2048, 4)
    at = fg.moe_dispatch(Q, sa, ids, 64, layout=fg.make_moe_layout(2048, 4, 64, rows=8192))[2]
    return inputs, lambda **kw: fg.moe_gather(Q, sa, at, weights=w, **kw)


def combine(dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    Y, w = torch.randn(6000, 1024, generator=g, device=dev).to(BF16), torch.rand(1500, 4, generator=g, device=dev)
    at = torch.randperm(6000, generator=g, device=dev).to(I32).view(1500, 4)
    return [Y, w], lambda **kw: (fg.moe_combine(Y, at, w, **kw),)


def combine_grad(dev, seed):
    (Y, w), _ = combine(dev, seed)
    g = torch.Generator(dev).manual_seed(seed)
    dO = torch.randn(1500, 1024, generator=g, device=dev).to(BF16)
    at = torch.randperm(6000, generator=g, device=dev).to(I32).view(1500, 4)
    return [Y, w, dO], lambda **kw: fg.moe_combine_backward(dO, Y, at, w, **kw)


def heads(dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    x, w = torch.randn(3000, 12, 128, generator=g, device=dev).to(BF16), torch.rand(128, generator=g, device=dev) + 0.5
    table = torch.rand(3000, 128, generator=g, device=dev)
    return [x, table], lambda **kw: fg.qk_norm_rope(x[:, :8], x[:, 8:], w, w, table, **kw)


def heads_grad(dev, seed):
    (x, table), _ = heads(dev, seed)
    g = torch.Generator(dev).manual_seed(seed)
    dy, w = torch.randn(3000, 12, 128, generator=g, device=dev).to(BF16), torch.rand(128, generator=g, device=dev) + 0.5
    return [x, dy], lambda **kw: fg.qk_norm_rope_backward(dy[:, :8], dy[:, 8:], x[:, :8], x[:, 8:], w, w, table, **kw)


CALLS = pytest.mark.parametrize("make", [route, route_grad, layout, layout_by_all, dispatch, dispatch_few, gather, combine, combine_grad, heads,
                                         heads_grad])


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@CALLS
def test_earlier_work_on_freed_memory(cuda_device, make):
    """Blocks freed with work still queued on them are what the allocator hands out next."""
    _, call = make(cuda_device, 1)
    go, side = busy(), torch.cuda.Stream()
    want = call()
    size = 0
    if make is heads_grad:
        size = moe._fn("fp8_qk_norm_rope_backward_workspace_size")(128)
    elif make is layout:
        size = moe._fn("fp8_moe_dispatch_workspace_size")(20000, 4, 50)
        assert size
    old = blocks_like(want, size)
    torch.cuda.synchronize()
    go()
    for t in old:
        t.view(torch.uint8).fill_(0x5A)
    del old, t
    got = call(stream=side)
    torch.cuda.synchronize()
    assert same(got, want)


@CALLS
def test_outputs_let_go_at_once(cuda_device, make):
    """What the caller does not keep is not handed out before the call has written it."""
    _, call = make(cuda_device, 2)
    go, side = busy(), torch.cuda.Stream()
    like = call()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        go()
    call(stream=side)
    new = blocks_like(like)
    for t in new:
        t.view(torch.uint8).fill_(0x5A)
    torch.cuda.synchronize()
    assert all(bool((t.view(torch.uint8) == 0x5A).all()) for t in new)


@CALLS
def test_outputs_that_the_current_stream_still_reads(cuda_device, make):
    (_, first), (_, second) = make(cuda_device, 3), make(cuda_device, 4)
    go, side = busy(), torch.cuda.Stream()
    want = [t.clone() for t in first()]
    copies = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    got = first(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    go()
    for c, t in zip(copies, got):
        c.copy_(t)
    del got, t
    second(stream=side)
    torch.cuda.synchronize()
    assert same(copies, want)


@CALLS
def test_on_a_side_stream_of_a_captured_graph(cuda_device, make):
    """Outputs allocated on a stream that a capture forks to belong to the graph, and replays follow
    the inputs, whatever eager calls run in between."""
    inputs, call = make(cuda_device, 6)
    side = torch.cuda.Stream()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    others, _ = make(cuda_device, 7)
    for turn in range(4):
        for a, b in zip(inputs, others):
            kept = a.clone()
            a.copy_(b)
            b.copy_(kept)
        for t in got:
            t.view(torch.uint8).fill_(0x5A)
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want), turn


def test_two_graphs_of_the_same_operators(cuda_device):
    """Each captures its own workspace: replayed one after the other, and at once on two streams."""
    made = [layout(cuda_device, s) for s in (1, 2)] + [heads_grad(cuda_device, s) for s in (1, 2)]
    want = [[t.clone() for t in call()] for _, call in made]
    torch.cuda.synchronize()
    graphs, got = [], []
    for _, call in made:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(call())
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(3):
        for out in got:
            for t in out:
                t.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


def test_streams_given_as_objects(cuda_device):
    _, call = heads(cuda_device, 5)
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    for s in (side, torch.cuda.ExternalStream(side.cuda_stream), Handle(), torch.cuda.current_stream(), torch.cuda.default_stream()):
        got = call(stream=s)
        torch.cuda.synchronize()
        assert torch.cuda.current_stream() == torch.cuda.default_stream() and same(got, want)


@pytest.mark.parametrize("cus", [1, 3, 100])
def test_on_fewer_compute_units(cuda_device, cus):
    """The gradient's sums are cut for the units in effect; everything else has no part in them."""
    x, dy = (torch.randn(500, 6, 64, generator=torch.Generator(cuda_device).manual_seed(s), device=cuda_device) for s in (1, 2))
    w = torch.ones(64, device=cuda_device)
    want = fg.qk_norm_rope_backward(dy[:, :4], dy[:, 4:], x[:, :4], x[:, 4:], w, w)
    fg.set_num_cus(cus)
    try:
        got = fg.qk_norm_rope_backward(dy[:, :4], dy[:, 4:], x[:, :4], x[:, 4:], w, w)
        again = fg.qk_norm_rope_backward(dy[:, :4], dy[:, 4:], x[:, :4], x[:, 4:], w, w)
    finally:
        fg.set_num_cus(0)
    assert same(got, again) and same(got[:2], want[:2])  # dx has no sums over heads
    xh = x.double() * torch.rsqrt(x.double().square().mean(2, keepdim=True) + 1e-6)
    for g, part in ((got[2], slice(0, 4)), (got[3], slice(4, 6))):
        terms = dy[:, part].double() * xh[:, part]
        assert bool(((g.double() - terms.sum((0, 1))).abs() <= (500 * 4 + 64) * 2.0 ** -24 * terms.abs().sum((0, 1))).all())
