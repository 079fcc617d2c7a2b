"""Calls on another stream than the current one, with work still queued on either: memory that a
call allocates is free of earlier work, stays the call's until it has run, and once handed over
is not given to a later call while the current stream still reads it."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def norm(dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    X, R = (torch.randn(1500, 2048, generator=g, device=dev).to(BF16) for _ in range(2))
    w = torch.ones(2048, device=dev)
    return lambda **kw: fg.rmsnorm_quantize_1x128(X, w, residual=R, **kw)


def grad(dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    dY, H = (torch.randn(3000, 2048, generator=g, device=dev).to(BF16) for _ in range(2))
    w, rstd = torch.ones(2048, device=dev), torch.ones(3000, device=dev)
    return lambda **kw: fg.rmsnorm_backward(dY, H, rstd, w, **kw)


def few_grad(dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    dY, H = (torch.randn(500, 2048, generator=g, device=dev) for _ in range(2))
    w, rstd = torch.ones(2048, device=dev), torch.ones(500, device=dev)
    return lambda **kw: fg.rmsnorm_backward(dY, H, rstd, w, **kw)


def sequences(dev):
    table = torch.arange(64, dtype=I32, device=dev).view(1, 64)
    return table, torch.tensor([2048], dtype=I32, device=dev), torch.tensor([0, 2048], dtype=I32, device=dev)


def append(dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    q, k, v = (torch.randn(2048, h, 128, generator=g, device=dev).to(BF16) for h in (8, 1, 1))
    cache, rot = fg.make_paged_kv_cache(64, 1, 32, 128, device=dev), torch.rand(2048, 128, generator=g, device=dev)
    seqs = sequences(dev)
    return lambda **kw: (fg.rope_append_paged_kv(q, k, v, rot, cache, *seqs, **kw),)


def attend(dev, seed):
    g = torch.Generator(dev).manual_seed(seed)
    q = torch.randn(2048, 8, 128, generator=g, device=dev).to(BF16)
    cache = fg.make_paged_kv_cache(64, 1, 32, 128, device=dev)
    for t in (cache.k, cache.v):
        t.copy_(torch.randint(0, 0x40, t.shape, generator=g, device=dev, dtype=torch.uint8))
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(0.5)
    seqs = sequences(dev)
    return lambda **kw: (fg.paged_attention(q, cache, *seqs, **kw),)


CALLS = pytest.mark.parametrize("make", [norm, grad, few_grad, append, attend])


def busy(times=60):
    """Queues some tens of milliseconds of work on the current stream."""
    x = torch.zeros(1 << 28, device="cuda")

    def go():
        for _ in range(times):
            x.add_(1.0)
    return go


def blocks_like(tensors, workspace=0):
    old = [torch.empty_like(t) for t in tensors]
    return old + ([torch.empty(workspace, dtype=torch.uint8, device="cuda")] if workspace else [])


@CALLS
def test_earlier_work_on_freed_memory(cuda_device, make):
    """Blocks freed with work still queued on them are what the allocator hands out next."""
    call, go, side = make(cuda_device, 1), busy(), torch.cuda.Stream()
    want = call()
    size = 0
    if make in (grad, few_grad):
        size = fg.layer._fn("fp8_rmsnorm_backward_workspace_size")(*want[0].shape)
    old = blocks_like(want, size)
    torch.cuda.synchronize()
    go()
    for t in old:
        t.view(torch.uint8).fill_(0x5A)
    del old, t
    got = call(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@CALLS
def test_outputs_let_go_at_once(cuda_device, make):
    """What the caller does not keep is not handed out before the call has written it."""
    call, go, side = make(cuda_device, 2), busy(), torch.cuda.Stream()
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
    first, second, go, side = make(cuda_device, 3), make(cuda_device, 4), busy(), torch.cuda.Stream()
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
    for a, b in zip(copies, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_any_stream_object_and_a_stream_of_its_own_handle(cuda_device):
    call = norm(cuda_device, 5)
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    for s in (side, torch.cuda.ExternalStream(side.cuda_stream), Handle(), torch.cuda.current_stream(), torch.cuda.default_stream()):
        got = call(stream=s)
        torch.cuda.synchronize()
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@CALLS
def test_on_a_side_stream_of_a_captured_graph(cuda_device, make):
    """Outputs allocated on a stream that a capture forks to belong to the graph: replays write them."""
    call, side = make(cuda_device, 6), torch.cuda.Stream()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(3):
        for t in (*got, *copies):
            t.view(torch.uint8).fill_(0x5A)
        other = call()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c, d in zip(got, copies, want, other):
            assert torch.equal(a.view(torch.uint8), c.view(torch.uint8)) and torch.equal(b.view(torch.uint8), c.view(torch.uint8))
            assert torch.equal(d.view(torch.uint8), c.view(torch.uint8))
