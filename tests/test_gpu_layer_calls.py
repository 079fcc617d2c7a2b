"""What the layer operators' Python calls refuse, and that a call keeps nothing of its
arguments."""
import sys

import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg

pytestmark = pytest.mark.gpu
BF16, FP32, I32 = torch.bfloat16, torch.float32, torch.int32


def norm_args(dev):
    return dict(X=torch.randn(5, 256, device=dev).to(BF16), weight=torch.ones(256, device=dev), residual=torch.zeros(5, 256, dtype=BF16, device=dev),
                Q=torch.empty(5, 256, dtype=torch.uint8, device=dev), sa=torch.empty(2, 8, device=dev), rstd=torch.empty(5, device=dev),
                H=torch.empty(5, 256, dtype=BF16, device=dev), Y=torch.empty(5, 256, dtype=BF16, device=dev))


def grad_args(dev):
    return dict(dY=torch.randn(5, 256, device=dev), H=torch.randn(5, 256, device=dev), rstd=torch.ones(5, device=dev),
                weight=torch.ones(256, device=dev), dH=torch.zeros(5, 256, device=dev), dX=torch.empty(5, 256, device=dev),
                dW=torch.empty(256, device=dev), workspace=torch.empty(1 << 20, dtype=torch.uint8, device=dev))


def sequences(dev):
    return dict(cache=fg.make_paged_kv_cache(4, 2, 16, 64, device=dev), block_table=torch.arange(4, dtype=I32, device=dev).view(2, 2),
                seq_lens=torch.tensor([3, 20], dtype=I32, device=dev), cu_q=torch.tensor([0, 2, 3], dtype=I32, device=dev))


def append_args(dev):
    return dict(q=torch.randn(3, 4, 64, device=dev).to(BF16), k=torch.randn(3, 2, 64, device=dev).to(BF16),
                v=torch.randn(3, 2, 64, device=dev).to(BF16), cos_sin=torch.rand(64, 64, device=dev), **sequences(dev),
                positions=torch.zeros(3, dtype=I32, device=dev), q_out=torch.empty(3, 4, 64, dtype=BF16, device=dev))


def attend_args(dev):
    return dict(q=torch.randn(3, 4, 64, device=dev).to(BF16), **sequences(dev), out=torch.empty(3, 4, 64, dtype=BF16, device=dev),
                lse=torch.empty(3, 4, device=dev), workspace=fg.make_attention_workspace(dev))


CALLS = {"norm": (fg.rmsnorm_quantize_1x128, norm_args), "grad": (fg.rmsnorm_backward, grad_args),
         "append": (fg.rope_append_paged_kv, append_args), "attend": (fg.paged_attention, attend_args)}


def other_type(t):
    return t.to(torch.float16) if t.is_floating_point() else t.to(torch.int64)


def other_place(t):
    return t.cpu()


def other_shape(t):
    return torch.cat([t, t])


@pytest.mark.parametrize("change", [other_type, other_place, other_shape])
@pytest.mark.parametrize("name", CALLS)
def test_types_places_and_shapes_are_refused(cuda_device, name, change):
    fn, make = CALLS[name]
    for key, value in make(cuda_device).items():
        if change is not other_place and key == "workspace" or change is other_shape and key == "cos_sin":
            continue  # any type and size will do; more positions are right
        for i in range(4) if key == "cache" else [None]:
            args = make(cuda_device)
            if i is None:
                args[key] = change(value)
            else:
                args[key] = fg.PagedKVCache(*(change(t) if i == j else t for j, t in enumerate(args[key])))
            with pytest.raises(ValueError):
                fn(**args)


@pytest.mark.parametrize("name", CALLS)
def test_what_is_no_tensor_is_refused(cuda_device, name):
    fn, make = CALLS[name]
    for key in make(cuda_device):
        with pytest.raises(TypeError):
            fn(**{**make(cuda_device), key: 7})


def strided(t):
    wide = torch.stack([t, t], dim=-1)
    return wide.as_strided(t.shape, [2 * s for s in t.stride()])


@pytest.mark.parametrize("name", CALLS)
def test_inner_strides_are_refused(cuda_device, name):
    fn, make = CALLS[name]
    for key, value in make(cuda_device).items():
        for i in range(4) if key == "cache" else [None]:
            args = make(cuda_device)
            if i is None:
                args[key] = strided(value)
            else:
                args[key] = fg.PagedKVCache(*(strided(t) if i == j else t for j, t in enumerate(args[key])))
            with pytest.raises(ValueError):
                fn(**args)


def test_numbers_that_the_library_refuses(cuda_device):
    for name, bad in (("norm", dict(eps=-1.0)), ("norm", dict(eps=float("nan"))), ("attend", dict(window=-1)),
                      ("attend", dict(softmax_scale=float("inf"))), ("append", dict(cos_sin=torch.zeros(0, 64, device=cuda_device))),
                      ("append", dict(cos_sin=torch.zeros(64, 24, device=cuda_device)))):
        fn, make = CALLS[name]
        with pytest.raises(fg.Fp8GemmError):
            fn(**{**make(cuda_device), **bad})
    args = attend_args(cuda_device)
    with pytest.raises(ValueError):
        fg.paged_attention(**{**args, "window": 1 << 40})
    with pytest.raises(TypeError):
        fg.paged_attention(**{**args, "window": "all"})
    with pytest.raises(ValueError):
        fg.rope_append_paged_kv(**{**append_args(cuda_device), "q": None})  # q_out without q
    with pytest.raises(ValueError):
        fg.rmsnorm_quantize_1x128(**{**norm_args(cuda_device), "residual": None})  # H without a residual
    with pytest.raises(AttributeError):
        fg.paged_attention(**args, stream=object())


@pytest.mark.parametrize("name", CALLS)
def test_a_call_keeps_nothing_of_its_arguments(cuda_device, name):
    fn, make = CALLS[name]
    args = make(cuda_device)
    held = [t for v in args.values() for t in (v if isinstance(v, tuple) else (v,))]
    fn(**args)
    torch.cuda.synchronize()
    counts = [sys.getrefcount(t) for t in held]
    memory = torch.cuda.memory_allocated()
    for _ in range(5):
        fn(**args)
    for key in args:
        with pytest.raises(TypeError):
            fn(**{**args, key: 7})
    torch.cuda.synchronize()
    assert [sys.getrefcount(t) for t in held] == counts
    assert torch.cuda.memory_allocated() == memory


def test_given_outputs_come_back_and_new_ones_are_whole(cuda_device):
    n = norm_args(cuda_device)
    Q, sa, H, rstd = fg.rmsnorm_quantize_1x128(**n)
    assert Q is n["Q"] and sa is n["sa"] and H is n["H"] and rstd is n["rstd"]
    Q2, sa2, H2, rstd2 = fg.rmsnorm_quantize_1x128(n["X"], n["weight"], n["residual"])
    assert torch.equal(Q, Q2) and torch.equal(sa[:, :5], sa2[:, :5]) and torch.equal(H, H2) and torch.equal(rstd, rstd2)
    assert fg.rmsnorm_quantize_1x128(n["X"], n["weight"])[2] is n["X"]
    g = grad_args(cuda_device)
    dX, dW = fg.rmsnorm_backward(**g)
    assert dX is g["dX"] and dW is g["dW"]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    dX2, dW2 = fg.rmsnorm_backward(g["dY"], g["H"], g["rstd"], g["weight"], g["dH"], stream=side)
    side.synchronize()
    assert torch.equal(dX, dX2) and torch.equal(dW, dW2)
    a = attend_args(cuda_device)
    assert fg.paged_attention(**a) is a["out"]
    p = append_args(cuda_device)
    assert fg.rope_append_paged_kv(**p) is p["q_out"]
    del p["q_out"]
    assert fg.rope_append_paged_kv(**{**p, "q": None}) is None
