"""examples/expert_layer.py runs, also with fewer experts than it chooses by default."""
import pytest
import torch

from examples.expert_layer import serve

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts", [2, 4, 12, 64])
def test_it_serves(cuda_device, experts):
    with torch.no_grad():
        y = serve(3, 20, 3, hidden=256, heads=4, kv_heads=2, dim=64, ffn=128, experts=experts)
    assert y.shape == (3, 256) and bool(y.isfinite().all())
