"""Ends of the ranges of the packed products and adapters, through the Python calls."""
import pytest
import torch

from test_gpu_adapter import gq, make_adapters, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [0, 5, 1100])
def test_a_layer_without_rows(n):
    c = 64
    X = normal((n, c), 1).bfloat16()
    ad = make_adapters(2, 8, 0, c, n, torch.bfloat16, 3)
    layer = (torch.empty((0, c // 8), dtype=torch.uint32, device="cuda"), torch.empty((0, 1), device="cuda"),
             torch.empty((0, 1), dtype=torch.int32, device="cuda"), 4, -1)
    for low in ({}, ad):
        assert gq().packed_linear(X, *layer, **low).shape == (n, 0)
    assert gq().adapter_add(torch.empty((n, 0), dtype=torch.bfloat16, device="cuda"), X, **ad).shape == (n, 0)
