"""The int8 matrix product at the ends of the sizes that it takes."""
import ctypes

import pytest
import torch

import dispatch_expert_gemm_amd as dm
from few_util import check, linear64, quant_weight, to_int8

gpu = pytest.mark.gpu
DEV = "cuda:0"


@gpu
@pytest.mark.parametrize("M", [1 << 24, (1 << 20) + 3])
def test_the_most_rows(M):
    """bf16 rows: 2^24 of them, and a few more than the quantiser's grid has on its first axis."""
    print(f"[linear int8] {M} rows", flush=True)
    K, N = 16, 3
    g = torch.Generator(device=DEV).manual_seed(90)
    x = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    w = quant_weight((torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16))
    out = dm.linear_int8(x, w)
    q, s = to_int8(x.float())
    check("rows", out, *linear64((q, s[:, 0]), w))


def test_sizes_that_are_refused():
    n = ctypes.c_size_t()
    size = lambda *a: dm.lib().moe_linear_int8_workspace_size(*a, ctypes.byref(n))   # noqa: E731
    assert size(1 << 24, 1 << 14, 131072) == 0
    assert size(1 << 24, (1 << 14) + 1, 16) == -5
    assert size((1 << 14) + 1, 1 << 24, 16) == -5
