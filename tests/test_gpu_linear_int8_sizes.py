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


@gpu
@pytest.mark.parametrize("M", [1, 20, 70])
def test_codes_at_minus_128(M):
    """Both operands, at the longest rows whose sums stay below 2^31."""
    N, K = 19, 131056
    xq = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    wq = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    wq[1::2] = 127
    wq[4, ::3] = 126
    xs, ws = torch.full((M,), 2.0 ** -12, device=DEV), torch.full((N,), 2.0 ** -9, device=DEV)
    v, bound = linear64((xq, xs), (wq, ws))
    check("-128", dm.linear_int8(xq, (wq, ws), x_scales=xs), v, bound)
