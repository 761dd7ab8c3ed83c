"""Sizes that the few-token layer refuses before it launches anything (no GPU)."""
import ctypes

import pytest
import torch

import dispatch_expert_gemm_amd as dm

UNSUP, WS = -5, -6


def call(workspace_bytes, **kw):
    """moe_few_tokens with addresses that nothing reads, unless it launched."""
    p = ctypes.c_void_p(0x1000)
    s = dm.make_shape(**kw)
    return dm.lib().moe_few_tokens(ctypes.byref(s), p, p, p, None, p, p, p, 0, None, None, None, None, None, None, None, p,
                                   p, p, workspace_bytes, None)


@pytest.mark.parametrize("H,F", [(8, 2 ** 20 - 32), (968, 2 ** 18)])
def test_a_grid_of_two_to_the_32_threads_is_refused(H, F):
    """1024 experts times F / 64 workgroups of 256 threads (F / 16 where H is long)."""
    if torch.cuda.is_available():
        pytest.skip("on the CPU, where a launch is refused too")
    assert call(1 << 40, T=64, H=H, K=16, num_experts=1024, F=F) == UNSUP


def test_one_below_is_not():
    """(nothing is launched: the workspace is too small)"""
    n = ctypes.c_size_t()
    s = dm.make_shape(T=64, H=8, K=16, num_experts=1024, F=2 ** 20 - 64)
    assert dm.lib().moe_few_tokens_workspace_size(ctypes.byref(s), 0, 0, ctypes.byref(n)) == 0
    assert call(256, T=64, H=8, K=16, num_experts=1024, F=2 ** 20 - 64) == WS
