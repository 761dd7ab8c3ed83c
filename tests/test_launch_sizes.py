"""CPU checks: entries refuse sizes whose launch would hold 2^32 threads or more, of which only a part would run."""
import ctypes
import os

import pytest

import dispatch_expert_gemm_amd as dm

UNSUPPORTED = -5
N = None
P = ctypes.c_void_p(0x10000)  # a non-NULL stand-in: never dereferenced (refused first)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dm.LIB_PATH):
        pytest.skip("libmoe.so not built (run __graft_entry__.build())")
    return dm.lib()


@pytest.mark.parametrize("T,H,K", [(1 << 26, 8, 1), ((1 << 31) - 1, 8, 1), (1 << 24, 4096, 4)])
def test_a_wave_or_more_a_token(L, T, H, K):
    s = ctypes.byref(dm.make_shape(T, H, K, 16, capacity=T * K))
    assert L.moe_combine(s, *[P] * 5, *[N] * 6, P, N) == UNSUPPORTED
    assert L.moe_dispatch_bwd(s, *[P] * 4, N, P, N, N, P, N) == UNSUPPORTED
    if T >= 1 << 26:
        assert L.moe_combine_bwd(s, *[P] * 6, *[N] * 5, P, P, N) == UNSUPPORTED
        assert L.moe_combine_bwd_weights(s, *[P] * 6, *[N] * 5, P, P, N) == UNSUPPORTED


def test_router(L):
    for T in (1 << 26, 1 << 31):
        assert L.moe_router(T, 16, 2, 1, P, P, P, N) == UNSUPPORTED
        assert L.moe_router_bwd(T, 16, 2, 1, P, P, P, P, P, N) == UNSUPPORTED


def test_quantisers(L):
    assert L.moe_quant_rows_int8(1 << 26, 8, P, N, P, P, N) == UNSUPPORTED
    assert L.moe_quant_rows_mx(1 << 30, 32, P, N, P, P, N) == UNSUPPORTED
    assert L.moe_quant_rows_fp8(1 << 34, 256, P, N, P, P, N) == UNSUPPORTED
    assert L.moe_quantize_weights_mx(1 << 15, 1024, 1024, P, P, P, P, P, N) == UNSUPPORTED
    assert L.moe_quantize_weights_fp8(1 << 19, 1024, 512, P, P, P, P, N) == UNSUPPORTED
    assert L.moe_quant_cols_fp8(1 << 31, 128, 1, P, P, P, P, N) == UNSUPPORTED
