"""The int8 matrix product (moe_linear_int8, moe_linear_int8_dynamic, linear_int8) against the
plain 64-bit form, element by element."""
import ctypes

import pytest
import torch

import dispatch_expert_gemm_amd as dm
from few_util import check, linear64, quant_weight, to_int8

gpu = pytest.mark.gpu
DEV = "cuda:0"


def make(M, N, K, seed, bias=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    w = quant_weight((torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16))
    b = torch.randn(N, generator=g, device=DEV) if bias else None
    return x, w, b


SIZES = [(1, 1, 16), (1, 7168, 2048), (2, 17, 48), (3, 16, 64), (5, 100, 1040), (15, 33, 512), (16, 64, 528), (17, 63, 80),
         (31, 250, 16), (33, 1, 4096), (47, 128, 272), (64, 512, 128), (65, 96, 144), (127, 129, 1040), (128, 256, 512),
         (129, 255, 400), (200, 1000, 96), (255, 384, 2048), (256, 256, 256), (300, 777, 336), (513, 512, 1024),
         (1000, 130, 64), (1, 40, 131072), (70, 300, 16400), (1, 8200, 96), (2, 300, 8192), (1, 64, 8208), (4, 4100, 64),
         (12, 4100, 272), (20, 4096, 144), (25, 4112, 272), (40, 4080, 400), (48, 4100, 144), (60, 4090, 272), (64, 4112, 272),
         (250, 510, 272), (2000, 128, 144), (500, 7100, 1040), (1001, 7160, 1040), (2041, 8190, 1040), (2048, 8192, 528)]


@gpu
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_against_64_bits(M, N, K):
    print(f"[linear int8] M={M} N={N} K={K}", flush=True)
    x, w, b = make(M, N, K, 31, bias=(M + N) % 2 == 0)
    q, s = to_int8(x.float())
    v, bound = linear64((q, s[:, 0].float()), w, b)
    out = dm.linear_int8(q.to(torch.int8), w, x_scales=s[:, 0].float().contiguous(), bias=b)
    check("codes", out, v, bound)
    check("bf16 rows", dm.linear_int8(x, dm.Int8Weights(*w), bias=b), v, bound)


@gpu
@pytest.mark.parametrize("M", [1, 40, 200])
def test_largest_sums_are_exact(M):
    """Every code at 127: sums up to 127^2 K, far beyond 2^24."""
    N, K = 48, 131072 if M == 1 else 16384
    xq = torch.full((M, K), 127, dtype=torch.int8, device=DEV)
    wq = torch.full((N, K), 127, dtype=torch.int8, device=DEV)
    wq[1::2] = -127
    wq[5, ::2] = 126
    xs, ws = torch.full((M,), 2.0 ** -12, device=DEV), torch.full((N,), 2.0 ** -9, device=DEV)
    v, bound = linear64((xq, xs), (wq, ws))
    check("largest", dm.linear_int8(xq, (wq, ws), x_scales=xs), v, bound)


@gpu
@pytest.mark.parametrize("M", [3, 70, 300])
def test_rows_of_zeros_tiny_and_large_values(M):
    x, w, _ = make(M, 96, 256, 32)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e30
    x[2, ::3] = 0
    if M > 3:
        x[7] = 0
        x[7, 5] = 2.0 ** -133        # the smallest bf16: a zero beside it keeps code 0
    q, s = to_int8(x.float())
    v, bound = linear64((q, s[:, 0]), w)
    # 2^-133 / 127 lies below the normal range: its scale is rounded to 2^-149, and so is the product
    bound = bound + 127 * 127 * 256 * 2.0 ** -149
    check("rows", dm.linear_int8(x, w), v, bound)


@gpu
@pytest.mark.parametrize("K", [256, 16400])
@pytest.mark.parametrize("M", [2, 40, 300])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_row_that_is_not_finite_does_not_reach_the_others(bad, M, K):
    x, w, b = make(M, 96, K, 41)
    clean = dm.linear_int8(x, w, bias=b)
    x[1, 17] = bad
    out = dm.linear_int8(x, w, bias=b)
    keep = [m for m in range(M) if m != 1]
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out[1]).any()


@gpu
@pytest.mark.parametrize("M,N,K", [(3, 140000, 16384), (40, 140000, 16384), (300000, 16, 8192), (70000, 32768, 32)])
def test_offsets_past_32_bits(M, N, K):
    """Weights, rows and outputs of more than 2^31 bytes or elements: the last rows and columns."""
    g = torch.Generator(device=DEV).manual_seed(42)
    wq = torch.zeros(N, K, dtype=torch.int8, device=DEV)
    wq[-200:] = torch.randint(-127, 128, (min(200, N), K), generator=g, device=DEV, dtype=torch.int8)
    xq = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    xq[-200:] = torch.randint(-127, 128, (min(200, M), K), generator=g, device=DEV, dtype=torch.int8)
    xs, ws = torch.rand(M, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    out = dm.linear_int8(xq, (wq, ws), x_scales=xs)
    v, bound = linear64((xq[-200:], xs[-200:]), (wq[-200:], ws[-200:]))
    check("last", out[-200:, -200:], v, bound)
    assert (out[:-200, :200] == 0).all() and (out[:200, :-200] == 0).all()


@gpu
def test_leading_dimensions_and_no_rows():
    x, w, b = make(24, 80, 96, 33)
    want = dm.linear_int8(x, w, bias=b)
    assert torch.equal(dm.linear_int8(x.view(2, 3, 4, 96), w, bias=b).view(24, 80), want)
    assert torch.equal(dm.linear_int8(x[5], w, bias=b), dm.linear_int8(x[5:6], w, bias=b)[0])
    assert dm.linear_int8(x[:0], w).shape == (0, 80)
    assert dm.linear_int8(x.view(2, 12, 96)[:, :0], w).shape == (2, 0, 80)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 200, 512), (40, 130, 80), (300, 260, 1040)])
def test_nothing_is_written_past_the_output(M, N, K):
    x, w, b = make(M, N, K, 34)
    q, s = quant_weight(x)     # rows by the same rule
    out = torch.full((M * N + 512,), 3.0, dtype=torch.bfloat16, device=DEV)
    dm.moe_linear_int8(q, s, *w, b, out)
    torch.cuda.synchronize()
    assert torch.equal(out[:M * N].view(M, N), dm.linear_int8(q, w, x_scales=s, bias=b))
    assert (out[M * N:] == 3.0).all()
    n = dm.moe_linear_int8_workspace_size(M, N, K)
    ws = torch.full((n + 256,), 0xff, dtype=torch.uint8, device=DEV)
    out.fill_(3.0)
    dm.moe_linear_int8_dynamic(x, *w, b, out, ws[:n])
    torch.cuda.synchronize()
    assert torch.equal(out[:M * N].view(M, N), dm.linear_int8(q, w, x_scales=s, bias=b))
    assert (out[M * N:] == 3.0).all() and (ws[n:] == 0xff).all()


@gpu
@pytest.mark.parametrize("M", [2, 40, 300])
def test_an_output_off_the_vector_boundary(M):
    x, w, b = make(M, 264, 512, 40)
    flat = torch.full((M * 264 + 9,), 3.0, dtype=torch.bfloat16, device=DEV)
    out = flat[1:1 + M * 264]
    q, s = quant_weight(x)
    dm.moe_linear_int8(q, s, *w, b, out)
    assert torch.equal(out.view(M, 264), dm.linear_int8(x, w, bias=b))
    assert flat[0] == 3.0 and (flat[1 + M * 264:] == 3.0).all()


@gpu
@pytest.mark.parametrize("M", [2, 48, 260])
def test_another_stream_and_a_captured_call(M):
    x, w, b = make(M, 272, 512, 35)
    want = dm.linear_int8(x, w, bias=b)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = dm.linear_int8(x, w, bias=b, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        out = dm.linear_int8(x, w, bias=b)
    for seed in (36, 37, 38):
        x.copy_(make(M, 272, 512, seed)[0])
        eager = dm.linear_int8(x, w, bias=b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@gpu
def test_refusals_of_tensors():
    x, w, b = make(4, 32, 64, 39)
    q, s = dm.quant_rows_int8(x)

    def refused(x, w, **kw):
        with pytest.raises(dm.MoeError):
            dm.linear_int8(x, w, **kw)

    refused(x.cpu(), w)
    refused(x.float(), w)
    refused(x, w, x_scales=s)                                  # scales go with codes
    refused(q, w)
    refused(x.t().contiguous().t(), w)
    refused(x[:, :48].contiguous(), w)
    refused(x, (w[0][:, :8].contiguous(), w[1]))
    refused(x, (w[0].view(1, 32, 64), w[1]))
    refused(x, (w[0], w[1][:31].contiguous()))
    refused(x, w, bias=b.double())
    refused(x, w, bias=b[:16].contiguous())
    refused(q, w, x_scales=s[:3].contiguous())
    flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device=DEV)
    refused(flat[1:].view(4, 64), w)                           # not on a 16-byte boundary
    refused(torch.zeros(4, 24, dtype=torch.bfloat16, device=DEV), (w[0].view(-1)[:32 * 24].view(32, 24), w[1]))


def test_refusals_of_the_entries():
    L = dm.lib()
    P = lambda v=0x1000: ctypes.c_void_p(v)   # noqa: E731  (never read: the checks come first)
    N = None
    NULL, SHAPE, UNSUP, WS = -1, -2, -5, -6

    def lin(M=4, n=32, K=64, xq=P(), xs=P(), wq=P(), ws=P(), out=P()):
        return L.moe_linear_int8(M, n, K, xq, xs, wq, ws, N, out, N)

    assert lin(M=-1) == SHAPE and lin(n=0) == SHAPE and lin(K=0) == SHAPE and lin(K=24) == SHAPE
    assert lin(K=131088) == UNSUP and lin(M=(1 << 24) + 1) == UNSUP and lin(n=(1 << 24) + 1) == UNSUP
    for a in ("xq", "xs", "wq", "ws", "out"):
        assert lin(**{a: N}) == NULL, a
    assert lin(xq=P(0x1008)) == SHAPE and lin(wq=P(0x1004)) == SHAPE
    assert lin(M=0, xq=N, xs=N, out=N) == 0
    n = ctypes.c_size_t()
    assert L.moe_linear_int8_workspace_size(4, 32, 60, ctypes.byref(n)) == SHAPE
    assert L.moe_linear_int8_workspace_size(4, 32, 64, N) == NULL
    assert L.moe_linear_int8_workspace_size(4, 32, 64, ctypes.byref(n)) == 0 and n.value >= 4 * 64 + 16

    def dyn(x=P(), ws=P(), nb=1 << 20, M=4):
        return L.moe_linear_int8_dynamic(M, 32, 64, x, P(), P(), N, P(), ws, nb, N)

    assert dyn(x=N) == NULL and dyn(ws=N) == WS and dyn(nb=16) == WS and dyn(x=P(0x1002)) == SHAPE
    assert dyn(M=0, x=N, ws=N, nb=0) == 0
