"""Every kernel that the int8 matrix product chooses from, at sizes that reach it: the name
that the library gives for a size is checked with the result, so a change of the rule that
takes a kernel's sizes away shows here."""
import ctypes
import random

import pytest
import torch

import dispatch_expert_gemm_amd as dm
from few_util import check, linear64, quant_weight, to_int8

gpu = pytest.mark.gpu
DEV = "cuda:0"

ROWS = {
    "k_linear_rows<1, 1, 1, 2, 8>": [(1, 1, 16), (5, 100, 1040)],
    "k_linear_rows<1, 2, 1, 2, 4>": [(7, 4100, 144)],
    "k_linear_rows<1, 1, 2, 2, 8>": [(15, 33, 528)],
    "k_linear_rows<1, 2, 2, 2, 4>": [(12, 4113, 272)],
    "k_linear_rows<2, 1, 2, 2, 8>": [(17, 63, 80)],
    "k_linear_rows<2, 2, 2, 2, 4>": [(25, 4112, 272)],
    "k_linear_rows<3, 1, 2, 2, 8>": [(47, 129, 272)],
    "k_linear_rows<3, 2, 2, 1, 8>": [(45, 4101, 144)],
    "k_linear_rows<4, 1, 2, 2, 8>": [(49, 43, 48), (255, 384, 2064)],
    "k_linear_rows<4, 2, 2, 1, 8>": [(194, 4, 32), (591, 33, 1040), (513, 512, 1024)],
    "k_linear_rows<4, 4, 2, 2, 4>": [(105, 4803, 6496), (112, 4800, 6512)],
}
# of the contraction's 128-byte steps: fewer than the kernel's stages, as many, more; whole and partial last ones
TILES = {
    "k_linear_tiles<64, 128, 2, 4, 128, 3>": [(65, 4781, 16), (66, 4227, 144), (65, 4208, 288), (65, 4181, 400), (518, 2000, 160),
                                              (341, 3051, 784), (500, 4096, 1024)],
    "k_linear_tiles<128, 128, 2, 4, 128, 4>": [(325, 5423, 144), (324, 5685, 272), (326, 5512, 400), (324, 5403, 528),
                                               (2312, 776, 1040)],
    "k_linear_tiles<128, 256, 2, 4, 128, 3>": [(717, 5406, 16), (775, 5063, 144), (649, 5976, 272), (2180, 1793, 400),
                                               (708, 5426, 1040)],
    "k_linear_tiles<256, 256, 2, 4, 128, 2>": [(2243, 4523, 16), (2086, 4875, 144), (2052, 4896, 272), (1930, 5257, 400)],
}
KERNELS = {**ROWS, **TILES}
CASES = [(name, *s) for name, sizes in KERNELS.items() for s in sizes]
# one of each that stages tiles, its columns a multiple of 8 (stored by 16 bytes where the output allows it)
VECTORS = [(name, *next(s for s in sizes if s[1] % 8 == 0)) for name, sizes in TILES.items()]


def make(M, N, K, seed, bias=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    w = quant_weight((torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16))
    return x, w, torch.randn(N, generator=g, device=DEV) if bias else None


@pytest.mark.parametrize("name,M,N,K", CASES)
def test_the_choice(name, M, N, K):
    assert dm.moe_linear_int8_kernel(M, N, K) == name


def test_every_kernel_of_the_rule_is_tested():
    r = random.Random(92)
    size = lambda hi: int(2 ** r.uniform(0, hi))   # noqa: E731
    seen = {dm.moe_linear_int8_kernel(size(14), size(14), 16 * size(9)) for _ in range(50000)}
    seen.add(dm.moe_linear_int8_kernel(1 << 24, 16, 16))
    assert seen == set(KERNELS)


def test_the_name_of_no_kernel():
    assert dm.moe_linear_int8_kernel(0, 8, 16) == ""
    for bad in ((-1, 8, 16), (4, 0, 16), (4, 8, 24), (4, 8, 131088), ((1 << 24) + 1, 8, 16)):
        with pytest.raises(dm.MoeError):
            dm.moe_linear_int8_kernel(*bad)
    assert dm.lib().moe_linear_int8_kernel(4, 8, 16, ctypes.POINTER(ctypes.c_char_p)()) == -1


@gpu
@pytest.mark.parametrize("name,M,N,K", CASES)
def test_product_of_each_kernel(name, M, N, K):
    print(f"[linear int8] {name} M={M} N={N} K={K}", flush=True)
    x, w, b = make(M, N, K, 93, bias=(M + N) % 2 == 0)
    q, s = to_int8(x.float())
    codes, xs = q.to(torch.int8), s[:, 0].float().contiguous()
    v, bound = linear64((codes, xs), w, b)
    check("codes", dm.linear_int8(codes, w, x_scales=xs, bias=b), v, bound)
    check("bf16 rows", dm.linear_int8(x, w, bias=b), v, bound)


@gpu
@pytest.mark.parametrize("name,M,N,K", VECTORS)
@pytest.mark.parametrize("at", [0, 1, 8])
def test_outputs_off_the_vector_boundary_and_nothing_past_them(name, M, N, K, at):
    x, w, b = make(M, N, K, 94)
    q, s = quant_weight(x)
    want = dm.linear_int8(q, w, x_scales=s, bias=b)
    flat = torch.full((M * N + 512,), 3.0, dtype=torch.bfloat16, device=DEV)
    out = flat[at:at + M * N]
    dm.moe_linear_int8(q, s, *w, b, out)
    assert torch.equal(out.view(M, N), want)
    assert (flat[:at] == 3.0).all() and (flat[at + M * N:] == 3.0).all()
    n = dm.moe_linear_int8_workspace_size(M, N, K)
    ws = torch.full((n + 256,), 0xff, dtype=torch.uint8, device=DEV)
    flat.fill_(3.0)
    dm.moe_linear_int8_dynamic(x, *w, b, out, ws[:n])
    assert torch.equal(out.view(M, N), want)
    assert (flat[:at] == 3.0).all() and (flat[at + M * N:] == 3.0).all() and (ws[n:] == 0xff).all()


@gpu
@pytest.mark.parametrize("name,M,N,K", VECTORS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_row_that_is_not_finite_does_not_reach_the_others(name, M, N, K, bad):
    x, w, b = make(M, N, K, 95)
    clean = dm.linear_int8(x, w, bias=b)
    at = M - 2
    x[at, 9] = bad
    out = dm.linear_int8(x, w, bias=b)
    keep = torch.arange(M, device=DEV) != at
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out[at]).any()


@gpu
@pytest.mark.parametrize("name,M,N", [("k_linear_tiles<64, 128, 2, 4, 128, 3>", 4097, 256),
                                      ("k_linear_rows<4, 4, 2, 2, 4>", 4000, 520),
                                      ("k_linear_tiles<128, 128, 2, 4, 128, 4>", 2048, 2044),
                                      ("k_linear_tiles<128, 256, 2, 4, 128, 3>", 2048, 4096),
                                      ("k_linear_tiles<256, 256, 2, 4, 128, 2>", 4096, 4096)])
def test_largest_sums_are_exact(name, M, N):
    """Codes at 127: sums up to 127^2 K, far beyond 2^24."""
    K = 16384
    assert dm.moe_linear_int8_kernel(M, N, K) == name
    xq = torch.full((M, K), 127, dtype=torch.int8, device=DEV)
    wq = torch.full((N, K), 127, dtype=torch.int8, device=DEV)
    wq[1::2] = -127
    wq[5, ::2] = 126
    xq[3, 1::2] = 125
    xs, ws = torch.full((M,), 2.0 ** -12, device=DEV), torch.full((N,), 2.0 ** -9, device=DEV)
    out = dm.linear_int8(xq, (wq, ws), x_scales=xs)
    # the rows are alike but row 3: two of them in 64 bits
    v, bound = linear64((xq[2:4], xs[2:4]), (wq, ws))
    check("largest", out[2:4], v, bound)
    keep = torch.arange(M, device=DEV) != 3
    assert (out[keep] == out[2]).all()


@gpu
@pytest.mark.parametrize("name,M,N,K", VECTORS)
def test_a_captured_call(name, M, N, K):
    x, w, b = make(M, N, K, 96)
    dm.linear_int8(x, w, bias=b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = dm.linear_int8(x, w, bias=b)
    for seed in (97, 98, 99):
        x.copy_(make(M, N, K, seed)[0])
        eager = dm.linear_int8(x, w, bias=b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
