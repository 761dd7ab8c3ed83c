"""GPU tests of the checkpoints in 8 bits: SwiGLU with its [G | U] kept, the combine with its rows kept, against the
64-bit forms on the values that the rule keeps."""
import pytest
import torch

import dispatch_expert_gemm_amd as dm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


def rule(v):
    """(codes, scales) of rows (R, W) by the rule's own 32-bit steps, on the CPU."""
    v = v.detach().cpu().float()
    R, W = v.shape
    nb = -(-W // 32)
    pad = torch.zeros(R, nb * 32)
    pad[:, :W] = v
    b = pad.view(R, nb, 32)
    amax = b.abs().amax(-1)
    s = (amax / 127).bfloat16()
    s = torch.where(s.float() < 2.0 ** -126, torch.zeros_like(s), s)
    s = torch.where(torch.isfinite(b).all(-1), s, torch.full_like(s, float("nan")))
    inv = torch.where(s.float() > 0, 1.0 / s.float(), torch.zeros_like(amax))
    q = (b * inv[..., None]).round()
    q = torch.where(torch.isfinite(s.float())[..., None] & (s.float() > 0)[..., None], q, torch.zeros_like(q))
    assert q.abs().max() <= 127 if q.numel() else True
    return q.view(R, nb * 32)[:, :W].to(torch.int8), s


def kept(codes, scales):
    s = scales.float().repeat_interleave(32, 1)[:, :codes.shape[1]]
    return codes.double() * s.double()


def halves(gu):
    F = gu.shape[1] // 2
    (a, s), (b, t) = rule(gu[:, :F]), rule(gu[:, F:])
    return torch.cat([a, b], 1), torch.cat([s, t], 1)


def same(a, b):
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    if a.is_floating_point():
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        a, b = torch.nan_to_num(a), torch.nan_to_num(b)
    assert torch.equal(a, b)


def near(name, got, want, mag):
    """bf16 results: half a step of the rounding, and 2^-18 of `mag`, the size of the terms: exp and the reciprocal are
    within 2^-22 and its argument's rounding |g| 2^-24, |g| < 60 here."""
    got, want = got.detach().cpu().double(), want.double()
    bound = BF16_HALF * want.abs() + 2.0 ** -18 * (1 + BF16_HALF) * mag + 2.0 ** -133
    bad = (got - want).abs() > bound
    assert not bad.any(), f"{name}: {int(bad.sum())} off, worst {float(((got - want).abs() / bound).max())}"


def swiglu64(g, u, d=None):
    sg = 1 / (1 + torch.exp(-g))
    h = g * sg * u
    if d is None:
        return h, h.abs()
    dg, du = d * u * sg * (1 + g * (1 - sg)), d * g * sg
    return torch.cat([dg, du], 1), torch.cat([(d * u).abs() * sg * (1 + (g * (1 - sg)).abs()), du.abs()], 1)


def gate_up(R, F, seed, std=1.0):
    return (torch.randn(R, 2 * F, generator=torch.Generator().manual_seed(seed)) * std).bfloat16()


def check_swiglu(gu, seed=0):
    R, F = gu.shape[0], gu.shape[1] // 2
    x = gu.to(DEV)
    d = (torch.randn(R, F, generator=torch.Generator().manual_seed(seed + 50)) * 0.3).bfloat16()
    h = torch.empty(R, F, dtype=torch.bfloat16, device=DEV)
    codes, scales = dm.checkpoint_buffers(R, F, DEV, halves=2)
    dm.moe_swiglu_checkpoint_fwd(x, h, codes, scales)
    qc, qs = halves(gu)
    same(codes, qc)
    same(scales, qs)
    near("h", h, *swiglu64(gu[:, :F].double(), gu[:, F:].double()))
    v = kept(qc[:, :F], qs[:, :qs.shape[1] // 2]), kept(qc[:, F:], qs[:, qs.shape[1] // 2:])
    grad = torch.empty_like(x)
    dm.moe_swiglu_checkpoint_bwd(codes, scales, d.to(DEV), grad)
    near("grad", grad, *swiglu64(*v, d.double()))
    # and through autograd
    leaf = x.clone().requires_grad_()
    out = dm.swiglu_checkpoint(leaf)
    same(out.detach(), h)
    same(torch.autograd.grad(out, leaf, d.to(DEV))[0], grad)


@pytest.mark.parametrize("F", [1, 2, 7, 8, 31, 32, 33, 40, 64, 96, 100, 480, 1000, 1001, 2048])
@pytest.mark.parametrize("R", [1, 3, 70])
def test_swiglu_sizes(R, F):
    check_swiglu(gate_up(R, F, R * 1000 + F, 3.0), F)


@pytest.mark.parametrize("R,F", [(2000, 480), (5, 14336), (4099, 32), (300, 1001)])
def test_swiglu_more_rows(R, F):
    check_swiglu(gate_up(R, F, F, 2.0), F)


def test_every_scale_and_every_tie():
    """Every bf16 magnitude as a block's largest value, with values at and beside the steps' borders."""
    top = torch.arange(0x0000, 0x7f80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    R = top.numel()
    frac = torch.rand(R, 64, generator=torch.Generator().manual_seed(1)) * 2 - 1
    frac[:, 1::4] = (torch.arange(16) * 8 + 0.5) / 127 * 1.0  # near the borders between two codes
    v = (frac * top.float()[:, None]).bfloat16()
    v[:, 0] = top
    v[:, 37] = -top
    codes, scales = dm.checkpoint_buffers(R, 32, DEV, halves=2)
    dm.moe_swiglu_checkpoint_fwd(v.to(DEV), torch.empty(R, 32, dtype=torch.bfloat16, device=DEV), codes, scales)
    qc, qs = halves(v)
    same(scales, qs)
    same(codes, qc)
    # each kept value is within half a step (the scales' own rounding leaves no code past 127)
    x, s = v.double(), qs.double().repeat_interleave(32, 1)
    err = (kept(qc, qs) - x).abs()
    assert (err <= s / 2 + 1.5e-36).all()


def test_the_rule_of_32_bits_is_the_division():
    """amax times fp32(1/127) rounds to the same bf16 as amax / 127, for every mantissa (CPU arithmetic of the kernel)."""
    a = torch.arange(128, 256).float()
    assert torch.equal((a * (torch.tensor(1.0) / 127)).bfloat16(), (a.double() / 127).bfloat16())


@pytest.mark.parametrize("F", [64, 50])
def test_infinities_and_nans_mark_their_block_only(F):
    gu = gate_up(6, F, 3)
    gu[0, 5], gu[1, F + 40], gu[2, 33], gu[3, 0] = float("inf"), -float("inf"), float("nan"), -float("nan")
    x = gu.to(DEV)
    codes, scales = dm.checkpoint_buffers(6, F, DEV, halves=2)
    h = torch.empty(6, F, dtype=torch.bfloat16, device=DEV)
    dm.moe_swiglu_checkpoint_fwd(x, h, codes, scales)
    qc, qs = halves(gu)
    same(codes, qc)
    same(scales, qs)
    assert int(torch.isnan(scales.float()).sum()) == 4
    grad = torch.empty_like(x)
    bad = torch.isnan(scales.float()).cpu().view(6, 2, -1).repeat_interleave(32, 2)[:, :, :F].reshape(6, 2 * F)
    dm.moe_swiglu_checkpoint_bwd(codes, scales, torch.ones(6, F, dtype=torch.bfloat16, device=DEV), grad)
    either = bad[:, :F] | bad[:, F:]
    assert torch.equal(torch.isnan(grad[:, :F].float()).cpu(), either)      # dG takes both
    assert torch.equal(torch.isnan(grad[:, F:].float()).cpu(), bad[:, :F])  # dU takes G alone
    want = torch.nn.functional.silu(gu[:, :F].double()) * gu[:, F:].double()
    assert torch.equal(torch.isfinite(h.float()).cpu(), torch.isfinite(want))


def test_far_gates():
    """Gates where the sigmoid is 0 or 1 in fp32, up to the type's largest."""
    g = torch.tensor([-3e38, -1e30, -200.0, -90.0, -88.0, -20.0, 0.0, 20.0, 88.0, 200.0, 1e30, 2e38]).bfloat16()
    gu = torch.zeros(12, 64).bfloat16()
    gu[:, :32], gu[:, 32:] = g[:, None], 0.5
    d = torch.full((12, 32), 0.25).bfloat16()
    x = gu.to(DEV).requires_grad_()
    h = dm.swiglu_checkpoint(x)
    grad, = torch.autograd.grad(h, x, d.to(DEV))
    assert torch.isfinite(h.float()).all() and torch.isfinite(grad.float()).all()
    grad = grad.cpu().double()
    assert (grad[:4, :32].abs() < 1e-30).all() and (grad[9:, :32] == 0.125).all()


@pytest.mark.parametrize("F", [96, 33])
@pytest.mark.parametrize("n", [0, 1, 7, 64, 99])
def test_rows_behind_the_last_are_left(F, n):
    R = 64
    gu, nrows = gate_up(R, F, n).to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    used = min(n, R)
    codes, scales = dm.checkpoint_buffers(R, F, DEV, halves=2)
    h, grad = (torch.empty(R, w, dtype=torch.bfloat16, device=DEV) for w in (F, 2 * F))
    for t in (codes, scales, h, grad):
        t.fill_(9)
    dm.moe_swiglu_checkpoint_fwd(gu, h, codes, scales, nrows=nrows)
    dm.moe_swiglu_checkpoint_bwd(codes, scales, gu[:, :F].contiguous(), grad, nrows=nrows)
    for t in (codes, scales, h, grad):
        assert (t[used:] == 9).all()
    if used:
        qc, qs = halves(gu[:used])
        same(codes[:used], qc)
        same(scales[:used], qs)


def test_misaligned_rows():
    """The same bits from matrices that begin on 2 bytes."""
    R, F = 37, 96
    gu = gate_up(R, F, 5).to(DEV)

    def odd(shape, dtype):
        n = 1
        for k in shape:
            n *= k
        return torch.empty(n + 1, dtype=dtype, device=DEV)[1:].view(shape)

    x = odd((R, 2 * F), torch.bfloat16).copy_(gu)
    want = [torch.empty(R, F, dtype=torch.bfloat16, device=DEV), *dm.checkpoint_buffers(R, F, DEV, halves=2)]
    got = [odd(t.shape, t.dtype) for t in want]
    dm.moe_swiglu_checkpoint_fwd(gu, *want)
    dm.moe_swiglu_checkpoint_fwd(x, *got)
    for a, b in zip(want, got):
        same(a, b)
    d = gu[:, F:].contiguous()
    g1, g2 = torch.empty_like(gu), odd(gu.shape, gu.dtype)
    dm.moe_swiglu_checkpoint_bwd(want[1], want[2], d, g1)
    dm.moe_swiglu_checkpoint_bwd(got[1], got[2], d, g2)
    assert float((g1.float() - g2.float()).abs().max()) <= BF16_HALF * 2 * float(g1.float().abs().max())


def test_swiglu_leading_dimensions_strides_and_none():
    gu = gate_up(24, 64, 2).to(DEV)
    x = gu.view(2, 3, 4, 128).requires_grad_()
    h = dm.swiglu_checkpoint(x)
    assert h.shape == (2, 3, 4, 64)
    g, = torch.autograd.grad(h, x, torch.ones_like(h))
    flat = gu.clone().requires_grad_()
    g2, = torch.autograd.grad(dm.swiglu_checkpoint(flat), flat, torch.ones(24, 64, dtype=torch.bfloat16, device=DEV))
    same(g.view(24, 128), g2)
    wide = torch.randn(24, 200, device=DEV).bfloat16().requires_grad_()
    part = wide[:, 3:131]
    g3, = torch.autograd.grad(dm.swiglu_checkpoint(part).sum(), wide)  # an expanded gradient
    flat = part.detach().clone().requires_grad_()
    g4, = torch.autograd.grad(dm.swiglu_checkpoint(flat).sum(), flat)
    same(g3[:, 3:131], g4)
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    h = dm.swiglu_checkpoint(empty)
    assert h.shape == (0, 32) and torch.autograd.grad(h.sum(), empty)[0].shape == (0, 64)


def test_swiglu_gradient_against_differences():
    """On values that the codes hold exactly the gradient is the function's own."""
    g = torch.Generator().manual_seed(4)
    q = torch.randint(-127, 128, (4, 128), generator=g)
    q[:, ::32] = 127
    gu = (q.double() / 32)
    x = gu.bfloat16().to(DEV).requires_grad_()
    assert torch.equal(x.detach().cpu().double(), gu)
    d = torch.randn(4, 64, generator=g).bfloat16()
    grad, = torch.autograd.grad(dm.swiglu_checkpoint(x), x, d.to(DEV))
    e = 1e-5
    up, down = ((swiglu64(gu[:, :64] + a, gu[:, 64:] + b)[0] - swiglu64(gu[:, :64] - a, gu[:, 64:] - b)[0]) / (2 * e)
                * d.double() for a, b in ((e, 0), (0, e)))
    want = torch.cat([up, down], 1)
    err = (grad.cpu().double() - want).abs()
    assert (err <= BF16_HALF * want.abs() + 1e-5).all()


def test_kept_memory_of_swiglu():
    """1.0625 bytes a value of [G | U], and nothing else."""
    gu = gate_up(4096, 480, 1).to(DEV).requires_grad_()
    held = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: held.append(t.numel() * t.element_size()) or t, lambda t: t):
        h = dm.swiglu_checkpoint(gu)
    assert sum(held) == 4096 * 960 * 17 // 16
    del h


def test_swiglu_streams_and_captured():
    R, F = 500, 480
    gu, d = gate_up(R, F, 1).to(DEV), gate_up(R, F, 2)[:, :F].contiguous().to(DEV)

    def step(x):
        x = x.detach().requires_grad_()
        h = dm.swiglu_checkpoint(x)
        return h.detach(), torch.autograd.grad(h, x, d)[0]

    want = step(gu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(gu)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        same(a, b)
    static = gu.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(static)
    for seed in (5, 6, 7):
        new = gate_up(R, F, seed).to(DEV)
        static.copy_(new)
        graph.replay()
        eager = step(new)
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            same(a, b)


def test_swiglu_differentiable_once():
    x = gate_up(6, 32, 1).to(DEV).requires_grad_()
    g, = torch.autograd.grad(dm.swiglu_checkpoint(x).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        g.float().square().sum().backward()
    with torch.no_grad():
        assert not dm.swiglu_checkpoint(x).requires_grad


def test_swiglu_refusals():
    x = gate_up(6, 32, 1).to(DEV)
    for bad, match in ((x.float(), "gate_up must be torch.bfloat16"), (x[:, :63], "shape"), (x[:, :0], "shape"),
                       (x[0, 0], "shape")):
        with pytest.raises(dm.MoeError, match=match):
            dm.swiglu_checkpoint(bad)
    codes, scales = dm.checkpoint_buffers(6, 32, DEV, halves=2)
    h = torch.empty(6, 32, dtype=torch.bfloat16, device=DEV)
    for f in (lambda: dm.moe_swiglu_checkpoint_fwd(x, h, codes[:5], scales),
              lambda: dm.moe_swiglu_checkpoint_fwd(x, h, codes, scales[:5]),
              lambda: dm.moe_swiglu_checkpoint_fwd(x, h, codes, scales.float()),
              lambda: dm.moe_swiglu_checkpoint_fwd(x, None, codes, scales),
              lambda: dm.moe_swiglu_checkpoint_fwd(x, h[:5], codes, scales),
              lambda: dm.moe_swiglu_checkpoint_fwd(x.t(), h, codes, scales),
              lambda: dm.moe_swiglu_checkpoint_bwd(codes, scales, x[:, :32], x),
              lambda: dm.moe_swiglu_checkpoint_bwd(codes, scales, x[:3, :32].contiguous(), x),
              lambda: dm.moe_swiglu_checkpoint_bwd(codes, scales, h, x[:5]),
              lambda: dm.moe_swiglu_checkpoint_bwd(codes, scales, h, x, nrows=torch.ones(1, device=DEV))):
        with pytest.raises(dm.MoeError):
            f()


# ----------------------------------------------------------------------------- combine


def routing(T, E, K, special, masked, seed):
    g = torch.Generator().manual_seed(seed)
    Z, C, Q = (2, 1, 2) if special else (0, 0, 0)
    ids = E + Z + C + Q
    idx = torch.rand(T, ids, generator=g).topk(K)[1].to(torch.int32) if T else torch.zeros(0, K, dtype=torch.int32)
    w = torch.randn(T, K, generator=g)
    mask = None
    if masked:
        mask = torch.rand(T, K, generator=g) >= 0.3
        mask[::4] = False  # tokens without a slot
        mask = mask.to(torch.uint8)
    return idx, w, mask, (Z, C, Q)


@pytest.mark.parametrize("T,H,E,K,special,masked,shared", [
    (1, 8, 2, 1, False, False, False), (5, 24, 4, 2, True, True, True), (33, 40, 8, 3, True, False, False),
    (64, 1536, 64, 2, False, False, False), (130, 1000, 16, 8, True, True, True), (40, 2048, 32, 8, False, True, True),
    (17, 7168, 32, 8, True, True, True), (9, 4096, 64, 16, True, True, False), (50, 520, 3, 3, False, False, True),
    (0, 64, 4, 2, False, False, False)])
def test_combine(T, H, E, K, special, masked, shared):
    idx, w, mask, (Z, C, Q) = routing(T, E, K, special, masked, T + H)
    g = torch.Generator().manual_seed(H)
    nd = 2 if masked else 0
    shape = dm.make_shape(T, H, K, E, zero_expert_num=Z, copy_expert_num=C, const_expert_num=Q, mask_ndim=nd)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    y, x, d = r(shape.capacity, H), r(T, H), r(T, H)
    sx = r(T, H) if shared else None
    consts = [r(Q, H) for _ in range(3)] if Q else [None] * 3
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    idx, w, mask, y, x, d, sx = (dev(t) for t in (idx, w, mask, y, x, d, sx))
    consts = [dev(t) for t in consts]
    route = dm.route(shape, idx, mask)
    args = (idx, w, route.assist_info_for_combine, route.ep_recv_counts, mask)
    out, want = torch.empty_like(x), torch.empty_like(x)
    codes, scales = dm.checkpoint_buffers(shape.capacity, H, DEV)
    codes.fill_(99)
    scales.fill_(99)
    dm.moe_combine_checkpoint(shape, y, *args, sx, x, *consts, out, codes, scales)
    dm.moe_combine(shape, y, *args, sx, x, *consts, want)
    same(out, want)  # bit for bit the plain combine
    rows = int(route.ep_recv_counts[-1]) if T else 0
    qc, qs = rule(y)
    same(codes[:rows], qc[:rows])
    same(scales[:rows], qs[:rows])
    assert (codes[rows:] == 99).all() and (scales[rows:] == 99).all()
    gw, gw2 = torch.empty_like(w), torch.empty_like(w)
    roww = torch.full((shape.capacity,), 5.0, device=DEV)
    dm.moe_combine_bwd_weights_checkpoint(shape, d, codes, scales, *args, x, *consts, gw, roww)
    dm.moe_combine_bwd_weights_checkpoint(shape, d, codes, scales, *args, x, *consts, gw2)
    same(gw, gw2)
    # 64 bits on the kept values; the bound counts one 2^-24 for each of a lane's sums, the butterfly's and the product
    slot = route.assist_info_for_combine[:T * K].cpu().view(T, K)
    v = torch.zeros(T, K, H, dtype=torch.float64)
    k64 = kept(qc, qs)
    for t in range(T):
        for k in range(K):
            c = int(slot[t, k])
            if c >= 0:
                v[t, k] = k64[c]
                assert float(roww[c]) == float(w[t, k])
            elif c == -2:
                v[t, k] = x[t].cpu().double()
            elif c <= -3:
                a1, a2, cv = (t_[-c - 3].cpu().double() for t_ in consts)
                v[t, k] = a1 * x[t].cpu().double() + a2 * cv
    assert (roww[rows:] == 5).all()
    prod = v * d.cpu().double()[:, None]
    bound = (H / 64 + 8 + 4) * 2.0 ** -24 * prod.abs().sum(-1) * 2
    assert ((gw.cpu().double() - prod.sum(-1)).abs() <= bound + 1e-30).all()


def test_combine_rows_that_are_not_finite():
    T, H, E, K = 12, 96, 4, 2
    idx, w, _, _ = routing(T, E, K, False, False, 1)
    shape = dm.make_shape(T, H, K, E)
    y = torch.randn(T * K, H, generator=torch.Generator().manual_seed(1)).bfloat16()
    y[3, 40], y[5, 95] = float("nan"), float("inf")
    idx, w, y = idx.to(DEV), w.to(DEV), y.to(DEV)
    route = dm.route(shape, idx)
    args = (idx, w, route.assist_info_for_combine, route.ep_recv_counts, None)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    want = torch.empty_like(out)
    codes, scales = dm.checkpoint_buffers(T * K, H, DEV)
    dm.moe_combine_checkpoint(shape, y, *args, None, None, None, None, None, out, codes, scales)
    dm.moe_combine(shape, y, *args, None, None, None, None, None, want)
    same(out, want)
    qc, qs = rule(y)
    same(codes, qc)
    same(scales, qs)
    gw = torch.empty_like(w)
    dm.moe_combine_bwd_weights_checkpoint(shape, torch.ones_like(out), codes, scales, *args, None, None, None, None, gw)
    slots = route.assist_info_for_combine[:T * K].view(T, K)
    assert torch.equal(torch.isnan(gw), (slots == 3) | (slots == 5))


def test_combine_refusals_streams_and_captured():
    T, H, E, K = 20, 96, 4, 2
    idx, w, mask, _ = (t if t is None or isinstance(t, tuple) else t.to(DEV) for t in routing(T, E, K, False, True, 1))
    shape = dm.make_shape(T, H, K, E, mask_ndim=2)
    y = torch.randn(T * K, H, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    route = dm.route(shape, idx, mask)
    none = [None] * 5
    codes, scales = (t.zero_() for t in dm.checkpoint_buffers(T * K, H, DEV))  # (rows of masked slots are not written)
    out, gw = torch.empty(T, H, dtype=torch.bfloat16, device=DEV), torch.empty_like(w)

    def fwd(stream=None, **kw):
        a = dict(y=y, idx=idx, w=w, assist=route.assist_info_for_combine, counts=route.ep_recv_counts, mask=mask, out=out,
                 codes=codes, scales=scales)
        a.update(kw)
        dm.moe_combine_checkpoint(shape, a["y"], a["idx"], a["w"], a["assist"], a["counts"], a["mask"], *none, a["out"],
                                  a["codes"], a["scales"], stream=stream)

    def bwd(stream=None, **kw):
        a = dict(d=out, codes=codes, scales=scales, idx=idx, w=w, assist=route.assist_info_for_combine,
                 counts=route.ep_recv_counts, mask=mask, gw=gw, rw=None)
        a.update(kw)
        dm.moe_combine_bwd_weights_checkpoint(shape, a["d"], a["codes"], a["scales"], a["idx"], a["w"], a["assist"],
                                              a["counts"], a["mask"], None, None, None, None, a["gw"], a["rw"],
                                              stream=stream)

    fwd()
    bwd()
    want = out.clone(), codes.clone(), scales.clone(), gw.clone()
    for f, names in ((fwd, ("y", "idx", "w", "assist", "counts", "out", "codes", "scales")),
                     (bwd, ("d", "codes", "scales", "idx", "w", "assist", "counts", "gw"))):
        for name in names:
            t = dict(y=y, d=out, idx=idx, w=w, assist=route.assist_info_for_combine, counts=route.ep_recv_counts, out=out,
                     codes=codes, scales=scales, gw=gw)[name]
            for bad in (None, 3, t.cpu(), t.double(), t.flatten()[:-1], torch.stack([t, t], -1)[..., 0]):
                with pytest.raises(dm.MoeError):
                    f(**{name: bad})
        with pytest.raises(dm.MoeError):
            f(mask=mask.float())
        f(mask=mask.bool())
    with pytest.raises(dm.MoeError):
        bwd(rw=gw.flatten()[:-1])
    for a, b in zip((out, codes, scales, gw), want):
        same(a, b)
    side = torch.cuda.Stream()
    for t in (out, codes, scales, gw):
        t.zero_()
    torch.cuda.synchronize()
    fwd(side)
    bwd(side)
    side.synchronize()
    for a, b in zip((out, codes, scales, gw), want):
        same(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd()
        bwd()
    for seed in (2, 3, 4):
        y.copy_(torch.randn(T * K, H, generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        got = out.clone(), codes.clone(), scales.clone(), gw.clone()
        fwd()
        bwd()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, codes, scales, gw)):
            same(a, b)


# ----------------------------------------------------------------------------- large


def test_swiglu_past_32_bit_offsets():
    """2.3e9 codes, 4.6 GB of gate_up: the first and the last rows."""
    R, F = 1_120_000, 1024
    part = gate_up(1000, F, 1).to(DEV)
    gu = part.repeat(R // 1000, 1)
    h = torch.empty(R, F, dtype=torch.bfloat16, device=DEV)
    codes, scales = dm.checkpoint_buffers(R, F, DEV, halves=2)
    dm.moe_swiglu_checkpoint_fwd(gu, h, codes, scales)
    d = h  # (any gradient: its last rows repeat as well)
    grad = torch.empty_like(gu)
    dm.moe_swiglu_checkpoint_bwd(codes, scales, d, grad)
    for t in (h, codes, scales, grad):
        same(t[-1000:], t[:1000])
    qc, qs = halves(part.cpu())
    same(codes[-1000:], qc)
    same(scales[-1000:], qs)


def test_combine_past_32_bit_offsets():
    T, H, E, K = 40000, 7168, 8, 8
    shape = dm.make_shape(T, H, K, E)
    y = torch.randn(2000, H, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV).repeat(T * K // 2000, 1)
    idx = torch.arange(K, dtype=torch.int32, device=DEV).repeat(T, 1)
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(2)).to(DEV)
    route = dm.route(shape, idx)
    args = (idx, w, route.assist_info_for_combine, route.ep_recv_counts, None)
    out, want = (torch.empty(T, H, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    codes, scales = dm.checkpoint_buffers(T * K, H, DEV)
    dm.moe_combine_checkpoint(shape, y, *args, None, None, None, None, None, out, codes, scales)
    dm.moe_combine(shape, y, *args, None, None, None, None, None, want)
    assert torch.equal(out, want)
    same(codes[-2000:], codes[:2000])
    same(scales[-2000:], scales[:2000])
    qc, qs = rule(y[-50:])
    same(codes[-50:], qc)
    same(scales[-50:], qs)
    gw = torch.empty_like(w)
    dm.moe_combine_bwd_weights_checkpoint(shape, out, codes, scales, *args, None, None, None, None, gw)
    c = int(route.assist_info_for_combine[T * K - 1])
    p = kept(codes[c:c + 1].cpu(), scales[c:c + 1].cpu())[0] * out[T - 1].cpu().double()
    assert abs(float(gw[T - 1, K - 1]) - float(p.sum())) <= (H / 64 + 12) * 2.0 ** -23 * float(p.abs().sum())


def test_combine_of_more_tokens_than_a_launch_has_waves_for():
    """2^22 tokens of 16 column blocks and 2^24 of four are past the 2^32 threads of a launch at a wave for each block: fewer
    waves a token.  Every slot is empty, so rows, codes and scales are not touched and out is 0."""
    H, T, T2 = 8192, (1 << 22) + 5, (1 << 24) + 3
    room = torch.empty(max(T * H, T2 * H // 4), dtype=torch.bfloat16, device=DEV).fill_(1)
    some = torch.zeros(64, dtype=torch.int32, device=DEV)
    P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream

    def inputs(t):
        w = torch.full((t, 1), 2.0, device=DEV)
        return some, w, torch.full((2 * t,), -1, dtype=torch.int32, device=DEV), some, None

    args = inputs(T)
    shape = dm.make_shape(T, H, 1, 1)
    dm._check(dm.lib().moe_combine_checkpoint(dm.ctypes.byref(shape), P(some), *map(P, args), *[None] * 5, P(room), P(some),
                                              P(some), stream))
    out = room[:T * H].view(T, H)
    for a in range(0, T, 1 << 20):
        assert not out[a:a + (1 << 20)].any()
    room.fill_(1)
    args = inputs(T2)
    grad = torch.full((T2, 1), 5.0, device=DEV)
    shape = dm.make_shape(T2, H // 4, 1, 1)
    dm._check(dm.lib().moe_combine_bwd_weights_checkpoint(dm.ctypes.byref(shape), P(room), P(some), P(some), *map(P, args),
                                                          *[None] * 4, P(grad), None, stream))
    assert not grad.any()


# 2^20 units of eight columns and more: two a thread, kThreads apart.  The second one's columns carry over (256 is no
# multiple of a row's 60, 132, 1792 or 28 units), or stay (4 units of the narrow rows)
@pytest.mark.parametrize("R,F", [(17500, 480), (17500, 479), (8000, 1050), (600, 14336), (600, 14329), (40000, 224),
                                 (262200, 7), (262200, 31), (262144, 32)])
def test_swiglu_two_units_a_thread(R, F):
    assert R * (-(-F // 32) * 4) >= 1 << 20
    check_swiglu(gate_up(R, F, R + F, 2.0), F)


def test_swiglu_two_units_a_thread_rows_in_use():
    """nrows that ends between a thread's two units' rows."""
    R, F = 17500, 480
    gu = gate_up(R, F, 1).to(DEV)
    whole = [torch.empty(R, F, dtype=torch.bfloat16, device=DEV), *dm.checkpoint_buffers(R, F, DEV, halves=2)]
    grad = torch.empty_like(gu)
    dm.moe_swiglu_checkpoint_fwd(gu, *whole)
    dm.moe_swiglu_checkpoint_bwd(whole[1], whole[2], whole[0], grad)
    for n in (0, 1, 5, 8745, 17499):
        nrows = torch.tensor([n], dtype=torch.int32, device=DEV)
        part = [torch.full_like(t, 9) for t in whole]
        g = torch.full_like(grad, 9)
        dm.moe_swiglu_checkpoint_fwd(gu, *part, nrows=nrows)
        dm.moe_swiglu_checkpoint_bwd(part[1], part[2], whole[0], g, nrows=nrows)
        for a, b in zip([*whole, grad], [*part, g]):
            same(a[:n], b[:n])
            assert (b[n:] == 9).all()


@pytest.mark.parametrize("F", [96, 480, 33])
@pytest.mark.parametrize("R", [37, 17500])
def test_misaligned_rows_by_element(R, F):
    """Forward and backward from and to matrices that begin on 2 bytes (codes on 1), every element against the 64-bit form."""
    gu = gate_up(R, F, 5, 2.0)

    def odd(shape, dtype):
        return torch.empty(shape[0] * shape[1] + 1, dtype=dtype, device=DEV)[1:].view(shape)

    x = odd((R, 2 * F), torch.bfloat16).copy_(gu)
    h = odd((R, F), torch.bfloat16)
    codes, scales = (odd(t.shape, t.dtype) for t in dm.checkpoint_buffers(R, F, DEV, halves=2))
    dm.moe_swiglu_checkpoint_fwd(x, h, codes, scales)
    qc, qs = halves(gu)
    same(codes, qc)
    same(scales, qs)
    near("h", h, *swiglu64(gu[:, :F].double(), gu[:, F:].double()))
    d = gate_up(R, F, 6, 0.3)[:, :F]
    grad = odd((R, 2 * F), torch.bfloat16)
    dm.moe_swiglu_checkpoint_bwd(codes, scales, odd((R, F), torch.bfloat16).copy_(d), grad)
    nb = qs.shape[1] // 2
    near("grad", grad, *swiglu64(kept(qc[:, :F], qs[:, :nb]), kept(qc[:, F:], qs[:, nb:]), d.double()))


def test_an_error_of_a_callers_hook_is_its_own():
    def pack(t):
        raise TypeError("of the hook")

    x = gate_up(6, 32, 1).to(DEV).requires_grad_()
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        with pytest.raises(TypeError, match="of the hook"):
            dm.swiglu_checkpoint(x)
