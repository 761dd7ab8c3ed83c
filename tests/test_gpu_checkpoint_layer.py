"""GPU tests of the MoE layer with its activations kept in 8 bits, and of a training step of router, balance loss and
such a layer together."""
import pytest
import torch

import dispatch_expert_gemm_amd as dm
from test_gpu_balance import _mask
from test_gpu_checkpoint import kept, rule, same

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _layer(T, H, F, E, K, seed, special=False, masked=False, shared=0, ids=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().to(DEV)  # noqa: E731
    Z, C, Q = (1, 1, 2) if special else (0, 0, 0)
    n = E + Z + C + Q
    idx = (torch.rand(T, n, generator=g).topk(K)[1].to(torch.int32) if ids is None else
           torch.full((T, K), 0, dtype=torch.int32) + torch.tensor(ids, dtype=torch.int32)).to(DEV)
    d = dict(x=r(T, H), idx=idx, w=torch.rand(T, K, generator=g).to(DEV), wg=r(E, F, H, std=H ** -0.5),
             wu=r(E, F, H, std=H ** -0.5), wd=r(E, H, F, std=F ** -0.5), dout=r(T, H), kw={})
    d["shared"] = [r(1, shared, H, std=H ** -0.5), r(1, shared, H, std=H ** -0.5), r(1, H, shared, std=shared ** -0.5)] \
        if shared else [None] * 3
    if special:
        d["kw"].update(zero_expert_num=Z, copy_expert_num=C, const_expert_num=Q,
                       **{k: r(Q, H) for k in ("const_alpha_1", "const_alpha_2", "const_v")})
    if masked:
        d["kw"]["x_active_mask"] = _mask(2, T, K, seed)
    return d


def _step(d, keep, weights=True):
    leaves = [d[k].detach().clone().requires_grad_() for k in ("x", "w", "wg", "wu", "wd")]
    leaves[1].requires_grad_(weights)
    shared = [t if t is None else t.detach().clone().requires_grad_() for t in d["shared"]]
    out = dm.moe_layer(leaves[0], d["idx"], *leaves[1:], shared_w_gate=shared[0], shared_w_up=shared[1],
                       shared_w_down=shared[2], checkpoint_8bit=keep, **d["kw"])
    ins = [t for t in leaves + shared if t is not None and t.requires_grad]
    return out.detach(), torch.autograd.grad(out, ins, d["dout"])


# (T, H, F, E, K, special, masked, shared): both ways of the backward (F under and over 1024); more than 256 rows an
# expert, the last two of the first four, take the smaller forward tiles
CASES = [
    (200, 128, 64, 8, 2, False, False, 0), (130, 256, 480, 16, 4, True, True, 96), (700, 128, 96, 2, 2, False, True, 0),
    (1200, 256, 1056, 4, 2, True, True, 64), (65, 512, 1056, 4, 2, True, True, 64),
    (1, 128, 64, 8, 8, False, False, 0), (90, 136, 32, 3, 1, False, True, 32)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_is_the_same_and_gradients_are_near(case):
    """The forward's bits do not change.  The kept values are within half a step, s / 2 = amax / 254 of their block of 32:
    for normal values (amax near 2.1 sigma) 0.5 % of sigma at most, 0.3 % in the mean; the activation's slopes are below
    1.1, so each gradient is within 2 % (relative norm) of the bf16 one's, which is the bar of the 8-bit paths."""
    T, H, F, E, K, special, masked, shared = case
    d = _layer(T, H, F, E, K, T + F, special, masked, shared)
    out, grads = _step(d, False)
    out8, grads8 = _step(d, True)
    same(out8, out)
    for a, b in zip(grads, grads8):
        assert a.shape == b.shape and a.dtype == b.dtype and torch.isfinite(b.float()).all()
        if a.numel():
            assert float((a.double() - b.double()).norm()) <= 2e-2 * float(a.double().norm()) + 1e-30


@pytest.mark.parametrize("case", CASES[:5], ids=str)
def test_gradients_are_those_of_the_kept_values(case):
    """The plain entries' chain on kept [G | U] and y: the same gradients of x, the gate and up weights bit for bit; the
    down weights' from an h that is within one bf16 step of the chain's (the two SwiGLU formulas differ in fp32's
    last bits), and dw in 64 bits."""
    T, H, F, E, K, special, masked, _ = case
    d = _layer(T, H, F, E, K, T + F, special, masked)
    _, (gx, gw, gwg, gwu, gwd) = _step(d, True)
    kw = dict(d["kw"])
    mask = kw.pop("x_active_mask", None)
    consts = [kw.pop(k, None) for k in ("const_alpha_1", "const_alpha_2", "const_v")]
    shape = dm.make_shape(T, H, K, E, F=F, mask_ndim=0 if mask is None else 2, **kw)
    x, idx, w, dout = d["x"], d["idx"], d["w"], d["dout"]
    route = dm.route(shape, idx, mask)
    recv, assist = route.ep_recv_counts, route.assist_info_for_combine
    cap, rows = shape.capacity, int(recv[-1])
    gus, h, y = (torch.zeros(cap, n, dtype=torch.bfloat16, device=DEV) for n in (2 * F, F, H))
    dm.moe_ffn_gate_up_fwd_gather(shape, x, assist, d["wg"], d["wu"], recv, gus, h)
    dm.moe_ffn_down_fwd(shape, h, d["wd"], recv, y)
    # the GEMM that keeps: the codes of what the plain one writes, and its h
    codes, scales = dm.checkpoint_buffers(cap, F, DEV, halves=2)
    codes.fill_(9)
    scales.fill_(9)
    h8 = torch.zeros_like(h)
    dm.moe_ffn_gate_up_fwd_checkpoint(shape, x, assist, d["wg"], d["wu"], recv, codes, scales, h8)
    same(h8, h)
    (qg, sg), (qu, su) = (rule(t) for t in (gus[:, :F], gus[:, F:]))
    same(codes[:rows], torch.cat([qg, qu], 1)[:rows])
    same(scales[:rows], torch.cat([sg, su], 1)[:rows])
    assert (codes[rows:] == 9).all() and (scales[rows:] == 9).all()
    gus.copy_(torch.cat([kept(qg, sg), kept(qu, su)], 1).bfloat16())
    yk = kept(*rule(y))
    g64, u64 = gus[:, :F].cpu().double(), gus[:, F:].cpu().double()
    h64 = g64 / (1 + torch.exp(-g64)) * u64
    hk = h64.bfloat16().to(DEV)
    args = (idx, w, assist, recv, mask, x, *consts)
    roww = torch.empty(cap, device=DEV)
    ggu = torch.empty_like(gus)
    wg, wu, wd = (torch.empty(d[k].shape, device=DEV) for k in ("wg", "wu", "wd"))
    if dm.fold_combine_bwd(F):
        dm.moe_combine_bwd_weights(shape, dout, None, *args, None, roww)
        dm.moe_ffn_down_bwd_data_gather(shape, dout, assist, roww, d["wd"], gus, recv, ggu)
        dm.moe_ffn_down_bwd_weight_gather(shape, dout, assist, roww, hk, recv, wd)
    else:
        gy = torch.empty(cap, H, dtype=torch.bfloat16, device=DEV)
        dm.moe_combine_bwd(shape, dout, None, *args, gy, None)
        dm.moe_ffn_down_bwd_data(shape, gy, d["wd"], gus, recv, ggu)
        dm.moe_ffn_down_bwd_weight(shape, gy, hk, recv, wd)
    gxe, gx2 = torch.empty(cap, H, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    dm.moe_ffn_gate_up_bwd_data(shape, ggu, d["wg"], d["wu"], recv, gxe)
    dm.moe_dispatch_bwd(shape, gxe, assist, idx, w, mask, dout, consts[0], None, gx2)
    dm.moe_ffn_gate_up_bwd_weight_gather(shape, ggu, x, assist, recv, wg, wu)
    same(gx, gx2)
    same(gwg, wg.bfloat16())
    same(gwu, wu.bfloat16())
    # a step of h is 2^-7 of it at most: |grad_y|^T |h| 2^-7, and the result's rounding
    gy64 = torch.zeros(cap, H, dtype=torch.float64)
    slot = assist[:T * K].view(T, K).cpu()
    for t in range(T):
        for k in range(K):
            if int(slot[t, k]) >= 0:
                gy64[int(slot[t, k])] = w[t, k].cpu().double() * dout[t].cpu().double()
    ends = [0, *recv.tolist()]
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        mag = gy64[a:b].abs().t() @ h64[a:b].abs()
        err = (gwd[e].cpu().double() - wd[e].bfloat16().cpu().double()).abs()
        assert (err <= 2.0 ** -7 * mag + 2.0 ** -7 * wd[e].cpu().double().abs() + 1e-30).all()
    # dw: 64 bits on the kept rows
    for t in range(0, T, 7):
        for k in range(K):
            c = int(slot[t, k])
            if c >= 0:
                p = yk[c] * dout[t].cpu().double()
                assert abs(float(gw[t, k]) - float(p.sum())) <= (H / 64 + 12) * 2.0 ** -23 * float(p.abs().sum())


def test_what_is_kept():
    """2.125 F + 1.0625 H bytes a routed row (2.125 F without the weights' gradient) in place of 6 F + 2 H."""
    T, H, F, E, K = 512, 1536, 480, 16, 8
    d = _layer(T, H, F, E, K, 1)

    def held(keep, weights):
        sizes = {}
        inputs = {d[k].data_ptr() for k in ("x", "wg", "wu", "wd", "w")}
        leaves = [d[k].detach().requires_grad_() for k in ("x", "w", "wg", "wu", "wd")]
        leaves[1].requires_grad_(weights)

        def pack(t):
            if t.data_ptr() not in inputs and t.numel() > T * K * 2:
                sizes[t.data_ptr()] = t.numel() * t.element_size()
            return t

        with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
            out = dm.moe_layer(leaves[0], d["idx"], *leaves[1:], checkpoint_8bit=keep)
        return sum(sizes.values()), out

    rows = T * K
    assert held(False, True)[0] == rows * (6 * F + 2 * H)
    assert held(True, True)[0] == rows * (2 * F + H) * 17 // 16
    assert held(True, False)[0] == rows * 2 * F * 17 // 16


def test_weights_without_gradient():
    d = _layer(150, 128, 64, 8, 2, 3, True, True, 32)
    a, b = _step(d, True), _step(d, True, weights=False)
    same(a[0], b[0])
    for g1, g2 in zip([a[1][0], *a[1][2:]], b[1]):
        same(g1, g2)


def test_one_expert_takes_all():
    d = _layer(100, 128, 64, 4, 1, 5, ids=[2])
    out, grads = _step(d, False)
    out8, grads8 = _step(d, True)
    same(out, out8)
    for k in (0, 1, 3):  # the weight gradients of experts without rows are zero
        assert not grads8[2][k].any() and not grads8[4][k].any()


@pytest.mark.parametrize("kw", [dict(fp8=True), dict(fp8=True, mx=True), dict(comm_quant_mode=2)], ids=str)
def test_refused_with_the_8_bit_paths(kw):
    d = _layer(16, 128, 128, 4, 2, 5)
    with pytest.raises(dm.MoeError, match="checkpoint_8bit"):
        dm.moe_layer(d["x"], d["idx"], d["w"], d["wg"], d["wu"], d["wd"], checkpoint_8bit=True, **kw)


def _train(p, K):
    """A step: router, balance and z loss, the layer -> its results, and the gradients of x, the logits and the weights
    for given gradients of the layer's output and of both losses."""
    leaves = [p[k].detach().requires_grad_() for k in ("x", "logits", "wg", "wu", "wd")]
    x, logits, *ws = leaves
    idx, w = dm.router(logits, K)
    balance, z, counts = dm.balance_loss(logits, idx, seq_offsets=p["off"])
    out = dm.moe_layer(x, idx, w, *ws, checkpoint_8bit=True)
    return (out, balance, z, counts, idx, w), torch.autograd.grad((out, balance, z), leaves, p["ups"])


def _train_inputs(T, H, F, E, K, off):
    d = _layer(T, H, F, E, K, 9)
    p = {k: d[k] for k in ("x", "wg", "wu", "wd")}
    p["logits"] = torch.randn(T, E, generator=torch.Generator().manual_seed(4)).to(DEV)
    p["off"] = torch.tensor(off, dtype=torch.int32, device=DEV)
    p["ups"] = [d["dout"], torch.tensor(0.5, device=DEV), torch.tensor(0.1, device=DEV)]
    return p


def test_a_training_step():
    T, H, F, E, K = 300, 128, 96, 16, 4
    p = _train_inputs(T, H, F, E, K, [0, 100, 100, 290])
    (out, balance, z, counts, idx, w), grads = _train(p, K)
    assert counts.shape == (3, E) and int(counts.sum()) == 290 * K and int(counts[1].sum()) == 0
    assert all(torch.isfinite(t.float()).all() for t in grads)
    # the logits' gradient is the sum of its parts, each by itself
    lg = p["logits"].detach().requires_grad_()
    i2, w2 = dm.router(lg, K)
    same(i2, idx)
    b2, z2, c2 = dm.balance_loss(lg, i2, seq_offsets=p["off"])
    same(c2, counts)
    layer = dm.moe_layer(p["x"], i2, w2, p["wg"], p["wu"], p["wd"], checkpoint_8bit=True)
    same(layer.detach(), out.detach())
    parts = [torch.autograd.grad(t, lg, g, retain_graph=True)[0].double() for t, g in zip((layer, b2, z2), p["ups"])]
    err = (grads[1].double() - sum(parts)).abs()
    assert (err <= 4 * 2.0 ** -24 * sum(t.abs() for t in parts) + 1e-30).all()
    # without checkpoints the layer's output is the same, and the logits' gradient within the kept values' 2 %
    plain = dm.moe_layer(p["x"], i2, w2, p["wg"], p["wu"], p["wd"])
    same(plain.detach(), out.detach())
    g = torch.autograd.grad(plain, lg, p["ups"][0])[0].double()
    assert float((g - parts[0]).norm()) <= 2e-2 * float(g.norm())


def test_a_captured_training_step():
    """Captured while an eager step's graph is alive, with leaves of its own, and replayed with new tokens."""
    K = 2
    p = _train_inputs(256, 128, 64, 8, K, [0, 100, 250])
    alive = _train(p, K)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _train(p, K)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, grads = _train(p, K)
    for seed in (1, 2, 3):
        g = torch.Generator().manual_seed(seed)
        p["x"].copy_(torch.randn(p["x"].shape, generator=g).bfloat16())
        p["logits"].copy_(torch.randn(p["logits"].shape, generator=g))
        graph.replay()
        outs2, grads2 = _train(p, K)
        torch.cuda.synchronize()
        for a, b in zip([*outs, *grads], [*outs2, *grads2]):
            same(a.detach(), b.detach())
    del alive


def test_a_capture_refuses_leaves_of_a_living_eager_graph():
    """What the engine would end the process for is refused at the forward, and the capture ends as an empty one."""
    p = _train_inputs(64, 128, 64, 8, 2, [0, 64])
    x, logits = p["x"].clone().requires_grad_(), p["logits"].clone().requires_grad_()
    gate_up = torch.randn(8, 64, device=DEV).bfloat16().requires_grad_()
    idx, w = dm.router(p["logits"], 2)
    calls = [lambda: dm.balance_loss(logits, idx)[0], lambda: dm.swiglu_checkpoint(gate_up),
             lambda: dm.moe_layer(x, idx, w, p["wg"], p["wu"], p["wd"], checkpoint_8bit=True)]
    alive = [f() for f in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f in calls:
            with pytest.raises(dm.MoeError, match="leaves of its own"):
                f()
        with torch.no_grad():
            same_again = dm.swiglu_checkpoint(gate_up)
    graph.replay()
    torch.cuda.synchronize()
    same(same_again, alive[1].detach())
    del alive
    for f in calls:  # and eagerly, or captured once that graph is gone, they run
        f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [f().detach() for f in calls]
    graph.replay()
    for f, o in zip(calls, outs):
        same(f().detach(), o)


def _offset(t, k):
    """t's values in memory that begins k elements behind a boundary."""
    return None if t is None else torch.empty(t.numel() + k, dtype=t.dtype, device=t.device)[k:].view(t.shape).copy_(t)


@pytest.mark.parametrize("k", [1, 4])
@pytest.mark.parametrize("F", [64, 1056])
@pytest.mark.parametrize("special", [False, True])
def test_tensors_off_a_16_byte_boundary(special, F, k):
    """x, the shared term, the constants and the output's gradient may begin anywhere, as in the layer that keeps bf16:
    the same bits as from aligned ones."""
    T, H = 60, 128
    d = _layer(T, H, F, 8, 2, 11, special, special)
    g = torch.Generator().manual_seed(3)
    term = None if special else torch.randn(T, H, generator=g).bfloat16().to(DEV)

    def step(move):
        leaves = [d[n].detach().clone().requires_grad_() for n in ("w", "wg", "wu", "wd")]
        x = move(d["x"]).requires_grad_()
        kw = {n: move(v) if n.startswith("const_") and isinstance(v, torch.Tensor) else v for n, v in d["kw"].items()}
        out = dm.moe_layer(x, d["idx"], *leaves, shared_expert_x=None if term is None else move(term),
                           checkpoint_8bit=True, **kw)
        return [out.detach(), *torch.autograd.grad(out, [x, *leaves], move(d["dout"]))]

    for a, b in zip(step(lambda t: t.detach().clone()), step(lambda t: _offset(t, k))):
        same(a, b)


def test_rows_are_kept_only_for_a_backward(monkeypatch):
    """y's codes are written where the routing weights' gradient will read them, so neither without gradients nor for
    weights that need none."""
    d = _layer(90, 128, 64, 8, 2, 7)
    kept_calls = []
    keep = dm.moe_combine_checkpoint
    monkeypatch.setattr(dm, "moe_combine_checkpoint", lambda *a, **k: kept_calls.append(1) or keep(*a, **k))

    def call(weights):
        w = d["w"].detach().requires_grad_(weights)
        x = d["x"].detach().requires_grad_()
        return dm.moe_layer(x, d["idx"], w, d["wg"], d["wu"], d["wd"], checkpoint_8bit=True)

    out = call(True)
    assert len(kept_calls) == 1 and out.requires_grad
    assert call(False).requires_grad and len(kept_calls) == 1
    with torch.no_grad():
        bare = call(True)
    assert len(kept_calls) == 1 and not bare.requires_grad
    same(bare, out.detach())


@pytest.mark.parametrize("op", ["balance", "swiglu", "router", "layer", "layer with checkpoints"])
def test_a_captured_backward_refuses_what_an_eager_graph_left(op):
    """A weight behind the operator's input whose eager graph still lives: the engine would end the process, so the
    backward is refused before it gets there.  A forward alone, and a backward that stops before that weight, run."""
    p = _train_inputs(64, 128, 64, 8, 2, [0, 64])
    idx, w = dm.router(p["logits"], 2)
    base = {"swiglu": torch.randn(8, 64, device=DEV).bfloat16(), "layer": p["x"], "layer with checkpoints": p["x"]}
    base = base.get(op, p["logits"]).detach()
    weight = torch.full((base.shape[1],), 0.5, dtype=base.dtype, device=DEV, requires_grad=True)
    layer = lambda x, keep: dm.moe_layer(x, idx, w, p["wg"], p["wu"], p["wd"], checkpoint_8bit=keep)  # noqa: E731
    call = {"balance": lambda x: dm.balance_loss(x, idx)[0], "swiglu": dm.swiglu_checkpoint,
            "router": lambda x: dm.router(x, 2)[1], "layer": lambda x: layer(x, False),
            "layer with checkpoints": lambda x: layer(x, True)}[op]

    def step(wrt, at=base):
        at = at * weight
        out = call(at)
        return out.detach(), *torch.autograd.grad(out, weight if wrt else at, torch.ones_like(out))

    want = [t.clone() for t in step(False)]
    alive = call(base * weight)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="leaves of its own"):
            step(True)
        forward = call(base * weight).detach()
        part = step(False)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        same(forward, alive.detach())
        for a, b in zip(want, part):
            same(a, b)
    del alive
    # with that graph gone, or a leaf of its own, the whole backward is captured
    whole = [t.clone() for t in step(True)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(True)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, whole):
            same(a, b)
