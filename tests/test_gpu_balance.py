"""GPU tests of the router's balance loss, z loss and counts with their gradient, against the 64-bit form."""
import pytest
import torch

import dispatch_expert_gemm_amd as dm
from balance_util import compare, reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs(T, n, K, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, n, generator=g) * std + torch.randn(n, generator=g)
    idx = l.topk(K, 1)[1].to(torch.int32) if T else torch.zeros(0, K, dtype=torch.int32)
    return l.to(dtype).to(DEV), idx.to(DEV)


def _mask(kind, T, K, seed):
    g = torch.Generator().manual_seed(seed + 100)
    if kind == 0:
        return None
    if kind == 1:
        return (torch.arange(T) < T - T // 3).to(DEV)
    m = torch.rand(T, K, generator=g) >= 0.3
    m[::5] = False  # whole tokens without a slot
    return m.to(torch.uint8).to(DEV)


def _offsets(S, T, seed, lead=0, tail=0):
    g = torch.Generator().manual_seed(seed + 200)
    cuts = (torch.rand(S - 1, generator=g) * max(T - lead - tail, 0)).long().sort()[0] + lead
    return torch.cat([torch.tensor([min(lead, T)]), cuts.clamp(max=T),
                      torch.tensor([max(min(lead, T), T - tail)])]).to(torch.int32).to(DEV)


def _run(l, idx, mask=None, offsets=None, g=0.7, gz=0.3):
    l = l.detach().requires_grad_()
    loss, z, counts = dm.balance_loss(l, idx, x_active_mask=mask, seq_offsets=offsets)
    assert loss.shape == () and z.shape == () and loss.dtype == torch.float32
    ups = [v if isinstance(v, torch.Tensor) else torch.tensor(v, device=DEV) for v in (g, gz)]
    grad, = torch.autograd.grad((loss, z), l, ups)
    assert grad.dtype == l.dtype and grad.shape == l.shape
    return loss.detach(), z.detach(), counts, grad


def _check(name, l, idx, mask=None, offsets=None, g=0.7, gz=0.3):
    got = _run(l, idx, mask, offsets, g, gz)
    g, gz = float(torch.tensor(g)), float(torch.tensor(gz))
    compare(name, got, reference(l, idx, mask, offsets, g, gz, l.dtype))
    return got


# every number of columns that changes the lanes or runs of a token, odd ones among them
COLUMNS = [1, 2, 3, 4, 5, 16, 17, 32, 33, 63, 64, 65, 100, 128, 129, 256, 257, 260, 384, 385, 512, 513, 1024, 1025, 2048, 2051, 4096]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("n", COLUMNS)
def test_columns(n, dtype):
    T, K = 97, min(n, 8)
    l, idx = _inputs(T, n, K, n, dtype=dtype)
    _check(f"n={n}", l, idx, _mask(2, T, K, n))


@pytest.mark.parametrize("T", [0, 1, 2, 15, 16, 17, 64, 255, 1000, 4099, 16384])
def test_tokens(T):
    l, idx = _inputs(T, 64, 8, T + 1)
    _check(f"T={T}", l, idx)
    _check(f"T={T} bf16", l.bfloat16(), idx, _mask(1, T, 8, T))


@pytest.mark.parametrize("mask", [0, 1, 2])
@pytest.mark.parametrize("T,n,K,S,lead,tail", [
    (1, 64, 8, 1, 0, 0), (1, 8, 2, 5, 0, 0), (300, 64, 8, 1, 7, 11), (300, 64, 8, 300, 0, 0), (513, 100, 3, 64, 0, 40),
    (513, 100, 3, 65, 3, 0), (2000, 260, 8, 37, 0, 61), (4096, 16, 1, 1000, 100, 100), (4000, 64, 16, 2, 3999, 0),
    (70, 1024, 16, 9, 0, 3), (16, 64, 8, 5000, 0, 0)])
def test_sequences(T, n, K, S, lead, tail, mask):
    """Ragged, empty and one-token sequences, tokens before the first and behind the last."""
    l, idx = _inputs(T, n, K, S)
    got = _check(f"S={S}", l, idx, _mask(mask, T, K, S), _offsets(S, T, S, lead, tail))
    assert got[2].shape == (S, n)


@pytest.mark.parametrize("mask", [0, 1, 2])
@pytest.mark.parametrize("T,n,K,S,lead,tail", [(70, 1500, 8, 9, 0, 3), (4100, 1028, 8, 37, 5, 61), (2100, 4093, 3, 700, 0, 0)])
def test_sequences_of_wide_rows(T, n, K, S, lead, tail, mask):
    """Rows that a whole workgroup holds: items and runs of several tokens that sequences end inside."""
    l, idx = _inputs(T, n, K, S)
    for x in (l, l.bfloat16()):
        _check(f"S={S} {x.dtype}", x, idx, _mask(mask, T, K, S), _offsets(S, T, S, lead, tail))


def test_sequences_are_each_by_themselves():
    """Two sequences give the token-weighted mean of their own losses, and the gradient of a token does not see the
    other sequence's logits."""
    l, idx = _inputs(200, 64, 8, 5)
    off = torch.tensor([0, 60, 200], dtype=torch.int32, device=DEV)
    loss, z, counts, grad = _run(l, idx, None, off)
    a, b = _run(l[:60], idx[:60]), _run(l[60:], idx[60:])
    assert abs(float(loss) - (0.3 * float(a[0]) + 0.7 * float(b[0]))) < 1e-6 * float(loss)
    assert torch.equal(counts, torch.stack([a[2], b[2]]))
    other = l.clone()
    other[60:] = other[60:].flip(0)
    assert torch.equal(_run(other, idx, None, off)[3][:60], grad[:60])


def test_even_load_is_one():
    l = torch.zeros(64, 32, device=DEV)
    idx = ((torch.arange(64)[:, None] * 4 + torch.arange(4)) % 32).to(torch.int32).to(DEV)
    loss, _, counts, _ = _run(l, idx)
    assert float(loss) == 1.0 and (counts == 8).all()


@pytest.mark.parametrize("mask", [1, 2])
def test_masks_that_leave_nothing(mask):
    l, idx = _inputs(50, 64, 8, 3)
    m = torch.zeros((50,) if mask == 1 else (50, 8), dtype=torch.bool, device=DEV)
    loss, z, counts, grad = _run(l, idx, m)
    assert float(loss) == 0 and float(z) == 0 and not counts.any() and not grad.any()


def test_masked_tokens_hold_anything():
    """NaN and infinities in tokens that take no part change nothing and get gradient 0."""
    l, idx = _inputs(120, 64, 8, 9)
    m = torch.rand(120, 8, generator=torch.Generator().manual_seed(1)).to(DEV) >= 0.5
    m[40:80] = False
    want = _run(l, idx, m)
    bad = l.clone()
    bad[40:60] = float("nan")
    bad[60:70] = float("inf")
    bad[70:80] = -float("inf")
    got = _run(bad, idx, m)
    for a, b in zip(want[:3], got[:3]):
        assert torch.equal(a, b)
    assert torch.equal(want[3][:40], got[3][:40]) and torch.equal(want[3][80:], got[3][80:])
    assert not got[3][40:80].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_impossible_and_extreme_logits(dtype):
    l, idx = _inputs(90, 72, 6, 4, dtype=dtype)
    l[:, 7] = -float("inf")                       # an id that no token may take
    l[3, :71] = -float("inf")                     # one id left
    l[4] = -float("inf")                          # nothing left: adds nothing
    l[5, 10] = float("nan")                       # read as -inf
    l[6] = torch.finfo(dtype).min                 # the type's lowest value everywhere
    l[7, 3] = torch.finfo(dtype).min
    l[8] = l[8] * 30
    gz = 0.0                                      # lse^2 of the lowest value is an infinity: the z loss by itself below
    loss, z, counts, grad = _run(l, idx, gz=gz)
    ref = reference(l, idx, None, None, float(torch.tensor(0.7)), gz, dtype)
    assert torch.equal(counts.cpu().long(), ref["counts"])
    assert abs(float(loss) - ref["loss"]) <= ref["loss_bound"]
    keep = torch.ones(90, dtype=torch.bool)
    keep[6] = False                               # 0 * lse is 0 * -3e38: finite, but its bound is not
    err = (grad.cpu().double() - ref["grad"]).abs()
    assert (err[keep] <= ref["bound"][keep]).all()
    assert not grad[4].any() and not grad[keep.to(DEV), 7].any() and float(grad[5, 10]) == 0  # (row 6 has an id 7)
    l[6] = 0
    _check("extreme", l, idx)


def test_wide_rows_with_anything_in_them():
    l, idx = _inputs(90, 1500, 6, 4)
    l[:, 7] = -float("inf")
    l[3, :1499] = -float("inf")                   # one id left, in the last wave
    l[4] = -float("inf")
    l[5, 1300] = float("nan")
    l[8] = l[8] * 30
    mask = _mask(1, 90, 6, 2)
    mask[:10] = True
    mask[20:23] = False
    l[20], l[21], l[22] = float("nan"), float("inf"), -float("inf")
    got = _check("wide", l, idx, mask)
    assert not got[3][4].any() and not got[3][20:23].any() and float(got[3][5, 1300]) == 0
    for a, b in zip(got, _run(l, idx, mask)):
        assert torch.equal(a, b)


def test_plus_infinity_is_seen():
    l, idx = _inputs(33, 16, 2, 4)
    l[3, 5] = float("inf")
    loss, z, _, grad = _run(l, idx)
    assert not torch.isfinite(loss) and not torch.isfinite(z) and not torch.isfinite(grad[3]).any()


def test_ids_outside_are_not_counted_and_repeated_ids_are():
    l, idx = _inputs(64, 32, 4, 6)
    idx[3] = torch.tensor([-1, 32, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    idx[4] = 5
    _check("ids", l, idx)


@pytest.mark.parametrize("offsets", [[0, -5, 40, 64], [50, 20, 10, 64], [-9, 10, 5000, 70], [64, 64, 0, 0], [2 ** 31 - 1, -2 ** 31, 3, 9]])
def test_offsets_that_decrease_or_leave_the_batch_stay_in_bounds(offsets):
    l, idx = _inputs(64, 32, 4, 6)
    room = torch.full((64 + 2, 32), 7.0, device=DEV)
    grad = room[1:-1]
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    loss, z = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    counts, tokens = torch.empty(3 * 32, dtype=torch.int32, device=DEV), torch.empty(4, dtype=torch.int32, device=DEV)
    ws = torch.zeros(dm.moe_balance_workspace_size(64, 32, 3), dtype=torch.uint8, device=DEV)
    dm.moe_balance_fwd(l, idx, None, off, loss, z, counts, tokens, ws)
    dm.moe_balance_bwd(l, 4, None, off, counts, tokens, loss, z, grad)
    torch.cuda.synchronize()
    assert (room[0] == 7).all() and (room[-1] == 7).all()


def test_views_and_misaligned_rows():
    big, idx = _inputs(50, 80, 4, 8)
    idx = idx.clamp(max=63)
    view = big[:, 5:69]                                  # strides: laid out by the call
    want = _run(view.contiguous(), idx)
    for a, b in zip(want, _run(view, idx)):
        assert torch.equal(a, b)
    flat = torch.empty(50 * 64 + 1, device=DEV)[1:].view(50, 64)  # rows that begin on 4 bytes
    flat.copy_(view)
    got = _run(flat, idx)
    for a, b in zip(want[:3], got[:3]):
        assert torch.equal(a, b)
    assert torch.equal(want[3], got[3])


def test_one_upstream_gradient_alone():
    l, idx = _inputs(70, 48, 4, 2)
    x = l.clone().requires_grad_()
    loss, z, _ = dm.balance_loss(x, idx)
    ga, = torch.autograd.grad(loss, x, retain_graph=True)
    gb, = torch.autograd.grad(z, x)
    ra, rb = reference(l, idx, g=1.0, gz=0.0), reference(l, idx, g=0.0, gz=1.0)
    for got, ref in ((ga, ra), (gb, rb)):
        assert ((got.cpu().double() - ref["grad"]).abs() <= ref["bound"]).all()


def test_gradient_against_differences():
    l, idx = _inputs(12, 10, 3, 7)
    m = _mask(2, 12, 3, 7)
    off = torch.tensor([0, 5, 5, 11], dtype=torch.int32, device=DEV)
    grad = _run(l, idx, m, off, 1.0, 0.5)[3].cpu().double()
    h = 1e-4

    def value(x):
        r = reference(x, idx, m, off)
        return r["loss"] + 0.5 * r["z"]

    base = l.cpu().double()
    for t, e in [(0, 0), (1, 3), (4, 9), (6, 2), (10, 5), (11, 1)]:
        a, b = base.clone(), base.clone()
        a[t, e] += h
        b[t, e] -= h
        # the difference quotient's own error is h^2 / 6 of a third derivative (the terms are of the order of 10 / N)
        assert abs((value(a) - value(b)) / (2 * h) - float(grad[t, e])) < 1e-6 + 10 * h * h


def test_bitwise_repeatable_and_whole_workspace_uninitialised():
    l, idx = _inputs(3000, 160, 8, 1)
    off = _offsets(11, 3000, 2)
    a = _run(l, idx, None, off)
    torch.empty(1 << 24, dtype=torch.uint8, device=DEV).fill_(255)  # what the allocator hands out next
    b = _run(l, idx, None, off)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_other_stream_and_captured_calls():
    T, n, K = 2000, 64, 8
    l, idx = _inputs(T, n, K, 1)
    want = _run(l, idx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _run(l, idx)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # two captured calls with workspaces of their own, replayed with new inputs and eager work between
    static = l.clone()
    ups = [torch.tensor(0.7, device=DEV), torch.tensor(0.3, device=DEV)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [_run(static, idx, None, None, *ups), _run(static * 1.0, idx, None, None, *ups)]
    for seed in (2, 3, 4):
        new, _ = _inputs(T, n, K, seed)
        static.copy_(new)
        graph.replay()
        eager = _run(new, idx)
        torch.cuda.synchronize()
        for o in outs:
            for a, b in zip(o, eager):
                assert torch.equal(a, b)


def test_large_batch():
    """Offsets past 2^31 bytes, many items and the most columns."""
    T, n, K = 140000, 4096, 4
    l = torch.randn(1000, n, generator=torch.Generator().manual_seed(1)).to(DEV).repeat(140, 1)
    idx = l[:1000].topk(K, 1)[1].to(torch.int32).repeat(140, 1)
    loss, z, counts, grad = _run(l, idx)
    small = _run(l[:1000], idx[:1000])
    assert torch.equal(counts, small[2] * 140)
    # every copy is the same batch: the losses agree to their rounding, the gradients to 1/140
    assert abs(float(loss) - float(small[0])) < 1e-4 * float(loss)
    assert abs(float(z) - float(small[1])) < 1e-4 * float(z)
    part = grad[-1000:] * 140
    assert float((part - small[3]).abs().max()) < 1e-4 * float(small[3].abs().max())


def test_differentiable_once():
    """A second derivative raises; a step that merely builds the graph of its first does not."""
    l, idx = _inputs(20, 16, 2, 1)
    x = l.clone().requires_grad_()
    loss, z, _ = dm.balance_loss(x, idx)
    g, = torch.autograd.grad(loss + z, x, create_graph=True)
    assert torch.equal(g.detach(), _run(l, idx, g=1.0, gz=1.0)[3])
    with pytest.raises(RuntimeError, match="differentiable once"):
        g.square().sum().backward()


def test_without_gradients():
    l, idx = _inputs(20, 16, 2, 1)
    loss, z, counts = dm.balance_loss(l, idx)
    assert not loss.requires_grad and not z.requires_grad
    with torch.no_grad():
        assert not dm.balance_loss(l.clone().requires_grad_(), idx)[0].requires_grad
    x = l.clone().requires_grad_()
    loss, z, counts = dm.balance_loss(x, idx)
    assert loss.requires_grad and z.requires_grad and not counts.requires_grad
    main = x.sum()
    main += 0.01 * loss + 1e-3 * z  # as a training loop adds them
    main.backward()
    assert x.grad.shape == x.shape


@pytest.mark.parametrize("change,match", [
    (dict(logits=lambda l: l.half()), "logits must be float32 or bfloat16"), (dict(logits=lambda l: l[0]), "logits must be"),
    (dict(idx=lambda i: i.long()), "topk_idx must be torch.int32"), (dict(idx=lambda i: i[:5]), "topk_idx must be a tensor"),
    (dict(idx=lambda i: i.cpu()), "topk_idx must be a GPU tensor"), (dict(idx=lambda i: i.t().contiguous().t()), "contiguous"),
    (dict(idx=lambda i: i.repeat(1, 9)), "status -2"), (dict(mask=torch.ones(19)), "x_active_mask must be a tensor"),
    (dict(mask=torch.ones(20, 3)), "x_active_mask must be a tensor"), (dict(mask=torch.ones(20)), "uint8 or torch.bool"),
    (dict(off=torch.zeros(1, dtype=torch.int32)), "seq_offsets must hold"), (dict(off=torch.zeros(3)), "seq_offsets must be"),
    (dict(off=torch.zeros(2, 2, dtype=torch.int32)), "seq_offsets must hold")])
def test_refusals(change, match):
    l, idx = _inputs(20, 16, 2, 1)
    l, idx = change.get("logits", lambda t: t)(l), change.get("idx", lambda t: t)(idx)
    mask, off = (None if change.get(k) is None else change[k].to(DEV) for k in ("mask", "off"))
    with pytest.raises(dm.MoeError, match=match):
        dm.balance_loss(l, idx, x_active_mask=mask, seq_offsets=off)


def test_entry_refusals():
    """The C entries' Python forms: short buffers and other types."""
    l, idx = _inputs(20, 16, 2, 1)
    f = torch.empty(1, device=DEV)
    i = torch.empty(64, dtype=torch.int32, device=DEV)
    ws = torch.empty(dm.moe_balance_workspace_size(20, 16), dtype=torch.uint8, device=DEV)
    for bad in (dict(counts=i[:15]), dict(seq_tokens=i[:1]), dict(workspace=ws[:100]), dict(loss=f.double()),
                dict(topk_idx=idx[:10])):
        a = dict(logits=l, topk_idx=idx, x_active_mask=None, seq_offsets=None, loss=f, z_loss=f, counts=i, seq_tokens=i,
                 workspace=ws)
        a.update(bad)
        with pytest.raises(dm.MoeError):
            dm.moe_balance_fwd(**a)
    with pytest.raises(dm.MoeError, match="grad_logits"):
        dm.moe_balance_bwd(l, 2, None, None, i, i, f, f, l[:10])


def _backward_us(l, K, off, counts, tokens, grad, passes=5):
    """The fastest of some passes of the backward, in us."""
    one = torch.ones(1, device=DEV)
    best = float("inf")
    for _ in range(passes):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        dm.moe_balance_bwd(l, K, None, off, counts, tokens, one, one, grad)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


@pytest.mark.parametrize("n", [64, 1500])
@pytest.mark.parametrize("lead", [0, 5])
def test_padded_offsets(n, lead):
    """Offsets padded to a fixed number of sequences, before the first tokens, between them and behind the last, and
    tokens behind them all: the gradient, and that a token's sequence is searched for, not walked to (131072 offsets
    one by one took 14 ms)."""
    T, K, S = 70, 4, 1 << 17
    l, idx = _inputs(T, n, K, n)
    off = torch.full((S + 1,), 40, dtype=torch.int32)
    off[:1000] = lead
    off[1000:50000] = 9
    off[50000:60000] = 23
    off = off.to(DEV)
    loss, z = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    counts, tokens = (torch.empty(k, dtype=torch.int32, device=DEV) for k in (S * n, S + 1))
    ws = torch.empty(dm.moe_balance_workspace_size(T, n, S), dtype=torch.uint8, device=DEV)
    dm.moe_balance_fwd(l, idx, None, off, loss, z, counts, tokens, ws)
    grad = torch.empty_like(l)
    us = _backward_us(l, K, off, counts, tokens, grad)
    few = torch.tensor([lead, 9, 23, 40], dtype=torch.int32, device=DEV)
    want = _run(l, idx, None, few, 1.0, 1.0)
    compare("padded", (loss, z, want[2], grad), reference(l, idx, None, few, 1.0, 1.0))
    assert torch.equal(grad, want[3])
    # (the last sequences that are not empty hold the counts)
    assert torch.equal(counts.view(S, n)[[999, 49999, 59999]], want[2])
    assert us < 2000, us


def _even(T, n, K):
    """Choices that give every id the same count (T K a multiple of n)."""
    return (torch.arange(T * K) % n).view(T, K).to(torch.int32)


# (T, n, K): the lanes of a token from 4 to a whole workgroup
EVEN = [(4096, 16, 4), (2048, 64, 8), (65536, 64, 8), (520, 260, 3), (4096, 1024, 8), (4096, 2048, 4), (8192, 4096, 16)]


@pytest.mark.parametrize("T,n,K", EVEN)
def test_an_even_load_has_no_gradient(T, n, K):
    """sum_j p_j = 1, so equal counts give c - sum_j p_j c_j = 0 whatever the logits; masked tokens, whose counts are
    not the tokens' share, do not change that."""
    l, _ = _inputs(T, n, K, T + n, std=2.0)
    idx = _even(T, n, K).to(DEV)
    assert not _run(l, idx, gz=0.0)[3].any()
    wide = torch.cat([l, l])
    on = torch.arange(2 * T, device=DEV) < T
    off = torch.tensor([0, T, 2 * T], dtype=torch.int32, device=DEV)
    assert not _run(wide, torch.cat([idx, idx]), on, None, gz=0.0)[3].any()
    assert not _run(wide, torch.cat([idx, idx]), None, off, gz=0.0)[3].any()


@pytest.mark.parametrize("T,n,K", EVEN)
def test_the_gradient_near_an_even_load(T, n, K):
    """Two ids one choice off the mean: the error goes by the counts' distance from the mean, not by the counts.
    With c' = c - mean (whole numbers) and p within e = (span + 16) 2^-23 of itself, d = sum_j p_j c'_j is within
    (e + n 2^-24) sum_j p_j |c'_j|, and an element, p share (c' - d), within 2 e + 4 2^-24 of its parts and that."""
    l, _ = _inputs(T, n, K, T + n)
    idx = _even(T, n, K)
    k = int((idx[0] == 0).nonzero()[0])
    idx[0, k] = next(e for e in range(n) if not (idx[0] == e).any())
    grad = _run(l, idx.to(DEV), g=1.0, gz=0.0)[3].cpu().double()
    p = torch.softmax(l.cpu().double(), 1)
    c = torch.bincount(idx.flatten().long(), minlength=n).double() - T * K // n
    assert c.abs().max() == 1 and c.sum() == 0
    share = n / (K * T * T)
    want = share * p * (c - (p * c).sum(1, keepdim=True))
    span = float((l.max(1)[0] - l.min(1)[0]).max())
    bound = (3 * (span + 16) + n / 2 + 4) * 2.0 ** -23 * share * p * (c.abs() + (p * c.abs()).sum(1, keepdim=True))
    err = (grad - want).abs()
    assert (err <= bound + 2.0 ** -126 * 4).all(), float((err / bound).max())


@pytest.mark.parametrize("T,n,K,S", [(300, 64, 8, 0), (3000, 160, 8, 0), (3000, 160, 8, 11), (20000, 33, 3, 0), (513, 1001, 4, 40),
                                     (4100, 1028, 8, 37), (2100, 4093, 3, 0), (0, 64, 4, 3), (0, 2000, 4, 0)])
def test_whatever_the_workspace_holds(T, n, K, S):
    """The same bits from workspaces of their exact size whose bytes are all 0, 0x7f or 0xff, and nothing written behind them."""
    l, idx = _inputs(T, n, K, n)
    off = _offsets(S, T, S, T // 50, T // 20) if S else None
    size = dm.moe_balance_workspace_size(T, n, S)
    got = []
    for byte in (0, 0x7F, 0xFF):
        room = torch.full((size + 4096,), byte, dtype=torch.uint8, device=DEV)
        outs = [torch.full((k,), 7, dtype=t, device=DEV) for k, t in
                ((1, torch.float32), (1, torch.float32), (max(S, 1) * n, torch.int32), (max(S, 1) + 1, torch.int32))]
        dm.moe_balance_fwd(l, idx, None, off, *outs, room[:size])
        assert (room[size:] == byte).all()
        got.append(outs)
    for outs in got[1:]:
        for a, b in zip(got[0], outs):
            assert torch.equal(a, b)
    ref = reference(l, idx, None, off)
    assert torch.equal(got[0][2].cpu().long().view(ref["counts"].shape), ref["counts"])
    assert abs(float(got[0][0]) - ref["loss"]) <= ref["loss_bound"] and abs(float(got[0][1]) - ref["z"]) <= ref["z_bound"]


@pytest.mark.parametrize("T,n,S", [(100, 64, 0), (5000, 64, 0), (5000, 260, 7), (3000, 1500, 0)])
def test_the_counts_are_the_callers(T, n, S):
    """What a step does to the counts before its backward (a sum over ranks in place, which leaves no trace on the tensor,
    or a bias update) does not reach the gradient."""
    l, idx = _inputs(T, n, 4, n)
    off = _offsets(S, T, S) if S else None
    want = _run(l, idx, None, off, 1.0, 1.0)
    for change in (lambda c: c.data.mul_(8), lambda c: c.mul_(8), lambda c: c.zero_()):
        x = l.clone().requires_grad_()
        loss, z, counts = dm.balance_loss(x, idx, seq_offsets=off)
        assert torch.equal(counts, want[2])
        change(counts)
        grad, = torch.autograd.grad(loss + z, x)
        assert torch.equal(grad, want[3])


def test_entries_refuse_what_is_no_tensor():
    l, idx = _inputs(20, 16, 2, 1)
    f = torch.empty(1, device=DEV)
    i = torch.empty(64, dtype=torch.int32, device=DEV)
    ws = torch.empty(dm.moe_balance_workspace_size(20, 16), dtype=torch.uint8, device=DEV)
    for bad in (None, 3, [1], torch.tensor(2, dtype=torch.int32, device=DEV)):
        with pytest.raises(dm.MoeError, match="topk_idx"):
            dm.moe_balance_fwd(l, bad, None, None, f, f, i, i, ws)
        if bad is not None:
            with pytest.raises(dm.MoeError, match="x_active_mask"):
                dm.moe_balance_fwd(l, idx, bad, None, f, f, i, i, ws)
            with pytest.raises(dm.MoeError, match="seq_offsets"):
                dm.moe_balance_fwd(l, idx, None, bad, f, f, i, i, ws)
            with pytest.raises(dm.MoeError, match="x_active_mask"):
                dm.moe_balance_bwd(l, 2, bad, None, i, i, f, f, l)
        with pytest.raises(dm.MoeError):
            dm.balance_loss(l, bad)


def test_an_even_load_of_masked_slots():
    """K n_s holds the masked slots of active tokens: a quarter of them masked, and an even load is 0.75."""
    l = torch.zeros(64, 32, device=DEV)
    idx = ((torch.arange(64)[:, None] * 3 + torch.arange(4)) % 32).to(torch.int32).to(DEV)
    mask = torch.ones(64, 4, dtype=torch.bool, device=DEV)
    mask[:, 3] = False
    loss, _, counts, _ = _run(l, idx, mask)
    assert (counts == 6).all() and float(loss) == 0.75


def test_large_even_counts_have_no_gradient():
    """Counts past 2^24 and their sum near 2^31, given to the backward."""
    n, T, c = 127, 8, 16909319
    l, _ = _inputs(T, n, 4, 1)
    counts = torch.full((n,), c, dtype=torch.int32, device=DEV)
    tokens = torch.full((2,), T, dtype=torch.int32, device=DEV)
    one = torch.ones(1, device=DEV)
    grad = torch.full_like(l, 7)
    dm.moe_balance_bwd(l, 4, None, None, counts, tokens, one, None, grad)
    assert not grad.any()
