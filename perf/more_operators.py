"""What the router's balance loss and the 8-bit activation checkpoints are measured on.

Each case is one pass of a training step through one operator, forward and backward:

* ``balance``  logits, choices -> balance loss, z loss, per-expert counts, and the gradient to the logits
* ``swiglu``   h = silu(G) * U of [G | U] rows that are kept in 8 bits, and [dG | dU] from the kept values
* ``combine``  out[t] = sum_k w[t, k] * row(t, k) (+ shared term), the experts' rows kept in 8 bits, and the routing
               weights' gradient <grad_out[t], kept row(t, k)>

Rows are kept as int8 codes with a bf16 scale for every 32 columns: scale = bf16(amax / 127), code =
rint(v * fp32(1 / scale)).

``run`` computes them in plain torch operations, or, where ``own`` is true, through dispatch_expert_gemm_amd.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLOCK = 32


# ----------------------------------------------------------------------------- cases


def _balance(name, T, n, K, seqs=0, mask=0, dtype="fp32"):
    return dict(name=name, op="balance", T=T, n=n, K=K, seqs=seqs, mask=mask, dtype=dtype)


def _swiglu(name, R, F):
    return dict(name=name, op="swiglu", R=R, F=F)


def _combine(name, T, H, E, K, special=False, mask=False, shared=False):
    return dict(name=name, op="combine", T=T, H=H, E=E, K=K, special=special, mask=mask, shared=shared)


def listed():
    return [
        # a small micro-batch: latency counts
        _balance("balance 256 tokens", 256, 64, 8),
        # the benchmark layer's batch: 8192 tokens, 64 experts, top 8
        _balance("balance 8192 tokens", 8192, 64, 8),
        # a packed batch of ragged sequences, each with its own balance; special experts among 260 ids, masked slots
        _balance("balance 37 sequences", 8192, 260, 8, seqs=37, mask=2),
        # a long batch whose logits come in bf16, padded at its end
        _balance("balance 65536 tokens bf16", 65536, 64, 8, mask=1, dtype="bf16"),
        # many fine-grained experts: the most logits
        _balance("balance 1024 experts", 32768, 1024, 16, seqs=8),
        # one token's eight rows of narrow experts: latency counts
        _swiglu("swiglu 8 rows", 8, 480),
        # odd sizes: 1000 rows of width 2 x 1001
        _swiglu("swiglu odd", 1000, 1001),
        # the benchmark layer's routed rows: 8192 tokens, top 8
        _swiglu("swiglu 65536 rows", 65536, 480),
        # 4096 tokens, top 8, through experts 2048 wide: the most bytes
        _swiglu("swiglu 32768 rows wide", 32768, 2048),
        # a small batch, top 2
        _combine("combine 64 tokens", 64, 1536, 64, 2),
        # the benchmark layer's batch
        _combine("combine 8192 tokens", 8192, 1536, 64, 8),
        # wide rows with zero, copy and constant experts, masked slots and a shared expert's term
        _combine("combine wide special", 4096, 7168, 32, 8, special=True, mask=True, shared=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "swiglu", "combine"])
    if op == "balance":
        n = _log_int(rng, 2, 1024)
        K = rng.randint(1, min(16, n))
        T = min(_log_int(rng, 1, 65536), 32768 * 1024 // n)
        c = _balance("", T, n, K, rng.choice([0, 0, _log_int(rng, 1, 256)]), rng.choice([0, 1, 2]),
                     rng.choice(["fp32", "fp32", "bf16"]))
    elif op == "swiglu":
        F = rng.choice([32 * _log_int(rng, 1, 128), _log_int(rng, 1, 4096)])
        R = max(1, min(_log_int(rng, 1, 65536), 32768 * 2048 // F))
        c = _swiglu("", R, F)
    else:
        H = 8 * _log_int(rng, 8, 896)
        E = _log_int(rng, 2, 64)
        K = rng.randint(1, min(8, E))
        T = max(1, min(_log_int(rng, 1, 16384), 4096 * 7168 * 8 // (H * K)))
        c = _combine("", T, H, E, K, rng.random() < 0.4, rng.random() < 0.4, rng.random() < 0.5)
    del c["name"]
    return c


# ----------------------------------------------------------------------------- inputs


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "balance":
        T, n, K, S = (case[k] for k in ("T", "n", "K", "seqs"))
        # some experts are liked better than others
        l = torch.randn(T, n, generator=g, device=DEV) + torch.randn(n, generator=g, device=DEV)
        st["idx"] = l.topk(K)[1].to(torch.int32)
        st["logits"] = l.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32).requires_grad_()
        st["mask"] = None
        if case["mask"] == 1:
            st["mask"] = torch.arange(T, device=DEV) < T - T // 16
        elif case["mask"] == 2:
            st["mask"] = torch.rand(T, K, generator=g, device=DEV) >= 0.1
        st["offsets"] = None
        if S:
            # sequences of any length, empty ones too, and a few tokens behind the last
            cuts = (torch.rand(S - 1, generator=g, device=DEV) * (T - T // 32)).to(torch.int32).sort()[0]
            ends = torch.tensor([0, T - T // 32], dtype=torch.int32).to(DEV)
            st["offsets"] = torch.cat([ends[:1], cuts, ends[1:]])
        st["grads"] = [torch.rand((), generator=g, device=DEV) + 0.5 for _ in range(2)]
    elif case["op"] == "swiglu":
        R, F = case["R"], case["F"]
        st["gate_up"] = _normal(g, (R, 2 * F)).requires_grad_()
        st["grad_h"] = _normal(g, (R, F), 0.1)
    else:
        T, H, E, K = (case[k] for k in ("T", "H", "E", "K"))
        Z, C, Q = (1, 1, 2) if case["special"] else (0, 0, 0)
        st["ids"] = (Z, C, Q)
        p, i = torch.randn(T, E + Z + C + Q, generator=g, device=DEV).softmax(-1).topk(K)
        st["idx"], st["w"] = i.to(torch.int32), (p / p.sum(-1, keepdim=True)).contiguous()
        st["mask"] = (torch.rand(T, K, generator=g, device=DEV) >= 0.1).to(torch.uint8) if case["mask"] else None
        st["y"], st["x"], st["grad_out"] = (_normal(g, s) for s in ((T * min(E, K), H), (T, H), (T, H)))
        st["shared"] = _normal(g, (T, H)) if case["shared"] else None
        st["const"] = [_normal(g, (Q, H)) for _ in range(3)] if Q else [None] * 3
        # the routing that the layer's dispatch left: each expert's rows in slot order
        idx = st["idx"].reshape(-1)
        on = torch.ones_like(idx, dtype=torch.bool) if st["mask"] is None else st["mask"].reshape(-1) != 0
        routed = on & (idx < E)
        key = torch.where(routed, idx, torch.full_like(idx, E))
        order = key.sort(stable=True)[1].to(torch.int32)
        row = torch.empty_like(order)
        row[order.long()] = torch.arange(T * K, dtype=torch.int32, device=DEV)
        none = torch.full_like(row, -1)
        special = torch.where(idx < E + Z, none, torch.where(idx < E + Z + C, none - 1, none * (3 - E - Z - C) - idx))
        st["assist"] = torch.cat([torch.where(routed, row, torch.where(on, special, none)),
                                  order[:T * min(E, K)]]).contiguous()
        st["counts"] = (key[:, None] == torch.arange(E, device=DEV)).sum(0).cumsum(0).to(torch.int32)
    return st


# ----------------------------------------------------------------------------- one pass


def run(st):
    op = st["case"]["op"]
    if own:
        return {"balance": _own_balance, "swiglu": _own_swiglu, "combine": _own_combine}[op](st)
    with torch.no_grad():
        return {"balance": _plain_balance, "swiglu": _plain_swiglu, "combine": _plain_combine}[op](st)


def _own_balance(st):
    import dispatch_expert_gemm_amd as dm
    loss, z_loss, counts = dm.balance_loss(st["logits"], st["idx"], x_active_mask=st["mask"],
                                           seq_offsets=st["offsets"])
    grad, = torch.autograd.grad((loss, z_loss), st["logits"], st["grads"])
    return loss.detach(), z_loss.detach(), counts, grad


def _own_swiglu(st):
    import dispatch_expert_gemm_amd as dm
    h = dm.swiglu_checkpoint(st["gate_up"])
    grad, = torch.autograd.grad(h, st["gate_up"], st["grad_h"])
    return h.detach(), grad


def _own_combine(st):
    import dispatch_expert_gemm_amd as dm
    case, x = st["case"], st["x"]
    T, H, E, K = (case[k] for k in ("T", "H", "E", "K"))
    Z, C, Q = st["ids"]
    shape = dm.make_shape(T, H, K, E, zero_expert_num=Z, copy_expert_num=C, const_expert_num=Q,
                          mask_ndim=2 if case["mask"] else 0)
    out = torch.empty_like(x)
    codes, scales = dm.checkpoint_buffers(shape.capacity, H, x.device)
    args = (st["idx"], st["w"], st["assist"], st["counts"], st["mask"])
    dm.moe_combine_checkpoint(shape, st["y"], *args, st["shared"], x, *st["const"], out, codes, scales)
    grad_w = torch.empty_like(st["w"])
    dm.moe_combine_bwd_weights_checkpoint(shape, st["grad_out"], codes, scales, *args, x, *st["const"], grad_w, None)
    return out, grad_w


def _plain_balance(st):
    l, idx, off = st["logits"].float(), st["idx"].long(), st["offsets"]
    (T, n), K = l.shape, idx.shape[1]
    if off is None:
        off = torch.tensor([0, T], dtype=torch.int32, device=l.device)
    S = off.shape[0] - 1
    t = torch.arange(T, device=l.device)
    seq = (t[:, None] >= off[None, 1:]).sum(1)
    inside = (t >= off[0]) & (seq < S)
    seq = seq.clamp(max=S - 1)
    slots = inside[:, None].expand(T, K)
    if st["mask"] is not None:
        slots = slots & (st["mask"] if st["mask"].dim() == 2 else st["mask"][:, None])
    tokens = slots.any(1)
    m = l.max(-1, keepdim=True)[0]
    e = torch.exp(l - m)
    total = e.sum(-1, keepdim=True)
    p = e / total * tokens[:, None]
    lse = (m + torch.log(total))[:, 0] * tokens
    counts = torch.zeros(S * n, dtype=torch.int32, device=l.device)
    counts = counts.scatter_add_(0, (seq[:, None] * n + idx).reshape(-1), slots.reshape(-1).to(torch.int32)).reshape(S, n)
    # sums over a sequence, as products with the tokens that belong to it
    member = ((seq[:, None] == torch.arange(S, device=l.device)) & tokens[:, None]).float().t()
    P, each = member @ p, member.sum(1)
    N = each.sum().clamp(min=1)
    share = n / (K * N) / each.clamp(min=1)
    loss = (share[:, None] * counts * P).sum()
    z_loss = lse.square().sum() / N
    g, gz = st["grads"]
    a = (g * share)[seq][:, None]
    c = counts.float()[seq]
    grad = a * p * (c - (p * c).sum(-1, keepdim=True)) + (2 * gz / N) * lse[:, None] * p
    return loss, z_loss, counts if st["offsets"] is not None else counts[0], grad.to(st["logits"].dtype)


def _kept(v):
    """The values that rows (..., W) are kept as."""
    W = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, -W % BLOCK)).unflatten(-1, (-1, BLOCK))
    s = (b.abs().amax(-1, keepdim=True) / 127.0).to(torch.bfloat16).float()
    q = (b * torch.where(s > 0, 1.0 / s, torch.zeros_like(s))).round().clamp(-127, 127)
    return (q * s).flatten(-2)[..., :W]


def _plain_swiglu(st):
    gu, dh = st["gate_up"].float(), st["grad_h"].float()
    F = dh.shape[-1]
    g, u = gu[:, :F], gu[:, F:]
    h = g * torch.sigmoid(g) * u
    g, u = _kept(g), _kept(u)
    sig = torch.sigmoid(g)
    grad = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], -1)
    return h.to(torch.bfloat16), grad.to(torch.bfloat16)


def _plain_combine(st):
    case, x, d = st["case"], st["x"].float(), st["grad_out"].float()
    T, H, K, E = (case[k] for k in ("T", "H", "K", "E"))
    Z, C, Q = st["ids"]
    row = st["assist"][:T * K].reshape(T, K)
    w = st["w"]
    routed = row >= 0
    v = st["y"].float()[row.clamp(min=0).long()]
    out = (v * (w * routed)[:, :, None]).sum(1)
    grad_w = (_kept(v) * d[:, None, :]).sum(-1) * routed
    if C or Q:
        copied = row == -2
        out = out + (w * copied).sum(1, keepdim=True) * x
        grad_w = grad_w + copied * (x * d).sum(-1, keepdim=True)
        a1, a2, c = (t.float() for t in st["const"])
        const = row[:, :, None] == -3 - torch.arange(Q, device=x.device)
        share = (w[:, :, None] * const).sum(1)
        out = out + (share @ a1) * x + share @ (a2 * c)
        grad_w = grad_w + (const * ((x * d) @ a1.t() + d @ (a2 * c).t())[:, None, :]).sum(-1)
    if st["shared"] is not None:
        out = out + st["shared"].float()
    return out.to(torch.bfloat16), grad_w


# ----------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "balance":
        T, n, K = case["T"], case["n"], case["K"]
        each = 2 if case["dtype"] == "bf16" else 4
        mask = {0: 0, 1: T, 2: T * K}[case["mask"]]
        # the logits are an input of both directions; the gradient is written once
        return dict(bytes=3 * each * T * n + 4 * T * K + mask + 4 * n * max(1, case["seqs"]), flops=14 * T * n)
    if case["op"] == "swiglu":
        R, F = case["R"], case["F"]
        kept = 2 * (F + 2 * -(-F // BLOCK))
        return dict(bytes=R * (4 * F + 2 * F + kept + kept + 2 * F + 4 * F), flops=R * F * 40)
    T, H, E, K = (case[k] for k in ("T", "H", "E", "K"))
    rows = T * K * E / (E + (4 if case["special"] else 0)) * (0.9 if case["mask"] else 1.0)
    kept = H + 2 * -(-H // BLOCK)
    tokens = T * H * 2 * (2 + (1 if case["shared"] else 0) + (2 if case["special"] else 0))
    return dict(bytes=rows * (2 * H + 2 * kept) + tokens + 16 * T * K, flops=rows * H * 9)


# ----------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return {"balance": _exact_balance, "swiglu": _exact_swiglu, "combine": _exact_combine}[case["op"]](st)


def _exact_balance(st):
    case, idx = st["case"], st["idx"].long()
    l = st["logits"].detach().double().requires_grad_()
    T, n, K = case["T"], case["n"], case["K"]
    mask = torch.ones(T, K, dtype=torch.bool, device=l.device) if st["mask"] is None else st["mask"]
    mask = mask if mask.dim() == 2 else mask[:, None].expand(T, K)
    ends = [0, T] if st["offsets"] is None else st["offsets"].tolist()
    if T * n * 8 * 6 > 16 << 30 or len(ends) > 2000:
        return None
    here = torch.zeros(T, dtype=torch.bool, device=l.device)
    here[ends[0]:ends[-1]] = True
    mask = mask & here[:, None]
    on = mask.any(1)
    N = max(1, int(on.sum()))
    p = torch.softmax(l, -1)
    loss, counts = l.new_zeros(()), torch.zeros(len(ends) - 1, n, dtype=torch.int64, device=l.device)
    for s, (a, b) in enumerate(zip(ends, ends[1:])):
        picked = idx[a:b][mask[a:b]]
        counts[s] = torch.bincount(picked, minlength=n)
        if picked.numel():
            tokens = on[a:b].double()
            f = counts[s].double() * n / (K * tokens.sum())
            loss = loss + (f * (tokens @ p[a:b])).sum() / N
    z_loss = (torch.logsumexp(l, -1)[on] ** 2).sum() / N
    grad, = torch.autograd.grad(loss * st["grads"][0].double() + z_loss * st["grads"][1].double(), l)
    counts = counts if st["offsets"] is not None else counts[0]
    return loss.detach(), z_loss.detach(), counts.to(torch.int32), grad


def _stand_for(rows):
    """What bf16 rows are kept as, in 64 bits: the whole numbers are fixed by 32-bit products (the rule's own), so a
    value next to a border goes the same way."""
    out = torch.empty_like(rows, dtype=torch.float64)
    W = rows.shape[-1]
    for a in range(0, W, BLOCK * 64):
        part = rows[:, a:a + BLOCK * 64].float()
        full = part.shape[1] // BLOCK * BLOCK
        for lo, hi, blocks in ((0, full, full // BLOCK), (full, part.shape[1], 1)):
            if hi == lo:
                continue
            v = part[:, lo:hi].reshape(part.shape[0], blocks, (hi - lo) // blocks)
            step = torch.linalg.vector_norm(v, float("inf"), dim=-1).div(127).bfloat16().float()
            back = torch.where(step == 0, step, step.reciprocal())
            whole = torch.round(v * back[..., None]).double()
            out[:, a + lo:a + hi] = (whole * step.double()[..., None]).reshape(part.shape[0], hi - lo)
    return out


def _exact_swiglu(st):
    F = st["case"]["F"]
    gu = st["gate_up"].detach()
    g = gu[:, :F].double()
    h = g / (1 + torch.exp(-g)) * gu[:, F:].double()
    g, d = _stand_for(gu[:, :F]), st["grad_h"].double()
    low = 1 / (1 + torch.exp(-g))
    dg = (low + g * low * (1 - low)).mul_(d).mul_(_stand_for(gu[:, F:]))
    return h, torch.cat([dg, g * low * d], 1)


def _exact_combine(st):
    case, x, d = st["case"], st["x"].double(), st["grad_out"].double()
    T, E, K = case["T"], case["E"], case["K"]
    Z, C, Q = st["ids"]
    out = torch.zeros_like(x) if st["shared"] is None else st["shared"].double()
    grad_w = torch.zeros(T, K, dtype=torch.float64, device=x.device)
    for k in range(K):
        i, w = st["idx"][:, k], st["w"][:, k].double()[:, None]
        on = torch.ones_like(i, dtype=torch.bool) if st["mask"] is None else st["mask"][:, k] != 0
        t = torch.nonzero(on & (i < E))[:, 0]
        rows = st["y"][st["assist"][t * K + k].long()]
        out[t] += w[t] * rows.double()
        grad_w[t, k] = (d[t] * _stand_for(rows)).sum(-1)
        for e in range(E + Z, E + Z + C + Q):
            t = torch.nonzero(on & (i == e))[:, 0]
            v = x[t]
            if e >= E + Z + C:
                a1, a2, c = (p[e - E - Z - C].double() for p in st["const"])
                v = a1 * v + a2 * c
            out[t] += w[t] * v
            grad_w[t, k] = (d[t] * v).sum(-1)
    return out, grad_w
