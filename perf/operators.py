"""What the int8 matrix product and the few-token MoE layer are measured on.

Each case is one call as a serving loop makes it:

* ``linear``     out = bf16(int(xq . wq) * xs * ws (+ bias)): a dense projection on 8-bit operands, the
                 activations either int8 codes with their scales or bf16 rows quantised in the call
* ``moe``        a whole MoE layer forward (experts' SwiGLU FFN, weighted sum, special experts, shared
                 expert) of a decode step with a few tokens, bf16 weights
* ``moe_int8``   the same layer on int8 weights: rows (times the expert's smooth scales) and h quantised per row

``run`` computes them in plain torch operations, or, where ``own`` is true, through dispatch_expert_gemm_amd.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------- cases


def _linear(name, M, N, K, dynamic, bias):
    return dict(name=name, op="linear", M=M, N=N, K=K, dynamic=dynamic, bias=bias)


def _moe(name, op, T, H, F, E, K, shared=0, special=False, mask=False, smooth=False):
    return dict(name=name, op=op, T=T, H=H, F=F, E=E, K=K, shared=shared, special=special, mask=mask, smooth=smooth)


def listed():
    return [
        # one token through a square projection at the decode workload's hidden size: latency counts
        _linear("linear 1 token", 1, 7168, 7168, True, False),
        # a ragged batch of sequences through a down projection with a bias, codes from an earlier quantiser
        _linear("linear 37 tokens", 37, 7168, 2048, False, True),
        # a prefill chunk through a shared expert's gate|up product
        _linear("linear 512 tokens", 512, 4096, 7168, True, False),
        # a long prefill through a wide FFN product
        _linear("linear 8192 tokens", 8192, 14336, 4096, False, False),
        # one token of a fine-grained layer (64 narrow experts, top 8): little to read, latency counts
        _moe("moe 1 token narrow", "moe", 1, 1536, 480, 64, 8),
        # one token of the decode workload's layer with its shared expert
        _moe("moe 1 token shared", "moe", 1, 7168, 2048, 32, 8, shared=2048),
        # a ragged batch with padded slots and zero, copy and constant experts among the ids
        _moe("moe 13 tokens special", "moe", 13, 7168, 2048, 32, 8, special=True, mask=True),
        # a full few-token batch on eight wide experts, top 2: the most bytes
        _moe("moe 64 tokens wide", "moe", 64, 4096, 14336, 8, 2),
        # the int8 layer: one token, shared expert, no smooth scales
        _moe("int8 moe 1 token shared", "moe_int8", 1, 7168, 2048, 32, 8, shared=2048),
        # a small batch with smooth scales and special experts
        _moe("int8 moe 9 tokens smooth", "moe_int8", 9, 7168, 2048, 32, 8, special=True, smooth=True),
        # narrow experts, an ordinary batch, every expert in use
        _moe("int8 moe 48 tokens narrow", "moe_int8", 48, 1536, 480, 64, 8, smooth=True, mask=True),
        # the largest int8 batch: every expert streams once for about 16 rows
        _moe("int8 moe 64 tokens", "moe_int8", 64, 7168, 2048, 32, 8, shared=2048, smooth=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "moe", "moe_int8"])
    if op == "linear":
        K = 16 * _log_int(rng, 8, 448)
        N = _log_int(rng, 64, 14336)
        M = _log_int(rng, 1, 8192)
        M = max(1, min(M, 8192 * 14336 * 4096 // (N * K)))
        c = _linear("", M, N, K, rng.random() < 0.5, rng.random() < 0.5)
    else:
        H = 16 * _log_int(rng, 32, 448)
        F = 32 * _log_int(rng, 4, 128)
        E = _log_int(rng, 4, 64)
        E = max(4, min(E, 8 * 14336 * 4096 // (F * H)))
        K = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 64)
        shared = rng.choice([0, 0, 32 * _log_int(rng, 4, 64)])
        c = _moe("", op, T, H, F, E, K, shared, rng.random() < 0.4, rng.random() < 0.4,
                 op == "moe_int8" and rng.random() < 0.5)
    del c["name"]
    return c


# ----------------------------------------------------------------------------- inputs


def _normal(g, shape, std):
    """bf16 N(0, std^2), drawn a slice at a time."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for o in out.reshape(shape[0], -1):
        o.copy_(torch.randn(o.shape, generator=g, device=DEV, dtype=torch.float32).mul_(std))
    return out


def _codes(w):
    """int8 codes and one scale for each row of the last dimension."""
    codes, scales = torch.empty(w.shape, dtype=torch.int8, device=DEV), torch.empty(w.shape[:-1], device=DEV)
    n = w.shape[-1]
    for c, s, r in zip(codes.reshape(w.shape[0], -1), scales.reshape(w.shape[0], -1), w.reshape(w.shape[0], -1)):
        q, a = _quant(r.reshape(-1, n).float())
        c.copy_(q.reshape(-1))
        s.copy_(a.reshape(-1))
    return codes, scales


def _quant(v):
    """Rows of fp32 values to (codes as fp32, scales): clamp(rint(v * (127 / amax))), amax / 127."""
    amax = v.abs().amax(-1, keepdim=True)
    some = amax > 0
    inv = torch.where(some, 127.0 / amax, torch.zeros_like(amax))
    return (v * inv).round().clamp(-127, 127), torch.where(some, amax / 127.0, torch.ones_like(amax))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        st["wq"] = _codes(_normal(g, (N, K), K ** -0.5).reshape(1, N, K))
        st["wq"] = tuple(t[0] for t in st["wq"])
        x = _normal(g, (M, K), 1.0)
        if case["dynamic"]:
            st["x"] = x
        else:
            q, s = _quant(x.float())
            st["x"], st["xs"] = q.to(torch.int8), s[:, 0].contiguous()
        st["bias"] = torch.randn(N, generator=g, device=DEV) if case["bias"] else None
        return st
    T, H, F, E, K = (case[k] for k in ("T", "H", "F", "E", "K"))
    Z, C, Q = (1, 1, 2) if case["special"] else (0, 0, 0)
    st["ids"] = (Z, C, Q)
    st["x"] = _normal(g, (T, H), 1.0)
    p, i = torch.randn(T, E + Z + C + Q, generator=g, device=DEV).softmax(-1).topk(K)
    st["idx"], st["w"] = i.to(torch.int32), (p / p.sum(-1, keepdim=True)).contiguous()
    st["mask"] = (torch.rand(T, K, generator=g, device=DEV) >= 0.1).to(torch.uint8) if case["mask"] else None
    ws = [_normal(g, (E, F, H), H ** -0.5), _normal(g, (E, F, H), H ** -0.5), _normal(g, (E, H, F), F ** -0.5)]
    sw = None
    if case["shared"]:
        S = case["shared"]
        sw = [_normal(g, (1, S, H), H ** -0.5), _normal(g, (1, S, H), H ** -0.5), _normal(g, (1, H, S), S ** -0.5)]
    if case["op"] == "moe_int8":
        ws = [_codes(w) for w in ws]
        sw = [_codes(w) for w in sw] if sw else None
    st["ws"], st["sw"] = ws, sw
    st["smooth"] = torch.randn(E, H, generator=g, device=DEV).mul_(0.5).exp_() if case["smooth"] else None
    st["const"] = [_normal(g, (Q, H), 1.0) for _ in range(3)] if Q else [None] * 3
    return st


# ----------------------------------------------------------------------------- one pass


def run(st):
    case = st["case"]
    if own:
        return _own_linear(st) if case["op"] == "linear" else _own_moe(st)
    return _plain_linear(st) if case["op"] == "linear" else _plain_moe(st)


def _own_linear(st):
    import dispatch_expert_gemm_amd as dm
    return dm.linear_int8(st["x"], st["wq"], x_scales=st.get("xs"), bias=st["bias"])


def _own_moe(st):
    import dispatch_expert_gemm_amd as dm
    Z, C, Q = st["ids"]
    sw = st["sw"] or (None, None, None)
    return dm.moe_layer_few_tokens(st["x"], st["idx"], st["w"], *st["ws"], smooth_scales=st["smooth"],
                                   x_active_mask=st["mask"], shared_w_gate=sw[0], shared_w_up=sw[1],
                                   shared_w_down=sw[2], const_alpha_1=st["const"][0], const_alpha_2=st["const"][1],
                                   const_v=st["const"][2], zero_expert_num=Z, copy_expert_num=C, const_expert_num=Q)


def _plain_linear(st):
    wq, ws = st["wq"]
    if st["case"]["dynamic"]:
        x, xs = _quant(st["x"].float())
    else:
        x, xs = st["x"].float(), st["xs"][:, None]
    y = (x @ wq.float().t()) * (xs * ws)
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(torch.bfloat16)


def _ffn(x, ws, pick, smooth):
    """SwiGLU of x (B, R, H) by the B experts `pick` of ws (all of them, in order, where it is None): (B, R, H) fp32."""
    def weight(w):
        w = w if pick is None else w[pick]
        return w.float()

    def product(v, w):
        if isinstance(w, torch.Tensor):
            return torch.bmm(v, weight(w).transpose(1, 2))
        q, s = _quant(v)
        return torch.bmm(q, weight(w[0]).transpose(1, 2)) * (s * weight(w[1])[:, None, :])

    if smooth is not None:
        x = x * weight(smooth)[:, None, :]
    g, u = product(x, ws[0]), product(x, ws[1])
    return product(g * torch.sigmoid(g) * u, ws[2])


def _plain_moe(st):
    case, idx, x = st["case"], st["idx"].long(), st["x"].float()
    T, H, E, K = (case[k] for k in ("T", "H", "E", "K"))
    Z, C, Q = st["ids"]
    w = st["w"] if st["mask"] is None else st["w"] * (st["mask"] != 0)
    if T * K <= E:
        # fewer choices than experts: each choice's expert is picked out
        pick = idx.clamp(max=E - 1).reshape(-1)
        y = _ffn(x.repeat_interleave(K, 0)[:, None, :], st["ws"], pick, st["smooth"])
        out = (y.reshape(T, K, H) * (w * (idx < E))[:, :, None]).sum(1)
    else:
        # every token through every expert, weighted by what it gives that expert
        y = _ffn(x.expand(E, T, H), st["ws"], None, st["smooth"])
        share = torch.zeros(T, E + Z + C + Q, device=x.device).scatter_add_(1, idx, w)
        out = (y * share[:, :E].t()[:, :, None]).sum(0)
    if C or Q:
        copied = (idx >= E + Z) & (idx < E + Z + C)
        out = out + (w * copied).sum(1, keepdim=True) * x
        a1, a2, v = (t.float() for t in st["const"])
        share = (w[:, :, None] * (idx[:, :, None] == E + Z + C + torch.arange(Q, device=x.device))).sum(1)
        out = out + (share @ a1) * x + share @ (a2 * v)
    if st["sw"] is not None:
        out = out + _ffn(x[None], st["sw"], None, None)[0]
    return out.to(torch.bfloat16)


# ----------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        read = N * K + 4 * N * (2 if case["bias"] else 1) + (2 * M * K if case["dynamic"] else M * K + 4 * M)
        return dict(bytes=read + 2 * M * N, flops=2 * M * N * K)
    T, H, F, E, K, S = (case[k] for k in ("T", "H", "F", "E", "K", "shared"))
    ids = E + (4 if case["special"] else 0)
    rows = T * K * E / ids * (0.9 if case["mask"] else 1.0)
    # experts that some row of a uniform choice goes to
    used = E * (1 - (1 - rows / (T * E)) ** T)
    each = 1 if case["op"] == "moe_int8" else 2
    per = 3 * F * H * each + (4 * (2 * F + H) if each == 1 else 0) + (4 * H if case["smooth"] else 0)
    sper = (3 * S * H * each + (4 * (2 * S + H) if each == 1 else 0)) if S else 0
    other = 4 * T * H + 8 * T * K + (12 * H if case["special"] else 0) + (T * K if case["mask"] else 0)
    return dict(bytes=used * per + sper + other, flops=6 * H * (rows * F + T * S))


# ----------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_linear(st) if case["op"] == "linear" else _exact_moe(st)


def _rows_to_int8(v):
    """The quantiser's rule on rows: whole numbers and the row's step, in 64 bits.  Where the rows are given in
    32 bits the whole numbers are fixed by 32-bit products, so a value next to a border goes the same way."""
    top = torch.linalg.vector_norm(v, float("inf"), dim=-1, keepdim=True)
    whole = torch.round(v * (127 / top.clamp(min=torch.finfo(v.dtype).tiny))).clamp_(-127, 127).double()
    return whole, torch.where(top > 0, top.double() / 127, torch.ones_like(top).double())


def _exact_linear(st):
    if st["case"]["dynamic"]:
        x, step = _rows_to_int8(st["x"].float())
    else:
        x, step = st["x"].double(), st["xs"].double()[:, None]
    out = torch.matmul(x, st["wq"][0].double().t())
    out *= step
    out *= st["wq"][1].double()
    return out if st["bias"] is None else out.add_(st["bias"].double())


def _exact_expert(rows, ws, e, smooth):
    if isinstance(ws[0], torch.Tensor):
        wg, wu, wd = (w[e].double() for w in ws)
        g, u = rows.double() @ wg.t(), rows.double() @ wu.t()
        return (g / (1 + torch.exp(-g)) * u) @ wd.t()
    q, s = _rows_to_int8(rows.float() if smooth is None else rows.float() * smooth[e])
    g, u = (q @ w[0][e].double().t() * s * w[1][e].double() for w in ws[:2])
    q, s = _rows_to_int8(g / (1 + torch.exp(-g)) * u)
    return q @ ws[2][0][e].double().t() * s * ws[2][1][e].double()


def _exact_moe(st):
    case, x = st["case"], st["x"].double()
    Z, C, Q = st["ids"]
    E = case["E"]
    out = torch.zeros_like(x)
    w = st["w"].double()
    if st["mask"] is not None:
        w = torch.where(st["mask"] != 0, w, torch.zeros_like(w))
    for e in range(E):
        t, k = torch.nonzero(st["idx"] == e, as_tuple=True)
        if t.numel():
            out.index_add_(0, t, _exact_expert(st["x"][t], st["ws"], e, st["smooth"]) * w[t, k][:, None])
    for e in range(E + Z, E + Z + C + Q):
        t, k = torch.nonzero(st["idx"] == e, as_tuple=True)
        v = x[t]
        if e >= E + Z + C:
            a1, a2, c = (p[e - E - Z - C].double() for p in st["const"])
            v = a1 * v + a2 * c
        out.index_add_(0, t, v * w[t, k][:, None])
    if st["sw"] is not None:
        out += _exact_expert(st["x"], st["sw"], 0, None)
    return out
