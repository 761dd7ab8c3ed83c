"""Plain 64-bit forms of the few-token layer and of the int8 matrix product, with
the error their kernels may make, element by element.

A sum of n products held in fp32 is within n 2^-23 of the sum of the magnitudes
(2^-24 for each product's and each addition's rounding).  An output is rounded to
bf16 once: 2^-8 of its value.  The rest is written at the lines it belongs to."""
from __future__ import annotations

import torch

BF16_STEP = 2.0 ** -8
U = 2.0 ** -23


def to_int8(v):
    """Rows of fp32 values -> (codes, scales) in double; the codes by the rule's fp32 operations:
    127 / amax is 127 times the rounded reciprocal."""
    assert v.dtype == torch.float32
    amax = v.abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, (127.0 * (torch.ones_like(amax) / amax)).clamp(max=torch.finfo(torch.float32).max),
                      torch.zeros_like(amax))
    q = (v * inv).round().clamp(-127, 127)
    return q.double(), torch.where(amax > 0, amax.double() / 127, torch.ones_like(amax, dtype=torch.float64))


def quant_weight(w):
    """bf16 weights (..., K) -> (int8 codes, fp32 scales)."""
    q, s = to_int8(w.float())
    return q.to(torch.int8).contiguous(), s[..., 0].float().contiguous()


def linear64(x, w, bias=None):
    """(value, error) of x (codes, scales) times w (codes, scales); exact integer sums, then a
    conversion to fp32, two products and an addition: 4 roundings of 2^-24."""
    isum = x[0].double() @ w[0].double().t()
    v = isum * x[1].double()[:, None] * w[1].double()
    mag = v.abs()
    if bias is not None:
        v = v + bias.double()
        mag = mag + bias.double().abs()
    return v, v.abs() * BF16_STEP + 2 * U * mag


def ffn64(x, ws, smooth=None):
    """One expert's FFN of rows x (n, H) bf16: (y, |error| of y), doubles."""
    if isinstance(ws[0], torch.Tensor):
        wg, wu, wd = (w.double() for w in ws)
        xd = x.double()
        n = x.shape[1]
        g, u = xd @ wg.t(), xd @ wu.t()
        dg, du = n * U * (xd.abs() @ wg.abs().t()), n * U * (xd.abs() @ wu.abs().t())
    else:
        v = x.float() if smooth is None else x.float() * smooth
        q, s = to_int8(v)
        (wg, sg), (wu, su), (wd, sd) = ((c.double(), t.double()) for c, t in ws)
        g, u = q @ wg.t() * s * sg, q @ wu.t() * s * su
        dg, du = 4 * U * g.abs(), 4 * U * u.abs()     # conversion, scale products
    silu = g / (1 + torch.exp(-g))
    h = silu * u
    # |silu'| <= 1.1; the exponential's argument and the quotient: (|g| + 8) 2^-22
    dh = 1.1 * u.abs() * dg + silu.abs() * du + 2 * U * (g.abs() + 8) * h.abs()
    if isinstance(ws[0], torch.Tensor):
        # two bf16 parts: 2^-17 of h
        dh = dh + 2.0 ** -17 * h.abs()
        n = h.shape[1]
        return h @ wd.t(), dh @ wd.abs().t() + n * U * (h.abs() @ wd.abs().t())
    amax = h.abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, 127 / amax.clamp(min=1e-300), torch.zeros_like(amax))
    q = (h * inv).round().clamp(-127, 127)
    step = torch.where(amax > 0, amax / 127, torch.ones_like(amax))
    y = q @ wd.t() * step * sd
    # the row's step moves with its largest value, and a code whose value lies next to a border may
    # be its neighbour: within the error of h, of the step and of the product
    damax = torch.where(amax > 0, dh.amax(-1, keepdim=True) / amax.clamp(min=1e-300), torch.zeros_like(amax))
    flip = ((h * inv - q).abs() > 0.5 - (dh * inv + 127 * (damax + 2 * U))).double()
    dy = (flip @ wd.abs().t() + q.abs() @ wd.abs().t() * (damax + 6 * U)) * step * sd
    return y, dy


def layer64(x, idx, w, ws, *, smooth=None, mask=None, shared_x=None, shared_w=None, const=None, Z=0, C=0, Q=0):
    """(out before its rounding, error bound of the rounded out, err flag) of the whole layer."""
    T, H = x.shape
    K = idx.shape[1]
    int8 = not isinstance(ws[0], torch.Tensor)
    E = (ws[0][0] if int8 else ws[0]).shape[0]
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    mag = torch.zeros_like(out)
    flag = 0
    ids = idx.cpu().tolist()
    act = [[True] * K for _ in range(T)]
    if mask is not None:
        m = mask.cpu().tolist()
        for t in range(T):
            for k in range(K):
                act[t][k] = bool(m[t][k] if mask.dim() == 2 else m[t])
        if mask.dim() == 1 and any(m[t] and not m[t - 1] for t in range(1, T)):
            flag |= 4
    rows = {}
    for t in range(T):
        for k in range(K):
            e = ids[t][k]
            if not 0 <= e < E + Z + C + Q:
                flag |= 1
            elif e in ids[t][:k]:
                flag |= 2
            elif act[t][k]:
                rows.setdefault(e, []).append((t, k))
    for e, tk in sorted(rows.items()):
        t = torch.tensor([a for a, _ in tk], device=x.device)
        k = torch.tensor([b for _, b in tk], device=x.device)
        wt = w[t, k].double()[:, None]
        if e < E:
            pick = [(c[e], s[e]) for c, s in ws] if int8 else [v[e] for v in ws]
            y, dy = ffn64(x[t], pick, None if smooth is None else smooth[e])
        elif e < E + Z:
            continue
        else:
            y = x[t].double()
            dy = torch.zeros_like(y)
            if e >= E + Z + C:
                a1, a2, cv = (p[e - E - Z - C].double() for p in const)
                dy = 4 * U * ((a1 * y).abs() + (a2 * cv).abs())
                y = a1 * y + a2 * cv
        out.index_add_(0, t, wt * y)
        err.index_add_(0, t, wt.abs() * dy)
        mag.index_add_(0, t, (wt * y).abs())
    if shared_w is not None:
        pick = [(c[0], s[0]) for c, s in shared_w] if int8 else [v[0] for v in shared_w]
        y, dy = ffn64(x, pick)
        out, err, mag = out + y, err + dy, mag + y.abs()
    if shared_x is not None:
        out, mag = out + shared_x.double(), mag + shared_x.double().abs()
    # K + 9 terms joined in fp32 (the waves' parts and the special experts)
    err = err + (K + 10) * U * mag
    return out, out.abs() * BF16_STEP + err * (1 + BF16_STEP) + 1e-38, flag


def check(name, got, ref, bound):
    got = got.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    if got.numel():
        # (an exact zero has a bound of zero)
        ratio = ((got - ref).abs() / bound.clamp(min=1e-300)).max().item()
        print(f"[{name}] worst err/bound {ratio:.3f}", flush=True)
        assert ratio <= 1, f"{name}: error {ratio:.3f} of its bound"
