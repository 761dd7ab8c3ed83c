"""Plain 64-bit form of the balance loss and its gradient, with an error bound for each element, for the tests of
balance_loss.

Bound: an fp32 exponential of x = l - m costs |x| 2^-24 for the product with log2(e) and a few units 2^-23 for the
rest, a sum of positive terms one 2^-24 for each addition on its path.  With `span` the largest m - l of the rows
(terms under exp(-span) count less than their own rounding) a softmax value is within (span + 16 + adds) 2^-23 of
itself; the losses and the gradient follow term by term, the differences c - sum_j p_j c_j by the size of their parts.
"""
import torch

STEP = 2.0 ** -23


def reference(logits, idx, mask=None, offsets=None, g=1.0, gz=1.0, out=torch.float32):
    """Everything in float64 on the CPU -> dict of values and bounds."""
    l = logits.detach().cpu().double()
    l = torch.where(torch.isnan(l), torch.full_like(l, -torch.inf), l)
    idx = idx.cpu().long()
    T, n = l.shape
    K = idx.shape[1]
    ends = [0, T] if offsets is None else offsets.cpu().tolist()
    S = len(ends) - 1
    on = torch.ones(T, K, dtype=torch.bool)
    if mask is not None:
        m = mask.cpu().bool()
        on = m.clone() if m.dim() == 2 else m[:, None].expand(T, K).clone()
    inside = torch.zeros(T, dtype=torch.bool)
    for a, b in zip(ends, ends[1:]):
        inside[a:b] = True
    on &= inside[:, None]
    active = on.any(1)
    some = (l > -torch.inf).any(1)
    top = l.max(1)[0] if n else l.new_zeros(T)
    p = torch.zeros_like(l)
    lse = l.new_zeros(T)
    use = active & some
    p[use] = torch.softmax(l[use], 1)
    lse[use] = torch.logsumexp(l[use], 1)
    N = int(active.sum())
    counts = torch.zeros(S, n, dtype=torch.int64)
    loss, grad, bound = 0.0, torch.zeros_like(l), torch.zeros_like(l)
    finite = l[use]
    span = 0.0
    if finite.numel():
        x = top[use][:, None] - finite
        span = float(x[torch.isfinite(x)].max()) if torch.isfinite(x).any() else 0.0
        span = min(span, 104.0)  # exp(-104) is 0 in fp32
    k = span + 16 + 512
    for s, (a, b) in enumerate(zip(ends, ends[1:])):
        if b <= a:
            continue
        picked = idx[a:b][on[a:b]]
        picked = picked[(picked >= 0) & (picked < n)]
        counts[s] = torch.bincount(picked, minlength=n)
        ns = int(active[a:b].sum())
        if not ns:
            continue
        c = counts[s].double()
        share = n / (K * N * ns)
        loss = loss + share * float((c * p[a:b].sum(0)).sum())
        d = (p[a:b] * c).sum(1, keepdim=True)
        grad[a:b] = g * share * p[a:b] * (c - d) + gz * 2 / N * lse[a:b, None] * p[a:b]
        bound[a:b] = (span + 64 + n ** 0.5) * STEP * p[a:b] * (
            3 * abs(g) * share * (c + d) + abs(gz) * 2 / N * (3 * lse[a:b, None].abs() + top[a:b, None].abs() + 16))
        grad[a:b][~use[a:b]] = 0
        bound[a:b][~use[a:b]] = 0
    z = float((lse ** 2).sum()) / N if N else 0.0
    zt = float(((lse.abs() + top.nan_to_num(0, 0, 0).abs() * use + 8) * lse.abs()).sum()) / N if N else 0.0
    bound = torch.nan_to_num(bound) + 2.0 ** -126 * 4
    if out is torch.bfloat16:
        bound = bound + torch.finfo(out).eps / 2 * (grad.abs() + bound)
    return dict(loss=float(loss), loss_bound=abs(float(loss)) * k * STEP, z=z, z_bound=2 * zt * k * STEP,
                counts=counts if offsets is not None else counts[0], grad=grad, bound=bound)


def compare(name, got, ref):
    """got: (loss, z_loss, counts, grad) on any device."""
    loss, z, counts, grad = got
    assert torch.equal(counts.cpu().long(), ref["counts"]), name
    for what, v, r, b in (("loss", loss, ref["loss"], ref["loss_bound"]), ("z_loss", z, ref["z"], ref["z_bound"])):
        assert abs(float(v) - r) <= b + 1e-30, f"{name}: {what} {float(v)} against {r}, bound {b}"
    err = (grad.detach().cpu().double() - ref["grad"]).abs()
    assert torch.isfinite(err).all(), name
    worst = (err / ref["bound"]).max() if err.numel() else 0
    assert (err <= ref["bound"]).all(), f"{name}: gradient off by {float(worst)} of its bound"
