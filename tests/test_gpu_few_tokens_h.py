"""The few-token layer in bf16 holds h in fp32: values of h that differ in their last bits
cancel in the down product, so that a bit of h that is lost is the whole output."""
import pytest
import torch

import dispatch_expert_gemm_amd as dm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(T, H, F, E, Fs, seed):
    """Experts whose h is 32 x0^2 (1 + a 2^-9 + b 2^-20), a odd: with its 21 significant bits, exactly,
    since x, the weights and the sums are whole numbers of a step, and silu(g) is g in fp32 from
    g = 32 on (1 + e^-32 is 1).  Every output takes h of one row minus h of another with the same
    a and b = 0: what is left is 2^-15 b.  Returns x, weights, shared weights and outs(e), the
    expert's output for x0 = 1 (the shared expert's: e = E), in doubles."""
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(T, H)
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 2.0 ** -9, 2.0 ** -20
    x *= 2.0 ** (torch.arange(T) % 3)[:, None]

    def expert(F):
        wg, wu, wd = torch.zeros(F, H), torch.zeros(F, H), torch.zeros(H, F)
        wg[:, 0] = 32.0
        order = torch.randperm(F, generator=g)
        up, down = order[:F // 2], order[F // 2:]
        a = 2.0 * torch.randint(0, 64, (F // 2,), generator=g) + 1
        b = torch.randint(1, 16, (F // 2,), generator=g).float()
        wu[:, 0] = 1.0
        wu[up, 1], wu[down, 1], wu[up, 2] = a, a, b
        pick = torch.randint(0, F // 2, (H,), generator=g)
        sign = torch.randint(0, 2, (H,), generator=g) * 2.0 - 1
        c = torch.arange(H)
        wd[c, up[pick]], wd[c, down[pick]] = sign, -sign
        return (wg, wu, wd), sign.double() * b[pick].double() * 2.0 ** -15

    every = [expert(F) for _ in range(E)] + ([expert(Fs)] if Fs else [])
    bf16 = lambda t: t.to(torch.bfloat16).to(DEV)   # noqa: E731
    ws = [bf16(torch.stack([every[e][0][i] for e in range(E)])) for i in range(3)]
    sw = [bf16(every[E][0][i][None]) for i in range(3)] if Fs else [None] * 3
    return bf16(x), ws, sw, [o for _, o in every]


@pytest.mark.parametrize("T,H,F,Fs", [(1, 16, 32, 0), (1, 1536, 480, 64), (2, 4112, 352, 96), (9, 208, 96, 0), (13, 4112, 2080, 32),
                                      (16, 272, 2624, 96), (6, 208, 5184, 64), (20, 64, 160, 2592), (24, 2064, 5152, 0),
                                      (40, 160, 2528, 32), (64, 128, 96, 64), (50, 272, 5152, 96)])
def test_every_bit_of_h_is_kept(T, H, F, Fs):
    """Two experts for each token, weights 1 and 1/2, in all batch sizes up to a whole batch on one
    expert.  Sums of a wave, an expert and a token are whole numbers of 2^-16 below 2^8 times
    x0^2, so fp32 holds each of them exactly, in any order, and so does the output in bf16."""
    print(f"[h] T={T} H={H} F={F} Fs={Fs}", flush=True)
    E = 5
    x, ws, sw, outs = make(T, H, F, E, Fs, 80 + T)
    idx = torch.tensor([[3, 1] if t % 4 else [1, 4] for t in range(T)], dtype=torch.int32, device=DEV)
    w = torch.tensor([1.0, 0.5], device=DEV).repeat(T, 1)
    got = dm.moe_layer_few_tokens(x, idx, w, *ws, shared_w_gate=sw[0], shared_w_up=sw[1], shared_w_down=sw[2])
    want = torch.stack([outs[i] + 0.5 * outs[j] + (outs[E] if Fs else 0) for i, j in idx.tolist()])
    want = want * 4.0 ** (torch.arange(T) % 3)[:, None]
    assert torch.equal(want, want.to(torch.bfloat16).double())
    assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("T", [1, 9, 40])
@pytest.mark.parametrize("F", [96, 5152])
def test_h_at_the_end_of_the_range(T, F):
    """h = 2^127 (2 - 2^-9), which bf16 would round to infinity, is a number; h past the range is an
    infinity of its sign.  The other tokens keep their values."""
    H, E = 16, 2
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 1.0
    x[0, 0] = 2.0 ** 60
    x[0, 1] = 2.0 ** 52
    wg, wu, wd = (torch.zeros(E, *s, dtype=torch.bfloat16) for s in ((F, H), (F, H), (H, F)))
    wg[:, :, 0] = 64.0                       # g = 2^66
    wu[0, 0, 0], wu[0, 0, 1] = 4.0, -1.0     # u = 2^62 - 2^52 = 2^61 (2 - 2^-9)
    wu[1, 0, 0] = 4.0                        # u = 2^62: h = 2^128
    wd[0, :, 0] = 2.0 ** -100
    wd[1, :8, :], wd[1, 8:, :] = 1.0, -1.0
    idx = torch.zeros(T, 1, dtype=torch.int32)
    args = [t.to(DEV) for t in (x, idx, torch.ones(T, 1))], [t.to(DEV) for t in (wg, wu, wd)]
    out = dm.moe_layer_few_tokens(*args[0], *args[1]).cpu()
    # 2^27 (2 - 2^-9) rounds to 2^28 in bf16
    assert (out[0] == 2.0 ** 28).all()
    assert (out[1:] == 64.0 * 4 * 2.0 ** -100).all()
    args[0][1].fill_(1)
    out = dm.moe_layer_few_tokens(*args[0], *args[1]).cpu()
    # (h of the other rows of the expert is 0)
    assert (out[0, :8] == float("inf")).all() and (out[0, 8:] == float("-inf")).all()
    assert (out[1:, :8] == 256.0).all() and (out[1:, 8:] == -256.0).all()
