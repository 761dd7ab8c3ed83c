"""The few-token layer: what a token's result depends on in a batch, and batches of 17 to 32 rows
for one expert with long contractions."""
import pytest
import torch

import dispatch_expert_gemm_amd as dm
from few_util import check, layer64, quant_weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(T, H, F, E, K, seed, int8, shared=0, same=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *s: (torch.randn(*s, generator=g, device=DEV) * s[-1] ** -0.5).to(torch.bfloat16)   # noqa: E731
    form = quant_weight if int8 else (lambda w: w)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    w, idx = torch.rand(T, E, generator=g, device=DEV).topk(K)
    if same:
        idx = torch.arange(K, device=DEV).repeat(T, 1)
    ws = [form(normal(*s)) for s in ((E, F, H), (E, F, H), (E, H, F))]
    sw = [form(normal(*s)) for s in ((1, shared, H), (1, shared, H), (1, H, shared))] if shared else None
    return x, idx.to(torch.int32).contiguous(), w.contiguous(), ws, sw


def call(x, idx, w, ws, sw):
    s = sw or (None, None, None)
    return dm.moe_layer_few_tokens(x, idx, w, *ws, shared_w_gate=s[0], shared_w_up=s[1], shared_w_down=s[2])


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T,H,F,E,K,shared", [(17, 2064, 5152, 2, 2, 0), (32, 1040, 5152, 3, 2, 96), (24, 208, 5184, 4, 1, 2592),
                                              (32, 2064, 96, 2, 2, 64), (30, 80, 160, 3, 3, 0), (16, 4112, 5152, 2, 2, 32)])
def test_one_expert_takes_every_token(T, H, F, E, K, shared, int8):
    print(f"[few tokens] T={T} H={H} F={F} int8={int8}", flush=True)
    x, idx, w, ws, sw = make(T, H, F, E, K, 100 + T, int8, shared, same=True)
    v, bound, _ = layer64(x, idx, w, ws, shared_w=sw)
    check("one expert", call(x, idx, w, ws, sw), v, bound)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T,H,F", [(2, 512, 160), (11, 512, 160), (16, 4112, 96), (7, 208, 2624), (29, 512, 160), (64, 272, 5152)])
def test_other_tokens_values_do_not_change_a_token(T, H, F, int8):
    """Other rows and weights, the same ids: the same bits, whichever token is looked at."""
    x, idx, w, ws, sw = make(T, H, F, 6, 3, 110 + T, int8, 64)
    out = call(x, idx, w, ws, sw)
    for t in {0, T // 2, T - 1}:
        y, v = make(T, H, F, 6, 3, 120 + t, int8)[0] * 7, torch.rand(T, 3, device=DEV)
        y[t], v[t] = x[t], w[t]
        assert torch.equal(call(y, idx, v, ws, sw)[t], out[t])


def test_most_rows_of_the_longest_h():
    """1024 slots of F = 2^20 - 32 columns: a plane of h ends at offset 2^31.  All but eight columns
    of each expert are 0, the last among the eight, and what is 0 adds nothing to a sum: the value
    and its bound are those of a layer of 16 columns, the eight (each of them three additions, a
    product's parts) and eight of the others."""
    T, H, F, E, K = 64, 8, 2 ** 20 - 32, 17, 16
    print(f"[few tokens] T={T} F={F}", flush=True)
    x, idx, w, ws, _ = make(T, H, F, E, K, 130, False)
    keep = torch.zeros(E, F, dtype=torch.bool, device=DEV)
    for e in range(E):
        keep[e, [0, 31 + e, 64 * e + 32, F // 2, F // 2 + 977 * e + 1, F - 65, F - 33, F - 1]] = True
    ws[1].masked_fill_(~keep[:, :, None], 0)
    ws[2].mul_(keep[:, None, :] * 1000)
    small = []
    for e in range(E):
        c = torch.cat([keep[e].nonzero()[:, 0], torch.arange(2, 10, device=DEV)])
        small.append((ws[0][e, c], ws[1][e, c], ws[2][e][:, c]))
    v, bound, _ = layer64(x, idx, w, [torch.stack(t) for t in zip(*small)])
    assert bound.mean() < 0.02 * v.abs().mean()
    check("longest h", call(x, idx, w, ws, None), v, bound)
