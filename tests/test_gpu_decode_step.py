"""A decode step as a model runs it: projection in, gate, router, the layer for a few
tokens, projection out; and the shared expert of moe_layer_int8.  Each stage is held
against the plain 64-bit form of what the stage before it wrote."""
import pytest
import torch

import dispatch_expert_gemm_amd as dm
from few_util import check, layer64, linear64, quant_weight, to_int8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Step:
    def __init__(self, D, H, F, Fs, E, K, int8, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def normal(*shape):
            return (torch.randn(*shape, generator=g, device=DEV) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.K, self.D, self.g = K, D, g
        self.w_in, self.w_gate, self.w_out = (dm.Int8Weights(*quant_weight(normal(*s))) for s in ((H, D), (E, H), (D, H)))
        self.bias = torch.randn(D, generator=g, device=DEV)
        form = (lambda v: dm.Int8Weights(*quant_weight(v))) if int8 else (lambda v: v)
        self.ws = [form(normal(*s)) for s in ((E, F, H), (E, F, H), (E, H, F))]
        self.sw = [form(normal(*s)) for s in ((1, Fs, H), (1, Fs, H), (1, H, Fs))]

    def rows(self, T):
        return torch.randn(T, self.D, generator=self.g, device=DEV).to(torch.bfloat16)

    def __call__(self, x):
        a = dm.linear_int8(x, self.w_in)
        logits = dm.linear_int8(a, self.w_gate).float()
        idx, w = dm.router(logits, self.K)
        y = dm.moe_layer_few_tokens(a, idx, w, *self.ws, shared_w_gate=self.sw[0], shared_w_up=self.sw[1],
                                    shared_w_down=self.sw[2])
        return a, logits, idx, w, y, dm.linear_int8(y, self.w_out, bias=self.bias)


def plain(x, w, bias=None):
    q, s = to_int8(x.float())
    return linear64((q, s[:, 0]), (w.codes, w.scales), bias)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T", [1, 2, 13, 64])
def test_decode_step(T, int8):
    step = Step(384, 512, 160, 96, 12, 3, int8, 50 + T)
    x = step.rows(T)
    a, logits, idx, w, y, out = step(x)
    check("in", a, *plain(x, step.w_in))
    check("gate", logits, *plain(a, step.w_gate))
    assert torch.equal(logits.gather(1, idx.long()).sort(-1).values, logits.topk(step.K).values.sort(-1).values)
    pair = (lambda v: (v.codes, v.scales)) if int8 else (lambda v: v)
    v, bound, _ = layer64(a, idx, w, [pair(t) for t in step.ws], shared_w=[pair(t) for t in step.sw])
    check("layer", y, v, bound)
    check("out", out, *plain(y, step.w_out, step.bias))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T", [1, 24])
def test_a_captured_decode_step(T, int8):
    step = Step(256, 512, 96, 64, 8, 2, int8, 60 + T)
    x = step.rows(T)
    step(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(x)
    for _ in range(4):
        x.copy_(step.rows(T))
        want = step(x)
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)


@pytest.mark.parametrize("T", [1, 70, 300])
def test_shared_expert_of_the_int8_layer(T):
    H, F, Fs, E, K = 512, 256, 128, 4, 2
    g = torch.Generator(device=DEV).manual_seed(70 + T)

    def weights(*shape):
        return dm.Int8Weights.quantize((torch.randn(*shape, generator=g, device=DEV) * shape[-1] ** -0.5).to(torch.bfloat16))

    ws = [weights(E, F, H), weights(E, F, H), weights(E, H, F)]
    sw = [weights(1, Fs, H), weights(1, Fs, H), weights(1, H, Fs)]
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    w, idx = torch.rand(T, E, generator=g, device=DEV).topk(K)
    idx = idx.to(torch.int32)
    kw = dict(shared_wq_gate=sw[0], shared_wq_up=sw[1], shared_wq_down=sw[2])
    out = dm.moe_layer_int8(x, idx, w, *ws, **kw)
    # the shared expert alone: h as the grouped product writes it, its down product in 64 bits
    shape = dm.make_shape(T, H, 1, 1, F=Fs)
    gus = torch.empty(T, 2 * Fs, dtype=torch.bfloat16, device=DEV)
    h = torch.empty(T, Fs, dtype=torch.bfloat16, device=DEV)
    dm.moe_ffn_gate_up_fwd_int8(shape, *dm.quant_rows_int8(x), sw[0].codes, sw[0].scales, sw[1].codes, sw[1].scales,
                                torch.full((1,), T, dtype=torch.int32, device=DEV), gus, h)
    q, s = to_int8(h.float())
    v, bound = linear64((q, s[:, 0]), (sw[2].codes[0], sw[2].scales[0]))
    shared = dm.linear_int8(h, (sw[2].codes[0], sw[2].scales[0]))
    check("shared", shared, v, bound)
    assert torch.equal(out, dm.moe_layer_int8(x, idx, w, *ws, shared_expert_x=shared))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        again = dm.moe_layer_int8(x, idx, w, *ws, **kw)
    st.synchronize()
    assert torch.equal(out, again)
    with pytest.raises(dm.MoeError):
        dm.moe_layer_int8(x, idx, w, *ws, shared_expert_x=shared, **kw)
    with pytest.raises(dm.MoeError):
        dm.moe_layer_int8(x, idx, w, *ws, shared_wq_gate=sw[0])
