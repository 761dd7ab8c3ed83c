"""Arguments that the few-token layer's and the int8 product's Python calls refuse: tensors that
are large enough and of another shape."""
import pytest
import torch

import dispatch_expert_gemm_amd as dm
from few_util import quant_weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, H, F, E, K, Q, FS = 4, 128, 64, 5, 2, 2, 32


def layer(int8=False, **kw):
    g = torch.Generator(device=DEV).manual_seed(91)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)   # noqa: E731
    form = quant_weight if int8 else (lambda w: w)
    args = dict(x=r(T, H), topk_idx=torch.tensor([[0, 1], [2, E], [E + 1, 3], [4, 0]], dtype=torch.int32, device=DEV),
                topk_weights=torch.rand(T, K, generator=g, device=DEV), w_gate=form(r(E, F, H)), w_up=form(r(E, F, H)),
                w_down=form(r(E, H, F)), const_alpha_1=r(Q, H), const_alpha_2=r(Q, H), const_v=r(Q, H), const_expert_num=Q)
    args.update(kw)
    return dm.moe_layer_few_tokens(**args)


def bf(*shape):
    return torch.ones(*shape, dtype=torch.bfloat16, device=DEV)


def ones(*shape):
    return torch.ones(*shape, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("name,shape", [
    ("x_active_mask", (T, K + 1)), ("x_active_mask", (K, T)), ("x_active_mask", (T + 1,)), ("x_active_mask", (T, 1)),
    ("x_active_mask", (T, K, 1)), ("x_active_mask", ()), ("shared_expert_x", (T + 1, H)), ("shared_expert_x", (H, T)),
    ("shared_expert_x", (T * H,)), ("const_alpha_1", (Q + 1, H)), ("const_alpha_2", (H, Q)), ("const_v", (Q, 2 * H)),
    ("x", (1, T, H)), ("topk_idx", (T * K,)), ("w_gate", (E * F * H,))])
@pytest.mark.parametrize("int8", [False, True])
def test_another_shape_is_refused(name, shape, int8):
    layer(int8=int8)
    dtype = {"x_active_mask": torch.uint8, "topk_idx": torch.int32}.get(name, torch.bfloat16)
    bad = torch.ones(shape, dtype=dtype, device=DEV)
    if int8 and name == "w_gate":
        bad = (bad.to(torch.int8), torch.ones(E * F, device=DEV))
    with pytest.raises(dm.MoeError):
        layer(int8=int8, **{name: bad})


@pytest.mark.parametrize("shape", [(E, 2 * H), (H, E), (E + 1, H), (E * H,)])
def test_smooth_scales_of_another_shape_are_refused(shape):
    layer(int8=True, smooth_scales=torch.ones(E, H, device=DEV))
    with pytest.raises(dm.MoeError):
        layer(int8=True, smooth_scales=torch.ones(*shape, device=DEV))


def test_weight_scales_of_another_shape_are_refused():
    q, s = quant_weight(bf(E, F, H))
    for bad in (torch.ones(E, 2 * F, device=DEV), torch.ones(E * F, device=DEV), torch.ones(F, E, device=DEV)):
        with pytest.raises(dm.MoeError):
            layer(int8=True, w_gate=(q, bad))
    sw = [quant_weight(bf(*shape)) for shape in ((1, FS, H), (1, FS, H), (1, H, FS))]
    layer(int8=True, shared_w_gate=sw[0], shared_w_up=sw[1], shared_w_down=sw[2])
    with pytest.raises(dm.MoeError):
        layer(int8=True, shared_w_gate=sw[0], shared_w_up=sw[1], shared_w_down=(sw[2][0], torch.ones(H, device=DEV)))


def test_masks_of_the_documented_shapes_are_taken():
    """A mask of ones, of either shape and type, changes nothing; constants are not looked at without
    constant experts."""
    want = layer()
    for m in (ones(T), ones(T, K), ones(T).bool(), ones(T, K).bool()):
        assert torch.equal(layer(x_active_mask=m), want)
    idx = torch.tensor([[0, 1], [2, 3], [4, 1], [4, 0]], dtype=torch.int32, device=DEV)
    layer(topk_idx=idx, const_expert_num=0, const_v=bf(1))


@pytest.mark.parametrize("int8", [False, True])
def test_weights_of_two_kinds_are_refused(int8):
    """A bf16 weight among int8 ones and the other way round, also the shared expert's; what is neither."""
    form = (lambda w: w) if int8 else quant_weight
    own = quant_weight if int8 else (lambda w: w)
    sw = [bf(1, FS, H), bf(1, FS, H), bf(1, H, FS)]
    names = ("shared_w_gate", "shared_w_up", "shared_w_down")
    layer(int8=int8, **{n: own(w) for n, w in zip(names, sw)})
    for kw in (dict(w_up=form(bf(E, F, H))), dict(w_gate=form(bf(E, F, H))), dict(w_down=form(bf(E, H, F))),
               {n: form(w) for n, w in zip(names, sw)}, dict(w_up=None), dict(w_down=(1, 2)),
               dict(w_gate=quant_weight(bf(E, F, H))[:1])):
        with pytest.raises(dm.MoeError):
            layer(int8=int8, **kw)


def test_product_arguments_of_another_shape_are_refused():
    """linear_int8: scales and bias that are large enough; moe_linear_int8 and its dynamic form: weights
    with more columns than the rows, which were read with the rows' length."""
    x = bf(2, 3, 64)
    q, s = quant_weight(x)
    w, b = quant_weight(bf(40, 64)), torch.ones(40, device=DEV)
    want = dm.linear_int8(x, w, bias=b)
    assert torch.equal(dm.linear_int8(q, w, x_scales=s, bias=b), want)
    for kw in (dict(x_scales=s.view(3, 2)), dict(x_scales=s.view(6)), dict(x_scales=torch.ones(2, 4, device=DEV)),
               dict(x_scales=s.view(2, 3, 1)), dict(x_scales=s, bias=torch.ones(41, device=DEV)),
               dict(x_scales=s, bias=b.view(1, 40))):
        with pytest.raises(dm.MoeError):
            dm.linear_int8(q, w, **kw)
    for pair in ((w[0], torch.ones(41, device=DEV)), (w[0], w[1].view(40, 1)), w[0], (w[0], None)):
        with pytest.raises(dm.MoeError):
            dm.linear_int8(x, pair)
    with pytest.raises(dm.MoeError):
        dm.linear_int8(x[0, 0, 0], w)
    wide = quant_weight(bf(40, 128))
    out = bf(6, 40)
    ws = torch.empty(dm.moe_linear_int8_workspace_size(6, 40, 64), dtype=torch.uint8, device=DEV)
    rows, (rq, rs) = x.view(6, 64), quant_weight(x.view(6, 64))
    dm.moe_linear_int8_dynamic(rows, *w, b, out, ws)
    assert torch.equal(out.view(2, 3, 40), want)
    for c, sc in (wide, (w[0].view(20, 128), w[1]), (w[0].view(-1), w[1])):
        with pytest.raises(dm.MoeError):
            dm.moe_linear_int8_dynamic(rows, c, sc, b, out, ws)
        with pytest.raises(dm.MoeError):
            dm.moe_linear_int8(rq, rs, c, sc, b, out)
    with pytest.raises(dm.MoeError):
        dm.moe_linear_int8(q, s, *w, b, out)              # three dimensions
    with pytest.raises(dm.MoeError):
        dm.moe_linear_int8_dynamic(x, *w, b, out, ws)
