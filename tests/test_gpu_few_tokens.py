"""The whole MoE layer for a few tokens (moe_few_tokens, moe_few_tokens_int8,
moe_layer_few_tokens) against the plain 64-bit form, element by element."""
import ctypes

import pytest
import torch

import dispatch_expert_gemm_amd as dm
from few_util import check, layer64, quant_weight

gpu = pytest.mark.gpu
DEV = "cuda:0"


def make(T, H, F, E, K, seed, int8=False, shared=0, Z=0, C=0, Q=0, mask=None, smooth=False, one_expert=False):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(torch.bfloat16)

    p = dict(x=normal(T, H))
    if one_expert:
        idx = torch.full((T, K), 2, dtype=torch.int32, device=DEV)
        for k in range(1, K):
            idx[:, k] = 2 + k
        w = torch.rand(T, K, generator=g, device=DEV)
    else:
        w, idx = torch.randn(T, E + Z + C + Q, generator=g, device=DEV).softmax(-1).topk(K)
    p["idx"], p["w"] = idx.to(torch.int32).contiguous(), w.float().contiguous()
    ws = [normal(E, F, H, std=H ** -0.5), normal(E, F, H, std=H ** -0.5), normal(E, H, F, std=F ** -0.5)]
    sw = [normal(1, shared, H, std=H ** -0.5), normal(1, shared, H, std=H ** -0.5),
          normal(1, H, shared, std=shared ** -0.5)] if shared else None
    if int8:
        ws, sw = [quant_weight(v) for v in ws], [quant_weight(v) for v in sw] if sw else None
    p["ws"], p["sw"] = ws, sw
    p["smooth"] = (torch.randn(E, H, generator=g, device=DEV) * 0.5).exp() if smooth else None
    p["const"] = [normal(Q, H) for _ in range(3)] if Q else None
    p["mask"] = None
    if mask == "1d":
        p["mask"] = (torch.arange(T, device=DEV) < (T + 1) // 2).to(torch.uint8)
    elif mask == "2d":
        p["mask"] = torch.rand(T, K, generator=g, device=DEV) >= 0.3
    elif mask == "none left":
        p["mask"] = torch.zeros(T, K, dtype=torch.uint8, device=DEV)
    p.update(Z=Z, C=C, Q=Q, shared_x=None)
    return p


def call(p, **kw):
    sw = p["sw"] or (None, None, None)
    c = p["const"] or (None, None, None)
    return dm.moe_layer_few_tokens(
        p["x"], p["idx"], p["w"], *p["ws"], smooth_scales=p["smooth"], x_active_mask=p["mask"],
        shared_expert_x=p["shared_x"], shared_w_gate=sw[0], shared_w_up=sw[1], shared_w_down=sw[2], const_alpha_1=c[0],
        const_alpha_2=c[1], const_v=c[2], zero_expert_num=p["Z"], copy_expert_num=p["C"], const_expert_num=p["Q"], **kw)


def ref(p):
    return layer64(p["x"], p["idx"], p["w"], p["ws"], smooth=p["smooth"], mask=p["mask"], shared_x=p["shared_x"],
                   shared_w=p["sw"], const=p["const"], Z=p["Z"], C=p["C"], Q=p["Q"])


CASES = {
    "one token": dict(T=1, H=1536, F=480, E=64, K=8),
    "one of everything": dict(T=1, H=16, F=32, E=1, K=1),
    "tails": dict(T=5, H=208, F=96, E=6, K=3),
    "shared": dict(T=3, H=512, F=128, E=8, K=2, shared=320),
    "special": dict(T=13, H=272, F=64, E=5, K=4, Z=1, C=1, Q=2),
    "prefix mask": dict(T=17, H=256, F=160, E=7, K=2, mask="1d", shared=64),
    "slot mask": dict(T=31, H=336, F=224, E=16, K=4, mask="2d", C=1),
    "nothing left": dict(T=9, H=128, F=64, E=4, K=2, mask="none left"),
    "nothing left but shared": dict(T=9, H=128, F=64, E=4, K=2, mask="none left", shared=32),
    "full tile": dict(T=16, H=640, F=256, E=3, K=3),
    "over a tile": dict(T=33, H=384, F=96, E=4, K=2, one_expert=True),
    "largest batch, one expert": dict(T=64, H=256, F=128, E=19, K=16, one_expert=True),
    "largest batch": dict(T=64, H=1024, F=512, E=32, K=8, shared=512),
    "many experts": dict(T=50, H=128, F=32, E=1024, K=16, Z=3, Q=1, mask="2d"),
    "three tiles": dict(T=47, H=160, F=64, E=2, K=2, shared=96),
    "two tokens": dict(T=2, H=512, F=160, E=6, K=3, shared=96, mask="2d", C=1),
    "longest held row": dict(T=2, H=8192, F=96, E=3, K=2),
    "a row too long to hold": dict(T=1, H=8208, F=64, E=2, K=2, shared=64),
    "too many rows of h to hold": dict(T=2, H=256, F=4096, E=8, K=8),
    "more columns than 16 for each CU": dict(T=7, H=4112, F=64, E=4, K=2, shared=32),
    "one token, wide": dict(T=1, H=4112, F=352, E=4, K=2, shared=32),
    "h rows past 8192": dict(T=3, H=160, F=8224, E=2, K=1, shared=32),
    "shared h rows past 8192": dict(T=18, H=160, F=64, E=4, K=2, shared=8224),
    "narrow, by expert": dict(T=12, H=592, F=1120, E=33, K=6, shared=64, mask="2d", Z=1, C=1, Q=1),
    "narrow, long": dict(T=6, H=208, F=5184, E=12, K=4),
    "narrow, full tile": dict(T=16, H=272, F=2624, E=5, K=3, one_expert=False, mask="1d"),
    "short contractions": dict(T=40, H=64, F=32, E=3, K=2, shared=32),
    "long contractions": dict(T=20, H=2064, F=5152, E=2, K=1),
    "long contractions, four tiles": dict(T=64, H=2064, F=5152, E=3, K=2, one_expert=False, shared=2592),
}


@gpu
@pytest.mark.parametrize("form", ["bf16", "int8", "int8 smooth"])
@pytest.mark.parametrize("name", list(CASES))
def test_layer_against_64_bits(name, form):
    print(f"[few tokens] {name} {form}", flush=True)
    p = make(seed=11, int8=form != "bf16", smooth=form == "int8 smooth", **CASES[name])
    flag = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    out = call(p, err_flag=flag)
    torch.cuda.synchronize()
    v, bound, f = ref(p)
    check(f"{name} {form}", out, v, bound)
    assert flag.item() == f


@gpu
@pytest.mark.parametrize("T,H,F,int8", [(1, 1 << 20, 32, False), (50, 1 << 20, 32, False), (1, 8, 1 << 20, False),
                                        (50, 8, 1 << 20, False), (2, 131072, 32, True), (50, 131072, 32, True),
                                        (2, 16, 131072, True), (50, 16, 131072, True)])
def test_longest_rows(T, H, F, int8):
    p = make(T, H, F, 3, 2, 45, int8=int8, smooth=int8, shared=32)
    v, bound, _ = ref(p)
    check("longest rows", call(p), v, bound)


@gpu
@pytest.mark.parametrize("T", [2, 20])
@pytest.mark.parametrize("int8", [False, True])
def test_weights_past_32_bits(int8, T):
    """Weight tensors of more than 2^32 bytes; the first and the last experts are used."""
    H, F, E = 8192, 4096, 68 if not int8 else 132
    p = make(T, H, F, 4, 2, 44, int8=int8)

    def spread(w):
        big = torch.zeros(E, *w.shape[1:], dtype=w.dtype, device=DEV)
        big[:2], big[-2:] = w[:2], w[2:]
        return big

    p["ws"] = [(spread(w[0]), spread(w[1])) if int8 else spread(w) for w in p["ws"]]
    p["idx"] = torch.where(p["idx"] < 2, p["idx"], p["idx"] + E - 4)
    v, bound, _ = ref(p)
    check("large weights", call(p), v, bound)


@gpu
@pytest.mark.parametrize("int8", [False, True])
def test_given_shared_term(int8):
    p = make(7, 256, 96, 5, 2, 12, int8=int8, C=1)
    p["shared_x"] = torch.randn(7, 256, device=DEV).to(torch.bfloat16)
    v, bound, _ = ref(p)
    check("shared_expert_x", call(p), v, bound)


@gpu
@pytest.mark.parametrize("int8", [False, True])
def test_bad_ids_are_flagged_and_dropped(int8):
    p = make(6, 256, 64, 5, 3, 13, int8=int8, Z=1)
    p["idx"][0, 1] = p["idx"][0, 0]
    p["idx"][2, 0] = -1
    p["idx"][3, 2] = 6
    p["idx"][4, 1] = 2 ** 31 - 1
    p["idx"][5, :] = -2 ** 31
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = call(p, err_flag=flag)
    v, bound, f = ref(p)
    check("bad ids", out, v, bound)
    assert flag.item() == f == dm.MOE_FLAG_ID_RANGE | dm.MOE_FLAG_ID_DUPLICATE


@gpu
def test_mask_that_is_no_prefix_is_flagged():
    p = make(4, 128, 32, 4, 2, 14)
    p["mask"] = torch.tensor([1, 0, 1, 0], dtype=torch.uint8, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = call(p, err_flag=flag)
    v, bound, f = ref(p)
    check("not a prefix", out, v, bound)
    assert flag.item() == f == dm.MOE_FLAG_MASK_NOT_PREFIX


@gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.3e38])
def test_what_no_active_slot_uses_does_not_matter(int8, bad):
    """A masked token's row and weights, an unused expert's weights and scales."""
    p = make(19, 256, 64, 6, 2, 15, int8=int8, smooth=int8)
    p["idx"] = (p["idx"] % 5).contiguous()                 # expert 5 unused
    p["idx"][:, 1] = (p["idx"][:, 0] + 1) % 5
    p["mask"] = torch.ones(19, 2, dtype=torch.uint8, device=DEV)
    p["mask"][4] = 0
    p["mask"][7, 1] = 0
    v, bound, _ = ref(p)
    p["x"][4] = bad
    p["w"][4] = bad
    p["w"][7, 1] = bad
    for w in p["ws"]:
        (w[1] if int8 else w)[5] = bad
    if int8:
        p["smooth"][5] = bad
    out = call(p)
    check("unused values", out, v, bound)
    assert (out[4] == 0).all()


@gpu
@pytest.mark.parametrize("T", [2, 8, 40])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_token_that_is_not_finite_does_not_reach_the_others(bad, int8, T):
    p = make(T, 256, 64, 4, 2, 16, int8=int8, smooth=int8)
    clean = call(p)
    p["x"][1, 77] = bad
    out = call(p)
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out[1]).any()


@gpu
@pytest.mark.parametrize("int8", [False, True])
def test_same_call_same_bits_whatever_the_workspace_held(int8):
    """Two calls, a third on a workspace full of NaN, and nothing written past the outputs."""
    p = make(29, 512, 160, 12, 4, 17, int8=int8, smooth=int8, shared=96, mask="2d")
    first = call(p)
    assert torch.equal(first, call(p))
    shape = dm.make_shape(29, 512, 4, 12, F=160, mask_ndim=2)
    n = dm.moe_few_tokens_workspace_size(shape, 96, int8)
    ws = torch.full((n + 256,), 0xff, dtype=torch.uint8, device=DEV)
    out = torch.full((29 * 512 + 64,), 5.0, dtype=torch.bfloat16, device=DEV)
    flag = torch.full((3,), 9, dtype=torch.int32, device=DEV)
    rest = (p["sw"], None, None, None, None, out, flag, ws[:n])
    if int8:
        dm.moe_few_tokens_int8(shape, p["x"], p["idx"], p["w"], p["mask"], p["smooth"], p["ws"], *rest)
    else:
        dm.moe_few_tokens(shape, p["x"], p["idx"], p["w"], p["mask"], *p["ws"], *rest)
    torch.cuda.synchronize()
    assert torch.equal(out[:29 * 512].view(29, 512), first)
    assert (out[29 * 512:] == 5.0).all() and (ws[n:] == 0xff).all()
    assert flag.tolist() == [0, 9, 9]


@gpu
def test_rows_do_not_depend_on_the_batch():
    """A token alone gives the bits it gives in a batch of one expert tile."""
    p = make(16, 512, 128, 4, 2, 18)
    out = call(p)
    for t in (0, 7, 15):
        q = dict(p, x=p["x"][t:t + 1].contiguous(), idx=p["idx"][t:t + 1].contiguous(), w=p["w"][t:t + 1].contiguous())
        v, bound, _ = ref(q)
        check("alone", call(q), v, bound)
        check("in the batch", out[t:t + 1], v, bound)


@gpu
@pytest.mark.parametrize("int8", [False, True])
def test_no_tokens(int8):
    p = make(1, 128, 32, 4, 2, 19, int8=int8, shared=64)
    p["x"], p["idx"], p["w"] = p["x"][:0], p["idx"][:0], p["w"][:0]
    flag = torch.full((1,), 3, dtype=torch.int32, device=DEV)
    assert call(p, err_flag=flag).shape == (0, 128)
    assert flag.item() == 0


@gpu
@pytest.mark.parametrize("int8", [False, True])
def test_another_stream_and_a_captured_call(int8):
    """On a stream of its own; captured once and replayed with other inputs between eager calls."""
    p = make(9, 512, 96, 8, 3, 20, int8=int8, shared=64)
    want = call(p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(p, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = call(p)
    for seed in (21, 22, 23):
        q = make(9, 512, 96, 8, 3, seed, int8=int8, shared=64)
        for k in ("x", "idx", "w"):
            p[k].copy_(q[k])
        eager = call(p)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@gpu
def test_two_streams_at_once():
    ps = [make(32, 1024, 256, 8, 2, s, int8=True) for s in (24, 25)]
    want = [call(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[call(p, stream=s) for p, s in zip(ps, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("int8", [False, True])
def test_two_graphs_at_once(int8):
    """Each captured call has a workspace of its own."""
    ps = [make(T, 512, 256, 8, 2, s, int8=int8, smooth=int8) for T, s in ((2, 28), (24, 29))]
    want = [call(p) for p in ps]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in ps]
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(p))
        graphs.append(g)
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@gpu
def test_refusals_of_tensors():
    p = make(4, 128, 64, 4, 2, 26)

    def refused(**kw):
        with pytest.raises(dm.MoeError):
            call(dict(p, **kw))

    refused(x=p["x"].float())
    refused(x=p["x"].cpu())
    refused(x=torch.empty(128, 4, dtype=torch.bfloat16, device=DEV).t())
    refused(idx=p["idx"].long())
    refused(idx=p["idx"][:3].contiguous())
    refused(w=p["w"].double())
    refused(w=p["w"][:, :1].contiguous())
    refused(mask=torch.ones(3, dtype=torch.uint8, device=DEV))
    refused(ws=[p["ws"][0], p["ws"][1], p["ws"][2][:3].contiguous()])
    refused(ws=[p["ws"][0], p["ws"][1], p["ws"][1]])
    refused(smooth=torch.ones(4, 128, device=DEV))            # bf16 weights
    refused(C=0, Q=1, idx=p["idx"])                           # constant experts without their tensors
    refused(x=p["x"].repeat(20, 1)[:65].contiguous(), idx=p["idx"].repeat(20, 1)[:65].contiguous(),
            w=p["w"].repeat(20, 1)[:65].contiguous())         # more than 64 tokens
    buf = torch.zeros(4 * 128 + 1, dtype=torch.bfloat16, device=DEV)
    refused(x=buf[1:].view(4, 128))                           # not on a 16-byte boundary
    sw = make(1, 128, 64, 4, 2, 27, shared=32)["sw"]
    refused(sw=sw, shared_x=p["x"])                           # both forms of the shared term
    refused(sw=[sw[0], None, sw[2]])
    refused(sw=[None, sw[1], sw[2]])
    q = make(4, 128, 64, 4, 2, 26, int8=True)
    flat = torch.ones(4 * 128 + 1, device=DEV)
    q["smooth"] = flat[1:].view(4, 128)                       # not on a 16-byte boundary
    with pytest.raises(dm.MoeError):
        call(q)


def test_refusals_of_the_entries():
    L = dm.lib()
    P = lambda v=0x1000: ctypes.c_void_p(v)   # noqa: E731  (never read: the checks come first)
    N = None

    def S(**kw):
        return ctypes.byref(dm.make_shape(**dict(dict(T=4, H=128, K=2, num_experts=4, F=64), **kw)))

    def bf16(s=None, Fs=0, sw=(N, N, N), x=P(), sx=N, cs=(N, N, N), out=P(), flag=P(), ws=P(), nb=1 << 30, mask=N, w=None):
        return L.moe_few_tokens(s or S(), x, P(), P(), mask, *(w or (P(), P(), P())), Fs, *sw, sx, *cs, out, flag, ws, nb, N)

    NULL, SHAPE, RANGE, UNSUP, WS = -1, -2, -3, -5, -6
    assert bf16(s=S(T=65)) == UNSUP
    assert bf16(s=S(comm_quant_mode=2)) == UNSUP
    assert bf16(s=S(F=48)) == SHAPE
    assert bf16(s=S(H=100)) == SHAPE
    assert bf16(s=S(K=17)) == SHAPE
    assert bf16(s=S(mask_ndim=1)) == NULL
    assert bf16(s=S(const_expert_num=1)) == NULL
    assert bf16(Fs=40, sw=(P(), P(), P())) == SHAPE
    assert bf16(Fs=-32) == SHAPE
    assert bf16(Fs=64) == NULL
    assert bf16(Fs=64, sw=(P(), P(), P()), sx=P()) == RANGE
    assert bf16(x=N) == NULL and bf16(out=N) == NULL and bf16(flag=N) == NULL and bf16(w=(P(), N, P())) == NULL
    assert bf16(x=P(0x1008)) == SHAPE and bf16(w=(P(), P(0x1002), P())) == SHAPE and bf16(ws=P(0x1001)) == SHAPE
    assert bf16(ws=N) == WS and bf16(nb=1024) == WS
    n = ctypes.c_size_t()
    size = L.moe_few_tokens_workspace_size
    assert size(S(), 0, 2, ctypes.byref(n)) == RANGE
    assert size(S(), 0, 0, N) == NULL
    assert size(S(H=136), 0, 1, ctypes.byref(n)) == SHAPE      # int8: H a multiple of 16
    assert size(S(H=136), 0, 0, ctypes.byref(n)) == 0
    assert size(S(H=1 << 18, F=32), 0, 1, ctypes.byref(n)) == UNSUP   # the int32 sums
    w = (dm.MoeInt8Weight * 3)(*[dm.MoeInt8Weight(0x1000, 0x1000)] * 3)
    half = (dm.MoeInt8Weight * 3)(*[dm.MoeInt8Weight(0x1000, None)] * 3)

    def i8(s=None, ww=w, Fs=0, sw=N, nb=1 << 30):
        return L.moe_few_tokens_int8(s or S(), P(), P(), P(), N, N, ww, Fs, sw, N, N, N, N, P(), P(), P(), nb, N)

    assert i8(ww=N) == NULL and i8(ww=half) == NULL and i8(Fs=64) == NULL and i8(Fs=64, sw=half) == NULL
    assert i8(s=S(H=136)) == SHAPE
    assert i8(nb=64) == WS
