"""CPU checks of the balance loss and the checkpoints: the C entries return the documented status for bad arguments
before anything is launched, the Python calls refuse tensors of another kind, and the workspace's size."""
import ctypes
import os

import pytest
import torch

import dispatch_expert_gemm_amd as dm

OK, NULL_ARG, BAD_SHAPE, BAD_RANGE, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3, -5, -6
N = None


def P(v=0x10000):
    return ctypes.c_void_p(v)  # a non-NULL stand-in: never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dm.LIB_PATH):
        pytest.skip("libmoe.so not built (run __graft_entry__.build())")
    return dm.lib()


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), BAD_SHAPE), (dict(T=1 << 31), BAD_SHAPE), (dict(n=0), BAD_SHAPE), (dict(n=4097), BAD_SHAPE),
    (dict(K=0), BAD_SHAPE), (dict(K=17), BAD_SHAPE), (dict(n=4, K=5), BAD_SHAPE), (dict(T=1 << 28, K=8), BAD_SHAPE),
    (dict(S=-1), BAD_SHAPE), (dict(S=(1 << 20) + 1), BAD_SHAPE), (dict(S=1 << 20, n=4096), BAD_SHAPE),
    (dict(mask=3), BAD_RANGE), (dict(mask=-1), BAD_RANGE), (dict(dtype=2), BAD_RANGE), (dict(dtype=-1), BAD_RANGE),
    (dict(logits=N), NULL_ARG), (dict(idx=N), NULL_ARG), (dict(mask=1, m=N), NULL_ARG), (dict(S=2, off=N), NULL_ARG),
    (dict(loss=N), NULL_ARG), (dict(z=N), NULL_ARG), (dict(counts=N), NULL_ARG), (dict(tokens=N), NULL_ARG),
    (dict(ws=N), WORKSPACE), (dict(ws_bytes=255), WORKSPACE), (dict(ws=P(0x10008)), BAD_SHAPE),
    (dict(ws=P(0x10001)), BAD_SHAPE)])
def test_balance_forward_refuses(L, kw, expect):
    a = dict(T=64, n=32, K=4, S=0, mask=0, dtype=1, logits=P(), idx=P(), m=P(), off=P(), loss=P(), z=P(), counts=P(),
             tokens=P(), ws=P(), ws_bytes=1 << 40)
    a.update(kw)
    st = L.moe_balance_fwd(a["T"], a["n"], a["K"], a["S"], a["mask"], a["dtype"], a["logits"], a["idx"], a["m"], a["off"],
                           a["loss"], a["z"], a["counts"], a["tokens"], a["ws"], a["ws_bytes"], N)
    assert st == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(n=0), BAD_SHAPE), (dict(K=17), BAD_SHAPE), (dict(mask=3), BAD_RANGE), (dict(dtype=7), BAD_RANGE),
    (dict(logits=N), NULL_ARG), (dict(mask=2, m=N), NULL_ARG), (dict(S=3, off=N), NULL_ARG), (dict(counts=N), NULL_ARG),
    (dict(tokens=N), NULL_ARG), (dict(grad=N), NULL_ARG), (dict(T=0, grad=N, logits=N), OK)])
def test_balance_backward_refuses(L, kw, expect):
    a = dict(T=64, n=32, K=4, S=0, mask=0, dtype=1, logits=P(), m=P(), off=P(), counts=P(), tokens=P(), grad=P())
    a.update(kw)
    st = L.moe_balance_bwd(a["T"], a["n"], a["K"], a["S"], a["mask"], a["dtype"], a["logits"], a["m"], a["off"],
                           a["counts"], a["tokens"], P(), P(), a["grad"], N)
    assert st == expect


def test_balance_workspace(L):
    assert L.moe_balance_workspace_size(8, 8, 0, N) == NULL_ARG
    with pytest.raises(dm.MoeError):
        dm.moe_balance_workspace_size(8, 0, 0)
    for T, n, S in ((0, 1, 0), (1, 64, 0), (65536, 64, 0), (1000, 4096, 77), ((1 << 31) - 1, 64, 1 << 20)):
        size = dm.moe_balance_workspace_size(T, n, S)
        assert size % 256 == 0 and size >= 2 * 4 * n * max(S, 1)


@pytest.mark.parametrize("kw,expect", [
    (dict(R=-1), BAD_SHAPE), (dict(R=(1 << 40) + 1), BAD_SHAPE), (dict(F=0), BAD_SHAPE), (dict(F=(1 << 20) + 1), BAD_SHAPE),
    (dict(R=0, a=N, b=N, c=N, d=N), OK), (dict(a=N), NULL_ARG), (dict(b=N), NULL_ARG), (dict(c=N), NULL_ARG),
    (dict(d=N), NULL_ARG),
    (dict(R=1 << 38, F=32), UNSUPPORTED), (dict(R=1 << 33, F=7), UNSUPPORTED)])
def test_swiglu_entries_refuse(L, kw, expect):
    a = dict(R=8, F=64, a=P(), b=P(), c=P(), d=P())
    a.update(kw)
    R, F = a["R"], a["F"]
    assert L.moe_swiglu_checkpoint_fwd(R, F, a["a"], N, a["d"], a["b"], a["c"], N) == expect
    assert L.moe_swiglu_checkpoint_bwd(R, F, a["a"], a["b"], N, a["c"], a["d"], N) == expect


def test_gemm_entries_refuse(L):
    def fwd(shape, **kw):
        a = dict(x=P(), assist=P(), wg=P(), wu=P(), recv=P(), c=P(), s=P(), h=P())
        a.update(kw)
        return L.moe_ffn_gate_up_fwd_checkpoint(ctypes.byref(shape), *a.values(), N)

    def bwd(shape, **kw):
        a = dict(x=P(), assist=P(), rw=P(), wd=P(), c=P(), s=P(), recv=P(), ggu=P(), h=P())
        a.update(kw)
        return L.moe_ffn_down_bwd_data_checkpoint(ctypes.byref(shape), *a.values(), N)

    ok = dm.make_shape(8, 64, 2, 4, F=64)
    for f, names in ((fwd, ("x", "wg", "wu", "recv", "c", "s", "h")),
                     (bwd, ("x", "rw", "wd", "c", "s", "recv", "ggu", "h"))):
        for name in names:
            assert f(ok, **{name: N}) == NULL_ARG, name
        assert f(dm.make_shape(8, 64, 2, 4, F=48)) == BAD_SHAPE
        assert f(ok, c=P(0x10004)) == BAD_SHAPE
        assert f(dm.make_shape(1 << 20, 1024, 2, 4, F=64)) == UNSUPPORTED  # 31-bit offsets into gathered rows


def test_combine_entries_refuse(L):
    def fwd(shape, **kw):
        a = dict(y=P(), idx=P(), w=P(), assist=P(), counts=P(), m=N, sx=N, ox=N, a1=N, a2=N, v=N, out=P(), c=P(), s=P())
        a.update(kw)
        return L.moe_combine_checkpoint(ctypes.byref(shape), *a.values(), N)

    def bwd(shape, **kw):
        a = dict(d=P(), c=P(), s=P(), idx=P(), w=P(), assist=P(), counts=P(), m=N, ox=N, a1=N, a2=N, v=N, gw=P(), rw=N)
        a.update(kw)
        return L.moe_combine_bwd_weights_checkpoint(ctypes.byref(shape), *a.values(), N)

    ok = dm.make_shape(8, 64, 2, 4)
    for f, names in ((fwd, ("y", "idx", "w", "assist", "counts", "out", "c", "s")),
                     (bwd, ("d", "c", "s", "idx", "w", "assist", "counts", "gw"))):
        for name in names:
            assert f(ok, **{name: N}) == NULL_ARG, name
        assert f(dm.make_shape(8, 60, 2, 4)) == BAD_SHAPE
        assert f(dm.make_shape(8, 64, 2, 4, comm_quant_mode=2)) == UNSUPPORTED
        assert f(dm.make_shape(8, 64, 2, 4, mask_ndim=2)) == NULL_ARG
        assert f(dm.make_shape(8, 64, 2, 4, copy_expert_num=1)) == NULL_ARG
        assert f(dm.make_shape(8, 64, 2, 4, const_expert_num=1), ox=P(), a1=P(), a2=P()) == NULL_ARG
        assert f(dm.make_shape(8, 64, 2, 4, capacity=15)) == -4
        assert f(ok, c=P(0x10004)) == BAD_SHAPE
        assert f(dm.make_shape(0, 64, 2, 4), **{n: N for n in names}) == OK
    for name in ("y", "sx", "out"):
        assert fwd(ok, **{name: P(0x10002)}) == BAD_SHAPE, name
    assert fwd(dm.make_shape(8, 64, 2, 4, copy_expert_num=1), ox=P(0x10002)) == BAD_SHAPE
    assert bwd(ok, d=P(0x10008)) == BAD_SHAPE


def test_python_calls_refuse_cpu_tensors():
    with pytest.raises(dm.MoeError, match="GPU tensor"):
        dm.balance_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(dm.MoeError, match="GPU tensor"):
        dm.swiglu_checkpoint(torch.zeros(4, 64, dtype=torch.bfloat16))
    for bad in (None, [1.0], 3):
        with pytest.raises(dm.MoeError, match="GPU tensors"):
            dm.balance_loss(bad, torch.zeros(4, 2, dtype=torch.int32))
        with pytest.raises(dm.MoeError, match="GPU tensors"):
            dm.swiglu_checkpoint(bad)
    with pytest.raises(dm.MoeError, match="GPU tensor"):
        dm.moe_swiglu_checkpoint_bwd(torch.zeros(4, 64, dtype=torch.int8), N, N, N)


def test_combine_calls_refuse_other_shapes():
    for bad in (None, (8, 64), ctypes.c_int64(8)):
        with pytest.raises(dm.MoeError, match="MoeShape"):
            dm.moe_combine_checkpoint(bad, *[N] * 14)
        with pytest.raises(dm.MoeError, match="MoeShape"):
            dm.moe_combine_bwd_weights_checkpoint(bad, *[N] * 13)


def test_checkpoint_buffers():
    c, s = dm.checkpoint_buffers(3, 100, "cpu")
    assert c.shape == (3, 100) and s.shape == (3, 4) and c.dtype == torch.int8 and s.dtype == torch.bfloat16
    c, s = dm.checkpoint_buffers(3, 33, "cpu", halves=2)
    assert c.shape == (3, 66) and s.shape == (3, 4)


def test_combine_refuses_more_tokens_than_a_launch_has_waves(L):
    """A wave for a token is 2^32 threads at 2^26 tokens."""
    for T, expect in ((1 << 26, UNSUPPORTED), ((1 << 31) - 1, UNSUPPORTED)):
        s = ctypes.byref(dm.make_shape(T, 8, 1, 1))
        assert L.moe_combine_checkpoint(s, *[P()] * 5, *[N] * 6, *[P()] * 3, N) == expect
        assert L.moe_combine_bwd_weights_checkpoint(s, *[P()] * 7, *[N] * 5, P(), N, N) == expect
