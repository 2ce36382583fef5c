"""Argument checks of the decode-time products (qlora_fmt4_linear_fwd, qlora_moe_fwd) on the
host: every refusal returns before anything is launched, so no GPU is needed. The pointers are
made-up addresses that the checks only look at."""
import ctypes

import pytest
import torch

import bit_nf4_quantized_double_b200 as q

P = 1 << 20                # an aligned address


def fmt4(**kw):
    a = dict(X=P, M=1, codes=P, absmax=P, rows=64, cols=128, fmt=0, Y=P, ydt=q.QLORA_BF16)
    a.update(kw)
    return q.lib().qlora_fmt4_linear_fwd(a["X"], a["M"], a["codes"], a["absmax"], a["rows"], a["cols"], a["fmt"], a["Y"],
                                         a["ydt"], None)


@pytest.mark.parametrize("kw", [dict(X=0), dict(codes=0), dict(absmax=0), dict(Y=0), dict(X=P + 8), dict(codes=P + 1),
                                dict(absmax=P + 2), dict(Y=P + 4), dict(fmt=3), dict(fmt=-1), dict(ydt=2)])
def test_fmt4_linear_bad_arguments(kw):
    assert fmt4(**kw) == q.QLORA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(M=0), dict(M=-1), dict(M=65535 * 16 + 1), dict(rows=0), dict(rows=(1 << 30) + 1),
                                dict(cols=0), dict(cols=32), dict(cols=100), dict(cols=(1 << 27) + 64)])
def test_fmt4_linear_bad_shapes(kw):
    assert fmt4(**kw) == q.QLORA_ERR_UNSUPPORTED_SHAPE


def tensor(rows, cols, codes=P, scale8=P, scale2=P, offset=P):
    return q._Tensor(rows, cols, codes, scale8, scale2, offset)


def moe(T=2, d=128, f=192, E=4, k=2, ws_bytes=None, gate=None, up=None, down=None, **kw):
    a = dict(X=P, router=P, rdt=q.QLORA_F32, Y=P, experts=P, weights=P, ws=P)
    a.update(kw)
    gate = gate or tensor(E * f, d)
    up = up or tensor(E * f, d)
    down = down or tensor(E * d, f)
    if ws_bytes is None:
        ws_bytes = q.qlora_moe_fwd_workspace(T, d, f, E, k)
    return q.lib().qlora_moe_fwd(a["X"], T, a["router"], a["rdt"], E, ctypes.byref(gate), ctypes.byref(up),
                                 ctypes.byref(down), k, 1, a["Y"], a["experts"], a["weights"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(X=0), dict(X=P + 8), dict(router=0), dict(router=P + 4), dict(Y=0), dict(Y=P + 2),
                                dict(rdt=5), dict(experts=P + 2), dict(weights=P + 1),
                                dict(gate=tensor(768, 128, codes=P + 8)), dict(up=tensor(768, 128, scale8=0)),
                                dict(up=tensor(768, 128, scale8=P + 1)), dict(down=tensor(512, 192, scale2=P + 2)),
                                dict(down=tensor(512, 192, offset=0))])
def test_moe_bad_arguments(kw):
    assert moe(**kw) == q.QLORA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(T=0), dict(T=65), dict(E=257), dict(k=0), dict(k=5), dict(E=32, k=17),
                                dict(d=100), dict(f=96), dict(d=65600), dict(f=65600), dict(gate=tensor(767, 128)),
                                dict(up=tensor(768, 192)), dict(down=tensor(511, 192))])
def test_moe_bad_shapes(kw):
    kw.setdefault("ws_bytes", 1 << 30)
    assert moe(**kw) == q.QLORA_ERR_UNSUPPORTED_SHAPE


def test_moe_no_experts():
    t = dict(gate=tensor(192, 128), up=tensor(192, 128), down=tensor(128, 192))
    assert moe(E=0, ws_bytes=1 << 30, **t) == q.QLORA_ERR_UNSUPPORTED_SHAPE


def test_moe_workspace():
    need = q.qlora_moe_fwd_workspace(2, 128, 192, 4, 2)
    assert need > 0
    assert moe(ws_bytes=need - 1) == q.QLORA_ERR_WORKSPACE
    assert moe(ws=0) == q.QLORA_ERR_WORKSPACE
    assert moe(ws=P + 8) == q.QLORA_ERR_WORKSPACE
    # hidden values and partial outputs of every (token, choice), and more with more of either
    T, d, f, E, k = 16, 2048, 1024, 64, 8
    need = q.qlora_moe_fwd_workspace(T, d, f, E, k)
    assert need >= T * k * (f + d) * 4 + T * E * 8 + T * d * 2
    assert q.qlora_moe_fwd_workspace(2 * T, d, f, E, k) > need
    assert q.qlora_moe_fwd_workspace(T, d, 8 * f, E, k) > need
    for bad in ((0, d, f, E, k), (65, d, f, E, k), (T, d + 1, f, E, k), (T, d, f + 32, E, k), (T, d, f, 0, k), (T, d, f, 4, 5)):
        assert q.qlora_moe_fwd_workspace(*bad) == 0


def test_wrapper_refusals():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    codes, absmax = torch.zeros(64 * 64, dtype=torch.uint8), torch.zeros(128)
    with pytest.raises(ValueError):
        q.qlora_fmt4_linear_fwd(x.float(), codes, absmax, 64, "int4")
    with pytest.raises(ValueError):
        q.qlora_fmt4_linear_fwd(x, codes, absmax, 64, "nf4")
    with pytest.raises(ValueError):
        q.qlora_fmt4_linear_fwd(x, codes, absmax, 63, "int4")
    with pytest.raises(ValueError):
        q.qlora_fmt4_linear_fwd(x, codes, absmax.double(), 64, "int4")
    with pytest.raises(ValueError):
        q.qlora_fmt4_linear_fwd(x, codes, absmax, 64, "int4", Y=torch.zeros(2, 65))
    with pytest.raises(ValueError):                       # not on a GPU
        q.qlora_fmt4_linear_fwd(x, codes, absmax, 64, "int4")
    t = [q.nf4_empty(r, c, "cpu") for r, c in ((256, 128), (256, 128), (512, 64))]
    router = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        q.qlora_moe_fwd(x.half(), router, *t, 2)
    with pytest.raises(ValueError):
        q.qlora_moe_fwd(x, router[:, :64], *t, 2)
    with pytest.raises(ValueError):
        q.qlora_moe_fwd(x, router, *t, 2, Y=torch.zeros(2, 128))
    with pytest.raises(ValueError):                       # not on a GPU
        q.qlora_moe_fwd(x, router, *t, 2)
