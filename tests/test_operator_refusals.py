"""What the serving operators refuse, and what they size, without a GPU: every call below fails on the host before
anything is launched."""
import ctypes

import pytest
import torch

import post_weight_quantization_21_b200 as g
from post_weight_quantization_21_b200 import pipeline as P


@pytest.fixture(scope="module")
def lib():
    return g.lib()


P16 = ctypes.c_void_p(4096)   # aligned, never dereferenced
Q16 = ctypes.c_void_p(8192)
ODD = ctypes.c_void_p(4097)
OFF8 = ctypes.c_void_p(4104)
OK, ARG, UNSUP, WS = g.GPTQ_OK, g.GPTQ_ERR_ARG, g.GPTQ_ERR_UNSUPPORTED, g.GPTQ_ERR_WORKSPACE


def quantize(X=P16, dt=0, m=4, k=64, rows=1, Q=Q16, sc=P16):
    return g.lib().gptq_fp8_quantize(X, dt, m, k, rows, Q, sc, None)


@pytest.mark.parametrize("kw", [dict(m=-1), dict(k=0), dict(k=24), dict(k=(1 << 20) + 16), dict(dt=3), dict(rows=0),
                                dict(rows=64), dict(X=None), dict(Q=None), dict(sc=None), dict(X=OFF8), dict(Q=OFF8),
                                dict(sc=ODD), dict(Q=P16, X=P16)])
def test_fp8_quantize_refuses(lib, kw):
    assert quantize(**kw) == ARG


def from_packed(pk=P16, sc=P16, z=P16, m=4, k=256, bits=4, gs=0, Q=P16, qs=Q16):
    return g.lib().gptq_fp8_from_packed(pk, sc, z, m, k, bits, gs, Q, qs, None)


@pytest.mark.parametrize("kw,st", [(dict(m=-1), ARG), (dict(k=40), ARG), (dict(bits=5), ARG), (dict(bits=1), ARG),
                                   (dict(gs=-128), ARG), (dict(gs=96), ARG), (dict(gs=512), ARG), (dict(gs=32), UNSUP),
                                   (dict(gs=64), UNSUP), (dict(k=192, gs=192), UNSUP), (dict(pk=None), ARG),
                                   (dict(Q=OFF8), ARG), (dict(qs=P16), ARG), (dict(z=ODD), ARG)])
def test_fp8_from_packed_refuses(lib, kw, st):
    assert from_packed(**kw) == st


def matmul(A=P16, sa=P16, B=P16, sb=P16, rows=1, m=33, n=64, k=64, Y=P16, dt=0, st=P16, ws=P16, nb=1 << 40):
    return g.lib().gptq_fp8_matmul(A, sa, B, sb, rows, m, n, k, Y, dt, st, ws, nb, None)


@pytest.mark.parametrize("kw", [dict(m=-1), dict(n=0), dict(k=0), dict(k=72), dict(rows=2), dict(dt=9), dict(A=None),
                                dict(sa=None), dict(B=None), dict(sb=None), dict(Y=None), dict(st=None), dict(A=OFF8),
                                dict(B=OFF8), dict(Y=ODD), dict(m=(1 << 20) + 1), dict(n=(1 << 20) + 1)])
def test_fp8_matmul_refuses(lib, kw):
    assert matmul(**kw) == ARG


def test_fp8_matmul_workspace(lib):
    m, n, k = 64, 768, 11008  # few tiles, many blocks: split
    need = g.gptq_fp8_matmul_workspace_size(m, n, k)
    assert need >= 2 * m * n * 4
    assert matmul(m=m, n=n, k=k, ws=None) == WS
    assert matmul(m=m, n=n, k=k, nb=0) == WS
    assert matmul(m=m, n=n, k=k, ws=OFF8) == WS
    assert g.gptq_fp8_matmul_workspace_size(1, 4096, 4096) == 0
    assert g.gptq_fp8_matmul_workspace_size(0, 64, 64) == 0
    assert g.gptq_fp8_matmul_workspace_size(8, 64, 40) == 0


def moe(X=P16, dt=0, t=4, d=64, f=64, e=4, top=2, bits=4, gs=0, act=g.GPTQ_ACT_SILU_GATED, flags=0, router=P16, up=P16,
        gate=P16, down=P16, ids=P16, w=P16, Y=P16, ydt=0, st=P16, ws=P16, nb=1 << 40, cfg=True):
    mk = lambda p: None if p is None else ctypes.byref(g.MoeWeights(p.value, p.value, p.value) if p else g.MoeWeights())
    c = ctypes.byref(g.MoeCfg(e, top, bits, gs, act, flags)) if cfg else None
    return g.lib().gptq_moe_layer(X, dt, t, d, f, c, router, mk(up), mk(gate), mk(down), ids, w, Y, ydt, st, ws, nb, None)


NONE = ctypes.c_void_p(0)


@pytest.mark.parametrize("kw", [dict(cfg=False), dict(t=-1), dict(t=65), dict(d=48), dict(f=16), dict(e=0), dict(e=257),
                                dict(top=0), dict(top=5), dict(router=None, top=17), dict(bits=1), dict(gs=96),
                                dict(gs=-32), dict(d=128, gs=128), dict(act=2), dict(flags=2), dict(dt=4), dict(ydt=5),
                                dict(up=None), dict(down=None), dict(gate=None), dict(gate=NONE), dict(up=NONE),
                                dict(down=OFF8), dict(act=g.GPTQ_ACT_RELU), dict(X=None), dict(X=OFF8), dict(router=OFF8),
                                dict(ids=None), dict(w=None), dict(Y=None), dict(Y=ODD), dict(st=None)])
def test_moe_refuses(lib, kw):
    assert moe(**kw) == ARG


def test_moe_workspace(lib):
    need = g.gptq_moe_workspace_size(4, 64, 64, 4, 2)
    assert need > 0
    assert moe(ws=None) == WS and moe(nb=need - 1) == WS and moe(ws=OFF8) == WS
    assert g.gptq_moe_workspace_size(0, 64, 64, 4, 2) == 0
    assert g.gptq_moe_workspace_size(65, 64, 64, 4, 2) == 0
    assert g.gptq_moe_workspace_size(4, 64, 48, 4, 2) == 0
    assert g.gptq_moe_workspace_size(4, 64, 64, 257, 2) == 0
    assert moe(t=0, X=None, up=NONE, ws=None) == OK  # no tokens: nothing to do


def test_binding_refuses_wrong_tensors():
    """Shapes, types and devices are checked before pointers reach the library."""
    f8 = torch.float8_e4m3fn
    X, Q, s = torch.zeros(4, 256), torch.zeros(4, 256).to(f8), torch.zeros(4, 2)
    st, ws, i32 = torch.zeros(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8), torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        g.gptq_fp8_quantize(X, Q, s)
    with pytest.raises(ValueError, match="X: "):
        g.gptq_fp8_quantize(X.double(), Q, s)
    with pytest.raises(ValueError, match="block_rows"):
        g.gptq_fp8_quantize(X, Q, s, 64)
    with pytest.raises(ValueError, match="A: "):
        g.gptq_fp8_matmul(X, s, Q, s, 1, X, st, ws)
    with pytest.raises(ValueError, match="b_block_rows"):
        g.gptq_fp8_matmul(Q, s, Q, s, 64, X, st, ws)
    with pytest.raises(ValueError, match="Q: "):
        g.gptq_fp8_from_packed(torch.zeros(4, 32, dtype=i32), s, s.to(i32), 4, 0, X, s)
    w = (torch.zeros(2, 64, 32, dtype=i32), torch.zeros(2, 64, 1), torch.zeros(2, 64, 1, dtype=i32))
    ids, tw = torch.zeros(4, 1, dtype=i32), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="bits"):
        g.gptq_moe_layer(X, None, w, w, w, ids, tw, X, st, ws, 5)
    with pytest.raises(ValueError, match="CUDA"):
        g.gptq_moe_layer(X, None, w, w, w, ids, tw, X, st, ws, 4)


def test_pipeline_configuration():
    with pytest.raises(ValueError, match="linears"):
        P.BlockConfig(128, 4, 512, 64, linears="int8")
    with pytest.raises(ValueError, match="group_size"):
        P.BlockConfig(128, 4, 512, 64, group_size=64, linears="fp8")
    assert P.BlockConfig(128, 4, 512, 64).linears == "dense"
