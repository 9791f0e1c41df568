"""CPU checks of the training entry points' refusals: each returns before any
launch, so no GPU is needed."""
import ctypes

import pytest
import torch

from mixture_experts_routing_router_gb300 import build as B
from mixture_experts_routing_router_gb300 import native as N

P = ctypes.c_void_p
A, ODD, WS = P(4096), P(4100), P(1 << 20)          # never dereferenced: validation fails first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    B.build()
    return N.lib()


def shape(**kw):
    base = dict(tokens=64, hidden=256, experts=16, top_k=2, inter=512)
    base.update(kw)
    return N.make_shape(**base)


def fwd(L, rows=4, hidden=64, type=0, wtype=1, x=A, gamma=A, beta=A, eps=1e-5, y=A, mean=None, rstd=None):
    return L.moe_layernorm(rows, hidden, type, wtype, x, gamma, beta, eps, y, mean, rstd, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(hidden=0), dict(hidden=(1 << 20) + 1), dict(type=2), dict(type=-1), dict(wtype=7),
    dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF), dict(x=None), dict(x=ODD), dict(gamma=None), dict(beta=ODD),
    dict(y=None), dict(mean=ODD), dict(rstd=ODD), dict(rows=0, gamma=None)])
def test_layernorm_refusals(L, bad):
    assert fwd(L, **bad) == N.MOE_ERR_INVALID_ARG


def test_layernorm_without_rows_launches_nothing(L):
    assert fwd(L, rows=0, x=None, y=None) == N.MOE_OK


def test_layernorm_scratch_size(L):
    n = ctypes.c_size_t(0)
    assert L.moe_layernorm_scratch_size(100, 64, ctypes.byref(n)) == N.MOE_OK
    assert n.value >= 100 * 2 * 64 * 4
    small = n.value
    assert L.moe_layernorm_scratch_size(1 << 40, 64, ctypes.byref(n)) == N.MOE_OK
    assert small <= n.value <= 4 << 20                       # bounded in the rows
    assert L.moe_layernorm_scratch_size(100, 64, None) == N.MOE_ERR_INVALID_ARG
    assert L.moe_layernorm_scratch_size(-1, 64, ctypes.byref(n)) == N.MOE_ERR_INVALID_ARG
    assert L.moe_layernorm_scratch_size(1, 0, ctypes.byref(n)) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(hidden=0), dict(type=3), dict(wtype=3), dict(dy=None), dict(x=ODD), dict(gamma=None),
    dict(mean=None), dict(rstd=None), dict(dres=ODD), dict(dx=None), dict(dgamma=None), dict(dbeta=ODD),
    dict(scratch=None), dict(scratch=P(4096 + 16)), dict(bytes=100), dict(rows=0, dgamma=None)])
def test_layernorm_backward_refusals(L, bad):
    a = dict(rows=4, hidden=64, type=0, wtype=1, dy=A, x=A, gamma=A, mean=A, rstd=A, dres=None, dx=A, dgamma=A,
             dbeta=A, scratch=WS, bytes=1 << 20)
    a.update(bad)
    assert L.moe_layernorm_backward(*a.values(), None) == N.MOE_ERR_INVALID_ARG


def size(s):
    return N.moe_workspace_size(s)


@pytest.mark.parametrize("bad", [dict(dout=None), dict(dest=ODD), dict(w=None), dict(dy=None), dict(dw=ODD),
                                 dict(y=None), dict(y=ODD), dict(ws=P((1 << 20) + 16)), dict(bytes=4096)])
def test_combine_backward_refusals(L, bad):
    s = shape()
    a = dict(dout=A, y=A, dest=A, w=A, dy=A, dw=A, ws=WS, bytes=size(s))
    a.update(bad)
    assert L.moe_combine_backward(ctypes.byref(s), *a.values(), None) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(dx_perm=None), dict(dest=None), dict(add=ODD), dict(dx=ODD), dict(ws=None)])
def test_dispatch_backward_refusals(L, bad):
    s = shape()
    a = dict(dx_perm=A, dest=A, add=None, dx=A, ws=WS, bytes=size(s))
    a.update(bad)
    assert L.moe_dispatch_backward(ctypes.byref(s), *a.values(), None) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(ids=None), dict(w=ODD), dict(dw=None), dict(dl=ODD), dict(ws=None)])
def test_route_backward_refusals(L, bad):
    s = shape()
    a = dict(ids=A, w=A, dw=A, dl=A, ws=WS, bytes=size(s))
    a.update(bad)
    assert L.moe_route_backward(ctypes.byref(s), *a.values(), None) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(logits=None), dict(ids=ODD), dict(scale=NAN), dict(scale=INF), dict(dw=ODD),
                                 dict(dl=None)])
def test_route_sigmoid_backward_refusals(L, bad):
    s = shape()
    a = dict(logits=A, ids=A, scale=1.0, dw=A, dl=A, ws=WS, bytes=size(s))
    a.update(bad)
    assert L.moe_route_sigmoid_backward(ctypes.byref(s), *a.values(), None) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(dl=None), dict(x=None), dict(w=ODD), dict(g=None), dict(dx=ODD), dict(dw=ODD),
                                 dict(wgrad=3), dict(dx=None, dw=None), dict(ws=None), dict(bytes=100)])
def test_gate_backward_refusals(L, bad):
    s = shape()
    a = dict(dl=A, x=A, w=A, g=A, dx=A, dw=A, wgrad=0, ws=WS, bytes=size(s))
    a.update(bad)
    assert L.moe_gate_backward(ctypes.byref(s), *a.values(), None) == N.MOE_ERR_INVALID_ARG


UP_TRAIN = dict(x=A, offsets=A, w13=A, pre=A, h=A)
DOWN = dict(dy=A, offsets=A, w2=A, pre=A, h=A, dpre=A, dw2=A, wgrad=0)
UP = dict(dpre=A, offsets=A, x=A, w13=A, dx=A, dw13=A, wgrad=0)


@pytest.mark.parametrize("call,args,bad", [
    ("moe_expert_up_train", UP_TRAIN, b) for b in (dict(x=None), dict(offsets=ODD), dict(w13=None), dict(pre=ODD),
                                                   dict(h=None))] + [
    ("moe_expert_down_backward", DOWN, b) for b in (dict(dy=None), dict(offsets=None), dict(w2=None), dict(pre=ODD),
                                                    dict(h=None), dict(dpre=ODD), dict(dw2=ODD), dict(wgrad=3),
                                                    dict(wgrad=-1), dict(dpre=None, dw2=None))] + [
    ("moe_expert_up_backward", UP, b) for b in (dict(dpre=None), dict(offsets=ODD), dict(x=None), dict(w13=ODD),
                                                dict(dx=ODD), dict(dw13=ODD), dict(wgrad=5),
                                                dict(dx=None, dw13=None))])
def test_expert_ffn_refusals(L, call, args, bad):
    s = shape()
    a = dict(args, ws=WS, bytes=size(s))
    a.update(bad)
    assert getattr(L, call)(ctypes.byref(s), *a.values(), None) == N.MOE_ERR_INVALID_ARG
    a = dict(args, ws=WS, bytes=4096)
    assert getattr(L, call)(ctypes.byref(s), *a.values(), None) == N.MOE_ERR_INVALID_ARG
    assert getattr(L, call)(None, *a.values(), None) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("call,args", [("moe_expert_up_train", UP_TRAIN), ("moe_expert_down_backward", DOWN),
                                       ("moe_expert_up_backward", UP)])
def test_expert_ffn_training_takes_no_shared_experts(L, call, args):
    s = shape(shared=1, shared_inter=64)
    assert getattr(L, call)(ctypes.byref(s), *args.values(), WS, size(s), None) == N.MOE_ERR_UNSUPPORTED
    assert "shared" in N.last_error_message()


def test_binding_refuses_mismatched_tensors():
    x, g = torch.zeros(3, 8, dtype=torch.bfloat16), torch.ones(8)
    with pytest.raises(ValueError, match="weight of"):
        N.moe_layernorm(x, torch.ones(7), torch.ones(7), 1e-5, x)
    with pytest.raises(ValueError, match="beside an input"):
        N.moe_layernorm(x, g, g, 1e-5, torch.zeros(3, 8))
    with pytest.raises(ValueError, match="gamma and beta"):
        N.moe_layernorm(x, g, g.to(torch.bfloat16), 1e-5, x)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        N.moe_layernorm(x.half(), g, g, 1e-5, x.half())
    with pytest.raises(ValueError, match="mean must be float32"):
        N._stat(torch.zeros(2), 3, "mean")
    with pytest.raises(ValueError, match="accumulated in float32"):
        N._wgrad(x, True)
