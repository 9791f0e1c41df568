"""Refusals of group-limited routing and the block-scaled FP8 calls on the host (no GPU: they
return before any CUDA call), and the rules on their kernel's waits."""
import ctypes
import math
import re

import pytest
import torch

from mixture_experts_routing_router_gb300 import build as B
from mixture_experts_routing_router_gb300 import native as N

import test_wait_discipline as W

P = ctypes.c_void_p
OK, WS = P(4096), P(1 << 20)


@pytest.fixture(scope="module")
def L():
    B.build()
    return N.lib()


def shape(**kw):
    return N.make_shape(**{**dict(tokens=64, hidden=256, experts=16, top_k=2, inter=512), **kw})


def calls(L, s, router=None, **change):
    """Every call with plain addresses, `change` replacing arguments by name."""
    n = change.pop("ws_bytes", N.moe_workspace_size(s))
    r = ctypes.byref(router if router is not None else N.make_router())
    s = ctypes.byref(s)
    a = lambda name: change.get(name, OK)
    ws = change.get("ws", WS)
    return {
        "moe_route_grouped": lambda: L.moe_route_grouped(s, r, a("logits"), a("bias"), a("ids"), a("w"), ws, n, None),
        "moe_route_grouped_backward": lambda: L.moe_route_grouped_backward(s, r, a("logits"), a("ids"), a("dw"),
                                                                           a("dlogits"), ws, n, None),
        "moe_dispatch_fp8_block": lambda: L.moe_dispatch_fp8_block(s, a("x"), a("ids"), a("counts"), a("offsets"),
                                                                   a("dest"), a("sorted_pair"), a("x_perm"),
                                                                   a("x_scale"), ws, n, None),
        "moe_expert_up_fp8_block": lambda: L.moe_expert_up_fp8_block(s, a("x_perm"), a("x_scale"), a("offsets"),
                                                                     a("w13"), a("w13_scale"), a("h"), a("h_scale"),
                                                                     ws, n, None),
        "moe_expert_down_fp8_block": lambda: L.moe_expert_down_fp8_block(s, a("h"), a("h_scale"), a("offsets"),
                                                                         a("w2"), a("w2_scale"), a("y_perm"), ws, n,
                                                                         None),
        "moe_layer_fp8_block": lambda: L.moe_layer_fp8_block(s, a("logits"), None, None, a("x"), a("w13"),
                                                             a("w13_scale"), a("w2"), a("w2_scale"), None, a("out"),
                                                             ws, n, None),
    }


ARGS = {
    "moe_route_grouped": ["logits", "ids", "w"],
    "moe_route_grouped_backward": ["logits", "ids", "dw", "dlogits"],
    "moe_dispatch_fp8_block": ["x", "ids", "counts", "offsets", "dest", "sorted_pair", "x_perm", "x_scale"],
    "moe_expert_up_fp8_block": ["x_perm", "x_scale", "offsets", "w13", "w13_scale", "h", "h_scale"],
    "moe_expert_down_fp8_block": ["h", "h_scale", "offsets", "w2", "w2_scale", "y_perm"],
    "moe_layer_fp8_block": ["logits", "x", "w13", "w13_scale", "w2", "w2_scale", "out"],
}


@pytest.mark.parametrize("call,arg", [(c, a) for c, args in ARGS.items() for a in args])
def test_null_and_misaligned_pointers(L, call, arg):
    for bad in (P(4096 + 4), None):
        if arg == "logits" and bad is None and call == "moe_layer_fp8_block":
            continue                            # preselected ids, which are NULL too: refused as well
        assert calls(L, shape(), **{arg: bad})[call]() == N.MOE_ERR_INVALID_ARG, bad


@pytest.mark.parametrize("call", sorted(ARGS))
def test_workspace(L, call):
    s = shape()
    assert calls(L, s, ws=P((1 << 20) + 16))[call]() == N.MOE_ERR_INVALID_ARG
    assert calls(L, s, ws=None)[call]() == N.MOE_ERR_INVALID_ARG
    least = N.moe_workspace_size(s) if call == "moe_layer_fp8_block" else N.moe_workspace_stage_size(s)
    assert calls(L, s, ws_bytes=least - 1)[call]() == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [c for c in sorted(ARGS) if "fp8" in c])
def test_shapes(L, call):
    assert calls(L, shape(hidden=264))[call]() == N.MOE_ERR_INVALID_ARG
    assert calls(L, shape(inter=520))[call]() == N.MOE_ERR_INVALID_ARG
    assert "16" in N.last_error_message()
    assert calls(L, shape(shared=1, shared_inter=64))[call]() == N.MOE_ERR_UNSUPPORTED


def test_preselected_layer_needs_ids_and_weights(L):
    s = shape()
    n = N.moe_workspace_size(s)
    for ids, w in ((None, OK), (OK, None)):
        assert L.moe_layer_fp8_block(ctypes.byref(s), None, ids, w, OK, OK, OK, OK, OK, None, OK, WS, n,
                                     None) == N.MOE_ERR_INVALID_ARG


BAD_ROUTERS = [dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=32), dict(groups=-4),
               dict(groups=4, topk_groups=5), dict(groups=4, topk_groups=0), dict(group_top=0), dict(group_top=3),
               dict(scale=math.inf), dict(scale=math.nan), dict(groups=16, topk_groups=1)]


@pytest.mark.parametrize("bad", BAD_ROUTERS, ids=str)
@pytest.mark.parametrize("call", ["moe_route_grouped", "moe_route_grouped_backward"])
def test_routers(L, call, bad):
    assert calls(L, shape(), N.make_router(**bad))[call]() == N.MOE_ERR_INVALID_ARG
    assert "router" in N.last_error_message()


def test_router_renorm_and_null(L):
    r = N.make_router()
    r.renorm = 2
    s = shape()
    assert calls(L, s, r)["moe_route_grouped"]() == N.MOE_ERR_INVALID_ARG
    assert L.moe_route_grouped(ctypes.byref(s), None, OK, None, OK, OK, WS, N.moe_workspace_size(s),
                               None) == N.MOE_ERR_INVALID_ARG


def test_the_layer_s_codes_and_scales_fit_its_workspace():
    """A row of n codes and its scales lie where the BF16 layer keeps a row of n values."""
    for n in range(16, 4096, 16):
        assert n + 4 * N.fp8_blocks(n) <= 2 * n


class Ws:
    is_cuda, nbytes = True, 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0


BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
T, H, E, K, I = 5, 144, 12, 3, 272
R = T * K


def tensors(act):
    parts = 2 if act == N.MOE_ACT_SWIGLU else 1
    up = dict(x_perm=(U8, R * H), x_scale=(F32, R * 2), offsets=(I32, E + 1), w13=(U8, E * parts * I * H),
              w13_scale=(F32, E * parts * 3 * 2), h=(U8, R * I), h_scale=(F32, R * 3))
    return {
        "moe_route_grouped": dict(router=N.make_router(), logits=(F32, T * E), bias=(F32, E), topk_ids=(I32, R),
                                  topk_w=(F32, R)),
        "moe_route_grouped_backward": dict(router=N.make_router(), logits=(F32, T * E), topk_ids=(I32, R),
                                           dtopk_w=(F32, R), dlogits=(F32, T * E)),
        "moe_dispatch_fp8_block": dict(x=(BF16, T * H), topk_ids=(I32, R), counts=(I32, E), offsets=(I32, E + 1),
                                       dest=(I32, R), sorted_pair=(I32, R), x_perm=(U8, R * H), x_scale=(F32, R * 2)),
        "moe_expert_up_fp8_block": up,
        "moe_expert_down_fp8_block": dict(h=(U8, R * I), h_scale=(F32, R * 3), offsets=(I32, E + 1),
                                          w2=(U8, E * H * I), w2_scale=(F32, E * 2 * 3), y_perm=(BF16, R * H)),
        "moe_layer_fp8_block": dict(logits=(F32, T * E), ids_in=(I32, R), w_in=(F32, R), x=(BF16, T * H),
                                    w13=up["w13"], w13_scale=up["w13_scale"], w2=(U8, E * H * I),
                                    w2_scale=(F32, E * 2 * 3), out=(BF16, T * H), residual=(BF16, T * H)),
    }


@pytest.mark.parametrize("act,call,arg", [(act, c, a) for act in (N.MOE_ACT_SWIGLU, N.MOE_ACT_RELU2)
                                          for c, args in tensors(act).items() for a, v in args.items()
                                          if isinstance(v, tuple)])
def test_the_binding_refuses_tensors_that_do_not_fit(L, act, call, arg):
    s = N.make_shape(T, H, E, K, I, act=act)
    args = tensors(act)[call]
    dtype, n = args[arg]

    def go(t):
        kw = {a: (v if not isinstance(v, tuple) else 4096) for a, v in args.items()}
        kw[arg] = t
        return getattr(N, call)(s, ws=Ws(), stream=0, **kw)

    with pytest.raises(ValueError, match=arg):
        go(torch.empty(n - 1, dtype=dtype))
    with pytest.raises(ValueError, match=arg):
        go(torch.empty(n, dtype=torch.int64))
    with pytest.raises(ValueError, match="device tensor"):
        go(torch.empty(n, dtype=dtype))                          # large enough, but not on a GPU
    with pytest.raises(N.MoEError):
        go(4096)                                                  # a plain address: the C call refuses the workspace


@pytest.mark.parametrize("name", ["gemm_fp8.cu", "gemm_fp8_rows.cu"])
def test_waits_of_the_fp8_kernels(name):
    """The rules of the other GEMMs: a warp gives up a wait as a whole (a wait that is not the
    warp's stands in a block of one thread), and no barrier without a limit between roles."""
    (kernel, body), = W.kernels(name)
    alone = list(re.finditer(r"\b(mbar_wait_bounded|wait_armed_stages)\(", body))
    assert len(alone) == 2 and body.count("mbar_wait_warp(") == 5
    for m in alone:
        assert any(W.SINGLE.search(h) for h in W.enclosing(body, m.start())), body[m.start():m.start() + 70]
    roles = body[body.index("if (warp == 0) {"):body.rindex("tc_fence_before")]
    assert "bar.sync" not in roles and "__syncthreads" not in roles
