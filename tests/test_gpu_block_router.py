"""The trainable block with a group-limited router: its output and gradients against the
same block in 64-bit autograd (with the block's own routes), and its refusals."""
import copy

import pytest
import torch

import fp8_ref as ref
import test_gpu_block as plain
from mixture_experts_routing_router_gb300 import native as N
from mixture_experts_routing_router_gb300.block import MoEBlock

from gpu_util import dev

pytestmark = pytest.mark.gpu

D = torch.float64


def in_64_bits(block, x, ids):
    p = {n: t.detach().to(D).requires_grad_() for n, t in block.named_parameters()}
    xd = x.detach().to(D).requires_grad_()
    mu = xd.mean(1, keepdim=True)
    n = (xd - mu) / torch.sqrt(((xd - mu) ** 2).mean(1, keepdim=True) + block.eps) * p["gamma"] + p["beta"]
    r = block.router
    w = ref.weights(n @ p["w_gate"].t(), ids, r.score == N.MOE_SCORE_SOFTMAX, bool(r.renorm), r.scale)
    out = xd
    for e in range(block.experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g, u = (n[t] @ p["w13"][e].t()).chunk(2, 1)
        out = out.index_add(0, t, (g * torch.sigmoid(g) * u @ p["w2"][e].t()) * w[t, j].unsqueeze(1))
    return out, xd, p


def routes_of(block, x):
    n = torch.empty_like(x)
    N.moe_layernorm(x, block.gamma.detach(), block.beta.detach(), block.eps, n)
    shape, ws = block._layer(x.shape[0], x.device)
    logits = torch.empty(x.shape[0], block.experts, device=dev())
    ids = torch.empty(x.shape[0], block.top_k, dtype=torch.int32, device=dev())
    N.moe_gate(shape, n, block.w_gate.detach(), logits, ws)
    N.moe_route_grouped(shape, block.router, logits, block.route_bias, ids, torch.empty_like(ids, dtype=torch.float32), ws)
    return ids.long()


@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "plain"])
@pytest.mark.parametrize("score", [N.MOE_SCORE_SIGMOID, N.MOE_SCORE_SOFTMAX], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [(1, 64, 8, 2, 64, 4, 2), (300, 136, 30, 5, 72, 6, 2)], ids=str)
def test_gradients(size, score, renorm):
    T, H, E, k, I, G, tg = size
    gen = torch.Generator(device=dev()).manual_seed(T)
    block = MoEBlock(H, E, k, I, device=dev(), generator=gen, router=N.make_router(score, G, tg, 2, renorm, 2.5))
    block.route_bias += 0.05 * torch.randn(E, generator=gen, device=dev())
    x = torch.randn(T, H, generator=gen, device=dev()).to(torch.bfloat16).requires_grad_()
    dout = torch.randn(T, H, generator=gen, device=dev()).to(torch.bfloat16)
    out = block(x)
    out.backward(dout)
    block.check()
    assert "route_bias" in block.state_dict() and "route_bias" not in dict(block.named_parameters())
    want, xd, p = in_64_bits(block, x, routes_of(block, x.detach()))
    want.backward(dout.to(D))
    assert plain.rel(out, want.detach()) <= plain.TOL
    assert plain.rel(x.grad, xd.grad) <= plain.TOL
    for name, param in block.named_parameters():
        if float(p[name].grad.norm()) > 0:
            assert plain.rel(param.grad, p[name].grad) <= plain.TOL, name


def test_the_bias_moves_the_choice_and_nothing_else():
    """A bias that decides: only its experts are used, with the unbiased scores' weights."""
    gen = torch.Generator(device=dev()).manual_seed(1)
    block = MoEBlock(64, 16, 2, 64, device=dev(), generator=gen, router=N.make_router(groups=4, topk_groups=2))
    other = copy.deepcopy(block)
    x = torch.randn(50, 64, generator=gen, device=dev()).to(torch.bfloat16)
    block.route_bias[[5, 14]] = 10.0
    assert torch.all(torch.sort(routes_of(block, x), 1).values == torch.tensor([5, 14], device=dev()))
    assert not torch.equal(block(x), other(x))
    block.check()


def test_other_routers_and_biases_are_refused():
    with pytest.raises(ValueError, match="make_router"):
        MoEBlock(64, 4, 2, 64, device=dev(), router=2)
    block = MoEBlock(64, 4, 2, 64, device=dev(), router=N.make_router(groups=3))
    x = torch.randn(3, 64, device=dev()).to(torch.bfloat16)
    with pytest.raises(N.MoEError, match="router"):
        block(x)
    block = MoEBlock(64, 4, 2, 64, device=dev(), router=N.make_router())
    block.route_bias = block.route_bias.half()
    with pytest.raises(ValueError, match="route_bias"):
        block(x)


def test_the_backward_pass_uses_the_router_of_its_forward():
    gen = torch.Generator(device=dev()).manual_seed(2)
    block = MoEBlock(64, 16, 2, 64, device=dev(), generator=gen, router=N.make_router(groups=4, topk_groups=2, scale=2.0))
    x = torch.randn(40, 64, generator=gen, device=dev()).to(torch.bfloat16)
    grads = []
    for scale in (2.0, 8.0):
        block.router.scale = 2.0
        loss = block(x).float().square().sum()
        block.router.scale = scale                       # for the next batch
        grads.append(torch.autograd.grad(loss, [p for p in block.parameters()]))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
