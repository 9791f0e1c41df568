"""The trainable MoE block: its output and every gradient against the same block in
64-bit torch autograd (with the block's own routes), and a few training steps."""
import pytest
import torch

from mixture_experts_routing_router_gb300 import native as N
from mixture_experts_routing_router_gb300.block import MoEBlock

from gpu_util import dev

pytestmark = pytest.mark.gpu

D = torch.float64
# a chain of at most eight bf16 roundings (n, pre, h, y, dy, dpre, dx_perm, dn), each an
# independent relative error of 2^-9 / sqrt(3) at most in the 2-norm, then five times that
TOL = 5 * 8 ** 0.5 * 2.0 ** -9 / 3 ** 0.5


def block_in_64_bits(block, x, ids):
    p = {n: t.detach().to(D).requires_grad_() for n, t in block.named_parameters()}
    xd = x.detach().to(D).requires_grad_()
    mu = xd.mean(1, keepdim=True)
    n = (xd - mu) / torch.sqrt(((xd - mu) ** 2).mean(1, keepdim=True) + block.eps) * p["gamma"] + p["beta"]
    w = torch.softmax(torch.gather(n @ p["w_gate"].t(), 1, ids), 1)
    out = xd
    for e in range(block.experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        z = n[t] @ p["w13"][e].t()
        if block.act == N.MOE_ACT_SWIGLU:
            g, u = z.chunk(2, 1)
            a = g * torch.sigmoid(g) * u
        else:
            a = torch.clamp(z, min=0.0) ** 2
        out = out.index_add(0, t, (a @ p["w2"][e].t()) * w[t, j].unsqueeze(1))
    return out, xd, p


def routes_of(block, x):
    """The ids the block's own forward picks (routing is a discrete choice)."""
    n = torch.empty_like(x)
    N.moe_layernorm(x, block.gamma.detach(), block.beta.detach(), block.eps, n)
    shape, ws = block._layer(x.shape[0], x.device)
    logits = torch.empty(x.shape[0], block.experts, device=dev())
    ids = torch.empty(x.shape[0], block.top_k, dtype=torch.int32, device=dev())
    N.moe_gate(shape, n, block.w_gate.detach(), logits, ws)
    N.moe_route(shape, logits, ids, torch.empty_like(ids, dtype=torch.float32), ws)
    return ids.long()


def rel(a, b):
    return float((a.detach().to(D) - b).norm() / b.norm())


@pytest.mark.parametrize("size", [(1, 64, 4, 2, 64), (40, 256, 16, 2, 512), (300, 136, 33, 5, 72),
                                  (513, 320, 6, 3, 264)], ids=str)
@pytest.mark.parametrize("act", [N.MOE_ACT_SWIGLU, N.MOE_ACT_RELU2], ids=["swiglu", "relu2"])
def test_block_gradients(size, act):
    T, H, E, k, I = size
    gen = torch.Generator(device=dev()).manual_seed(T)
    block = MoEBlock(H, E, k, I, act=act, device=dev(), generator=gen)
    with torch.no_grad():
        block.gamma += 0.2 * torch.randn(H, generator=gen, device=dev())
        block.beta += 0.2 * torch.randn(H, generator=gen, device=dev())
    x = torch.randn(T, H, generator=gen, device=dev()).to(torch.bfloat16).requires_grad_()
    dout = torch.randn(T, H, generator=gen, device=dev()).to(torch.bfloat16)
    out = block(x)
    out.backward(dout)
    block.check()
    want, xd, p = block_in_64_bits(block, x, routes_of(block, x.detach()))
    want.backward(dout.to(D))
    assert rel(out, want.detach()) <= TOL
    assert rel(x.grad, xd.grad) <= TOL
    for name, param in block.named_parameters():
        assert param.grad.dtype == param.dtype
        if float(p[name].grad.norm()) > 0:
            assert rel(param.grad, p[name].grad) <= TOL, name


def test_frozen_weights_get_no_gradient():
    block = MoEBlock(64, 4, 2, 64, device=dev())
    block.w13.requires_grad_(False)
    block.w2.requires_grad_(False)
    x = torch.randn(9, 64, device=dev()).to(torch.bfloat16)
    block(x).float().square().sum().backward()
    block.check()
    assert block.w13.grad is None and block.w2.grad is None
    assert block.w_gate.grad is not None and block.gamma.grad is not None


def test_training_steps_reduce_the_loss():
    gen = torch.Generator(device=dev()).manual_seed(3)
    block = MoEBlock(128, 8, 2, 128, device=dev(), generator=gen)
    x = torch.randn(256, 128, generator=gen, device=dev()).to(torch.bfloat16)
    target = x.float() + torch.randn(256, 128, generator=gen, device=dev())
    opt = torch.optim.Adam(block.parameters(), lr=3e-3)
    losses = []
    for _ in range(40):
        opt.zero_grad()
        loss = (block(x).float() - target).square().mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    block.check()
    assert losses[-1] < 0.7 * losses[0], (losses[0], losses[-1])


def test_block_refuses_other_inputs():
    block = MoEBlock(64, 4, 2, 64, device=dev())
    with pytest.raises(ValueError, match="bfloat16"):
        block(torch.randn(3, 64, device=dev()))
    with pytest.raises(ValueError, match="tokens, 64"):
        block(torch.randn(3, 72, device=dev()).to(torch.bfloat16))
    with pytest.raises(N.MoEError):
        block(torch.empty(0, 64, device=dev(), dtype=torch.bfloat16))


def test_batches_of_several_sizes_share_the_workspace():
    """Gradients are those of each batch alone, bit for bit, whichever forward passes come
    between, and an error of any of them waits for check()."""
    gen = torch.Generator(device=dev()).manual_seed(5)
    block = MoEBlock(136, 7, 3, 72, device=dev(), generator=gen)
    sizes = [40, 513, 1, 300, 40]
    xs = [torch.randn(n, 136, generator=gen, device=dev()).to(torch.bfloat16).requires_grad_() for n in sizes]
    params = list(block.parameters())
    alone = [torch.autograd.grad(block(x).float().square().sum(), [x, *params]) for x in xs]
    outs = [block(x) for x in xs]
    for out, x, want in reversed(list(zip(outs, xs, alone))):
        got = torch.autograd.grad(out.float().square().sum(), [x, *params])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    block.check()
    fresh = MoEBlock(136, 7, 3, 72, device=dev(), generator=gen)
    nan = torch.full((40, 136), float("nan"), device=dev(), dtype=torch.bfloat16)
    fresh(nan)
    for n in (30, 2000):
        fresh(torch.randn(n, 136, generator=gen, device=dev()).to(torch.bfloat16))
    with pytest.raises(N.MoEError) as e:
        fresh.check()
    assert e.value.status == N.MOE_ERR_NONFINITE
    fresh.check()
