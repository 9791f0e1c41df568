"""What the trainable block refuses before it calls the library (CPU)."""
import pytest
import torch

from mixture_experts_routing_router_gb300 import block as block_module
from mixture_experts_routing_router_gb300 import native as N
from mixture_experts_routing_router_gb300.block import MoEBlock

BF16 = torch.bfloat16


def block(act=N.MOE_ACT_SWIGLU):
    return MoEBlock(24, 4, 2, 8, act=act, device="cpu")


@pytest.mark.parametrize("act", [N.MOE_ACT_SWIGLU, N.MOE_ACT_RELU2])
@pytest.mark.parametrize("name", ["w_gate", "w13", "w2"])
def test_weights_of_another_type_or_shape_are_refused(act, name):
    """Module.float() would otherwise have the kernels read float32 as bfloat16."""
    x = torch.zeros(3, 24, dtype=BF16)
    with pytest.raises(ValueError, match="w_gate must be bfloat16"):
        block(act).float()(x)
    for bad in (lambda w: w.float(), lambda w: w[:-1], lambda w: w.transpose(-1, -2)):
        b = block(act)
        w = getattr(b, name).detach()
        setattr(b, name, torch.nn.Parameter(bad(w).contiguous()))
        with pytest.raises(ValueError, match=f"{name} must be bfloat16"):
            b(x)


class FakeLibrary:
    """The native module with calls that compute nothing, for the block's own logic."""

    def __getattr__(self, name):
        if name.startswith("moe_"):
            return lambda *a, **k: None
        return getattr(N, name)

    def workspace(self, shape, device):               # zero-filled, as the library's
        return torch.zeros(self.moe_workspace_size(shape), dtype=torch.uint8)

    def moe_workspace_size(self, shape):
        return 2 * self.moe_workspace_stage_size(shape)

    def moe_workspace_stage_size(self, shape):
        return 8192 * shape.tokens

    def moe_workspace_init(self, ws):
        ws[:4096] = 0

    # the device status: the workspace's first word
    fails = ()                                        # (call, tokens) that raise one

    def raised(self, call, shape, ws):
        assert ws.nbytes >= self.moe_workspace_stage_size(shape)
        if (call, shape.tokens) in self.fails:
            ws.view(torch.int32)[0] = N.MOE_ERR_NONFINITE

    def moe_route(self, shape, *args):
        self.raised("forward", shape, args[-1])

    def moe_route_backward(self, shape, *args):
        self.raised("backward", shape, args[-1])

    def moe_status_read(self, ws):
        status = int(ws.view(torch.int32)[0])
        ws.view(torch.int32)[0] = 0
        return status

    def layernorm_scratch(self, rows, hidden, device):
        return torch.zeros(1)


def test_second_derivatives_raise(monkeypatch):
    """A gradient penalty would otherwise lose its gradient without a word."""
    monkeypatch.setattr(block_module, "N", FakeLibrary())
    b = block()
    b.w2.requires_grad_(False)
    x = torch.zeros(3, 24, dtype=BF16, requires_grad=True)
    params = [b.gamma, b.beta, b.w_gate, b.w13]
    for wrt in ([x], [b.gamma], [b.w_gate], [x, *params]):
        for dout_has_a_graph in (False, True):
            out = b(x).float()
            loss = out.square().sum() if dout_has_a_graph else out.sum()
            grads = torch.autograd.grad(loss, wrt, create_graph=True)
            assert all(g.shape == t.shape and g.dtype == t.dtype for g, t in zip(grads, wrt))
            with pytest.raises(RuntimeError, match="cannot be differentiated again"):
                (loss + sum(g.float().square().sum() for g in grads)).backward()


def test_a_graph_that_nothing_asks_for_does_not_matter(monkeypatch):
    monkeypatch.setattr(block_module, "N", FakeLibrary())
    b = block()
    x = torch.zeros(3, 24, dtype=BF16, requires_grad=True)
    scale = torch.ones((), requires_grad=True)
    loss = b(x).float().sum() * scale
    loss.backward(create_graph=True, inputs=[x, scale, *b.parameters()])
    assert all(p.grad is not None and p.grad.dtype == p.dtype for p in b.parameters())
    b.zero_grad()
    b(x.detach()).float().sum().backward()
    assert all(not p.grad.requires_grad for p in b.parameters())


@pytest.mark.parametrize("after", [2, 5, 9])
def test_a_status_survives_other_batch_sizes(monkeypatch, after):
    """An error of one batch is still there when check() comes after another one."""
    fake = FakeLibrary()
    monkeypatch.setattr(block_module, "N", fake)
    b = block()
    batch = lambda n: torch.zeros(n, 24, dtype=BF16, requires_grad=True)
    b(batch(5))
    b.check()
    fake.fails = (("forward", 5),)
    b(batch(5))
    fake.fails = ()
    b(batch(after))
    with pytest.raises(N.MoEError) as e:
        b.check()
    assert e.value.status == N.MOE_ERR_NONFINITE
    b.check()                                         # read and cleared
    # an error of a backward pass that runs after another batch's forward
    fake.fails = (("backward", 5),)
    out = b(batch(5))
    b(batch(after))
    b.check()
    out.float().sum().backward()
    with pytest.raises(N.MoEError):
        b.check()
    # and the batch before is read with its own shape
    fake.fails = ()
    x = batch(7)
    out = b(x)
    b(batch(after))
    out.float().sum().backward()
    assert x.grad.shape == x.shape
    b.check()


def test_the_workspace_is_that_of_the_calls_it_makes(monkeypatch):
    """Not moe_layer's, which holds x_perm, h and y_perm a second time; and it only grows."""
    fake = FakeLibrary()
    monkeypatch.setattr(block_module, "N", fake)
    b = block()
    size = lambda n: fake.moe_workspace_stage_size(N.make_shape(n, 24, 4, 2, 8))
    for n, want in ((5, 5), (3, 5), (9, 9), (5, 9)):
        b(torch.zeros(n, 24, dtype=BF16))
        assert b._ws.nbytes == size(want)
