"""A block that was pickled whole keeps running, with and without a router (CPU)."""
import pickle

import pytest
import torch

from mixture_experts_routing_router_gb300 import block as block_module
from mixture_experts_routing_router_gb300 import native as N
from mixture_experts_routing_router_gb300.block import MoEBlock
from test_block_host import FakeLibrary


class Fake(FakeLibrary):
    moe_router = N.moe_router           # a structure, not a call


@pytest.mark.parametrize("router", [False, True], ids=["softmax", "router"])
def test_a_pickled_block_runs(monkeypatch, router):
    b = MoEBlock(24, 4, 2, 8, device="cpu", router=N.make_router(scale=2.5) if router else None)
    saved = pickle.loads(pickle.dumps(b))
    assert (saved.router is not None) == router and (not router or saved.router.scale == 2.5)
    monkeypatch.setattr(block_module, "N", Fake())
    assert saved(torch.zeros(3, 24, dtype=torch.bfloat16)).shape == (3, 24)


def test_a_block_pickled_before_there_were_routers_runs(monkeypatch):
    state = MoEBlock(24, 4, 2, 8, device="cpu").__getstate__()
    state = {name: value for name, value in state.items() if name != "router"}
    old = MoEBlock.__new__(MoEBlock)
    old.__setstate__(state)
    monkeypatch.setattr(block_module, "N", Fake())
    out = old(torch.zeros(3, 24, dtype=torch.bfloat16, requires_grad=True))
    out.float().sum().backward()
