"""What the trainable block refuses before it calls the library (CPU)."""
import pytest
import torch

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
