"""The workspace's share of the split gradient reductions (CPU)."""
import random

import pytest

from mixture_experts_routing_router_gb300 import build as B
from mixture_experts_routing_router_gb300 import native as N

LIMIT = 70_000_000        # as the header says


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def up(v, a=1024):
    return (v + a - 1) // a * a


def partial_bytes(T, H, E, k, I, act):
    """What is left of moe_workspace_size without the regions of the forward calls."""
    R = T * k
    rest = 4096
    rest += up(-(-R // 1024) * E * 8) + up(R * 4) + up(0)                       # flags, ranks, no shared expert
    rest += up(E * 4) + up((E + 1) * 4) + 4 * up(R * 4)                         # counts, offsets, ids, w, dest, pairs
    rest += 2 * up(R * H * 2) + up(R * I * 2) + up((E + 4 * -(-H // 128) + 1) * 4)
    return N.moe_workspace_size(N.make_shape(T, H, E, k, I, act=act)) - rest


KNOWN = [(3292, 3304, 1, 1, 384, N.MOE_ACT_SWIGLU), (9944, 256, 1, 1, 3288, N.MOE_ACT_RELU2),
         (4288, 256, 1, 1, 3840, N.MOE_ACT_SWIGLU)]


@pytest.mark.parametrize("shape", KNOWN, ids=str)
def test_shapes_with_the_largest_partial_sums(shape):
    assert LIMIT // 2 < partial_bytes(*shape) <= LIMIT


def test_partial_sums_stay_within_the_stated_size():
    rng = random.Random(7)
    most = 0
    for _ in range(6000):
        draw = lambda lo, hi: int(lo * (hi / lo) ** rng.random())
        E = rng.choice((1, 1, 2, 3, draw(1, 64)))
        k = rng.randint(1, min(E, 4))
        T, H, I = draw(1, 30000), 8 * draw(1, 1000), 8 * draw(1, 1000)
        b = partial_bytes(T, H, E, k, I, rng.choice((N.MOE_ACT_SWIGLU, N.MOE_ACT_RELU2)))
        assert 0 <= b <= LIMIT, (T, H, E, k, I)
        most = max(most, b)
    assert most > LIMIT // 2            # the draws reach the shapes that matter


def test_stage_size():
    """What the calls on their own need: none of moe_layer's x_perm, h and y_perm, 4.3 GB at
    16384 tokens, k = 8, 7168 hidden."""
    for act in (N.MOE_ACT_SWIGLU, N.MOE_ACT_RELU2):
        s = N.make_shape(16384, 7168, 256, 8, 2048, act=act)
        whole, stage = N.moe_workspace_size(s), N.moe_workspace_stage_size(s)
        assert whole - stage > 2 * 16384 * 8 * 2 * 7168 and 4096 < stage < 100_000_000
    with pytest.raises(N.MoEError):
        N.moe_workspace_stage_size(N.make_shape(0, 64, 4, 2, 64))


def test_stage_size_is_what_the_stage_calls_ask_for():
    """One byte less is refused on the host, before anything is launched (the pointers are
    never followed: the second refusal is that of a null output)."""
    import ctypes
    L, P = N.lib(), ctypes.c_void_p
    s = N.make_shape(300, 136, 5, 2, 72)
    n = N.moe_workspace_stage_size(s)
    for bytes_, out in ((n - 1, P(4096)), (n, None)):
        assert L.moe_expert_down_backward(ctypes.byref(s), P(4096), P(4096), P(4096), P(4096), P(4096), out, None, 0,
                                          P(1 << 20), bytes_, None) == N.MOE_ERR_INVALID_ARG
