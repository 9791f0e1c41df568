"""The binding's checks of the training calls' tensors: a kernel reads and writes as
many elements as the shape says, so a tensor of fewer, or of another type, is refused
before the call.  The other arguments are plain addresses (never used: nothing is
launched), so no GPU is needed."""
import pytest
import torch

from mixture_experts_routing_router_gb300 import build as B
from mixture_experts_routing_router_gb300 import native as N

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
T, H, E, K, I = 5, 16, 13, 3, 8
R, E8 = T * K, 16


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


class Ws:
    """Stands for a workspace: an address and its size (none: the C call refuses it)."""
    is_cuda, nbytes = True, 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0


def calls(act):
    up = 2 * I if act == N.MOE_ACT_SWIGLU else I
    return {
        "moe_combine_backward": dict(dout=(BF16, T * H), y_perm=(BF16, R * H), dest=(I32, R), topk_w=(F32, R),
                                     dy_perm=(BF16, R * H), dtopk_w=(F32, R)),
        "moe_dispatch_backward": dict(dx_perm=(BF16, R * H), dest=(I32, R), dx=(BF16, T * H), add=(BF16, T * H)),
        "moe_route_backward": dict(topk_ids=(I32, R), topk_w=(F32, R), dtopk_w=(F32, R), dlogits=(F32, T * E)),
        "moe_route_sigmoid_backward": dict(logits=(F32, T * E), topk_ids=(I32, R), route_scale=2.5, dtopk_w=(F32, R),
                                           dlogits=(F32, T * E)),
        "moe_gate_backward": dict(dlogits=(F32, T * E), x=(BF16, T * H), w_gate=(BF16, E * H),
                                  dlogits_bf16=(BF16, T * E8), dx=(BF16, T * H), dw_gate=(None, E * H)),
        "moe_expert_up_train": dict(x_perm=(BF16, R * H), offsets=(I32, E + 1), w13=(BF16, E * up * H),
                                    pre=(BF16, R * up), h=(BF16, R * I)),
        "moe_expert_down_backward": dict(dy_perm=(BF16, R * H), offsets=(I32, E + 1), w2=(BF16, E * H * I),
                                         pre=(BF16, R * up), h=(BF16, R * I), dpre=(BF16, R * up),
                                         dw2=(None, E * H * I)),
        "moe_expert_up_backward": dict(dpre=(BF16, R * up), offsets=(I32, E + 1), x_perm=(BF16, R * H),
                                       w13=(BF16, E * up * H), dx_perm=(BF16, R * H), dw13=(None, E * up * H)),
    }


CASES = [(act, call, arg) for act in (N.MOE_ACT_SWIGLU, N.MOE_ACT_RELU2) for call, args in calls(act).items()
         for arg, want in args.items() if isinstance(want, tuple)]


@pytest.mark.parametrize("act,call,arg", CASES)
def test_a_tensor_that_does_not_fit_is_refused(act, call, arg):
    shape = N.make_shape(T, H, E, K, I, act=act)
    args = calls(act)[call]
    dtype, n = args[arg]

    def go(tensor):
        given = {a: v if not isinstance(v, tuple) else None if v[0] is None else 4096 for a, v in args.items()}
        given[arg] = tensor
        getattr(N, call)(shape, **given, ws=Ws(), stream=0)

    either = dtype is None                            # a weight gradient: bfloat16 or float32
    for good in (BF16, F32) if either else (dtype,):
        with pytest.raises(ValueError, match=rf"^{arg}\b.*{n} elements"):
            go(torch.zeros(n - 1, dtype=good))
        with pytest.raises(ValueError, match="device tensor expected"):       # fits, but not on the device
            go(torch.zeros(n, dtype=good))
    for other in (torch.float16, torch.float64) if either else (torch.float16, F32 if dtype is not F32 else BF16):
        with pytest.raises(ValueError, match="expected, got"):
            go(torch.zeros(2 * n, dtype=other))


def test_rounded_gate_gradients_of_the_unpadded_width_are_refused():
    """[T, E] with E no multiple of eight: the kernel writes whole 16-byte rows."""
    shape = N.make_shape(T, H, E, K, I)
    with pytest.raises(ValueError, match="dlogits_bf16"):
        N.moe_gate_backward(shape, 4096, 4096, 4096, torch.empty(T, E, dtype=BF16), 4096, None, Ws(), stream=0)
