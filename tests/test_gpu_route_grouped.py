"""Group-limited routing and its gradient against their definitions in 64 bits: ids bit
for bit, weights and gradients within the bounds of their FP32 arithmetic."""
import itertools

import pytest
import torch

import fp8_ref as ref
from mixture_experts_routing_router_gb300 import native as N

from gpu_util import dev
from test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu

F32, I32, D = torch.float32, torch.int32, torch.float64
SCORE = {True: N.MOE_SCORE_SOFTMAX, False: N.MOE_SCORE_SIGMOID}

#         T    E     k   G  topk_groups
SIZES = [(1, 256, 8, 8, 4), (70, 256, 8, 8, 4), (65, 160, 6, 8, 3), (33, 1, 1, 1, 1), (40, 7, 3, 7, 5),
         (50, 33, 5, 3, 2), (40, 48, 6, 16, 4), (30, 1024, 32, 32, 7), (37, 250, 9, 10, 10), (20, 512, 16, 4, 1),
         (45, 64, 6, 1, 1), (30, 96, 32, 32, 32), (260, 20, 4, 5, 2)]
KINDS = ["normal", "ties", "near", "wide"]


def make(T, E, kind, seed):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g)
    if kind == "ties":                                  # many equal logits, whole rows among them
        l = torch.randint(-1, 2, (T, E), generator=g).float()
        l[T // 2] = 0.5
    elif kind == "near":                                # neighbours a few units in the last place apart
        l = (torch.randint(0, 4, (T, E), generator=g) + torch.tensor(1.0).view(torch.int32)).to(I32).view(F32)
        l = l + torch.randint(0, 2, (T, E), generator=g).float()
    elif kind == "wide":                                # scores that saturate or underflow
        l = l * 60.0
    bias = 0.05 * torch.randn(E, generator=g)
    if kind == "ties":
        bias = 0.25 * torch.randint(-1, 2, (E,), generator=g).float()
    return l, bias


def gpu_route(shape, router, l, bias):
    T, k = shape.tokens, shape.top_k
    ws = N.workspace(shape, dev())
    ids, w = Guarded((T, k), I32), Guarded((T, k), F32)
    N.moe_route_grouped(shape, router, l.to(dev()), None if bias is None else bias.to(dev()), ids.t, w.t, ws)
    st = N.moe_status_read(ws)
    assert ids.intact() and w.intact()
    return ids.t.cpu(), w.t.cpu(), st


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_route(size, softmax, kind):
    T, E, k, G, tg = size
    shape = N.make_shape(T, 64, E, k, 64)
    l, bias = make(T, E, kind, seed=E + T)
    for with_bias, top, renorm in itertools.product((True, False), (1, 2), (True, False)):
        b = bias if with_bias else None
        ids, w, st = gpu_route(shape, N.make_router(SCORE[softmax], G, tg, top, renorm, 2.5), l, b)
        assert st == N.MOE_OK
        want, want_w = ref.route(l, b, k, softmax, G, tg, top, renorm, 2.5)
        assert torch.equal(ids.long(), want), (with_bias, top)
        over = (w.to(D) - want_w).abs() - (ref.W_REL * want_w.abs() + ref.W_ABS)
        assert (over <= 0).all(), (with_bias, top, renorm, float(over.max()))


def test_a_large_bias_decides():
    T, E = 40, 64
    shape = N.make_shape(T, 64, E, 4, 64)
    l, _ = make(T, E, "normal", 3)
    bias = torch.zeros(E)
    bias[::3], bias[1::3] = 1000.0, -1000.0              # a group's two largest may cancel
    for softmax, top in itertools.product((False, True), (1, 2)):
        ids, _, st = gpu_route(shape, N.make_router(SCORE[softmax], 8, 3, top), l, bias)
        assert st == N.MOE_OK
        assert torch.equal(ids.long(), ref.route(l, bias, 4, softmax, 8, 3, top, True, 1.0)[0])


def test_one_group_of_sigmoid_scores_is_the_ungrouped_route():
    T, E, k = 300, 240, 9
    shape = N.make_shape(T, 64, E, k, 64)
    l, bias = make(T, E, "normal", 5)
    ids, w, _ = gpu_route(shape, N.make_router(scale=2.5), l, bias)
    ws = N.workspace(shape, dev())
    ids2, w2 = torch.empty((T, k), dtype=I32, device=dev()), torch.empty((T, k), device=dev())
    N.moe_route_sigmoid(shape, l.to(dev()), bias.to(dev()), 2.5, ids2, w2, ws)
    assert torch.equal(ids, ids2.cpu())
    assert ((w - w2.cpu()).abs() <= 2 * ref.W_REL * w).all()


@pytest.mark.parametrize("where", ["logit", "bias"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_values_are_reported(where, bad):
    shape = N.make_shape(20, 64, 40, 3, 64)
    l, bias = make(20, 40, "normal", 7)
    (l[11] if where == "logit" else bias)[5] = bad
    for softmax in (False, True):
        assert gpu_route(shape, N.make_router(SCORE[softmax], 4, 2), l, bias)[2] == N.MOE_ERR_NONFINITE


def test_a_large_batch_on_a_stream_and_in_a_graph():
    """16384 tokens, ids against a vectorised restatement; then captured, with the logits replaced."""
    T, E, k, G, tg = 16384, 256, 8, 8, 4
    shape, router = N.make_shape(T, 64, E, k, 64), N.make_router(groups=G, topk_groups=tg, scale=2.5)
    ws = N.workspace(shape, dev())
    bias = 0.05 * torch.randn(E, generator=torch.Generator().manual_seed(1)).to(dev())
    l = torch.empty(T, E, device=dev())
    ids, w = torch.empty((T, k), dtype=I32, device=dev()), torch.empty((T, k), device=dev())

    def want():
        s = ref.scores(l, False)
        key = s.float() + bias
        two = torch.sort(key.view(T, G, -1), dim=2, descending=True).values
        gi = torch.sort(two[..., 0] + two[..., 1], dim=1, descending=True, stable=True).indices[:, :tg]
        held = torch.zeros((T, G), dtype=torch.bool, device=dev()).scatter_(1, gi, True).repeat_interleave(E // G, 1)
        return torch.sort(key.masked_fill(~held, float("-inf")), dim=1, descending=True, stable=True).indices[:, :k]

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        l.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(2)))
        N.moe_route_grouped(shape, router, l, bias, ids, w, ws)
    s.synchronize()
    assert torch.equal(ids.long(), want())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        N.moe_route_grouped(shape, router, l, bias, ids, w, ws)
    l.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(3)))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids.long(), want()) and N.moe_status_read(ws) == N.MOE_OK


# ---- gradient --------------------------------------------------------------------
def gpu_backward(shape, router, l, ids, dw):
    ws = N.workspace(shape, dev())
    d = Guarded((shape.tokens, shape.experts), F32)
    N.moe_route_grouped_backward(shape, router, l.to(dev()), ids.to(I32).to(dev()), dw.to(dev()), d.t, ws)
    st = N.moe_status_read(ws)
    assert d.intact()
    return d.t.cpu(), st


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "plain"])
@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, softmax, renorm, kind):
    T, E, k, G, tg = size
    shape, router = N.make_shape(T, 64, E, k, 64), N.make_router(SCORE[softmax], G, tg, 2, renorm, -1.5)
    l, bias = make(T, E, kind, seed=E + T)
    ids, _ = ref.route(l, bias, k, softmax, G, tg, 2, renorm, 1.0)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(9))
    d, st = gpu_backward(shape, router, l, ids, dw)
    assert st == N.MOE_OK
    want, mag = ref.route_backward(l, ids, dw, softmax, renorm, -1.5)
    # the weights' bound for each of the (up to three) scores in a term, and k terms' sum
    over = (d.to(D) - want).abs() - ((3 * ref.W_REL + 2 * k * ref.U_F32) * mag + ref.W_ABS)
    assert (over <= 0).all(), float(over.max())


@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "plain"])
@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
def test_backward_against_differences(softmax, renorm):
    """Central differences of the 64-bit weights along random directions."""
    T, E, k = 30, 24, 5
    shape, router = N.make_shape(T, 64, E, k, 64), N.make_router(SCORE[softmax], 4, 2, 2, renorm, 2.0)
    l, bias = make(T, E, "normal", 21)
    ids, _ = ref.route(l, bias, k, softmax, 4, 2, 2, renorm, 2.0)
    g = torch.Generator().manual_seed(4)
    dw, v = torch.randn(T, k, generator=g), torch.randn(T, E, generator=g, dtype=D)
    d, _ = gpu_backward(shape, router, l, ids, dw)
    f = lambda x: (ref.weights(x, ids, softmax, renorm, 2.0) * dw.to(D)).sum(1)
    h = 1e-5
    diff = (f(l.to(D) + h * v) - f(l.to(D) - h * v)) / (2 * h)
    # truncation h^2 |f'''| < 1e-8 and cancellation 1e-16 / h, beside the FP32 gradient
    assert torch.allclose((d.to(D) * v).sum(1), diff, rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("softmax", [False, True])
def test_one_dominant_expert_keeps_its_gradient(softmax, renorm):
    """A logit far above the rest: the differences that cancel are as small as the others' scores."""
    T, E, k = 8, 16, 4
    l = torch.linspace(-2, 2, E).repeat(T, 1)
    l[:, 3] = torch.linspace(8, 22, T)
    ids = torch.tensor([3, 15, 14, 13]).repeat(T, 1)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(2))
    d, st = gpu_backward(N.make_shape(T, 64, E, k, 64), N.make_router(SCORE[softmax], renorm=renorm), l, ids, dw)
    want, _ = ref.route_backward(l, ids, dw, softmax, renorm, 1.0)
    assert st == N.MOE_OK
    assert torch.allclose(d[:, 3].to(D), want[:, 3], rtol=1e-4, atol=0)


def test_backward_leaves_out_invalid_pairs():
    """An id out of range or repeated takes no part and is reported, as in the dispatch."""
    T, E, k = 12, 10, 3
    l, _ = make(T, E, "normal", 2)
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(T)])
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(3))
    ids[2, 1], ids[5, 0], ids[7, 2] = -1, E, ids[7, 0]
    shape = N.make_shape(T, 64, E, k, 64)
    for softmax, renorm in itertools.product((False, True), repeat=2):
        d, st = gpu_backward(shape, N.make_router(SCORE[softmax], renorm=renorm), l, ids, dw)
        assert st == N.MOE_ERR_INVALID_ROUTE
        for t, keep in ((2, [0, 2]), (5, [1, 2]), (7, [0, 1]), (0, [0, 1, 2])):
            want, mag = ref.route_backward(l[t:t + 1], ids[t:t + 1, keep], dw[t:t + 1, keep], softmax, renorm, 1.0)
            assert ((d[t:t + 1].to(D) - want).abs() <= 4 * ref.W_REL * mag + ref.W_ABS).all(), (t, softmax, renorm)
