"""Gradients of the combine, the dispatch and the routing against their formulas
in 64 bits, each element within the bound of its own arithmetic."""
import pytest
import torch

from mixture_experts_routing_router_gb300 import native as N

import train_ref as ref
from gpu_util import dev
from test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu

BF16, F32, D = torch.bfloat16, torch.float32, torch.float64


def check(got, want, bound, what):
    got = got.to(D)
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()} outside, worst by {over.max():.3e}"


def routes(T, E, k, seed, bad=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    if bad:                                   # negative, wide, repeated, a token with none left
        ids[0, 0], ids[T // 2, k - 1], ids[T - 1] = -3, E + 5, -1
        if k > 1:
            ids[T // 3, 1] = ids[T // 3, 0]
    dest, offsets = ref.dispatch(ids, E)
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    return ids.to(dev()), dest.to(dev()), offsets, w.to(dev())


#        T     H     E   k
SIZES = [(1, 8, 1, 1), (1, 7168, 16, 8), (3, 64, 4, 2), (64, 256, 16, 2), (37, 136, 33, 5), (50, 72, 40, 9),
         (40, 128, 8, 8), (300, 64, 1024, 32), (20, 2056, 17, 17), (700, 2048, 64, 6), (4, 20000, 6, 3)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("bad", [False, True], ids=["valid", "invalid"])
def test_combine_and_dispatch_backward(size, bad):
    T, H, E, k = size
    if bad and T < 4:
        pytest.skip("too few tokens for the invalid kinds")
    ids, dest, offsets, w = routes(T, E, k, seed=T + k, bad=bad)
    shape = N.make_shape(T, H, E, k, 8)
    ws = N.workspace(shape, dev())
    g = torch.Generator(device=dev()).manual_seed(1)
    dout = torch.randn(T, H, generator=g, device=dev()).to(BF16)
    y = torch.randn(T * k, H, generator=g, device=dev()).to(BF16)
    y[int(offsets[-1]):] = float("nan")                 # rows no pair points at
    dy, dw = Guarded((T * k, H), BF16), Guarded((T, k), F32)
    N.moe_combine_backward(shape, dout, y, dest, w, dy.t, dw.t, ws)
    assert N.moe_status_read(ws) == N.MOE_OK and dy.intact() and dw.intact()
    slot, want, want_w, mag = ref.combine_backward(dout, y, dest, w)
    check(dy.t[slot], want, ref.U_BF16 * want.abs() + ref.U_F32 * want.abs(), "dy_perm")
    check(dw.t, want_w, ref.sum_bound(H, mag), "dtopk_w")
    assert torch.all(dw.t[dest < 0] == 0)
    spare = dy.t[int(offsets[-1]):].contiguous().view(torch.uint8)
    assert torch.all(spare == 0xA5)
    # fixed weights; in place
    only = torch.empty(T * k, H, dtype=BF16, device=dev())
    N.moe_combine_backward(shape, dout, None, dest, w, only, None, ws)
    assert torch.equal(only[slot], dy.t[slot])
    over, dw2 = y.clone(), torch.empty_like(dw.t)
    N.moe_combine_backward(shape, dout, over, dest, w, over, dw2, ws)
    assert torch.equal(over[slot], dy.t[slot]) and torch.equal(dw2, dw.t)

    add = torch.randn(T, H, generator=g, device=dev()).to(BF16)
    for a in (None, add):
        dx = Guarded((T, H), BF16)
        N.moe_dispatch_backward(shape, y, dest, dx.t, ws, add=a)
        assert dx.intact()
        want, mag = ref.dispatch_backward(y, dest, a)
        check(dx.t, want, k * ref.U_F32 * mag + ref.U_BF16 * want.abs(), "dx")
    over = add.clone()
    N.moe_dispatch_backward(shape, y, dest, over, ws, add=over)
    assert torch.equal(over, dx.t)


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_route_backward(size):
    T, H, E, k = size
    shape = N.make_shape(T, H, E, k, 8)
    ws = N.workspace(shape, dev())
    logits = 3 * torch.randn(T, E, generator=torch.Generator().manual_seed(k)).to(dev())
    ids, w = torch.empty(T, k, dtype=torch.int32, device=dev()), torch.empty(T, k, device=dev())
    N.moe_route(shape, logits, ids, w, ws)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(T)).to(dev())
    dl = Guarded((T, E), F32)
    N.moe_route_backward(shape, ids, w, dw, dl.t, ws)
    assert N.moe_status_read(ws) == N.MOE_OK and dl.intact()
    want = ref.route_backward(ids, w, dw, E)
    check(dl.t, want, ref.U_F32 * want.abs(), "dlogits")          # terms in double, one rounding
    # sigmoid routing, a bias that selects, scores down to where they underflow
    bias = torch.randn(E, generator=torch.Generator().manual_seed(5)).to(dev())
    for lg in (logits, logits - 60.0, logits + 60.0):
        N.moe_route_sigmoid(shape, lg, bias, 2.5, ids, w, ws)
        N.moe_route_sigmoid_backward(shape, lg, ids, 2.5, dw, dl.t, ws)
        assert N.moe_status_read(ws) == N.MOE_OK and dl.intact()
        want = ref.route_sigmoid_backward(lg, ids, 2.5, dw)
        # terms in double: 1e-13 of the largest product covers 64-bit cancellation on both sides
        check(dl.t, want, ref.U_F32 * want.abs() + 1e-12 * dw.abs().max(), "sigmoid dlogits")


def test_route_backward_of_scores_that_underflow_keeps_their_ratios():
    shape = N.make_shape(2, 8, 8, 3, 8)
    ws = N.workspace(shape, dev())
    logits = torch.full((2, 8), -800.0, device=dev())
    logits[:, 2] = -799.0
    ids = torch.tensor([[2, 0, 5], [0, 2, 7]], dtype=torch.int32, device=dev())
    dw = torch.tensor([[1.0, -2.0, 0.5], [3.0, 1.0, -1.0]], device=dev())
    dl = torch.empty(2, 8, device=dev())
    N.moe_route_sigmoid_backward(shape, logits, ids, 1.0, dw, dl, ws)
    p = torch.softmax(torch.gather(logits.to(D), 1, ids.long()), 1)      # s_j / sum s in the limit
    want = torch.zeros(2, 8, dtype=D, device=dev()).scatter_(1, ids.long(),
                                                              p * (dw.to(D) - (p * dw.to(D)).sum(1, keepdim=True)))
    check(dl, want, ref.U_F32 * want.abs(), "dlogits")


def test_route_backward_reports_bad_ids_and_leaves_them_out():
    T, E, k = 40, 12, 4
    ids, _, _, w = routes(T, E, k, seed=3, bad=True)
    shape = N.make_shape(T, 8, E, k, 8)
    ws = N.workspace(shape, dev())
    dw = torch.randn(T, k, device=dev())
    dl = Guarded((T, E), F32)
    N.moe_route_backward(shape, ids, w, dw, dl.t, ws)
    assert N.moe_status_read(ws) == N.MOE_ERR_INVALID_ROUTE and dl.intact()
    dest, _ = ref.dispatch(ids.cpu(), E)
    ok = (dest >= 0).to(dev())
    safe = torch.where(ok, ids, torch.zeros_like(ids))
    want = torch.zeros(T, E, dtype=D, device=dev())
    wd, dd = torch.where(ok, w, 0.0).to(D), torch.where(ok, dw, 0.0).to(D)
    want.scatter_add_(1, safe.long(), wd * (dd - (wd * dd).sum(1, keepdim=True)))
    check(dl.t, want, ref.U_F32 * want.abs(), "dlogits")
    assert torch.all(dl.t[T - 1] == 0)


def test_combine_backward_of_a_nan_token_stays_in_it():
    T, H, E, k = 20, 264, 8, 3
    ids, dest, _, w = routes(T, E, k, seed=4)
    shape = N.make_shape(T, H, E, k, 8)
    ws = N.workspace(shape, dev())
    dout, y = torch.randn(T, H, device=dev()).to(BF16), torch.randn(T * k, H, device=dev()).to(BF16)
    dout[7] = float("nan")
    y[dest[3, 1]] = float("inf")
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    N.moe_combine_backward(shape, dout, y, dest, w, dy, dw, ws)
    bad = torch.zeros(T * k, dtype=torch.bool, device=dev())
    bad[dest[7].long()] = True
    assert torch.isnan(dy[bad]).all() and torch.isfinite(dy[~bad]).all()
    fin = torch.isfinite(dw)
    fin[7], fin[3, 1] = ~fin[7], ~fin[3, 1]
    assert fin.all()


def test_streams_and_graphs_agree():
    T, H, E, k = 200, 264, 16, 4
    ids, dest, _, w = routes(T, E, k, seed=5)
    shape = N.make_shape(T, H, E, k, 8)
    ws = N.workspace(shape, dev())
    dout, y = torch.randn(T, H, device=dev()).to(BF16), torch.randn(T * k, H, device=dev()).to(BF16)

    def outs():
        return (torch.zeros_like(y), torch.zeros_like(w), torch.zeros(T, E, device=dev()), torch.zeros_like(dout))

    def call(o, stream=None):
        N.moe_combine_backward(shape, dout, y, dest, w, o[0], o[1], ws, stream=stream)
        N.moe_route_backward(shape, ids, w, o[1], o[2], ws, stream=stream)
        N.moe_dispatch_backward(shape, o[0], dest, o[3], ws, stream=stream)

    a, b, c = outs(), outs(), outs()
    call(a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(b, s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c)
    g.replay()
    assert N.moe_status_read(ws) == N.MOE_OK
    for u, v, x in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, x)


def test_gradients_against_differences():
    """Central differences in 64 bits of combine(route(logits)) along random directions."""
    T, H, E, k = 13, 72, 9, 4
    gen = torch.Generator(device=dev()).manual_seed(6)
    logits = torch.randn(T, E, generator=gen, device=dev())
    shape = N.make_shape(T, H, E, k, 8)
    ws = N.workspace(shape, dev())
    ids, w = torch.empty(T, k, dtype=torch.int32, device=dev()), torch.empty(T, k, device=dev())
    N.moe_route(shape, logits, ids, w, ws)
    dest, _ = ref.dispatch(ids.cpu(), E)
    dest = dest.to(dev())
    dout, y = (torch.randn(n, H, generator=gen, device=dev()).to(BF16) for n in (T, T * k))

    def loss(lg, yp):
        wt = torch.softmax(torch.gather(lg, 1, ids.long()), 1)
        return ((wt.unsqueeze(2) * yp[dest.long().view(-1)].view(T, k, H)).sum(1) * dout.to(D)).sum()

    dy, dw, dl = torch.empty_like(y), torch.empty_like(w), torch.empty(T, E, device=dev())
    N.moe_combine_backward(shape, dout, y, dest, w, dy, dw, ws)
    N.moe_route_backward(shape, ids, w, dw, dl, ws)
    at = [logits.to(D), y.to(D)]
    for i, (grad, rel) in enumerate(((dl, 1e-5), (dy, 5 * 0.5 * ref.U_BF16))):
        v = torch.randn(at[i].shape, generator=gen, device=dev(), dtype=D)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 1e-4 * v, at[i] - 1e-4 * v
        diff = (loss(*up) - loss(*down)) / 2e-4
        # dl: FP32 sums, 1e-5 of |grad| |v|; dy: independent bf16 roundings, five sigma
        tol = rel * grad.to(D).norm() * (v.norm() if i == 0 else 1.0)
        assert abs((grad.to(D) * v).sum() - diff) <= tol
