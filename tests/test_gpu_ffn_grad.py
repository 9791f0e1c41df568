"""The expert FFN's training calls against their formulas in 64 bits.

Each output is held to the bound of its own arithmetic: one rounding to the
output type plus the FP32 sum over its products (tests/train_ref.py).  Buffers
are padded with NaN where no valid row may be read: rows past the last bucket.
"""
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


class Case:
    """Buckets of the given sizes (and `spare` pairs that went nowhere)."""

    def __init__(self, counts, H, I, glu, seed=0, spare=0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        E, R = len(counts), sum(counts) + spare
        self.E, self.R, self.H, self.I, self.glu, self.valid = E, R, H, I, glu, sum(counts)
        self.up = 2 * I if glu else I
        # the largest bucket is the number of tokens' lower bound; k pads to R pairs
        k = next(k for k in range(1, 33) if R % k == 0 and k <= E and R // k >= max(counts)) if R else 1
        self.shape = N.make_shape(R // k, H, E, k, I, act=N.MOE_ACT_SWIGLU if glu else N.MOE_ACT_RELU2)
        self.ws = N.workspace(self.shape, dev())
        self.offsets = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device=dev())

        def rows(n, std=1.0):
            t = (torch.randn(R, n, generator=g) * std).to(BF16)
            t[self.valid:] = float("nan")
            return t.to(dev())

        self.x, self.dy, self.pre, self.dpre_in = rows(H), rows(H), rows(self.up), rows(self.up)
        self.h = rows(I)
        self.w13 = (torch.randn(E, self.up, H, generator=g) / H ** 0.5).to(BF16).to(dev())
        self.w2 = (torch.randn(E, H, I, generator=g) / I ** 0.5).to(BF16).to(dev())

    def status(self):
        assert N.moe_status_read(self.ws) == N.MOE_OK

    def dpre_ref(self):
        dh, mag = ref.rows_times(self.dy, self.offsets, self.w2, False)
        pre = self.pre.to(D)
        want = ref.act_backward(pre, dh, self.glu)
        # the sum's error through |d act / d pre|, the sigmoid's few units, the rounding
        fac = ref.act_backward(pre, torch.ones_like(dh), self.glu).abs()
        e_dh = ref.sum_bound(self.H, mag)
        if self.glu:
            g, u = pre.chunk(2, 1)
            s = torch.sigmoid(g)
            # g in the exponent: an error of 2 units of |g| + 1; the terms' magnitudes, not their sum
            e_s = ref.U_F32 * (4 * g.abs() + 8)
            e_fac = torch.cat([u.abs() * s * (1 + g.abs()), g.abs() * s], 1) * torch.cat([e_s, e_s], 1)
            both = lambda t: torch.cat([t, t], 1)
        else:
            e_fac, both = 2 * ref.U_F32 * fac, (lambda t: t)
        bound = fac * both(e_dh) + e_fac * both(dh.abs()) + ref.U_BF16 * want.abs()
        v = self.valid
        return want[:v], bound[:v]


# every residue class of a 64-row step and its 16-row slices, several steps, empty buckets
COUNTS = {
    "ones": [1, 0, 1, 1, 0],
    "slices": [15, 16, 17, 31, 32, 33, 47, 48, 49],
    "steps": [63, 0, 64, 65, 127, 128, 129],
    "tiles": [255, 256, 257, 0, 300],
    "ring": [5 * 64 + 3, 6 * 64 + 60, 7 * 64, 13 * 64 + 1],   # around the six-stage ring
    "one_expert": [200],
}
SHAPES = [(8, 8), (64, 64), (136, 72), (256, 512), (320, 264), (1024, 264)]


@pytest.mark.parametrize("hi", SHAPES, ids=str)
@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("glu", [True, False], ids=["swiglu", "relu2"])
def test_backward_matches_the_formulas(counts, hi, glu):
    c = Case(COUNTS[counts], *hi, glu, seed=len(counts) + hi[0], spare=3 if counts == "steps" else 0)
    run_and_check(c, COUNTS[counts])


def run_and_check(c, counts):
    dpre = Guarded((c.R, c.up), BF16)
    dw2, dw13 = Guarded((c.E, c.H, c.I), BF16), Guarded((c.E, c.up, c.H), BF16)
    dx = Guarded((c.R, c.H), BF16)
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, c.pre, c.h, dpre.t, dw2.t, c.ws)
    N.moe_expert_up_backward(c.shape, c.dpre_in, c.offsets, c.x, c.w13, dx.t, dw13.t, c.ws)
    c.status()
    assert all(b.intact() for b in (dpre, dw2, dw13, dx))
    v, n = c.valid, max(counts)
    check(dpre.t[:v], *c.dpre_ref(), "dpre")
    want, mag = ref.weights_grad(c.dy, c.h, c.offsets)
    check(dw2.t, want, ref.sum_bound(n, mag) + ref.U_BF16 * want.abs(), "dw2")
    want, mag = ref.rows_times(c.dpre_in, c.offsets, c.w13, False)
    check(dx.t[:v], want[:v], (ref.sum_bound(c.up, mag) + ref.U_BF16 * want.abs())[:v], "dx_perm")
    want, mag = ref.weights_grad(c.dpre_in, c.x, c.offsets)
    check(dw13.t, want, ref.sum_bound(n, mag) + ref.U_BF16 * want.abs(), "dw13")
    # rows past the last bucket are not written
    canary = torch.full((2,), 0xA5, dtype=torch.uint8, device=dev()).view(BF16)
    if c.R > v:
        assert torch.equal(dx.t[v:].contiguous().view(torch.int16), canary.view(torch.int16).expand(c.R - v, c.H))


# few output tiles and long reductions: split over the CTA pairs, in every residue of the
# last 64-row step and with parts of no step at all
SPLIT = [([300], 4096, 64), ([2000], 64, 40), ([5], 6432, 416), ([1031, 1], 72, 1480), ([1400, 0, 2600], 136, 200),
         ([0, 1600], 8, 8), ([64 * 20], 256, 256), ([3, 2500], 520, 24)]


@pytest.mark.parametrize("case", SPLIT, ids=str)
@pytest.mark.parametrize("glu", [True, False], ids=["swiglu", "relu2"])
def test_split_reductions_match_the_formulas(case, glu):
    counts, H, I = case
    c = Case(counts, H, I, glu, seed=H + I, spare=0 if len(counts) == 1 else 2 * len(counts) - sum(counts) % len(counts))
    run_and_check(c, counts)
    # float32, stored and added, without the rows form
    want, mag = ref.weights_grad(c.dy, c.h, c.offsets)
    bound = ref.sum_bound(max(counts), mag) + 2 * ref.U_F32 * want.abs()
    dw = Guarded(tuple(want.shape), F32)
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, None, None, c.h, None, dw.t, c.ws)
    c.status()
    check(dw.t, want, bound, "dw2")
    old = torch.randn(want.shape, device=dev())
    dw.t.copy_(old)
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, None, None, c.h, None, dw.t, c.ws, add=True)
    c.status()
    check(dw.t, want + old.to(D), bound + 2 * ref.U_F32 * old.to(D).abs(), "dw2 +=")
    empty = [e for e, m in enumerate(counts) if m == 0]
    assert torch.equal(dw.t[empty], old[empty]) and dw.intact()
    # the rows form alone, and again: the same bits
    a, b = torch.zeros_like(c.pre), torch.zeros_like(c.pre)
    for t in (a, b):
        N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, c.pre, None, t, None, c.ws)
    c.status()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    check(a[:c.valid], *c.dpre_ref(), "dpre alone")


def test_calls_back_to_back_keep_their_bits():
    """The pair's last arrivals are in before a kernel ends: the next one, of another
    layout on the same SMs, gets the results it gets alone."""
    c = Case([77, 0, 300, 64, 9], 264, 136, True, seed=3)
    pre, h = torch.empty_like(c.pre), torch.empty_like(c.h)
    runs = []
    for _ in range(100):
        dpre, dx = torch.zeros_like(c.pre), torch.zeros_like(c.x)
        dw2, dw13 = torch.zeros_like(c.w2), torch.zeros_like(c.w13)
        N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, c.pre, c.h, dpre, dw2, c.ws)
        N.moe_expert_up_train(c.shape, c.x, c.offsets, c.w13, pre, h, c.ws)
        N.moe_expert_up_backward(c.shape, dpre, c.offsets, c.x, c.w13, dx, dw13, c.ws)
        runs.append((dpre, dx, dw2, dw13, pre.clone(), h.clone()))
    for got in runs[1:]:
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(runs[0], got))
    c.status()


@pytest.mark.parametrize("counts", ["ones", "steps", "ring"])
def test_float32_weight_gradients_and_accumulation(counts):
    c = Case(COUNTS[counts], 136, 72, True, seed=5)
    n = max(COUNTS[counts])
    for call, a, b in ((lambda dw, add: N.moe_expert_down_backward(c.shape, c.dy, c.offsets, None, None, c.h, None, dw,
                                                                   c.ws, add=add), c.dy, c.h),
                       (lambda dw, add: N.moe_expert_up_backward(c.shape, c.dpre_in, c.offsets, c.x, None, None, dw,
                                                                 c.ws, add=add), c.dpre_in, c.x)):
        want, mag = ref.weights_grad(a, b, c.offsets)
        bound = ref.sum_bound(n, mag) + ref.U_F32 * want.abs()
        dw = Guarded(tuple(want.shape), F32)
        call(dw.t, False)
        c.status()
        check(dw.t, want, bound, "dw")
        old = torch.randn(want.shape, device=dev())
        dw.t.copy_(old)
        call(dw.t, True)
        c.status()
        check(dw.t, want + old.to(D), bound + ref.U_F32 * (want + old.to(D)).abs(), "dw +=")
        assert dw.intact()
        empty = [e for e, m in enumerate(COUNTS[counts]) if m == 0]
        assert torch.equal(dw.t[empty], old[empty])


@pytest.mark.parametrize("glu", [True, False], ids=["swiglu", "relu2"])
@pytest.mark.parametrize("rows", [40, 300])          # a swapped tile; a full one and a swapped one
def test_saturated_pre_activations(rows, glu):
    c = Case([rows], 72, 64, glu, seed=12)
    pick = torch.tensor([-3e38, -1e4, -100.0, -88.0, -20.0, -0.0, 0.0, 20.0, 88.0, 100.0, 1e4])
    at = torch.randint(0, len(pick), c.pre.shape, generator=torch.Generator().manual_seed(1))
    c.pre.copy_(pick[at].to(BF16))
    if glu:                                          # up half and dy of ordinary size: the products stay finite
        c.pre[:, c.I:] = torch.randn(rows, c.I, device=dev()).to(BF16)
    else:
        c.pre.clamp_(max=1e4)
    dpre = torch.empty_like(c.pre)
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, c.pre, None, dpre, None, c.ws)
    c.status()
    want, bound = c.dpre_ref()
    # below 2^-126 a sigmoid may flush to zero: its value times |g| + 1, the largest factor here
    check(dpre, want, bound + 2.0 ** -126 * 4e2 * (want.abs() + 1), "dpre")


@pytest.mark.parametrize("bad", [[0, 60, 50, 100], [-1, 30, 60, 100], [0, 30, 60, 101], [0, 1 << 30, 60, 100],
                                 [0, 30, -(1 << 31), 100]], ids=str)
def test_bad_bucket_bounds_are_reported_and_move_nothing(bad):
    c = Case([30, 30, 40], 72, 40, True, seed=11)
    offsets = torch.tensor(bad, dtype=torch.int32, device=dev())
    dpre, dx = Guarded((c.R, c.up), BF16), Guarded((c.R, c.H), BF16)
    dw2, dw13 = Guarded((c.E, c.H, c.I), BF16), Guarded((c.E, c.up, c.H), BF16)
    N.moe_expert_down_backward(c.shape, c.dy, offsets, c.w2, c.pre, c.h, dpre.t, dw2.t, c.ws)
    assert N.moe_status_read(c.ws) == N.MOE_ERR_INVALID_ROUTE
    N.moe_expert_up_backward(c.shape, c.dpre_in, offsets, c.x, c.w13, dx.t, dw13.t, c.ws)
    assert N.moe_status_read(c.ws) == N.MOE_ERR_INVALID_ROUTE
    for b in (dpre, dx, dw2, dw13):
        assert b.intact()
    for b in (dpre, dx):
        assert torch.all(b.t.view(torch.uint8) == 0xA5)


def test_a_bucket_of_nan_rows_stays_in_its_expert():
    counts = [40, 70, 1, 130, 17]
    c = Case(counts, 200, 136, True, seed=6)
    lo, hi = int(c.offsets[1]), int(c.offsets[2])
    for t in (c.x, c.dy, c.pre, c.dpre_in, c.h):
        t[lo:hi] = float("nan")
    dpre, dx = torch.zeros(c.R, c.up, dtype=BF16, device=dev()), torch.zeros(c.R, c.H, dtype=BF16, device=dev())
    dw2, dw13 = torch.zeros_like(c.w2), torch.zeros_like(c.w13)
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, c.pre, c.h, dpre, dw2, c.ws)
    N.moe_expert_up_backward(c.shape, c.dpre_in, c.offsets, c.x, c.w13, dx, dw13, c.ws)
    c.status()
    others = [0, 2, 3, 4]
    rows = torch.cat([torch.arange(0, lo), torch.arange(hi, c.R)]).to(dev())
    for t in (dpre[rows], dx[rows], dw2[others], dw13[others]):
        assert torch.isfinite(t).all()
    for t in (dpre[lo:hi], dx[lo:hi], dw2[1], dw13[1]):
        assert torch.isnan(t).all()


def test_weights_of_nan_stay_in_their_expert():
    c = Case([33, 20, 50], 72, 40, True, seed=7)         # K tails: the next expert's rows follow in memory
    c.w13[1], c.w2[1] = float("nan"), float("nan")
    dpre, dx = torch.zeros(c.R, c.up, dtype=BF16, device=dev()), torch.zeros(c.R, c.H, dtype=BF16, device=dev())
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, c.pre, None, dpre, None, c.ws)
    N.moe_expert_up_backward(c.shape, c.dpre_in, c.offsets, None, c.w13, dx, None, c.ws)
    c.status()
    for t in (dpre, dx):
        assert torch.isfinite(t[:33]).all() and torch.isfinite(t[53:]).all() and torch.isnan(t[33:53]).all()


@pytest.mark.parametrize("glu", [True, False], ids=["swiglu", "relu2"])
@pytest.mark.parametrize("counts", ["ones", "steps", "tiles"])
def test_up_train_keeps_its_pre_activations(counts, glu):
    c = Case(COUNTS[counts], 136, 72, glu, seed=8, spare=3 if counts == "steps" else 0)
    pre, h = Guarded((c.R, c.up), BF16), Guarded((c.R, c.I), BF16)
    N.moe_expert_up_train(c.shape, c.x, c.offsets, c.w13, pre.t, h.t, c.ws)
    c.status()
    assert pre.intact() and h.intact()
    v = c.valid
    want, mag = ref.rows_times(c.x, c.offsets, c.w13, True)
    check(pre.t[:v], want[:v], (ref.sum_bound(c.H, mag) + ref.U_BF16 * want.abs())[:v], "pre")
    p = pre.t[:v].to(D)
    want = ref.act(p, glu)
    # the sigmoid's error is some units of (1 + |g|)
    e = 8 * ref.U_F32 * (1 + (p.chunk(2, 1)[0] if glu else p).abs())
    check(h.t[:v], want, (ref.U_BF16 + e) * want.abs(), "h")


@pytest.mark.parametrize("size", [(1, 8, 1), (5, 72, 3), (64, 256, 16), (300, 136, 33), (257, 1000, 240),
                                  (130, 64, 1024), (2000, 520, 100), (6000, 264, 40),
                                  (5000, 1032, 8)], ids=str)
def test_gate_backward(size):
    T, H, E = size
    g = torch.Generator().manual_seed(T)
    shape = N.make_shape(T, H, E, 1, 8)
    ws = N.workspace(shape, dev())
    dl = torch.randn(T, E, generator=g).to(dev())
    x, w = (torch.randn(n, H, generator=g).to(BF16).to(dev()) for n in (T, E))
    gb = Guarded((T, (E + 7) // 8 * 8), BF16)
    dx, dw, dw32 = Guarded((T, H), BF16), Guarded((E, H), BF16), Guarded((E, H), F32)
    N.moe_gate_backward(shape, dl, x, w, gb.t, dx.t, dw.t, ws)
    assert N.moe_status_read(ws) == N.MOE_OK and all(b.intact() for b in (gb, dx, dw))
    assert torch.equal(gb.t[:, :E], dl.to(BF16)) and torch.all(gb.t[:, E:] == 0)
    gd, xd, wd = gb.t[:, :E].to(D), x.to(D), w.to(D)
    want = gd @ wd
    check(dx.t, want, ref.sum_bound(E, gd.abs() @ wd.abs()) + ref.U_BF16 * want.abs(), "dx")
    want, mag = gd.t() @ xd, gd.abs().t() @ xd.abs()
    check(dw.t, want, ref.sum_bound(T, mag) + ref.U_BF16 * want.abs(), "dw_gate")
    old = torch.randn(E, H, device=dev())
    dw32.t.copy_(old)
    N.moe_gate_backward(shape, dl, x, None, gb.t, None, dw32.t, ws, add=True)
    assert N.moe_status_read(ws) == N.MOE_OK and dw32.intact()
    check(dw32.t, want + old.to(D), ref.sum_bound(T, mag) + 2 * ref.U_F32 * (want.abs() + old.to(D).abs()), "dw_gate +=")


def test_runs_on_the_given_stream_in_a_graph_and_repeats_bitwise():
    c = Case([70, 3, 0, 129], 136, 72, True, seed=9)
    outs = lambda: [torch.zeros(c.R, c.up, dtype=BF16, device=dev()), torch.zeros_like(c.w2),
                    torch.zeros(c.R, c.H, dtype=BF16, device=dev()), torch.zeros_like(c.w13)]

    def call(o, stream=None):
        N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, c.pre, c.h, o[0], o[1], c.ws, stream=stream)
        N.moe_expert_up_backward(c.shape, o[0], c.offsets, c.x, c.w13, o[2], o[3], c.ws, stream=stream)

    a, b, d = outs(), outs(), outs()
    call(a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(b, s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(d)
    g.replay()
    g.replay()
    c.status()
    for x, y, z in zip(a, b, d):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert torch.equal(x.view(torch.int16), z.view(torch.int16))


def test_gradients_against_differences():
    """Central differences of the FFN in 64 bits along random directions."""
    c = Case([21, 0, 64, 9], 72, 40, True, seed=10)
    b = c.offsets.tolist()

    def loss(x, w13, w2):
        y = torch.zeros(c.R, c.H, dtype=D, device=dev())
        for e in range(c.E):
            r = slice(b[e], b[e + 1])
            y[r] = ref.act(x[r] @ w13[e].t(), True) @ w2[e].t()
        return (y * c.dy.to(D)).sum()

    pre = torch.empty(c.R, c.up, dtype=BF16, device=dev())
    h = torch.empty(c.R, c.I, dtype=BF16, device=dev())
    dpre, dx = torch.empty_like(pre), torch.empty_like(c.x)
    dw13, dw2 = torch.empty(c.w13.shape, device=dev()), torch.empty(c.w2.shape, device=dev())
    N.moe_expert_up_train(c.shape, c.x, c.offsets, c.w13, pre, h, c.ws)
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, pre, h, dpre, dw2, c.ws)
    N.moe_expert_up_backward(c.shape, dpre, c.offsets, c.x, c.w13, dx, dw13, c.ws)
    c.status()
    at = [c.x.to(D), c.w13.to(D), c.w2.to(D)]
    gen = torch.Generator(device=dev()).manual_seed(1)
    for i, grad in enumerate((dx, dw13, dw2)):
        v = torch.randn(at[i].shape, generator=gen, device=dev(), dtype=D)
        step = 1e-4
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * v, at[i] - step * v
        diff = (loss(*up) - loss(*down)) / (2 * step)
        got = (grad.to(D) * v).sum()
        # pre, h, dpre and the gradient itself each rounded to bf16 (half a unit, as
        # independent errors of the gradient's own size): four of them, five sigma
        tol = 5 * 2 * 0.5 * ref.U_BF16 * grad.to(D).norm()
        assert abs(got - diff) <= tol, (i, float(got), float(diff), float(tol))


# in one piece, with the weights form split, with both forms split
@pytest.mark.parametrize("case", [([30, 30, 40], 72, 40), ([1950, 1950], 64, 40), ([2600], 2400, 64)], ids=str)
@pytest.mark.parametrize("bad", ["decreasing", "negative", "past the end"])
def test_refused_bounds_leave_the_weight_gradient_of_empty_buckets(case, bad):
    counts, H, I = case
    c = Case(counts, H, I, True, seed=11)
    b = c.offsets.tolist()
    if bad == "decreasing":
        b[0], b[1] = b[1], b[0]
    elif bad == "negative":
        b[0] = -1
    else:
        b[-1] = c.R + 1
    offsets = torch.tensor(b, dtype=torch.int32, device=dev())

    def calls(dw2, dw13, add=False):
        N.moe_expert_down_backward(c.shape, c.dy, offsets, c.w2, c.pre, c.h, torch.empty_like(c.pre), dw2, c.ws, add=add)
        assert N.moe_status_read(c.ws) == N.MOE_ERR_INVALID_ROUTE
        N.moe_expert_up_backward(c.shape, c.dpre_in, offsets, c.x, c.w13, torch.empty_like(c.x), dw13, c.ws, add=add)
        assert N.moe_status_read(c.ws) == N.MOE_ERR_INVALID_ROUTE
        N.moe_expert_up_backward(c.shape, c.dpre_in, offsets, c.x, None, None, dw13, c.ws, add=add)   # its own plan
        assert N.moe_status_read(c.ws) == N.MOE_ERR_INVALID_ROUTE

    for dtype in (BF16, F32):
        dw2, dw13 = Guarded((c.E, c.H, c.I), dtype), Guarded((c.E, c.up, c.H), dtype)
        calls(dw2.t, dw13.t)
        assert torch.all(dw2.t == 0) and torch.all(dw13.t == 0) and dw2.intact() and dw13.intact()
    old2, old13 = torch.randn(c.E, c.H, c.I, device=dev()), torch.randn(c.E, c.up, c.H, device=dev())
    dw2, dw13 = old2.clone(), old13.clone()
    calls(dw2, dw13, add=True)
    assert torch.equal(dw2, old2) and torch.equal(dw13, old13)


def many_buckets(E, seed):
    """Ragged and empty buckets, and two of several rounds of either ring plus a remainder."""
    g = torch.Generator().manual_seed(seed)
    sizes = torch.tensor([0, 0, 1, 2, 15, 16, 17, 33, 63, 64, 65, 100])
    counts = sizes[torch.randint(0, len(sizes), (E,), generator=g)].tolist()
    counts[E // 3], counts[E - 2] = 3 * 5 * 64 + 7, 2 * 6 * 64 + 60
    return counts


# around the change from six stages to five (up to 63 groups have room for six), up to the
# most experts; from 353 on a thread counts several groups' tiles
@pytest.mark.parametrize("E", [33, 63, 64, 65, 240, 352, 353, 705, 1024])
@pytest.mark.parametrize("glu", [True, False], ids=["swiglu", "relu2"])
def test_many_experts(E, glu):
    counts = many_buckets(E, E)
    c = Case(counts, 136 if E < 300 else 72, 72 if E < 300 else 40, glu, seed=E)
    run_and_check(c, counts)
    # each form alone: the same bits as together
    a, b = (dict(dpre=torch.zeros_like(c.pre), dw2=torch.zeros_like(c.w2), dx=torch.zeros_like(c.x),
                 dw13=torch.zeros_like(c.w13)) for _ in range(2))
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, c.pre, c.h, b["dpre"], b["dw2"], c.ws)
    N.moe_expert_up_backward(c.shape, c.dpre_in, c.offsets, c.x, c.w13, b["dx"], b["dw13"], c.ws)
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, c.w2, c.pre, None, a["dpre"], None, c.ws)
    N.moe_expert_down_backward(c.shape, c.dy, c.offsets, None, None, c.h, None, a["dw2"], c.ws)
    N.moe_expert_up_backward(c.shape, c.dpre_in, c.offsets, None, c.w13, a["dx"], None, c.ws)
    N.moe_expert_up_backward(c.shape, c.dpre_in, c.offsets, c.x, None, None, a["dw13"], c.ws)
    c.status()
    assert all(torch.equal(a[n].view(torch.int16), b[n].view(torch.int16)) for n in a)


@pytest.mark.parametrize("E", [63, 64, 65])
def test_split_reductions_of_many_experts(E):
    """Few rows an expert and a long reduction: the rows form split in either ring."""
    run_and_check(Case([1 + e % 2 for e in range(E)], 9216, 8, E % 2 == 0, seed=E), [2])
