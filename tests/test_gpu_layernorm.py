"""Layer norm, forward and backward, against the formulas in 64 bits: element by
element within the error bound of FP32 statistics and one rounding of the output."""
import pytest
import torch

from mixture_experts_routing_router_gb300 import native as N

import train_ref as ref
from gpu_util import dev
from test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu

BF16, F32, D = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-5


def check(got, want, bound, what):
    got = got.to(D)
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()} outside, worst by {over.max():.3e}"


def inputs(rows, H, dtype, wtype, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = (r(rows, H) * (1 + 7 * (torch.rand(H, generator=g) < 0.02)) + offset).to(dtype)
    return [t.to(dev()) for t in (x, (1 + 0.3 * r(H)).to(wtype), r(H).to(wtype), r(rows, H).to(dtype),
                                  r(rows, H).to(dtype))]


def run_both(x, gamma, beta, dy, dres):
    rows, H = x.numel() // x.shape[-1], x.shape[-1]
    y, dx = Guarded(tuple(x.shape), x.dtype), Guarded(tuple(x.shape), x.dtype)
    mean, rstd = Guarded((rows,), F32), Guarded((rows,), F32)
    dg, db = Guarded((H,), F32), Guarded((H,), F32)
    sc = Guarded((N.moe_layernorm_scratch_size(rows, H),), torch.uint8)
    N.moe_layernorm(x, gamma, beta, EPS, y.t, mean.t, rstd.t)
    N.moe_layernorm_backward(dy, x, gamma, mean.t, rstd.t, dx.t, dg.t, db.t, sc.t, dres=dres)
    torch.cuda.synchronize()
    assert all(b.intact() for b in (y, dx, mean, rstd, dg, db, sc))
    return y.t, mean.t, rstd.t, dx.t, dg.t, db.t


def verify(x, gamma, beta, dy, dres):
    y, mean, rstd, dx, dg, db = run_both(x, gamma, beta, dy, dres)
    rows = x.numel() // x.shape[-1]
    for got, want, bound, what in zip((y, mean, rstd), ref.layernorm(x, gamma, beta, EPS),
                                      ref.layernorm_bound(x, gamma, beta, EPS, x.dtype), ("y", "mean", "rstd")):
        check(got.view(want.shape), want, bound, what)
    m, r = mean.view(x.shape[:-1]), rstd.view(x.shape[:-1])
    for got, want, bound, what in zip((dx, dg, db), ref.layernorm_backward(dy, x, gamma, m, r, dres),
                                      ref.layernorm_backward_bound(dy, x, gamma, m, r, dres, x.dtype),
                                      ("dx", "dgamma", "dbeta")):
        check(got, want, bound, what)
    return rows


# widths around every vector and block size, odd ones, one column, very wide ones
WIDTHS = [1, 2, 7, 8, 31, 33, 64, 100, 255, 256, 257, 1001, 1024, 2040, 2048, 4096, 4104, 7168, 8192, 8200, 16384,
          40000]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_widths(H, dtype):
    x, gamma, beta, dy, dres = inputs(5, H, dtype, F32, seed=H)
    verify(x, gamma, beta, dy, dres)


@pytest.mark.parametrize("rows", [1, 2, 3, 151, 303, 304, 305, 609, 2000])
@pytest.mark.parametrize("H", [72, 1001])
def test_rows(rows, H):
    x, gamma, beta, dy, _ = inputs(rows, H, BF16, F32, seed=rows)
    verify(x, gamma, beta, dy, None)


@pytest.mark.parametrize("rows", [1, 7, 9, 20, 151, 153, 170])
@pytest.mark.parametrize("H", [509, 1023, 2046, 4089, 7167, 8185, 9001, 16381])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_odd_widths_at_every_thread_count(rows, H, dtype):
    x, gamma, beta, dy, dres = inputs(rows, H, dtype, F32, seed=rows + H)
    verify(x, gamma, beta, dy, dres)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("wtype", [BF16, F32], ids=["wbf16", "wf32"])
@pytest.mark.parametrize("H", [264, 7168, 515])
def test_types(dtype, wtype, H):
    x, gamma, beta, dy, dres = inputs(37, H, dtype, wtype, seed=3)
    verify(x, gamma, beta, dy, dres)


def test_leading_dimensions_are_rows():
    x, gamma, beta, dy, dres = inputs(24, 136, BF16, F32)
    verify(x.view(2, 3, 4, 136), gamma, beta, dy.view(2, 3, 4, 136), dres.view(2, 3, 4, 136))


@pytest.mark.parametrize("H", [264, 1001])
def test_a_large_offset_keeps_its_digits(H):
    x, gamma, beta, dy, dres = inputs(9, H, F32, F32, seed=4, offset=1000.0)
    verify(x, gamma, beta, dy, dres)


@pytest.mark.parametrize("H", [264, 1001])
def test_constant_rows(H):
    x, gamma, beta, dy, _ = inputs(3, H, F32, F32, seed=5)
    x[:] = 0.5                                   # exact in any order of summation
    y, mean, rstd, dx, dg, db = run_both(x, gamma, beta, dy, None)
    assert torch.equal(y, beta.expand_as(y)) and torch.all(mean == 0.5)
    want = torch.full_like(rstd, EPS).to(D).rsqrt()
    assert ((rstd.to(D) - want).abs() <= 4 * ref.U_F32 * want).all()
    assert torch.all(dg == 0)


@pytest.mark.parametrize("H", [264, 1001, 7168])
def test_a_row_of_nan_or_infinity_stays_in_its_row(H):
    x, gamma, beta, dy, dres = inputs(6, H, BF16, F32, seed=6)
    x[2, 3], x[4, 0] = float("nan"), float("inf")
    y, mean, rstd, dx, dg, db = run_both(x, gamma, beta, dy, dres)
    for t in (y, dx):
        assert torch.isnan(t[[2, 4]]).all() and torch.isfinite(t[[0, 1, 3, 5]]).all()
    assert torch.isnan(dg).all() and torch.isfinite(db).all()


def test_no_rows():
    H = 40
    x = torch.empty(0, H, dtype=BF16, device=dev())
    gamma = torch.ones(H, device=dev())
    N.moe_layernorm(x, gamma, gamma, EPS, torch.empty_like(x), torch.empty(0, device=dev()), None)
    dg, db = torch.full((H,), 7.0, device=dev()), torch.full((H,), 7.0, device=dev())
    e = torch.empty(0, device=dev())
    N.moe_layernorm_backward(x, x, gamma, e, e, torch.empty_like(x), dg, db, N.layernorm_scratch(0, H))
    assert torch.all(dg == 0) and torch.all(db == 0)


@pytest.mark.parametrize("H", [264, 1001, 7168, 40000])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_outputs_in_place(H, dtype):
    x, gamma, beta, dy, dres = inputs(700 if H < 8000 else 20, H, dtype, F32, seed=7)
    y, mean, rstd, dx, dg, db = run_both(x, gamma, beta, dy, dres)
    own = x.clone()
    N.moe_layernorm(own, gamma, beta, EPS, own)
    assert torch.equal(own, y)
    for which in range(3):
        b = [dy.clone(), x.clone(), dres.clone()]
        dg2, db2 = torch.empty_like(dg), torch.empty_like(db)
        N.moe_layernorm_backward(b[0], b[1], gamma, mean, rstd, b[which], dg2, db2,
                                 N.layernorm_scratch(x.shape[0], H), dres=b[2])
        assert torch.equal(b[which], dx) and torch.equal(dg2, dg) and torch.equal(db2, db)


def test_a_row_does_not_depend_on_its_batch_and_streams_and_graphs_agree():
    x, gamma, beta, dy, dres = inputs(333, 1032, BF16, F32, seed=8)
    y, mean, rstd, dx, dg, db = run_both(x, gamma, beta, dy, dres)
    one = [torch.empty_like(x[:1]) for _ in range(2)]
    N.moe_layernorm(x[100:101], gamma, beta, EPS, one[0])
    assert torch.equal(one[0], y[100:101])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dx2, dg2, db2, sc = torch.empty_like(dx), torch.empty_like(dg), torch.empty_like(db), N.layernorm_scratch(333, 1032)
    N.moe_layernorm_backward(dy, x, gamma, mean, rstd, dx2, dg2, db2, sc, dres=dres, stream=s)
    s.synchronize()
    assert torch.equal(dx2, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        N.moe_layernorm_backward(dy, x, gamma, mean, rstd, dx2, dg2, db2, sc, dres=dres)
    for t in (dx2, dg2, db2):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx2, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)


def test_gradient_against_differences():
    """Central differences of the 64-bit layer norm along random directions."""
    x, gamma, beta, dy, _ = inputs(11, 96, F32, F32, seed=9)
    _, _, _, dx, dg, db = run_both(x, gamma, beta, dy, None)
    loss = lambda x, g, b: (ref.layernorm(x, g, b, EPS)[0] * dy.to(D)).sum()
    at = [x.to(D), gamma.to(D), beta.to(D)]
    gen = torch.Generator(device=dev()).manual_seed(2)
    for i, grad in enumerate((dx, dg, db)):
        v = torch.randn(at[i].shape, generator=gen, device=dev(), dtype=D)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 1e-4 * v, at[i] - 1e-4 * v
        diff = (loss(*up) - loss(*down)) / 2e-4
        # the difference's own error is of order step^2; FP32 gradients: 1e-6 of their size
        assert abs((grad.to(D) * v).sum() - diff) <= 1e-5 * grad.to(D).norm() * v.norm()
