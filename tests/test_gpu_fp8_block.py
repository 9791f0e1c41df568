"""The expert path in block-scaled FP8 against its definition in 64 bits: codes and scales
of the dispatch bit for bit, the products within the bounds of FP32 sums and the output's
rounding; odd widths, buckets around the tile sizes, empty ones, rows behind the last."""
import pytest
import torch

import fp8_ref as ref
from mixture_experts_routing_router_gb300 import native as N

from gpu_util import dev
from test_gpu_guard import Guarded, guarded_workspace

pytestmark = pytest.mark.gpu

BF16, F32, I32, U8, D = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float64
ACT = {"swiglu": N.MOE_ACT_SWIGLU, "relu2": N.MOE_ACT_RELU2}


def gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def rows_of(g, R, H):
    """Rows as a residual stream has them: a few large channels, a zero row, a zero block, tiny values."""
    x = torch.randn(R, H, generator=g, device=dev()) * (1.0 + 30.0 * (torch.rand(H, generator=g, device=dev()) < 0.02))
    x = x.to(BF16)
    if R > 2:
        x[1] = 0
        x[2, :128] = 0
        x[R - 1] *= 2.0 ** -90
    return x


# ---- quantizing dispatch -----------------------------------------------------------
#         T    H     E   k
SIZES = [(1, 16, 1, 1), (1, 7168, 16, 8), (3, 48, 4, 2), (37, 144, 33, 5), (64, 256, 16, 2), (40, 1040, 8, 8),
         (300, 128, 1024, 32), (700, 2048, 64, 6), (3, 20000, 6, 3), (16, 1008, 9, 3),
         # one launch up to 12288 pairs, three from there on
         (1365, 64, 40, 9), (1366, 64, 40, 9), (384, 32, 64, 32), (385, 32, 64, 32), (12288, 16, 5, 1), (2400, 272, 300, 8)]


def dispatch_buffers(T, H, E, k):
    R = T * k
    return [Guarded((E,), I32), Guarded((E + 1,), I32), Guarded((R,), I32), Guarded((R,), I32), Guarded((R, H), U8),
            Guarded((R, ref.blocks(H)), F32)]


@pytest.mark.parametrize("bad", [False, True], ids=["valid", "invalid"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_dispatch(size, bad):
    T, H, E, k = size
    g = torch.Generator().manual_seed(T + H)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(I32)
    if bad:
        if T < 4:
            pytest.skip("too few tokens for the invalid kinds")
        ids[0, 0], ids[T // 2, k - 1], ids[T - 1] = -3, E + 5, -1
    ids = ids.to(dev())
    x = rows_of(gen(3), T, H)
    shape = N.make_shape(T, H, E, k, 16)
    ws = guarded_workspace(shape)
    out = dispatch_buffers(T, H, E, k)
    out[4].t.fill_(0x5A)
    N.moe_dispatch_fp8_block(shape, x, ids, *(o.t for o in out), ws.t)
    assert N.moe_status_read(ws.t) == (N.MOE_ERR_INVALID_ROUTE if bad else N.MOE_OK)
    assert all(o.intact() for o in out) and ws.intact()
    # placement: that of the unquantized dispatch
    i32 = lambda *s: torch.empty(s, dtype=I32, device=dev())
    plain = [i32(E), i32(E + 1), i32(T * k), i32(T * k), torch.empty((T * k, H), dtype=BF16, device=dev())]
    N.moe_dispatch(shape, x, ids, *plain, N.workspace(shape, dev()))
    n = int(plain[1][-1])
    for a, b in zip(out[:3], plain[:3]):
        assert torch.equal(a.t, b)
    assert torch.equal(out[3].t[:n], plain[3][:n])
    codes, scale = ref.quantize(plain[4][:n])
    assert torch.equal(ref.values(out[4].t[:n]), codes) and torch.equal(out[5].t[:n], scale)
    assert torch.all(out[4].t[n:] == 0x5A)                       # rows behind the last one


@pytest.mark.parametrize("size", [(20000, 16, 300, 3), (4099, 32, 1024, 32), (70001, 16, 33, 1), (5003, 16, 7, 7)], ids=str)
def test_dispatch_of_many_tiles(size):
    """More tiles of pairs than a scan has warps, tokens across the edges of warps and tiles,
    repeated and invalid ids everywhere, then a call over capacity and a valid one again, and the
    unquantized dispatch between them on the same workspace."""
    T, H, E, k = size
    g = torch.Generator().manual_seed(E)
    ids = torch.randint(-1, E + 1, (T, k), generator=g, dtype=I32)
    ids[T // 3:T // 2] = torch.arange(k, dtype=I32)[None] % E
    ids = ids.to(dev())
    x = rows_of(gen(4), T, H)
    shape = N.make_shape(T, H, E, k, 16)
    ws = guarded_workspace(shape)
    i32 = lambda *s: torch.empty(s, dtype=I32, device=dev())
    plain = [i32(E), i32(E + 1), i32(T * k), i32(T * k), torch.empty((T * k, H), dtype=BF16, device=dev())]
    for _ in range(2):
        out = dispatch_buffers(T, H, E, k)
        out[4].t.fill_(0x5A)
        N.moe_dispatch_fp8_block(shape, x, ids, *(o.t for o in out), ws.t)
        assert N.moe_status_read(ws.t) == N.MOE_ERR_INVALID_ROUTE
        assert all(o.intact() for o in out) and ws.intact()
        N.moe_dispatch(shape, x, ids, *plain, ws.t)
        assert N.moe_status_read(ws.t) == N.MOE_ERR_INVALID_ROUTE
        n = int(plain[1][-1])
        assert all(torch.equal(a.t, b) for a, b in zip(out[:3], plain[:3]))
        assert torch.equal(out[3].t[:n], plain[3][:n])
        codes, scale = ref.quantize(plain[4][:n])
        assert torch.equal(ref.values(out[4].t[:n]), codes) and torch.equal(out[5].t[:n], scale)
        assert torch.all(out[4].t[n:] == 0x5A)
        most = int(plain[0].max())
        before = out[4].t.clone()
        small = N.make_shape(T, H, E, k, 16, capacity=most - 1)
        N.moe_dispatch_fp8_block(small, x, ids, *(o.t for o in out), ws.t)
        assert N.moe_status_read(ws.t) in (N.MOE_ERR_CAPACITY, N.MOE_ERR_INVALID_ROUTE)
        assert torch.equal(out[4].t, before) and torch.equal(out[0].t, plain[0])


def test_dispatch_extremes():
    """The largest values, subnormals, rounding ties, and blocks that are not finite."""
    T, H = 6, 400
    x = torch.randn(T, H, generator=gen(5), device=dev()).to(BF16)
    x[0] *= 2.0 ** 120
    x[0, 7] = torch.finfo(BF16).max
    x[1] = 2.0 ** -133
    x[2] = torch.tensor([1.0 + i / 128 for i in range(128)] * 4, device=dev())[:H].to(BF16)   # ties of a power of two
    x[2, 0:H:128] = 1.75
    x[3, 130] = float("nan")
    x[4, 399], x[4, 3] = float("inf"), float("-inf")
    shape = N.make_shape(T, H, 1, 1, 16)
    ws = N.workspace(shape, dev())
    out = [o.t for o in dispatch_buffers(T, H, 1, 1)]
    N.moe_dispatch_fp8_block(shape, x, torch.zeros((T, 1), dtype=I32, device=dev()), *out, ws)
    codes, scale = ref.quantize(x)
    same = lambda a, b: torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    assert same(out[5], scale) and same(ref.values(out[4]), codes)
    assert torch.isnan(out[5][3]).tolist() == [False, True, False, False]
    assert N.moe_status_read(ws) == N.MOE_OK


def test_dispatch_over_capacity_moves_nothing():
    shape = N.make_shape(50, 64, 4, 2, 16, capacity=10)
    ids = torch.tensor([[0, 1]], dtype=I32, device=dev()).repeat(50, 1)
    out = [o.t for o in dispatch_buffers(50, 64, 4, 2)]
    before = out[4].clone()
    ws = N.workspace(shape, dev())
    N.moe_dispatch_fp8_block(shape, rows_of(gen(1), 50, 64), ids, *out, ws)
    assert N.moe_status_read(ws) == N.MOE_ERR_CAPACITY
    assert torch.equal(out[4], before) and out[0].tolist() == [50, 50, 0, 0]


# ---- products ------------------------------------------------------------------------
BUCKETS = {
    "one": [1], "few": [0, 3, 0, 8, 9, 1], "edges": [32, 33, 96, 97, 127, 128, 129], "big": [300, 0, 513],
    "mixed": [1, 8, 129, 200, 256, 257, 700, 1000],
    "many": [(7 * i) % 11 for i in range(300)], "thousand": [(5 * i) % 4 for i in range(1024)],
}
WIDTHS = [(16, 16), (128, 128), (144, 112), (272, 400), (1024, 640), (2064, 144)]


def problem(buckets, H, I, act, seed, extra=3):
    """Rows in buckets, `extra` rows behind the last one, weights and a shape that holds them."""
    g = gen(seed)
    R = sum(buckets) + extra
    E = len(buckets)
    bounds = [0]
    for b in buckets:
        bounds.append(bounds[-1] + b)
    x = rows_of(g, R, H)
    codes, scale = ref.quantize(x)
    d = dict(bounds=bounds, offsets=torch.tensor(bounds, dtype=I32, device=dev()),
             x=codes.to(torch.float32).to(ref.E4M3).view(U8), x_scale=scale, R=R)
    d["w13"], d["w13_scale"] = ref.random_weights(g, (E, 2 if act == "swiglu" else 1), I, H, dev())
    d["w2"], d["w2_scale"] = ref.random_weights(g, (E,), H, I, dev())
    d["shape"] = N.make_shape(R, H, E, 1, I, act=ACT[act])
    return d


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("width", WIDTHS, ids=str)
@pytest.mark.parametrize("name", sorted(BUCKETS))
def test_products(name, width, act):
    H, I = width
    if name in ("many", "thousand") and H * I > 40000:
        pytest.skip("covered by the smaller widths")
    d = problem(BUCKETS[name], H, I, act, seed=H + I)
    ws = guarded_workspace(d["shape"])
    h, hs, y = Guarded((d["R"], I), U8), Guarded((d["R"], ref.blocks(I)), F32), Guarded((d["R"], H), BF16)
    for o in (h, y):
        o.t.view(U8).fill_(0x5A)
    hs.t.fill_(7.0)
    N.moe_expert_up_fp8_block(d["shape"], d["x"], d["x_scale"], d["offsets"], d["w13"], d["w13_scale"], h.t, hs.t, ws.t)
    N.moe_expert_down_fp8_block(d["shape"], h.t, hs.t, d["offsets"], d["w2"], d["w2_scale"], y.t, ws.t)
    assert N.moe_status_read(ws.t) == N.MOE_OK
    assert h.intact() and hs.intact() and y.intact() and ws.intact()
    n = d["bounds"][-1]
    want, off = ref.up(d["x"][:n], d["x_scale"][:n], d["bounds"], d["w13"], d["w13_scale"], act == "swiglu")
    ref.check_quantized(h.t[:n], hs.t[:n], want, off, "h")
    want, off = ref.down(h.t[:n], hs.t[:n], d["bounds"], d["w2"], d["w2_scale"])
    over = (y.t[:n].to(D) - want).abs() - off
    assert (over <= 0).all(), f"y: {int((over > 0).sum())} outside, worst by {over.max():.3e}"
    # rows behind the last one
    assert torch.all(h.t[n:] == 0x5A) and torch.all(hs.t[n:] == 7.0) and torch.all(y.t[n:].view(U8) == 0x5A)


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("width", [(16, 16), (144, 112), (272, 400), (1024, 640), (2064, 144), (400, 1536)], ids=str)
@pytest.mark.parametrize("tokens", [1, 8, 9, 16, 17, 31, 33, 64])
def test_products_of_few_rows(tokens, width, act):
    """Few rows a group (decode): every group at most as many as there are tokens, and, with
    bounds that no dispatch of so few tokens makes, groups that span several tiles."""
    H, I = width
    E, k = 12, 5
    R, spread = tokens * k, [min(tokens, 1 + (3 * e) % 7) if e % 3 == 1 else 0 for e in range(E)]
    for buckets in (spread, [R - 3] + [0] * (E - 2) + [2]):
        d = problem(buckets, H, I, act, seed=H + I + tokens, extra=R - sum(buckets))
        shape = N.make_shape(tokens, H, E, k, I, act=ACT[act])
        ws = guarded_workspace(shape)
        h, hs, y = Guarded((R, I), U8), Guarded((R, ref.blocks(I)), F32), Guarded((R, H), BF16)
        for o in (h, y):
            o.t.view(U8).fill_(0x5A)
        hs.t.fill_(7.0)
        N.moe_expert_up_fp8_block(shape, d["x"], d["x_scale"], d["offsets"], d["w13"], d["w13_scale"], h.t, hs.t, ws.t)
        N.moe_expert_down_fp8_block(shape, h.t, hs.t, d["offsets"], d["w2"], d["w2_scale"], y.t, ws.t)
        assert N.moe_status_read(ws.t) == N.MOE_OK
        assert h.intact() and hs.intact() and y.intact() and ws.intact()
        n = d["bounds"][-1]
        want, off = ref.up(d["x"][:n], d["x_scale"][:n], d["bounds"], d["w13"], d["w13_scale"], act == "swiglu")
        ref.check_quantized(h.t[:n], hs.t[:n], want, off, "h")
        want, off = ref.down(h.t[:n], hs.t[:n], d["bounds"], d["w2"], d["w2_scale"])
        over = (y.t[:n].to(D) - want).abs() - off
        assert (over <= 0).all(), f"y: {int((over > 0).sum())} outside, worst by {over.max():.3e}"
        assert torch.all(h.t[n:] == 0x5A) and torch.all(hs.t[n:] == 7.0) and torch.all(y.t[n:].view(U8) == 0x5A)


def test_no_rows():
    d = problem([0, 0, 0], 128, 128, "swiglu", 1, extra=4)
    ws = N.workspace(d["shape"], dev())
    h, hs = torch.full((4, 128), 9, dtype=U8, device=dev()), torch.full((4, 1), 7.0, device=dev())
    y = torch.full((4, 128), 5.0, dtype=BF16, device=dev())
    N.moe_expert_up_fp8_block(d["shape"], d["x"], d["x_scale"], d["offsets"], d["w13"], d["w13_scale"], h, hs, ws)
    N.moe_expert_down_fp8_block(d["shape"], h, hs, d["offsets"], d["w2"], d["w2_scale"], y, ws)
    assert N.moe_status_read(ws) == N.MOE_OK
    assert torch.all(h == 9) and torch.all(hs == 7) and torch.all(y == 5)


@pytest.mark.parametrize("rows", [400, 1200])
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
def test_a_row_does_not_depend_on_its_company(act, rows):
    """A row alone and among 400 or 1200 others: the same bits."""
    H, I = 400, 272
    d = problem([rows, 17], H, I, act, seed=8, extra=0)

    def run(offsets, x, xs, R):
        shape = N.make_shape(R, H, 2, 1, I, act=ACT[act])
        ws = N.workspace(shape, dev())
        h, hs = torch.empty((R, I), dtype=U8, device=dev()), torch.empty((R, ref.blocks(I)), device=dev())
        y = torch.empty((R, H), dtype=BF16, device=dev())
        N.moe_expert_up_fp8_block(shape, x, xs, offsets, d["w13"], d["w13_scale"], h, hs, ws)
        N.moe_expert_down_fp8_block(shape, h, hs, offsets, d["w2"], d["w2_scale"], y, ws)
        assert N.moe_status_read(ws) == N.MOE_OK
        return h, hs, y

    whole = run(d["offsets"], d["x"], d["x_scale"], rows + 17)
    again = run(d["offsets"], d["x"], d["x_scale"], rows + 17)
    for a, b in zip(whole, again):
        assert torch.equal(a.view(U8), b.view(U8))
    for r, bounds in ((0, [0, 1, 1]), (131, [0, 1, 1]), (rows - 1, [0, 1, 1]), (rows + 5, [0, 0, 1])):
        alone = run(torch.tensor(bounds, dtype=I32, device=dev()), d["x"][r:r + 1].clone(), d["x_scale"][r:r + 1].clone(), 1)
        for a, b in zip(whole, alone):
            assert torch.equal(a[r:r + 1].view(U8), b.view(U8)), r


def test_a_row_that_is_not_finite_stays_alone():
    d = problem([40, 5], 272, 144, "swiglu", seed=4, extra=0)
    shape = d["shape"]

    def run():
        ws = N.workspace(shape, dev())
        h, hs = torch.empty((45, 144), dtype=U8, device=dev()), torch.empty((45, 2), device=dev())
        y = torch.empty((45, 272), dtype=BF16, device=dev())
        N.moe_expert_up_fp8_block(shape, d["x"], d["x_scale"], d["offsets"], d["w13"], d["w13_scale"], h, hs, ws)
        N.moe_expert_down_fp8_block(shape, h, hs, d["offsets"], d["w2"], d["w2_scale"], y, ws)
        assert N.moe_status_read(ws) == N.MOE_OK
        return y

    clean = run()
    d["x"][7, 128:256], d["x_scale"][7, 1] = 0x7F, float("nan")          # as the dispatch codes such a block
    y = run()
    assert torch.isnan(y[7].float()).all()
    keep = [r for r in range(45) if r != 7]
    assert torch.equal(y[keep].view(torch.int16), clean[keep].view(torch.int16))


def test_few_rows_of_a_thousand_experts():
    """64 tokens to 32 of 1024 experts: about two rows a group, the largest group lists."""
    H, I, E, k, T = 144, 112, 1024, 32, 64
    buckets = [2 if e % 5 else 1 for e in range(E)]
    d = problem(buckets, H, I, "swiglu", seed=3, extra=T * k - sum(buckets))
    shape = N.make_shape(T, H, E, k, I)
    ws = N.workspace(shape, dev())
    h, hs = torch.empty((T * k, I), dtype=U8, device=dev()), torch.empty((T * k, 1), device=dev())
    y = torch.empty((T * k, H), dtype=BF16, device=dev())
    N.moe_expert_up_fp8_block(shape, d["x"], d["x_scale"], d["offsets"], d["w13"], d["w13_scale"], h, hs, ws)
    N.moe_expert_down_fp8_block(shape, h, hs, d["offsets"], d["w2"], d["w2_scale"], y, ws)
    assert N.moe_status_read(ws) == N.MOE_OK
    n = d["bounds"][-1]
    ref.check_quantized(h[:n], hs[:n], *ref.up(d["x"][:n], d["x_scale"][:n], d["bounds"], d["w13"], d["w13_scale"], True), "h")
    want, off = ref.down(h[:n], hs[:n], d["bounds"], d["w2"], d["w2_scale"])
    assert ((y[:n].to(D) - want).abs() <= off).all()


@pytest.mark.parametrize("rows", [5, 200])
def test_nan_weights_reach_their_outputs_only(rows):
    """A NaN code of w2 makes its column of its expert NaN; one of w13 the rows of its expert."""
    d = problem([rows, rows], 272, 144, "swiglu", seed=2, extra=0)
    shape, R = N.make_shape(2 * rows, 272, 2, 1, 144), 2 * rows

    def run():
        ws = N.workspace(shape, dev())
        h, hs = torch.empty((R, 144), dtype=U8, device=dev()), torch.empty((R, 2), device=dev())
        y = torch.empty((R, 272), dtype=BF16, device=dev())
        N.moe_expert_up_fp8_block(shape, d["x"], d["x_scale"], d["offsets"], d["w13"], d["w13_scale"], h, hs, ws)
        N.moe_expert_down_fp8_block(shape, h, hs, d["offsets"], d["w2"], d["w2_scale"], y, ws)
        assert N.moe_status_read(ws) == N.MOE_OK
        return y

    clean = run()
    keep = d["w2"][1, 130, 77].clone()
    d["w2"][1, 130, 77] = 0x7F
    y = run()
    nan = torch.isnan(y)
    assert nan[rows:, 130].all() and int(nan.sum()) == rows
    assert torch.equal(y[~nan], clean[~nan])
    d["w2"][1, 130, 77], d["w13"][0, 1, 7, 9] = keep, 0xFF
    y = run()
    assert torch.isnan(y[:rows]).all() and torch.equal(y[rows:].view(torch.int16), clean[rows:].view(torch.int16))


def test_buckets_outside_the_rows_are_clamped():
    """Bounds that leave the rows or decrease: nothing outside the buffers is touched."""
    d = problem([20, 30], 128, 144, "relu2", seed=6, extra=0)
    offsets = torch.tensor([-5, 4000, 20], dtype=I32, device=dev())
    ws = guarded_workspace(d["shape"])
    h, hs, y = Guarded((50, 144), U8), Guarded((50, 2), F32), Guarded((50, 128), BF16)
    N.moe_expert_up_fp8_block(d["shape"], d["x"], d["x_scale"], offsets, d["w13"], d["w13_scale"], h.t, hs.t, ws.t)
    N.moe_expert_down_fp8_block(d["shape"], h.t, hs.t, offsets, d["w2"], d["w2_scale"], y.t, ws.t)
    torch.cuda.synchronize()
    assert h.intact() and hs.intact() and y.intact() and ws.intact()


# ---- the layer -------------------------------------------------------------------------
#         T    H    E   k   I   act       groups topk_groups
LAYERS = [(1, 272, 24, 6, 144, "relu2", 8, 4), (16, 128, 8, 2, 400, "swiglu", 4, 2), (70, 400, 32, 5, 128, "swiglu", 8, 3),
          (600, 256, 6, 2, 272, "relu2", 3, 2), (33, 1024, 240, 9, 640, "swiglu", 16, 4)]


def layer_inputs(T, H, E, k, I, act, seed):
    g = gen(seed)
    d = dict(x=torch.randn(T, H, generator=g, device=dev()).to(BF16),
             w_gate=(torch.randn(E, H, generator=g, device=dev()) / H ** 0.5).to(BF16),
             bias=0.05 * torch.randn(E, generator=g, device=dev()),
             residual=torch.randn(T, H, generator=g, device=dev()).to(BF16))
    d["w13"], d["w13_scale"] = ref.random_weights(g, (E, 2 if act == "swiglu" else 1), I, H, dev())
    d["w2"], d["w2_scale"] = ref.random_weights(g, (E,), H, I, dev())
    return d


def stages(shape, d, ids, w, residual, ws):
    T, H, E, k, I = shape.tokens, shape.hidden, shape.experts, shape.top_k, shape.inter
    R = T * k
    new = lambda *s, t=F32: torch.empty(s, dtype=t, device=dev())
    offsets, dest, xq, xs = new(E + 1, t=I32), new(R, t=I32), new(R, H, t=U8), new(R, ref.blocks(H))
    h, hs, y, out = new(R, I, t=U8), new(R, ref.blocks(I)), new(R, H, t=BF16), new(T, H, t=BF16)
    N.moe_dispatch_fp8_block(shape, d["x"], ids, new(E, t=I32), offsets, dest, new(R, t=I32), xq, xs, ws)
    N.moe_expert_up_fp8_block(shape, xq, xs, offsets, d["w13"], d["w13_scale"], h, hs, ws)
    N.moe_expert_down_fp8_block(shape, h, hs, offsets, d["w2"], d["w2_scale"], y, ws)
    N.moe_combine(shape, y, dest, w, None, out, ws, residual=residual)
    return out, offsets, dest, y


@pytest.mark.parametrize("size", LAYERS, ids=str)
def test_gate_route_and_layer(size):
    """gate -> group-limited route -> layer, as a model runs them: the layer gives the bits of
    the calls one by one, and those are right."""
    T, H, E, k, I, act, G, tg = size
    d = layer_inputs(T, H, E, k, I, act, 31)
    shape, router = N.make_shape(T, H, E, k, I, act=ACT[act]), N.make_router(groups=G, topk_groups=tg, scale=2.5)
    ws = guarded_workspace(shape)
    logits, w = torch.empty((T, E), device=dev()), torch.empty((T, k), device=dev())
    ids = torch.empty((T, k), dtype=I32, device=dev())
    N.moe_gate(shape, d["x"], d["w_gate"], logits, ws.t)
    N.moe_route_grouped(shape, router, logits, d["bias"], ids, w, ws.t)
    out = Guarded((T, H), BF16)
    N.moe_layer_fp8_block(shape, None, ids, w, d["x"], d["w13"], d["w13_scale"], d["w2"], d["w2_scale"], out.t, ws.t,
                          residual=d["residual"])
    assert N.moe_status_read(ws.t) == N.MOE_OK and ws.intact() and out.intact()
    want, want_w = ref.route(logits.cpu(), d["bias"].cpu(), k, False, G, tg, 2, True, 2.5)
    assert torch.equal(ids.cpu().long(), want)
    assert ((w.cpu().to(D) - want_w).abs() <= ref.W_REL * want_w).all()
    by_calls, offsets, dest, y = stages(shape, d, ids, w, d["residual"], ws.t)
    assert torch.equal(out.t.view(torch.int16), by_calls.view(torch.int16))
    # the rows' outputs from the definitions, then the combine's own rounding
    xq, xs = ref.quantize(d["x"])
    src = torch.empty_like(dest)
    src[dest.long()] = torch.arange(T * k, dtype=I32, device=dev()) // k
    codes = xq[src.long()].to(F32).to(ref.E4M3).view(U8)
    h, off = ref.up(codes, xs[src.long()], offsets.tolist(), d["w13"], d["w13_scale"], act == "swiglu")
    hq, hs = ref.quantize(h)
    ref_y, y_off = ref.down(hq.to(F32).to(ref.E4M3).view(U8), hs, offsets.tolist(), d["w2"], d["w2_scale"])
    # codes of h next to a border may go either way: a step (2^-3) on the few that do.  At most
    # half of it on every element at once would be sqrt-summed; the row norm is what is bounded.
    rel = (y.to(D) - ref_y).norm() / ref_y.norm()
    assert rel <= 2.0 ** -8 + 1e-3, float(rel)
    mix = (w.to(D).unsqueeze(2) * y.to(D)[dest.long()].view(T, k, H)).sum(1) + d["residual"].to(D)
    mag = (w.to(D).unsqueeze(2) * y.to(D)[dest.long()].view(T, k, H).abs()).sum(1) + d["residual"].to(D).abs()
    over = (out.t.to(D) - mix).abs() - (ref.U_BF16 * mix.abs() + ref.sum_bound(k + 1, mag))
    assert (over <= 0).all()


def test_layer_routes_logits_and_repeats_in_a_graph():
    """Softmax routing inside the layer; captured on a side stream, the batch replaced, replayed."""
    T, H, E, k, I = 48, 272, 16, 4, 144
    d = layer_inputs(T, H, E, k, I, "swiglu", 5)
    shape = N.make_shape(T, H, E, k, I)
    ws = N.workspace(shape, dev())
    logits, out = torch.randn(T, E, generator=gen(6), device=dev()), torch.empty((T, H), dtype=BF16, device=dev())

    def call():
        N.moe_layer_fp8_block(shape, logits, None, None, d["x"], d["w13"], d["w13_scale"], d["w2"], d["w2_scale"], out, ws)

    def expected():
        ids, w = torch.empty((T, k), dtype=I32, device=dev()), torch.empty((T, k), device=dev())
        ws2 = N.workspace(shape, dev())
        N.moe_route(shape, logits, ids, w, ws2)
        return stages(shape, d, ids, w, None, ws2)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(out.view(torch.int16), expected().view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for seed in (7, 8):
        d["x"].copy_(torch.randn(T, H, generator=gen(seed), device=dev()))
        logits.copy_(torch.randn(T, E, generator=gen(seed + 10), device=dev()))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), expected().view(torch.int16))
    assert N.moe_status_read(ws) == N.MOE_OK


def test_layer_over_capacity_leaves_out_as_it_was():
    T, H, E, k, I = 100, 128, 4, 1, 64
    d = layer_inputs(T, H, E, k, I, "swiglu", 9)
    shape = N.make_shape(T, H, E, k, I, capacity=50)
    ids, w = torch.zeros((T, k), dtype=I32, device=dev()), torch.ones((T, k), device=dev())
    out = torch.full((T, H), 3.0, dtype=BF16, device=dev())
    ws = N.workspace(shape, dev())
    args = (shape, None, ids, w, d["x"], d["w13"], d["w13_scale"], d["w2"], d["w2_scale"], out, ws)
    N.moe_layer_fp8_block(*args)
    assert N.moe_status_read(ws) == N.MOE_ERR_CAPACITY and torch.all(out == 3)
    ids[60:] = 2                                                 # the same workspace afterwards
    ids[50:60] = 1
    N.moe_layer_fp8_block(*args)
    assert N.moe_status_read(ws) == N.MOE_OK and not torch.any(torch.all(out == 3, 1))


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("size", [(1, 1024, 240, 9, 400), (5, 272, 7, 4, 144), (10, 128, 64, 32, 128), (64, 144, 1024, 5, 64),
                                  (11, 128, 64, 32, 128)], ids=str)
def test_small_layer_with_repeated_and_invalid_ids(size, act):
    """Up to 320 pairs the up projection counts its buckets from the ids: as the dispatch does,
    over capacity, and on one workspace with calls before."""
    T, H, E, k, I = size
    d = layer_inputs(T, H, E, k, I, act, 11)
    kind = N.MOE_ACT_SWIGLU if act == "swiglu" else N.MOE_ACT_RELU2
    shape, tight = N.make_shape(T, H, E, k, I, kind), N.make_shape(T, H, E, k, I, kind, capacity=1)
    ws, ws2 = guarded_workspace(shape), N.workspace(shape, dev())
    w = torch.rand(T, k, generator=gen(12), device=dev())
    out = torch.empty((T, H), dtype=BF16, device=dev())
    g = torch.Generator().manual_seed(13)
    for round_ in range(3):
        ids = torch.randint(-1, E + 1, (T, k), generator=g, dtype=I32)
        if round_ == 2:
            ids[:, 0] = E - 1                                    # a bucket of all tokens
            ids[0] = E - 1
        ids = ids.to(dev())
        call = lambda s: N.moe_layer_fp8_block(s, None, ids, w, d["x"], d["w13"], d["w13_scale"], d["w2"], d["w2_scale"],
                                               out, ws.t)
        call(shape)
        status = N.moe_status_read(ws.t)
        assert torch.equal(out.view(torch.int16), stages(shape, d, ids, w, None, ws2)[0].view(torch.int16)) and ws.intact()
        assert status == N.moe_status_read(ws2)
        if round_ == 2 and T > 1:
            out.fill_(3.0)
            call(tight)
            assert N.moe_status_read(ws.t) != N.MOE_OK and torch.all(out == 3) and ws.intact()


def test_small_layer_takes_weights_and_ids_written_just_before():
    """The layer's kernels start while earlier ones run: what those write is seen all the same."""
    T, H, E, k, I = 2, 1024, 16, 3, 512
    d = layer_inputs(T, H, E, k, I, "relu2", 14)
    shape = N.make_shape(T, H, E, k, I, N.MOE_ACT_RELU2)
    ws, w = N.workspace(shape, dev()), torch.ones((T, k), device=dev())
    sets, want = [], []
    for i in range(2):
        e = layer_inputs(T, H, E, k, I, "relu2", 15 + i)
        ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i))[:k] for _ in range(T)]).to(I32).to(dev())
        sets.append((e["w13"], e["w2"], ids))
        want.append(stages(shape, dict(d, w13=e["w13"], w2=e["w2"]), ids, w, None, ws)[0])
    w13, w2, ids = (t.clone() for t in sets[0])
    outs = [torch.empty((T, H), dtype=BF16, device=dev()) for _ in range(60)]
    for i, out in enumerate(outs):
        for a, b in zip((w13, w2, ids), sets[i % 2]):
            a.copy_(b)
        N.moe_layer_fp8_block(shape, None, ids, w, d["x"], w13, d["w13_scale"], w2, d["w2_scale"], out, ws)
    assert N.moe_status_read(ws) == N.MOE_OK
    for i, out in enumerate(outs):
        assert torch.equal(out.view(torch.int16), want[i % 2].view(torch.int16)), i
