"""The block-scaled weights of synth.py: scales by blocks and codes within half a step, on the CPU."""
import pytest
import torch

from fp8_ref import blocks, spread_cols, spread_rows, values
from mixture_experts_routing_router_gb300 import synth


@pytest.mark.parametrize("rows,cols", [(1, 16), (128, 128), (129, 144), (200, 272)])
def test_codes_are_within_half_a_step(rows, cols):
    g = torch.Generator().manual_seed(rows)
    w = torch.randn(2, rows, cols, generator=g) * 0.02
    w[1, :128, :128] = 0.0
    codes, scale = synth.quantize_blocks_fp8(w)
    assert codes.dtype == torch.uint8 and codes.shape == w.shape
    assert scale.dtype == torch.float32 and scale.shape == (2, blocks(rows), blocks(cols))
    assert scale[1, 0, 0] == 1.0 and not codes[1, :128, :128].any()
    for i in range(2):
        s = spread_cols(spread_rows(scale[i], rows), cols)
        v, want = values(codes[i]) * s, w[i].double()
        # half a step is 2^-4 of a value from 2^-6 up and 2^-10 below (before the scale); scale and
        # w / scale are rounded to FP32 first, which can move the value by 2^-23 of itself or so and
        # the largest one, 448, not at all beyond the clamp
        assert ((v - want).abs() <= 2.0 ** -4 * (1 + 2.0 ** -18) * want.abs() + 2.0 ** -10 * s).all()
        for b in range(scale.shape[1]):
            for c in range(scale.shape[2]):
                part = want[128 * b:128 * b + 128, 128 * c:128 * c + 128].abs().max()
                if part > 0:
                    assert abs(scale[i, b, c].item() * 448.0 - part) <= 2.0 ** -23 * part


def test_expert_weights_have_a_grid_per_matrix():
    wl = synth.Workload("small", 4, 144, 3, 2, 80)
    d = synth.make_fp8_block_weights(wl)
    assert d["w13"].shape == (3, 160, 144) and d["s13"].shape == (3, 2, 1, 2)
    assert d["w2"].shape == (3, 144, 80) and d["s2"].shape == (3, 2, 1)
    a, b = synth.expert_weights(wl, 2)
    # half a step is at most 2^-4 of a value, and less than 2^-4 of the largest below that
    up = values(d["w13"][2, 80:]) * spread_cols(spread_rows(d["s13"][2, 1], 80), 144)
    assert (up - a[80:].double()).abs().max() <= 2.0 ** -4 * a.abs().max().double()
    down = values(d["w2"][2]) * spread_cols(spread_rows(d["s2"][2], 144), 80)
    assert (down - b.double()).abs().max() <= 2.0 ** -4 * b.abs().max().double()


@pytest.mark.parametrize("amax", [2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 2.0 ** -118, 2.0 ** -117])
def test_blocks_of_tiny_weights(amax):
    """Largest values at which max / 448 is below FP32's normal range, zeros among them."""
    w = torch.zeros(130, 144)
    w[0, 0], w[5, 7], w[129, 143] = amax, -0.75 * amax, 0.5 * amax
    codes, scale = synth.quantize_blocks_fp8(w)
    v = values(codes) * spread_cols(spread_rows(scale, 130), 144)
    s = spread_cols(spread_rows(scale, 130), 144)
    assert ((v - w.double()).abs() <= 2.0 ** -4 * (1 + 2.0 ** -18) * w.double().abs() + 2.0 ** -10 * s).all()
    assert not codes[w == 0].any()
