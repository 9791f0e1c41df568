"""Plain 64-bit forms of group-limited routing and of the block-scaled FP8 expert path,
for the tests: each straight from its definition, sharing no code with the library.  The
bounds say, element by element, how far FP32 sums and the output's rounding may be off."""
import torch

from train_ref import U_BF16, U_F32, sum_bound

D, F32, U8, E4M3 = torch.float64, torch.float32, torch.uint8, torch.float8_e4m3fn
U_E4M3 = 2.0 ** -4          # half a step of a normal E4M3 value, relatively
STEP_E4M3 = 2.0 ** -10      # half a step of a subnormal one


def blocks(n):
    return (n + 127) // 128


def nearest_e4m3(v):
    """The E4M3 value nearest v, ties to even, |v| at most 448 afterwards (64 bits)."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def quantize(x):
    """(code values, scales in FP32) of rows; a block with a NaN or an infinity is NaN throughout."""
    x = x.to(D)
    codes, scales = torch.empty_like(x), []
    for c in range(0, x.shape[1], 128):
        b = x[:, c:c + 128]
        a = b.abs().amax(1, keepdim=True).clamp(min=2.0 ** -100)
        a = torch.where(torch.isfinite(b).all(1, keepdim=True), a, torch.full_like(a, float("nan")))
        codes[:, c:c + 128] = nearest_e4m3(b * 448.0 / a)
        scales.append((a / 448.0).to(F32))
    return codes, torch.cat(scales, 1)


def values(codes):
    """The values of E4M3 code bytes, in 64 bits."""
    return codes.view(E4M3).to(F32).to(D)


def spread_rows(scale, n):
    return scale.to(D).repeat_interleave(128, 0)[:n]


def spread_cols(scale, n):
    return scale.to(D).repeat_interleave(128, -1)[..., :n]


def random_weights(g, lead, rows, cols, device):
    """Random codes (no NaN) and scales that differ from block to block, values of about 1 / sqrt(cols)."""
    codes = torch.randint(0, 256, (*lead, rows, cols), generator=g, device=device, dtype=torch.int32).to(U8)
    codes[(codes & 127) == 127] = 0
    scale = torch.exp2(4.0 * torch.rand((*lead, blocks(rows), blocks(cols)), generator=g, device=device) - 2.0)
    return codes, scale / (128.0 * cols ** 0.5)


def product(a, w, w_scale):
    """(a w^T, |a| |w|^T) for rows a in 64 bits and coded weights."""
    wd = values(w) * spread_cols(spread_rows(w_scale, w.shape[0]), w.shape[1])
    return a @ wd.t(), a.abs() @ wd.abs().t()


def up(x, x_scale, bounds, w13, w13_scale, swiglu):
    """(h, bound on h before quantization) of the routed rows."""
    a = values(x) * spread_cols(x_scale, x.shape[1])
    h = torch.zeros((x.shape[0], w13.shape[2]), dtype=D, device=x.device)
    off = torch.zeros_like(h)
    K = x.shape[1]
    for e in range(w13.shape[0]):
        r = slice(bounds[e], bounds[e + 1])
        if r.start == r.stop:
            continue
        p, mag = product(a[r], w13[e, 0], w13_scale[e, 0])
        dp = sum_bound(K, mag)
        if swiglu:
            u, umag = product(a[r], w13[e, 1], w13_scale[e, 1])
            du = sum_bound(K, umag)
            s = p * torch.sigmoid(p)
            h[r] = s * u
            # |silu'| <= 1.1; the exponential's argument is rounded, then exp, division, two products
            off[r] = 1.1 * dp * (u.abs() + du) + s.abs() * du + (2 * p.abs() + 16) * U_F32 * h[r].abs()
        else:
            h[r] = torch.where(p > 0, p * p, torch.zeros_like(p))
            off[r] = 2 * p.abs() * dp + dp * dp + 2 * U_F32 * h[r]
    return h, off


def check_quantized(codes, scale, h, off, what):
    """Codes and scales against the values h, each known to `off`: half a step of the code, and `off`."""
    nb = blocks(h.shape[1])
    pad = lambda t: torch.nn.functional.pad(t, (0, nb * 128 - h.shape[1])).view(h.shape[0], nb, 128)
    amax, worst = pad(h.abs()).amax(2), pad(off).amax(2)
    want = amax.clamp(min=2.0 ** -100) / 448.0
    over = (scale.to(D) - want).abs() - (worst / 448.0 + 2 * U_F32 * want)
    assert (over <= 0).all(), f"{what}: scales off by {over.max():.3e}"
    s = spread_cols(scale, h.shape[1])
    got = values(codes) * s
    over = (got - h).abs() - (U_E4M3 * (h.abs() + off) + STEP_E4M3 * s + off + 8 * U_F32 * h.abs())
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} codes outside, worst by {over.max():.3e}"


def down(h, h_scale, bounds, w2, w2_scale):
    """(y, bound) of the routed rows."""
    a = values(h) * spread_cols(h_scale, h.shape[1])
    y = torch.zeros((h.shape[0], w2.shape[1]), dtype=D, device=h.device)
    off = torch.zeros_like(y)
    for e in range(w2.shape[0]):
        r = slice(bounds[e], bounds[e + 1])
        if r.start != r.stop:
            y[r], mag = product(a[r], w2[e], w2_scale[e])
            off[r] = sum_bound(h.shape[1], mag) + U_BF16 * y[r].abs()
    return y, off


# ---- routing -------------------------------------------------------------------
def scores(logits, softmax):
    l = logits.to(D)
    return torch.softmax(l, 1) if softmax else 1.0 / (1.0 + torch.exp(-l))


def route(logits, bias, k, softmax, groups, topk_groups, group_top, renorm, scale):
    """(ids, weights): a token at a time, by sorting (key, index) pairs."""
    s = scores(logits, softmax)
    key = s.to(F32) + (bias if bias is not None else torch.zeros(logits.shape[1]))
    T, E = logits.shape
    n = E // groups
    ids = torch.empty((T, k), dtype=torch.int64)
    keys = key.tolist()
    for t in range(T):
        row = keys[t]
        value = []
        for g in range(groups):
            top = sorted(row[g * n:(g + 1) * n], reverse=True)[:group_top]
            value.append(float((torch.tensor(top[0], dtype=F32) + torch.tensor(top[1], dtype=F32)))
                         if len(top) == 2 else top[0])
        held = sorted(range(groups), key=lambda g: (-value[g], g))[:topk_groups]
        pool = [e for g in held for e in range(g * n, (g + 1) * n)]
        ids[t] = torch.tensor(sorted(pool, key=lambda e: (-row[e], e))[:k])
    return ids, weights(logits, ids, softmax, renorm, scale)


def weights(logits, ids, softmax, renorm, scale):
    """Weights of a selection; renormalised ones through log scores, which do not underflow."""
    l = logits.to(D)
    # renormalised softmax weights: the normaliser over all experts drops out (and with it
    # gradients of 1e-19 for the others, where there are none)
    log = torch.nn.functional.logsigmoid(l) if not softmax else l if renorm else torch.log_softmax(l, 1)
    sel = torch.gather(log, 1, ids.long())
    return scale * (torch.softmax(sel, 1) if renorm else torch.exp(sel))


# Relative: 1024 terms of a sum, exponents of up to 127 rounded to FP32, a few operations.
W_REL = 2.0 ** -17
W_ABS = 2.0 ** -120        # where FP32 leaves its normal range


def route_backward(logits, ids, dw, softmax, renorm, scale):
    """(dlogits, magnitude): autograd on the 64-bit weights, and what its terms amount to."""
    l = logits.to(D).clone().requires_grad_()
    w = weights(l, ids, softmax, renorm, scale)
    d = torch.autograd.grad((w * dw.to(D)).sum(), l)[0]
    w = w.detach()
    mean = (w.abs() * dw.to(D).abs()).sum(1, keepdim=True) / (abs(scale) if renorm else 1.0)
    mag = torch.zeros_like(d).scatter(1, ids.long(), w.abs() * (dw.to(D).abs() + (mean if renorm else 0.0)))
    s = scores(logits, softmax)
    if softmax and not renorm:
        mag += s * mean
    elif not softmax:
        mag *= torch.sigmoid(-l.detach())        # 1 - s, which is 0 in 64 bits from l = 37 on if subtracted
    return d, mag
