"""Plain 64-bit forms of the training operators, for the tests: each one straight
from its formula, on whatever device its inputs are, sharing no code with the
library.  The ``*_bound`` functions give, element by element, how far a result
with FP32 sums and the stated output type may be from the 64-bit value."""
import torch

D = torch.float64
U_BF16 = 2.0 ** -8        # a bf16 rounding moves a value by at most half of this, relatively
U_F32 = 2.0 ** -23


def out_unit(dtype):
    return U_BF16 if dtype == torch.bfloat16 else U_F32


def sum_bound(n, mag):
    """FP32 sum of n products of total magnitude `mag`, in any order with at most
    n/8 + 8 dependent additions (tensor-core slices, shuffles, chunked loops)."""
    return (n / 8 + 8) * U_F32 * mag


# ---- layer norm ---------------------------------------------------------------
def layernorm(x, gamma, beta, eps):
    x = x.to(D)
    mu = x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    return (x - mu) * rstd * gamma.to(D) + beta.to(D), mu.squeeze(-1), rstd.squeeze(-1)


def layernorm_bound(x, gamma, beta, eps, dtype):
    """mean: a sum's error over H; rstd: relative; y: both carried through, plus the rounding."""
    H = x.shape[-1]
    xd, g, b = x.to(D), gamma.to(D).abs(), beta.to(D).abs()
    y, mu, rstd = layernorm(x, gamma, beta, eps)
    c = (xd - mu.unsqueeze(-1)).abs()
    e_mu = sum_bound(H, xd.abs().sum(-1)) / H + U_F32 * mu.abs()
    # var's error: the sum's, and the mean's error squared (its linear part cancels)
    var = (c * c).mean(-1)
    e_var = sum_bound(H, var * H) / H + 4 * U_F32 * var + e_mu ** 2 + 2 * e_mu * U_F32 * c.amax(-1)
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 4 * U_F32)
    r = rstd.unsqueeze(-1)
    e_y = g * (e_mu.unsqueeze(-1) * r + c * e_rstd.unsqueeze(-1) + 4 * U_F32 * (c + U_F32 * xd.abs()) * r) \
        + 2 * U_F32 * b + out_unit(dtype) * y.abs()
    return e_y, e_mu, e_rstd


def layernorm_backward(dy, x, gamma, mean, rstd, dres=None):
    dy, x, g = dy.to(D), x.to(D), gamma.to(D)
    xh = (x - mean.to(D).unsqueeze(-1)) * rstd.to(D).unsqueeze(-1)
    a = dy * g
    dx = rstd.to(D).unsqueeze(-1) * (a - a.mean(-1, keepdim=True) - xh * (a * xh).mean(-1, keepdim=True))
    if dres is not None:
        dx = dx + dres.to(D)
    flat = (dy * xh).reshape(-1, x.shape[-1]), dy.reshape(-1, x.shape[-1])
    return dx, flat[0].sum(0), flat[1].sum(0)


def layernorm_backward_bound(dy, x, gamma, mean, rstd, dres, dtype):
    H = x.shape[-1]
    dyd, xd, g = dy.to(D), x.to(D), gamma.to(D)
    mu, r = mean.to(D).unsqueeze(-1), rstd.to(D).unsqueeze(-1)
    xh = (xd - mu) * r
    e_xh = 3 * U_F32 * ((xd - mu).abs() + U_F32 * xd.abs()) * r      # per element, FP32
    a = (dyd * g).abs()
    ma = a.mean(-1, keepdim=True)
    mb = (a * xh.abs()).mean(-1, keepdim=True)
    e_ma = sum_bound(H, a.sum(-1, keepdim=True)) / H + 2 * U_F32 * ma
    e_mb = sum_bound(H, (a * xh.abs()).sum(-1, keepdim=True)) / H + 2 * U_F32 * mb + (a * e_xh).mean(-1, keepdim=True)
    dx = layernorm_backward(dy, x, gamma, mean, rstd, dres)[0]
    mag = a + ma + xh.abs() * mb
    e_dx = r * (4 * U_F32 * mag + e_ma + xh.abs() * e_mb + e_xh * mb) + out_unit(dtype) * dx.abs()
    if dres is not None:
        e_dx = e_dx + 2 * U_F32 * (dres.to(D).abs() + r * mag)
    rows = dyd.reshape(-1, H).shape[0]
    e_g = sum_bound(rows, (dyd * xh).abs().reshape(-1, H).sum(0)) + (dyd.abs() * e_xh).reshape(-1, H).sum(0)
    e_b = sum_bound(rows, dyd.abs().reshape(-1, H).sum(0))
    return e_dx, e_g, e_b


# ---- routes ---------------------------------------------------------------------
def dispatch(ids, E):
    """(dest [T, k], offsets [E+1]) of the stable expert-contiguous order; -1 for an
    invalid pair (out of range, or repeated inside its token)."""
    T, k = ids.shape
    rows = ids.tolist()
    buckets = [[] for _ in range(E)]
    dest = torch.full((T * k,), -1, dtype=torch.int32)
    for t, row in enumerate(rows):
        for j, e in enumerate(row):
            if 0 <= e < E and e not in row[:j]:
                buckets[e].append(t * k + j)
    offsets, at = [0], 0
    for b in buckets:
        for p in b:
            dest[p] = at
            at += 1
        offsets.append(at)
    return dest.view(T, k), torch.tensor(offsets, dtype=torch.int32)


def combine_backward(dout, y_perm, dest, w):
    """(slots written, their dy rows, dw [T, k])"""
    T, k = w.shape
    p = torch.nonzero(dest.reshape(-1) >= 0).squeeze(1)
    slot, tok = dest.reshape(-1)[p].long(), p // k
    dy = dout[tok].to(D) * w.reshape(-1)[p].to(D).unsqueeze(1)
    dw = torch.zeros(T * k, dtype=D, device=w.device)
    dw[p] = (dout[tok].to(D) * y_perm[slot].to(D)).sum(1)
    mag = torch.zeros(T * k, dtype=D, device=w.device)
    mag[p] = (dout[tok].to(D) * y_perm[slot].to(D)).abs().sum(1)
    return slot, dy, dw.view(T, k), mag.view(T, k)


def dispatch_backward(dx_perm, dest, add):
    T, k = dest.shape
    out = torch.zeros(T, dx_perm.shape[1], dtype=D, device=dx_perm.device)
    mag = torch.zeros_like(out)
    for j in range(k):
        ok = dest[:, j] >= 0
        rows = dx_perm[dest[ok, j].long()].to(D)
        out[ok] += rows
        mag[ok] += rows.abs()
    if add is not None:
        out = out + add.to(D)
        mag = mag + add.to(D).abs()
    return out, mag


def route_backward(ids, w, dw, E):
    w, dw = w.to(D), dw.to(D)
    out = torch.zeros(w.shape[0], E, dtype=D, device=w.device)
    out.scatter_(1, ids.long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return out


def route_sigmoid_weights(logits, ids, scale):
    s = torch.sigmoid(torch.gather(logits.to(D), 1, ids.long()))
    return scale * s / s.sum(1, keepdim=True)


def route_sigmoid_backward(logits, ids, scale, dw):
    l = torch.gather(logits.to(D), 1, ids.long())
    s = torch.sigmoid(l)
    p = s / s.sum(1, keepdim=True)
    out = torch.zeros(logits.shape, dtype=D, device=logits.device)
    out.scatter_(1, ids.long(), scale * p * torch.sigmoid(-l) * (dw.to(D) - (p * dw.to(D)).sum(1, keepdim=True)))
    return out


# ---- expert FFN -------------------------------------------------------------------
def act(pre, glu):
    if glu:
        g, u = pre.chunk(2, 1)
        return g * torch.sigmoid(g) * u
    return torch.clamp(pre, min=0.0) ** 2


def act_backward(pre, dh, glu):
    if glu:
        g, u = pre.chunk(2, 1)
        s = torch.sigmoid(g)
        return torch.cat([dh * u * (s + g * s * (1 - s)), dh * g * s], 1)
    return dh * 2 * torch.clamp(pre, min=0.0)


def rows_times(a, offsets, w, transpose):
    """C[r] = a[r] w[e] (or a[r] w[e]^T) and the products' magnitude, over the valid rows."""
    b = offsets.tolist()
    n = w.shape[1] if transpose else w.shape[2]
    c = torch.zeros(a.shape[0], n, dtype=D, device=a.device)
    mag = torch.zeros_like(c)
    for e in range(len(b) - 1):
        if b[e + 1] > b[e]:
            x, m = a[b[e]:b[e + 1]].to(D), w[e].to(D)
            m = m.t() if transpose else m
            c[b[e]:b[e + 1]] = x @ m
            mag[b[e]:b[e + 1]] = x.abs() @ m.abs()
    return c, mag


def weights_grad(a, b, offsets):
    o = offsets.tolist()
    E = len(o) - 1
    c = torch.zeros(E, a.shape[1], b.shape[1], dtype=D, device=a.device)
    mag = torch.zeros_like(c)
    for e in range(E):
        if o[e + 1] > o[e]:
            x, y = a[o[e]:o[e + 1]].to(D), b[o[e]:o[e + 1]].to(D)
            c[e] = x.t() @ y
            mag[e] = x.abs().t() @ y.abs()
    return c, mag
