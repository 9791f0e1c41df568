"""Cases for timing group-limited routing and the block-scaled FP8 expert path.

A layer that serves or trains with many experts limits each token to a few groups of
experts: scores (sigmoid or softmax), a bias that only selects, the best groups, the
best experts inside them, weights from the unbiased scores; and its gradient.  Its
experts' products run in 8-bit floating point: activations in E4M3 with an FP32 scale
per row and 128 columns, weights in E4M3 with an FP32 scale per 128 x 128 block, the
dispatch quantizing the rows it moves and the up projection the activations it writes.
Each case below is one of these operators, or the routed layer made of them, at sizes
of this repository's workloads (or generic odd ones).

``own`` selects what ``run`` does: False computes the operators with elementary
torch operations in 32 bits, rounded once at the end (the selection's scores in 64:
values next to a border decide which expert a token takes); True calls the library.
"""
import math

import torch

own = False

BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
BLOCK = 128                   # columns of an activation scale, rows and columns of a weight scale
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100      # a block of zeros (or of nothing larger) keeps a normal scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _route(op, tokens, experts, top_k, groups, topk_groups, score, renorm, group_top=2):
    return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, groups=groups, topk_groups=topk_groups,
                score=score, renorm=renorm, group_top=group_top)


def _dispatch(tokens, hidden, experts, top_k, zipf=False):
    return dict(op="dispatch_fp8", tokens=tokens, hidden=hidden, experts=experts, top_k=top_k, zipf=zipf)


def _ffn(tokens, hidden, experts, top_k, inter, act, zipf=False):
    return dict(op="expert_ffn_fp8", tokens=tokens, hidden=hidden, experts=experts, top_k=top_k, inter=inter, act=act,
                zipf=zipf)


def _layer(tokens, hidden, experts, top_k, inter, act, groups, topk_groups):
    return dict(op="layer_fp8", tokens=tokens, hidden=hidden, experts=experts, top_k=top_k, inter=inter, act=act,
                groups=groups, topk_groups=topk_groups, score="sigmoid", renorm=True, group_top=2)


def listed():
    return [
        # one decoded token's route: pure latency
        dict(name="route_decode", **_route("route_grouped", 1, 256, 8, 8, 4, "sigmoid", True)),
        # softmax scores, groups by their best expert, weights left as they are, an odd batch
        dict(name="route_softmax_mid", **_route("route_grouped", 1023, 160, 6, 8, 3, "softmax", False, 1)),
        # the large layer's batch
        dict(name="route_large", **_route("route_grouped", 16384, 256, 8, 8, 4, "sigmoid", True)),
        # the gradient that reaches every expert's logit (softmax over all of them), an odd batch
        dict(name="route_backward_softmax_mid",
             **_route("route_grouped_backward", 1023, 160, 6, 8, 3, "softmax", False, 1)),
        # the large layer's gradient
        dict(name="route_backward_large", **_route("route_grouped_backward", 16384, 256, 8, 8, 4, "sigmoid", True)),
        # 1024 tokens to 6 of 64 experts, quantized on the way
        dict(name="dispatch_mid", **_dispatch(1024, 2048, 64, 6)),
        # the large layer's dispatch with its skewed (hot-expert) routes
        dict(name="dispatch_large", **_dispatch(16384, 7168, 256, 8, zipf=True)),
        # decode: 8 tokens to 9 of 240 squared-ReLU experts, weights streamed for a row or two each
        dict(name="ffn_decode", **_ffn(8, 1024, 240, 9, 1536, "relu2")),
        # 1024 tokens to 6 of 64 experts, SwiGLU: about 96 rows an expert
        dict(name="ffn_mid", **_ffn(1024, 2048, 64, 6, 1408, "swiglu")),
        # the large layer's hidden and intermediate sizes over 32 experts, skewed routes: tensor-bound
        dict(name="ffn_large", **_ffn(4096, 7168, 32, 8, 2048, "swiglu", zipf=True)),
        # one decoded token through route and layer: latency and one token's experts
        dict(name="layer_decode", **_layer(1, 1024, 240, 9, 1536, "relu2", 8, 4)),
        # 2048 tokens to 8 of 128 experts through route and layer
        dict(name="layer_prefill", **_layer(2048, 2048, 128, 8, 768, "swiglu", 8, 4)),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_groups(rng, most):
    """(experts, top_k, groups, topk_groups): equal groups, enough experts in the chosen ones."""
    groups = rng.choice([1, 2, 3, 4, 8, 8, 16])
    experts = groups * max(1, _logu(rng, 4, most) // groups)
    topk_groups = rng.randint(1, groups)
    top_k = rng.randint(1, min(16, topk_groups * (experts // groups)))
    return experts, top_k, groups, topk_groups


def draw(rng):
    op = rng.choice(["route_grouped", "route_grouped_backward", "dispatch_fp8", "expert_ffn_fp8", "expert_ffn_fp8",
                     "layer_fp8"])
    if op.startswith("route"):
        experts, top_k, groups, topk_groups = _draw_groups(rng, 256)
        return _route(op, _logu(rng, 1, 16384), experts, top_k, groups, topk_groups,
                      rng.choice(["sigmoid", "softmax"]), rng.random() < 0.5, rng.choice([1, 2]))
    if op == "dispatch_fp8":
        experts = _logu(rng, 2, 256)
        return _dispatch(_logu(rng, 1, 16384), 16 * _logu(rng, 2, 448), experts, rng.randint(1, min(8, experts)),
                         zipf=rng.random() < 0.5)
    while True:
        act = rng.choice(["swiglu", "relu2"])
        tokens, hidden, inter = _logu(rng, 1, 4096), 16 * _logu(rng, 2, 448), 16 * _logu(rng, 2, 128)
        if op == "layer_fp8":
            experts, top_k, groups, topk_groups = _draw_groups(rng, 240)
            case = _layer(tokens, hidden, experts, min(top_k, 9), inter, act, groups, topk_groups)
        else:
            experts = _logu(rng, 1, 240)
            case = _ffn(tokens, hidden, experts, rng.randint(1, min(9, experts)), inter, act, zipf=rng.random() < 0.5)
        if experts * hidden * inter <= 32 * 7168 * 2048 and \
                tokens * case["top_k"] * hidden * inter <= 4096 * 8 * 7168 * 2048:
            return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _weights(g, lead, rows, cols):
    """E4M3 weights [*lead, rows, cols] of N(0, 1/cols) and the scale of each 128 x 128 block."""
    n = math.prod(lead)
    codes = torch.empty((n, rows, cols), dtype=E4M3, device="cuda")
    scale = torch.empty((n, _blocks(rows), _blocks(cols)), device="cuda")
    R, C = _blocks(rows) * BLOCK, _blocks(cols) * BLOCK
    step = max(1, (1 << 27) // (R * C))
    for i in range(0, n, step):
        m = min(n, i + step) - i
        w = torch.zeros((m, R, C), device="cuda")
        w[:, :rows, :cols] = torch.randn((m, rows, cols), generator=g, device="cuda") / math.sqrt(cols)
        t = w.view(m, R // BLOCK, BLOCK, C // BLOCK, BLOCK)
        s = t.abs().amax((2, 4)) / E4M3_MAX
        scale[i:i + m] = s
        codes[i:i + m] = (t / s[:, :, None, :, None]).view(m, R, C)[:, :rows, :cols].to(E4M3)
    return codes.view(*lead, rows, cols), scale.view(*lead, *scale.shape[1:])


def _experts(d, case, g):
    E, H, I = case["experts"], case["hidden"], case["inter"]
    parts = 2 if case["act"] == "swiglu" else 1          # gate and up, each with its own blocks
    d["w13"], d["w13_scale"] = _weights(g, (E, parts), I, H)
    d["w2"], d["w2_scale"] = _weights(g, (E,), H, I)


def _routes(case, g):
    """Distinct experts per token and the stable expert-contiguous order."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    logits = torch.randn((T, E), generator=g, device="cuda", dtype=F32)
    if case["zipf"]:
        rank = torch.argsort(torch.rand(E, generator=g, device="cuda"))
        logits -= 1.2 * torch.log(rank.float() + 1.0)
    ids = torch.topk(logits, k, dim=1).indices
    flat = ids.reshape(-1)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    return dict(ids=ids.to(torch.int32), offsets=offsets.to(torch.int32), bounds=offsets.tolist())


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T, E, k = case["op"], case["tokens"], case["experts"], case["top_k"]
    d = {}
    if op in ("route_grouped", "layer_fp8"):
        d["logits"] = torch.randn((T, E), generator=g, device="cuda")
        d["bias"] = 0.05 * torch.randn(E, generator=g, device="cuda") * (1.0 if case["score"] == "sigmoid" else 0.1)
        d["scale"] = 2.5
    if op == "layer_fp8":
        d["x"] = _randn(g, (T, case["hidden"]))
        _experts(d, case, g)
    elif op == "route_grouped_backward":
        d["logits"] = torch.randn((T, E), generator=g, device="cuda")
        d["scale"] = 2.5
        # the route's choice is its input here: the best experts of randomly chosen groups
        G, n = case["groups"], E // case["groups"]
        keep = torch.topk(torch.rand((T, G), generator=g, device="cuda"), case["topk_groups"], dim=1).indices
        held = torch.zeros((T, G), device="cuda", dtype=torch.bool).scatter_(1, keep, True)
        key = d["logits"].masked_fill(~held.repeat_interleave(n, 1), -math.inf)
        d["ids"] = torch.topk(key, k, dim=1).indices.to(torch.int32)
        d["dw"] = torch.randn((T, k), generator=g, device="cuda")
    elif op == "dispatch_fp8":
        H = case["hidden"]
        d.update(_routes(case, g))
        # a normalised residual stream: a few channels larger than the rest
        d["x"] = (torch.randn((T, H), generator=g, device="cuda")
                  * (1.0 + 7.0 * (torch.rand(H, generator=g, device="cuda") < 0.01))).to(BF16)
    elif op == "expert_ffn_fp8":
        d.update(_routes(case, g))
        d["x"], d["x_scale"] = _quantize(_randn(g, (T * k, case["hidden"])).float())
        _experts(d, case, g)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = case
    if own:
        _prepare_own(case, d)
    return d


def _prepare_own(case, d):
    """The output buffers, workspace and descriptions a program keeps."""
    from mixture_experts_routing_router_gb300 import native as N
    op, T, E, k = case["op"], case["tokens"], case["experts"], case["top_k"]
    H, I, R = case.get("hidden", 16), case.get("inter", 16), T * k
    act = N.MOE_ACT_RELU2 if case.get("act") == "relu2" else N.MOE_ACT_SWIGLU
    new = lambda *s, t=F32: torch.empty(s, dtype=t, device="cuda")
    d["shape"] = N.make_shape(T, H, E, k, I, act=act)
    d["ws"] = N.workspace(d["shape"])
    if "groups" in case:
        d["router"] = N.make_router(score=N.MOE_SCORE_SOFTMAX if case["score"] == "softmax" else N.MOE_SCORE_SIGMOID,
                                    groups=case["groups"], topk_groups=case["topk_groups"],
                                    group_top=case["group_top"], renorm=case["renorm"], scale=d["scale"])
    if op in ("route_grouped", "layer_fp8"):
        d["out"] = (new(T, k, t=torch.int32), new(T, k))
    if op == "layer_fp8":
        d["out"] += (new(T, H, t=BF16),)
    elif op == "route_grouped_backward":
        d["out"] = new(T, E)
    elif op == "dispatch_fp8":
        i32 = torch.int32
        d["out"] = (new(E, t=i32), new(E + 1, t=i32), new(R, t=i32), new(R, t=i32), new(R, H, t=E4M3),
                    new(R, _blocks(H)))
    elif op == "expert_ffn_fp8":
        d["out"] = (new(R, I, t=E4M3), new(R, _blocks(I)), new(R, H, t=BF16))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


def _run_own(s):
    from mixture_experts_routing_router_gb300 import native as N
    op, out = s["case"]["op"], s["out"]
    if op == "route_grouped":
        N.moe_route_grouped(s["shape"], s["router"], s["logits"], s["bias"], *out, s["ws"])
    elif op == "route_grouped_backward":
        N.moe_route_grouped_backward(s["shape"], s["router"], s["logits"], s["ids"], s["dw"], out, s["ws"])
    elif op == "dispatch_fp8":
        N.moe_dispatch_fp8_block(s["shape"], s["x"], s["ids"], *out, s["ws"])
    elif op == "expert_ffn_fp8":
        h, h_scale, y = out
        N.moe_expert_up_fp8_block(s["shape"], s["x"], s["x_scale"], s["offsets"], s["w13"], s["w13_scale"], h,
                                  h_scale, s["ws"])
        N.moe_expert_down_fp8_block(s["shape"], h, h_scale, s["offsets"], s["w2"], s["w2_scale"], y, s["ws"])
    else:
        ids, w, y = out
        N.moe_route_grouped(s["shape"], s["router"], s["logits"], s["bias"], ids, w, s["ws"])
        N.moe_layer_fp8_block(s["shape"], None, ids, w, s["x"], s["w13"], s["w13_scale"], s["w2"], s["w2_scale"], y,
                              s["ws"])
    return out


def _scores(logits, score):
    """In 64 bits: which of two experts a token takes can hang on the last bits."""
    l = logits.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _best(key, n):
    """Indices of the n largest, descending, ties to the lower index."""
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :n]


def _plain_route(s):
    case = s["case"]
    score = _scores(s["logits"], case["score"])
    key = score.float() + s["bias"]                     # the selection's keys are 32 bits wide
    G = case["groups"]
    T, E = key.shape
    if G > 1:
        top = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
        rank = top[..., 0] + top[..., 1] if case["group_top"] == 2 and E > G else top[..., 0]
        held = torch.zeros((T, G), dtype=torch.bool, device=key.device)
        held.scatter_(1, _best(rank, case["topk_groups"]), True)
        key = torch.where(held.repeat_interleave(E // G, 1), key, torch.full_like(key, -math.inf))
    ids = _best(key, case["top_k"])
    w = torch.gather(score, 1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (s["scale"] * w).float()


def _plain_route_backward(s):
    case, ids, g = s["case"], s["ids"].long(), s["dw"]
    score = _scores(s["logits"], case["score"])
    sel = torch.gather(score, 1, ids)
    p = sel / sel.sum(1, keepdim=True) if case["renorm"] else sel
    d = torch.zeros_like(score)
    if case["score"] == "softmax":
        mean = (p * g).sum(1, keepdim=True)
        if case["renorm"]:                              # a softmax over the selection
            d.scatter_(1, ids, p * (g - mean))
        else:                                           # every logit is in the normaliser
            d = d.scatter(1, ids, p * g) - score * mean
    else:
        ds = g - (p * g).sum(1, keepdim=True) if case["renorm"] else g
        d.scatter_(1, ids, p * (1.0 - sel) * ds)
    return (s["scale"] * d).float()


def _quantize(x):
    """FP32 rows to E4M3 codes and a scale per row and 128 columns.  The code is next to
    448 x / amax, taken as (0.875 x) / (amax / 512): for a BF16 x numerator and denominator are exact."""
    R, C = x.shape
    nb = _blocks(C)
    p = torch.zeros((R, nb * BLOCK), device=x.device)
    p[:, :C] = x
    p = p.view(R, nb, BLOCK)
    amax = torch.clamp(p.abs().amax(2), min=AMAX_FLOOR)
    codes = (0.875 * p / (amax / 512.0)[:, :, None]).view(R, nb * BLOCK)[:, :C].to(E4M3)
    return codes, amax / E4M3_MAX


def _spread(scale, n, dim):
    """Each scale over its 128 rows or columns."""
    return scale.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _plain_dispatch(s):
    case = s["case"]
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    flat = s["ids"].long().reshape(-1)
    order = torch.argsort(flat, stable=True)
    dest = torch.empty_like(order)
    dest[order] = torch.arange(T * k, device=flat.device)
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(counts, 0)
    codes, scale = _quantize(s["x"].float())
    i32 = torch.int32
    return (counts.to(i32), offsets.to(i32), dest.to(i32), order.to(i32),
            codes.view(torch.uint8)[order // k].view(E4M3), scale[order // k])


def _plain_ffn(case, d, x, x_scale, bounds):
    """(h codes, h scales, y) of the routed rows."""
    R, H, I = x.shape[0], case["hidden"], case["inter"]
    h = torch.zeros((R, I), dtype=E4M3, device=x.device)
    h_scale = torch.zeros((R, _blocks(I)), device=x.device)
    y = torch.zeros((R, H), dtype=BF16, device=x.device)
    for e in range(case["experts"]):
        r = slice(bounds[e], bounds[e + 1])
        if r.start == r.stop:
            continue
        xe = x[r].float() * _spread(x_scale[r], H, 1)
        w13 = d["w13"][e].float() * _spread(_spread(d["w13_scale"][e], I, 1), H, 2)
        a = xe @ w13[0].t()
        if case["act"] == "swiglu":
            a = a / (1.0 + torch.exp(-a)) * (xe @ w13[1].t())
        else:
            a = torch.clamp(a, min=0.0).square()
        h[r], h_scale[r] = _quantize(a)
        he = h[r].float() * _spread(h_scale[r], I, 1)
        y[r] = (he @ (d["w2"][e].float() * _spread(_spread(d["w2_scale"][e], H, 0), I, 1)).t()).to(BF16)
    return h, h_scale, y


def _plain_expert_ffn(s):
    return _plain_ffn(s["case"], s, s["x"], s["x_scale"], s["bounds"])


def _plain_layer(s):
    case = s["case"]
    T, k = case["tokens"], case["top_k"]
    ids, w = _plain_route(s)
    _, offsets, dest, _, x, x_scale = _plain_dispatch(dict(case=case, ids=ids, x=s["x"]))
    y = _plain_ffn(case, s, x, x_scale, offsets.tolist())[2]
    out = (w.view(T, k, 1) * y[dest.long()].view(T, k, -1).float()).sum(1)
    return ids, w, out.to(BF16)


_PLAIN = {"route_grouped": _plain_route, "route_grouped_backward": _plain_route_backward,
          "dispatch_fp8": _plain_dispatch, "expert_ffn_fp8": _plain_expert_ffn, "layer_fp8": _plain_layer}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _nearest_e4m3(v):
    """The E4M3 value next to v (ties to even), in 64 bits: 3 fraction bits, exponents from -6, 448 at most."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rows(a):
    """(code values, scales) of 64-bit rows."""
    codes, scales = torch.empty_like(a), []
    for c in range(0, a.shape[1], BLOCK):
        m = a[:, c:c + BLOCK].abs().amax(1, keepdim=True).clamp(min=AMAX_FLOOR)
        codes[:, c:c + BLOCK] = _nearest_e4m3(a[:, c:c + BLOCK] * E4M3_MAX / m)
        scales.append(m / E4M3_MAX)
    return codes, torch.cat(scales, 1)


def _exact_route(case, d):
    l = d["logits"].to(F64)
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    key = (s.to(F32) + d["bias"]).to(F64)               # keys are defined in 32 bits
    T, E = l.shape
    G, k = case["groups"], case["top_k"]
    n = E // G
    # rank by counting the ones that come before: larger, or equal with a lower index
    before = lambda v: ((v[:, None, :] > v[:, :, None])
                        | ((v[:, None, :] == v[:, :, None]) & torch.ones(v.shape[1], v.shape[1], dtype=torch.bool,
                                                                         device=v.device).tril(-1))).sum(2)
    ids = torch.empty((T, k), dtype=torch.int64, device=l.device)
    for t in range(0, T, 1024):
        q = key[t:t + 1024]
        if G > 1:
            m, at = q.view(-1, G, n).max(2)
            if case["group_top"] == 2 and n > 1:
                rest = q.view(-1, G, n).scatter(2, at.unsqueeze(2), -math.inf)
                m = (m.to(F32) + rest.amax(2).to(F32)).to(F64)
            out = before(m) >= case["topk_groups"]
            q = q.masked_fill(out.unsqueeze(2).expand(-1, G, n).reshape(-1, E), -math.inf)
        r = before(q)
        row, col = torch.nonzero(r < k, as_tuple=True)
        ids[t + row, r[row, col]] = col
    rows = torch.arange(T, device=l.device).unsqueeze(1)
    w = s[rows, ids]
    if case["renorm"]:
        w = w / torch.einsum("tk->t", w).unsqueeze(1)
    return ids, w * d["scale"]


def _exact_ffn(case, d, x, x_scale, bounds):
    R, H, I, E = x.shape[0], case["hidden"], case["inter"], case["experts"]
    h = torch.zeros((R, I), dtype=F64, device="cuda")
    hs = torch.zeros((R, _blocks(I)), dtype=F64, device="cuda")
    y = torch.zeros((R, H), dtype=F64, device="cuda")

    def product(a, a_scale, w, w_scale):
        """Block by block: the codes' products, then both scales."""
        out = torch.zeros((a.shape[0], w.shape[0]), dtype=F64, device="cuda")
        row = torch.arange(w.shape[0], device="cuda") // BLOCK
        for b, c in enumerate(range(0, a.shape[1], BLOCK)):
            part = a[:, c:c + BLOCK] @ w[:, c:c + BLOCK].to(F64).t()
            out += part * a_scale[:, b:b + 1] * w_scale[row, b].to(F64)
        return out

    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if hi <= lo:
            continue
        xe, xs = x[lo:hi].to(F64), x_scale[lo:hi].to(F64)
        a = product(xe, xs, d["w13"][e, 0], d["w13_scale"][e, 0])
        if case["act"] == "swiglu":
            a = torch.nn.functional.silu(a) * product(xe, xs, d["w13"][e, 1], d["w13_scale"][e, 1])
        else:
            a = torch.where(a > 0, a * a, torch.zeros_like(a))
        h[lo:hi], hs[lo:hi] = _exact_rows(a)
        y[lo:hi] = product(h[lo:hi], hs[lo:hi], d["w2"][e], d["w2_scale"][e])
    return h, hs, y


def exact(case, seed):
    d = _inputs(case, seed)
    op, T, k = case["op"], case["tokens"], case["top_k"]
    if op == "route_grouped":
        return _exact_route(case, d)
    if op == "route_grouped_backward":
        # differentiate sum_j dw_j w_j(logits) for the given choice
        l = d["logits"].to(F64).requires_grad_()
        s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        w = torch.gather(s, 1, d["ids"].long())
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return torch.autograd.grad((w * d["dw"].to(F64)).sum() * d["scale"], l)[0]
    if op == "dispatch_fp8":
        E, H = case["experts"], case["hidden"]
        flat = d["ids"].reshape(-1).cpu().tolist()
        rows = [[] for _ in range(E)]
        for p, e in enumerate(flat):
            rows[e].append(p)
        order = torch.tensor([p for r in rows for p in r], device="cuda")
        dest = torch.empty(T * k, dtype=torch.int64, device="cuda")
        dest[order] = torch.arange(T * k, device="cuda")
        counts = torch.tensor([len(r) for r in rows], device="cuda")
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        codes = torch.empty((T * k, H), dtype=F64, device="cuda")
        scale = torch.empty((T * k, _blocks(H)), dtype=F64, device="cuda")
        for r in range(0, T * k, 16384):
            codes[r:r + 16384], scale[r:r + 16384] = _exact_rows(d["x"][order[r:r + 16384] // k].to(F64))
        return counts, offsets, dest, order, codes, scale
    if work(case)["flops"] > 7e12:
        return None
    if op == "expert_ffn_fp8":
        return _exact_ffn(case, d, d["x"], d["x_scale"], d["bounds"])
    ids, w = _exact_route(case, d)
    order = torch.sort(ids.reshape(-1), stable=True).indices
    bounds = [0] + torch.bincount(ids.reshape(-1), minlength=case["experts"]).cumsum(0).tolist()
    x, x_scale = _exact_rows(d["x"].to(F64))
    y = _exact_ffn(case, d, x[order // k], x_scale[order // k], bounds)[2]
    out = torch.zeros((T, case["hidden"]), dtype=F64, device="cuda")
    out.index_add_(0, order // k, y * w.reshape(-1)[order].unsqueeze(1))
    return ids, w, out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, T, E, k = case["op"], case["tokens"], case["experts"], case["top_k"]
    R = T * k
    route = 4 * T * E + 4 * E + 8 * R
    if op == "route_grouped":
        return {"bytes": route, "flops": 6 * T * E}
    if op == "route_grouped_backward":
        dense = case["score"] == "softmax" and not case["renorm"]        # reads every logit
        # renormalised softmax or sigmoid weights need the selected logits only
        return {"bytes": 4 * T * E + 8 * R + (4 * T * E if dense else 4 * R), "flops": (6 * T * E if dense else 0) + 8 * R}
    H = case["hidden"]
    if op == "dispatch_fp8":
        return {"bytes": 2 * T * H + 4 * R + R * H + 4 * R * _blocks(H) + 8 * R + 8 * E + 4, "flops": 4 * T * H}
    I = case["inter"]
    up = 2 * I if case["act"] == "swiglu" else I
    hit = min(E, R)                                                      # experts that receive a row, at most
    weights = hit * (up * H + H * I + 4 * (up // I * _blocks(I) * _blocks(H) + _blocks(H) * _blocks(I)))
    flops = 2 * R * H * (up + I)
    if op == "layer_fp8":
        return {"bytes": int(route + 4 * T * H + weights), "flops": int(flops)}
    rows = R * H + 4 * R * _blocks(H) + 2 * R * H                        # x in, y out
    h = R * I + 4 * R * _blocks(I)                                       # an output too
    return {"bytes": int(rows + h + weights + 4 * (E + 1)), "flops": int(flops)}
