"""Cases for timing the training operators of the MoE block.

A training step of a pre-norm MoE block runs, besides the forward calls, the
layer norm in front of the router (forward and backward), the gradient of the
weighted combine with the router's softmax gradient behind it, the gradient of
the dispatch, and the backward pass of the grouped expert FFN.  Each case below
is one of them at sizes of this repository's workloads (or generic odd ones).

``own`` selects what ``run`` does: False computes the operators with elementary
torch operations in 32 bits, rounded once at the end; True calls the library.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _ln(op, rows, hidden, dtype, res=False):
    return dict(op=op, rows=rows, hidden=hidden, dtype=dtype, res=res)


def _perm(op, tokens, hidden, experts, top_k, zipf=False):
    return dict(op=op, tokens=tokens, hidden=hidden, experts=experts, top_k=top_k, zipf=zipf)


def _ffn(tokens, hidden, experts, top_k, inter, act, zipf=False):
    return dict(op="expert_ffn_backward", tokens=tokens, hidden=hidden, experts=experts, top_k=top_k, inter=inter,
                act=act, zipf=zipf)


def listed():
    return [
        # the norm in front of the router for one decoded token: pure latency
        dict(name="layernorm_decode", **_ln("layernorm", 1, 7168, "bf16")),
        # the same norm over a 16384-token batch of the large layer
        dict(name="layernorm_large", **_ln("layernorm", 16384, 7168, "bf16")),
        # an odd width and an odd number of rows in 32 bits (a small model's float training)
        dict(name="layernorm_backward_odd", **_ln("layernorm_backward", 4095, 1001, "f32")),
        # the norm's gradient in the large layer's block, the residual's gradient added on the way
        dict(name="layernorm_backward_large", **_ln("layernorm_backward", 16384, 7168, "bf16", res=True)),
        # the smallest layer: 64 tokens, a launch-bound gradient of combine and router
        dict(name="combine_backward_tiny", **_perm("combine_backward", 64, 256, 16, 2)),
        # the large layer's combine and router gradients, with its skewed (hot-expert) routes
        dict(name="combine_backward_large", **_perm("combine_backward", 16384, 7168, 256, 8, zipf=True)),
        # 1024 tokens to 6 of 64 experts
        dict(name="dispatch_backward_mid", **_perm("dispatch_backward", 1024, 2048, 64, 6)),
        # the large layer's dispatch gradient
        dict(name="dispatch_backward_large", **_perm("dispatch_backward", 16384, 7168, 256, 8, zipf=True)),
        # the smallest expert FFN: about 8 rows an expert
        dict(name="expert_ffn_backward_tiny", **_ffn(64, 256, 16, 2, 512, "swiglu")),
        # about 77 rows an expert, squared-ReLU experts: weights and their gradients dominate
        dict(name="expert_ffn_backward_relu2", **_ffn(2048, 1024, 240, 9, 1536, "relu2")),
        # 1024 tokens to 6 of 64 experts, SwiGLU: about 96 rows an expert
        dict(name="expert_ffn_backward_mid", **_ffn(1024, 2048, 64, 6, 1408, "swiglu")),
        # the large layer's hidden and intermediate sizes over 32 experts, skewed routes: tensor-bound
        dict(name="expert_ffn_backward_large", **_ffn(4096, 7168, 32, 8, 2048, "swiglu", zipf=True)),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layernorm", "layernorm_backward", "combine_backward", "dispatch_backward",
                     "expert_ffn_backward", "expert_ffn_backward"])
    if op.startswith("layernorm"):
        hidden = _logu(rng, 33, 7168)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        return _ln(op, _logu(rng, 1, 16384), hidden, rng.choice(["bf16", "f32"]) if hidden <= 3500 else "bf16",
                   res=op == "layernorm_backward" and rng.random() < 0.5)
    experts = _logu(rng, 2, 256)
    top_k = rng.randint(1, min(8, experts))
    hidden = 8 * _logu(rng, 4, 896)
    if op != "expert_ffn_backward":
        return _perm(op, _logu(rng, 1, 16384), hidden, experts, top_k, zipf=rng.random() < 0.5)
    while True:
        case = _ffn(_logu(rng, 1, 4096), 8 * _logu(rng, 4, 896), _logu(rng, 1, 240), 1, 8 * _logu(rng, 4, 256),
                    rng.choice(["swiglu", "relu2"]), zipf=rng.random() < 0.5)
        case["top_k"] = rng.randint(1, min(8, case["experts"]))
        weights = case["experts"] * case["hidden"] * case["inter"]
        if weights <= 32 * 7168 * 2048 and case["tokens"] * case["top_k"] * case["hidden"] * case["inter"] \
                <= 4096 * 8 * 7168 * 2048:
            return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _routes(case, g):
    """Distinct experts per token, softmax weights over them, and the stable
    expert-contiguous order: what routing and dispatch hand to the backward."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    logits = torch.randn((T, E), generator=g, device="cuda", dtype=F32)
    if case["zipf"]:
        rank = torch.argsort(torch.rand(E, generator=g, device="cuda"))
        logits -= 1.2 * torch.log(rank.float() + 1.0)
    top, ids = torch.topk(logits, k, dim=1)
    w = torch.softmax(top, dim=1)
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    dest = torch.empty_like(order)
    dest[order] = torch.arange(T * k, device="cuda")
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return dict(ids=ids.to(torch.int32), w=w, dest=dest.to(torch.int32), offsets=offsets.to(torch.int32),
                bounds=offsets.tolist())


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op.startswith("layernorm"):
        rows, H = case["rows"], case["hidden"]
        dt = BF16 if case["dtype"] == "bf16" else F32
        # a residual stream: unit scale, an offset per channel and a few large channels
        scale = 1.0 + 7.0 * (torch.rand(H, generator=g, device="cuda") < 0.01)
        x = (torch.randn((rows, H), generator=g, device="cuda") * scale
             + 0.5 * torch.randn(H, generator=g, device="cuda")).to(dt)
        d = dict(x=x, gamma=1.0 + _randn(g, (H,), 0.1, F32), beta=_randn(g, (H,), 0.1, F32), eps=1e-5)
        if op == "layernorm_backward":
            xf = x.float()
            mean = xf.mean(1)
            d["mean"] = mean
            d["rstd"] = torch.rsqrt((xf - mean[:, None]).square().mean(1) + d["eps"])
            d["dy"] = _randn(g, (rows, H), 1.0, dt)
            d["dres"] = _randn(g, (rows, H), 1.0, dt) if case["res"] else None
        return d
    T, H, E, k = case["tokens"], case["hidden"], case["experts"], case["top_k"]
    R = T * k
    d = _routes(case, g)
    if op == "combine_backward":
        d["dout"] = _randn(g, (T, H))
        d["y_perm"] = _randn(g, (R, H))
    elif op == "dispatch_backward":
        d["dx_perm"] = _randn(g, (R, H))
        d["add"] = _randn(g, (T, H))
    else:
        I = case["inter"]
        up = 2 * I if case["act"] == "swiglu" else I
        d["x_perm"] = _randn(g, (R, H))
        d["dy_perm"] = _randn(g, (R, H), 1.0 / k)
        d["pre"] = _randn(g, (R, up))
        pf = d["pre"].float()
        d["h"] = (pf[:, :I] * torch.sigmoid(pf[:, :I]) * pf[:, I:] if case["act"] == "swiglu"
                  else torch.clamp(pf, min=0.0).square()).to(BF16)
        d["w13"] = torch.randn((E, up, H), generator=g, device="cuda", dtype=BF16).mul_(1.0 / math.sqrt(H))
        d["w2"] = torch.randn((E, H, I), generator=g, device="cuda", dtype=BF16).mul_(1.0 / math.sqrt(I))
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"] = case
    if own:
        _prepare_own(case, d)
    return d


def _prepare_own(case, d):
    """The output buffers, workspace and layer description a training program keeps."""
    from mixture_experts_routing_router_gb300 import native as N
    op = case["op"]
    if op.startswith("layernorm"):
        rows, H = case["rows"], case["hidden"]
        out = torch.empty_like(d["x"])
        if op == "layernorm":
            d["out"] = (out, torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"))
        else:
            d["out"] = (out, torch.empty(H, device="cuda"), torch.empty(H, device="cuda"))
            d["scratch"] = N.layernorm_scratch(rows, H)
        return
    T, H, E, k = case["tokens"], case["hidden"], case["experts"], case["top_k"]
    R = T * k
    inter = case.get("inter", 8)
    act = N.MOE_ACT_RELU2 if case.get("act") == "relu2" else N.MOE_ACT_SWIGLU
    d["shape"] = N.make_shape(T, H, E, k, inter, act=act)
    d["ws"] = N.workspace(d["shape"])
    if op == "combine_backward":
        d["out"] = (torch.empty((R, H), dtype=BF16, device="cuda"), torch.empty((T, k), device="cuda"),
                    torch.empty((T, E), device="cuda"))
    elif op == "dispatch_backward":
        d["out"] = torch.empty((T, H), dtype=BF16, device="cuda")
    else:
        d["out"] = (torch.empty_like(d["pre"]), torch.empty((R, H), dtype=BF16, device="cuda"),
                    torch.empty_like(d["w13"]), torch.empty_like(d["w2"]))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


def _run_own(s):
    from mixture_experts_routing_router_gb300 import native as N
    op = s["case"]["op"]
    if op == "layernorm":
        y, mean, rstd = s["out"]
        N.moe_layernorm(s["x"], s["gamma"], s["beta"], s["eps"], y, mean, rstd)
    elif op == "layernorm_backward":
        dx, dgamma, dbeta = s["out"]
        N.moe_layernorm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], dx, dgamma, dbeta, s["scratch"],
                                 dres=s["dres"])
    elif op == "combine_backward":
        dy_perm, dw, dlogits = s["out"]
        N.moe_combine_backward(s["shape"], s["dout"], s["y_perm"], s["dest"], s["w"], dy_perm, dw, s["ws"])
        N.moe_route_backward(s["shape"], s["ids"], s["w"], dw, dlogits, s["ws"])
    elif op == "dispatch_backward":
        N.moe_dispatch_backward(s["shape"], s["dx_perm"], s["dest"], s["out"], s["ws"], add=s["add"])
    else:
        dpre, dx_perm, dw13, dw2 = s["out"]
        N.moe_expert_down_backward(s["shape"], s["dy_perm"], s["offsets"], s["w2"], s["pre"], s["h"], dpre, dw2,
                                   s["ws"])
        N.moe_expert_up_backward(s["shape"], dpre, s["offsets"], s["x_perm"], s["w13"], dx_perm, dw13, s["ws"])
    return s["out"]


def _plain_layernorm(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + s["eps"])
    y = c * rstd[:, None] * s["gamma"] + s["beta"]
    return y.to(s["x"].dtype), mean, rstd


def _plain_layernorm_backward(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    gy = dy * s["gamma"]
    dx = (gy - gy.mean(1, keepdim=True) - xhat * (gy * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dx.to(s["x"].dtype), (dy * xhat).sum(0), dy.sum(0)


def _plain_combine_backward(s):
    T, H = s["dout"].shape
    w, ids, dest = s["w"], s["ids"].long(), s["dest"].long()
    k, E = w.shape[1], s["case"]["experts"]
    dout = s["dout"].float().unsqueeze(1)
    dy = torch.empty((T * k, H), dtype=BF16, device=dout.device)
    dy[dest] = (dout * w.unsqueeze(2)).to(BF16).view(T * k, H)
    dw = (dout * s["y_perm"][dest].view(T, k, H).float()).sum(2)
    dlogits = torch.zeros((T, E), device=dout.device)
    dlogits.scatter_(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    return dy, dw, dlogits


def _plain_dispatch_backward(s):
    T = s["add"].shape[0]
    dest = s["dest"].long().view(T, -1)
    return (s["dx_perm"][dest].float().sum(1) + s["add"].float()).to(BF16)


def _plain_expert_ffn_backward(s):
    case, bounds = s["case"], s["bounds"]
    I = case["inter"]
    dpre, dx = torch.empty_like(s["pre"]), torch.empty_like(s["x_perm"])
    dw13, dw2 = torch.zeros_like(s["w13"]), torch.zeros_like(s["w2"])
    for e in range(case["experts"]):
        r = slice(bounds[e], bounds[e + 1])
        if r.start == r.stop:
            continue
        dy, p = s["dy_perm"][r].float(), s["pre"][r].float()
        w13, w2 = s["w13"][e].float(), s["w2"][e].float()
        dh = dy @ w2
        if case["act"] == "swiglu":
            g, u = p[:, :I], p[:, I:]
            sg = 1.0 / (1.0 + torch.exp(-g))
            dp = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], 1)
        else:
            dp = dh * 2.0 * torch.clamp(p, min=0.0)
        dw2[e] = (dy.t() @ s["h"][r].float()).to(BF16)
        dpre[r] = dp.to(BF16)
        dx[r] = (dp @ w13).to(BF16)
        dw13[e] = (dp.t() @ s["x_perm"][r].float()).to(BF16)
    return dpre, dx, dw13, dw2


_PLAIN = {"layernorm": _plain_layernorm, "layernorm_backward": _plain_layernorm_backward,
          "combine_backward": _plain_combine_backward, "dispatch_backward": _plain_dispatch_backward,
          "expert_ffn_backward": _plain_expert_ffn_backward}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    D = torch.float64
    if op == "layernorm":
        y = torch.empty(d["x"].shape, dtype=D, device="cuda")
        mean = torch.empty(d["x"].shape[0], dtype=D, device="cuda")
        rstd = torch.empty_like(mean)
        for r in range(0, len(mean), 2048):
            x = d["x"][r:r + 2048].to(D)
            var, mu = torch.var_mean(x, dim=1, correction=0)
            mean[r:r + 2048], rstd[r:r + 2048] = mu, (var + d["eps"]).pow(-0.5)
            y[r:r + 2048] = torch.addcmul(d["beta"].to(D), (x - mu.unsqueeze(1)) / (var + d["eps"]).sqrt().unsqueeze(1),
                                          d["gamma"].to(D))
        return y, mean, rstd
    if op == "layernorm_backward":
        # dx_i = rstd * (a_i - A/H - xhat_i B/H), a = dy gamma, A = sum a, B = sum a xhat
        rows, H = d["x"].shape
        dx = torch.empty((rows, H), dtype=D, device="cuda")
        dgamma, dbeta = torch.zeros(H, dtype=D, device="cuda"), torch.zeros(H, dtype=D, device="cuda")
        for r in range(0, rows, 2048):
            q = slice(r, min(rows, r + 2048))
            rs = d["rstd"][q].to(D).unsqueeze(1)
            xh = (d["x"][q].to(D) - d["mean"][q].to(D).unsqueeze(1)).mul_(rs)
            dy = d["dy"][q].to(D)
            dgamma += torch.einsum("rh,rh->h", dy, xh)
            dbeta += dy.sum(0)
            a = dy.mul_(d["gamma"].to(D))
            A, B = a.sum(1, keepdim=True), torch.einsum("rh,rh->r", a, xh).unsqueeze(1)
            dx[q] = rs / H * (H * a - A - xh * B)
            if d["dres"] is not None:
                dx[q] += d["dres"][q].to(D)
        return dx, dgamma, dbeta
    T, H, E, k = case["tokens"], case["hidden"], case["experts"], case["top_k"]
    if op == "combine_backward":
        tok = torch.empty(T * k, dtype=torch.long, device="cuda")       # token of each slot
        tok[d["dest"].long()] = torch.arange(T * k, device="cuda") // k
        ws = torch.empty(T * k, dtype=D, device="cuda")
        ws[d["dest"].long()] = d["w"].to(D).reshape(-1)
        dy = torch.empty((T * k, H), dtype=D, device="cuda")
        dws = torch.empty(T * k, dtype=D, device="cuda")
        for r in range(0, T * k, 16384):
            g = d["dout"][tok[r:r + 16384]].to(D)
            dws[r:r + 16384] = torch.einsum("rh,rh->r", g, d["y_perm"][r:r + 16384].to(D))
            dy[r:r + 16384] = g.mul_(ws[r:r + 16384, None])
        dw = dws[d["dest"].long()].view(T, k)
        w = d["w"].to(D)
        # Jacobian of the softmax over the selection: diag(w) - w w^T
        jac = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)
        dl = torch.zeros((T, E), dtype=D, device="cuda")
        dl[torch.arange(T, device="cuda").unsqueeze(1), d["ids"].long()] = torch.einsum("tij,tj->ti", jac, dw)
        return dy, dw, dl
    if op == "dispatch_backward":
        out = d["add"].to(D)
        tok = torch.empty(T * k, dtype=torch.long, device="cuda")
        tok[d["dest"].long()] = torch.arange(T * k, device="cuda") // k
        for r in range(0, T * k, 16384):
            out.index_add_(0, tok[r:r + 16384], d["dx_perm"][r:r + 16384].to(D))
        return out
    if work(case)["flops"] > 7e12:
        return None
    I, b = case["inter"], d["bounds"]
    glu = case["act"] == "swiglu"
    dpre = torch.zeros(d["pre"].shape, dtype=D, device="cuda")
    dx = torch.zeros(d["x_perm"].shape, dtype=D, device="cuda")
    dw13 = torch.zeros(d["w13"].shape, dtype=D, device="cuda")
    dw2 = torch.zeros(d["w2"].shape, dtype=D, device="cuda")
    for e in range(E):
        lo, hi = b[e], b[e + 1]
        if hi <= lo:
            continue
        dy, pre = d["dy_perm"][lo:hi].to(D), d["pre"][lo:hi].to(D)
        dh = torch.einsum("rh,hi->ri", dy, d["w2"][e].to(D))
        torch.mm(dy.t(), d["h"][lo:hi].to(D), out=dw2[e])
        if glu:
            gate, val = pre.split(I, 1)
            s = torch.sigmoid(gate)
            # d(g s)/dg = s + g s (1 - s)
            dpre[lo:hi, :I] = (s + gate * s * (1 - s)) * val * dh
            dpre[lo:hi, I:] = s * gate * dh
        else:
            dpre[lo:hi] = torch.where(pre > 0, 2 * pre * dh, torch.zeros_like(pre))
        torch.mm(dpre[lo:hi].t(), d["x_perm"][lo:hi].to(D), out=dw13[e])
        dx[lo:hi] = torch.einsum("ru,uh->rh", dpre[lo:hi], d["w13"][e].to(D))
    return dpre, dx, dw13, dw2


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _hit(case):
    """Experts that receive a row, at most."""
    return min(case["experts"], case["tokens"] * case["top_k"])


def work(case):
    op = case["op"]
    if op.startswith("layernorm"):
        rows, H = case["rows"], case["hidden"]
        el = 2 if case["dtype"] == "bf16" else 4
        if op == "layernorm":
            return {"bytes": 2 * rows * H * el + 8 * H + 8 * rows, "flops": 8 * rows * H}
        return {"bytes": (4 if case["res"] else 3) * rows * H * el + 12 * H + 8 * rows, "flops": 14 * rows * H}
    T, H, E, k = case["tokens"], case["hidden"], case["experts"], case["top_k"]
    R = T * k
    if op == "combine_backward":
        return {"bytes": 2 * T * H + 4 * R * H + 4 * (4 * R) + 4 * T * E, "flops": 3 * R * H + 5 * R}
    if op == "dispatch_backward":
        return {"bytes": 4 * T * H + 2 * R * H + 4 * R, "flops": R * H}
    I = case["inter"]
    up = 2 * I if case["act"] == "swiglu" else I
    weights = 2 * H * (up + I)
    # rows in and out, each used expert's weights, every expert's weight gradients
    rows = 2 * R * (H + up + I + H) + 2 * R * (up + H)
    return {"bytes": int(rows + _hit(case) * weights + E * weights + 4 * (E + 1)),
            "flops": int(4 * R * H * (up + I))}

