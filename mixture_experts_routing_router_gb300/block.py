"""A trainable pre-norm MoE block on the library's calls:

    n = layernorm(x);  logits = n w_gate^T;  (ids, w) = softmax top-k of logits
    out = x + sum_j w_j * FFN_{ids_j}(n)

(or, with a ``router``, group-limited routing: its scores, groups and weights).

Forward: moe_layernorm, moe_gate, moe_route (moe_route_grouped), moe_dispatch, moe_expert_up_train,
moe_expert_down, moe_combine (the residual x added there).  Backward:
moe_combine_backward, moe_route_backward (moe_route_grouped_backward),
moe_expert_down_backward, moe_expert_up_backward, moe_gate_backward, moe_dispatch_backward (the gate's part
of dn added there) and moe_layernorm_backward (the residual's gradient added
there).  torch carries memory, streams and the autograd graph; every number comes
from the library's kernels.  dn is rounded twice: the gate's part to BF16 (g w_gate), then
its sum with the experts' part.

Reference: DeepSeek fleet megakernel REPORT.md, the per-op table (MOE_GATE_TOPK,
EXPERT_W13_SILU, EXPERT_W2, MOE_COMBINE_RESIDUAL) for the block's forward chain.
"""
from __future__ import annotations

import torch

from . import native as N


class _SecondDerivative(torch.autograd.Function):
    @staticmethod
    def forward(ctx, anchor, *grads):
        return grads

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("MoEBlock: its gradients cannot be differentiated again")


def _differentiable_once(grads):
    """The gradients, in a graph whose only step raises: without one a loss on them (a
    gradient penalty) beside another term would lose its gradient without a word.
    (autograd's once_differentiable raises only where the incoming gradient has a graph.)"""
    some = [g for g in grads if g is not None]
    if some:
        some = iter(_SecondDerivative.apply(some[0].new_zeros((), requires_grad=True), *some))
    return tuple(None if g is None else next(some) for g in grads)


class _MoEBlockFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, w_gate, w13, w2, block):
        shape, ws = block._layer(x.shape[0], x.device)
        dev, bf16 = x.device, torch.bfloat16
        T, H, E, k, I = shape.tokens, shape.hidden, shape.experts, shape.top_k, shape.inter
        R, up = T * k, w13.shape[1]
        i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=dev)
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=dev)
        b16 = lambda *s: torch.empty(s, dtype=bf16, device=dev)
        n, mean, rstd = torch.empty_like(x), f32(T), f32(T)
        N.moe_layernorm(x, gamma, beta, block.eps, n, mean, rstd)
        logits, ids, w = f32(T, E), i32(T, k), f32(T, k)
        N.moe_gate(shape, n, w_gate, logits, ws)
        router = block.router and N.moe_router.from_buffer_copy(block.router)  # as it is now, for the backward pass too
        if router is None:
            N.moe_route(shape, logits, ids, w, ws)
        else:
            N.moe_route_grouped(shape, router, logits, block.route_bias, ids, w, ws)
        offsets, dest, x_perm = i32(E + 1), i32(R), b16(R, H)
        N.moe_dispatch(shape, n, ids, i32(E), offsets, dest, i32(R), x_perm, ws)
        pre, h, y_perm, out = b16(R, up), b16(R, I), b16(R, H), torch.empty_like(x)
        N.moe_expert_up_train(shape, x_perm, offsets, w13, pre, h, ws)
        N.moe_expert_down(shape, h, offsets, w2, None, y_perm, None, ws)
        N.moe_combine(shape, y_perm, dest, w, None, out, ws, residual=x)
        ctx.save_for_backward(x, gamma, w_gate, w13, w2, n, mean, rstd, ids, w, offsets, dest, x_perm, pre, h, y_perm,
                              logits if router is not None else None)
        ctx.block, ctx.router = block, router
        return out

    @staticmethod
    def backward(ctx, dout):
        with torch.no_grad():
            grads = _MoEBlockFn._gradients(ctx, dout)
        if torch.is_grad_enabled():           # create_graph
            grads = _differentiable_once(grads)
        return (*grads, None)

    @staticmethod
    def _gradients(ctx, dout):
        (x, gamma, w_gate, w13, w2, n, mean, rstd, ids, w, offsets, dest, x_perm, pre, h, y_perm,
         logits) = ctx.saved_tensors
        shape, ws = ctx.block._layer(x.shape[0], x.device)     # the block's, where check() looks
        want = ctx.needs_input_grad
        like = lambda t, on: torch.empty_like(t) if on else None
        dout = dout.contiguous()
        dy_perm, dw, dlogits = torch.empty_like(y_perm), torch.empty_like(w), w.new_empty(shape.tokens, shape.experts)
        N.moe_combine_backward(shape, dout, y_perm, dest, w, dy_perm, dw, ws)
        if ctx.router is None:
            N.moe_route_backward(shape, ids, w, dw, dlogits, ws)
        else:
            N.moe_route_grouped_backward(shape, ctx.router, logits, ids, dw, dlogits, ws)
        dpre, dx_perm = torch.empty_like(pre), torch.empty_like(x_perm)
        dw13, dw2, dw_gate = like(w13, want[4]), like(w2, want[5]), like(w_gate, want[3])
        N.moe_expert_down_backward(shape, dy_perm, offsets, w2, pre, h, dpre, dw2, ws)
        N.moe_expert_up_backward(shape, dpre, offsets, x_perm, w13, dx_perm, dw13, ws)
        dn = torch.empty_like(n)
        dl16 = n.new_empty(shape.tokens, (shape.experts + 7) // 8 * 8)
        N.moe_gate_backward(shape, dlogits, n, w_gate, dl16, dn, dw_gate, ws)
        N.moe_dispatch_backward(shape, dx_perm, dest, dn, ws, add=dn)
        dx = torch.empty_like(x)
        dgamma, dbeta = mean.new_empty(gamma.shape), mean.new_empty(gamma.shape)
        scratch = N.layernorm_scratch(x.shape[0], x.shape[1], x.device)
        N.moe_layernorm_backward(dn, x, gamma, mean, rstd, dx, dgamma, dbeta, scratch, dres=dout)
        return (dx if want[0] else None, dgamma.to(gamma.dtype) if want[1] else None,
                dbeta.to(gamma.dtype) if want[2] else None, dw_gate, dw13, dw2)


class MoEBlock(torch.nn.Module):
    """x [T, hidden] BF16 -> x + MoE(layernorm(x)), differentiable in x and every parameter.

    Parameters: gamma, beta [hidden] FP32; w_gate [experts, hidden], w13 [experts, up,
    hidden] (up = 2 * inter for SwiGLU, inter for ReLU^2), w2 [experts, hidden, inter]
    BF16 (of another type, say after ``float()``, the block refuses to run).  The block
    keeps one workspace, as large as the largest batch it saw needs, so its calls belong
    on one stream at a time.  Device-side errors (non-finite logits, a bounded wait that
    ran out), of any batch and either direction, stay there until ``check`` reads them.
    Differentiable once: a second
    derivative through the block raises.

    ``router`` (native.make_router) has the tokens routed by moe_route_grouped; the block
    then has a buffer ``route_bias`` [experts] FP32, zeros at first, that only selects: it
    has no gradient, and a program that balances its experts adds to it between steps."""

    router = None        # of blocks that were pickled whole before there was one, too

    def __init__(self, hidden, experts, top_k, inter, act=N.MOE_ACT_SWIGLU, eps=1e-5, device="cuda", generator=None,
                 router=None):
        super().__init__()
        if router is not None and not isinstance(router, N.moe_router):
            raise ValueError(f"MoEBlock: router must come from native.make_router, got {type(router).__name__}")
        self.router = router
        if router is not None:
            self.register_buffer("route_bias", torch.zeros(experts, device=device))
        up = 2 * inter if act == N.MOE_ACT_SWIGLU else inter
        self.hidden, self.experts, self.top_k, self.inter, self.act, self.eps = hidden, experts, top_k, inter, act, eps

        def draw(*shape):
            t = torch.randn(shape, generator=generator, device=device, dtype=torch.float32)
            return torch.nn.Parameter((t / shape[-1] ** 0.5).to(torch.bfloat16))

        self.gamma = torch.nn.Parameter(torch.ones(hidden, device=device))
        self.beta = torch.nn.Parameter(torch.zeros(hidden, device=device))
        self.w_gate, self.w13, self.w2 = draw(experts, hidden), draw(experts, up, hidden), draw(experts, hidden, inter)
        self._shape = self._ws = None
        self._bytes = 0                       # of workspace that _shape needs

    def _layer(self, tokens, device):
        """The shape of a batch and the block's workspace, grown where the shape needs more.
        The larger one takes over the header, so a status not yet read stays to be read."""
        if self._shape is None or self._shape.tokens != tokens:
            shape = N.make_shape(tokens, self.hidden, self.experts, self.top_k, self.inter, self.act)
            self._bytes = N.moe_workspace_stage_size(shape)
            self._shape = shape
        old = self._ws
        if old is None or old.device != device or old.nbytes < self._bytes:
            self._ws = torch.empty(self._bytes, dtype=torch.uint8, device=device)
            if old is None:
                N.moe_workspace_init(self._ws)
            else:
                self._ws[:N.WORKSPACE_HEADER].copy_(old[:N.WORKSPACE_HEADER])
        return self._shape, self._ws

    def forward(self, x):
        if x.dim() != 2 or x.shape[1] != self.hidden or x.dtype != torch.bfloat16:
            raise ValueError(f"MoEBlock: expected a bfloat16 [tokens, {self.hidden}] input, got {x.dtype} {tuple(x.shape)}")
        up = 2 * self.inter if self.act == N.MOE_ACT_SWIGLU else self.inter
        for name, want in (("w_gate", (self.experts, self.hidden)), ("w13", (self.experts, up, self.hidden)),
                           ("w2", (self.experts, self.hidden, self.inter))):
            w = getattr(self, name)
            if w.dtype != torch.bfloat16 or w.shape != want:        # the kernels read them as they lie
                raise ValueError(f"MoEBlock: {name} must be bfloat16 {want}, got {w.dtype} {tuple(w.shape)} "
                                 "(gamma and beta may be float32 or bfloat16)")
        if self.router is not None and (self.route_bias.dtype != torch.float32 or self.route_bias.shape != (self.experts,)):
            raise ValueError(f"MoEBlock: route_bias must be float32 ({self.experts},), got {self.route_bias.dtype} "
                             f"{tuple(self.route_bias.shape)}")
        return _MoEBlockFn.apply(x.contiguous(), self.gamma, self.beta, self.w_gate, self.w13, self.w2, self)

    def check(self):
        """Synchronise and raise if a kernel of this block's calls reported an error."""
        if self._ws is not None:
            st = N.moe_status_read(self._ws)
            if st != N.MOE_OK:
                raise N.MoEError(st, "MoEBlock")
