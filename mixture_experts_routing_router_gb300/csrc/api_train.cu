// api_train.cu -- the extern "C" entry points for training the MoE block: layer
// norm, the forward up projection that keeps its pre-activations, and the
// gradients of dispatch, combine, routing and the expert FFN.  Same manner as
// api.cu: host-side checks that launch nothing on an error, then kernels on the
// caller's stream.
#include "common.cuh"

#include <climits>
#include <cmath>

namespace moe {
namespace {

WsHeader* header(void* ws) { return static_cast<WsHeader*>(ws); }

float* partials(const moe_shape& s, void* ws) {
    return reinterpret_cast<float*>(static_cast<char*>(ws) + ws_layout(s).partials);
}

bool aligned_or_null(const void* p, uintptr_t a) { return p == nullptr || aligned(p, a); }

bool is_type(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }

int up_rows(const moe_shape& s) { return (s.act == MOE_ACT_SWIGLU ? 2 : 1) * s.inter; }

moe_status check_stage(const moe_shape* shape, const void* ws, size_t ws_bytes) {
    const moe_status r = validate_shape(shape);
    return r != MOE_OK ? r : check_ws(shape, ws, ws_bytes, false);
}

// The expert FFN's training calls take routed experts only.
moe_status check_ffn(const moe_shape* shape, const void* ws, size_t ws_bytes) {
    const moe_status r = check_stage(shape, ws, ws_bytes);
    if (r == MOE_OK && shape->shared > 0) {
        set_error("expert FFN training calls: shared experts are not supported (shape.shared must be 0; a shared "
                  "expert is a one-expert shape over all tokens)");
        return MOE_ERR_UNSUPPORTED;
    }
    return r;
}

bool is_wgrad(int32_t m) { return m == MOE_WGRAD_BF16 || m == MOE_WGRAD_F32 || m == MOE_WGRAD_F32_ADD; }

moe_status check_layernorm(int64_t rows, int32_t hidden, int32_t type, int32_t wtype) {
    if (rows < 0 || hidden < 1 || hidden > (1 << 20) || !is_type(type) || !is_type(wtype)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

size_t layernorm_scratch_bytes(int64_t rows, int32_t hidden) {
    return align_up((size_t)layernorm_parts(rows) * 2 * (size_t)hidden * sizeof(float), kAlign);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_layernorm(int64_t rows, int32_t hidden, int32_t type, int32_t wtype, const void* x, const void* gamma,
                         const void* beta, float eps, void* y, float* mean, float* rstd, void* stream) {
    clear_error();
    const moe_status r = check_layernorm(rows, hidden, type, wtype);
    if (r != MOE_OK) return r;
    if (!(eps >= 0.0f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (!aligned(gamma, 16) || !aligned(beta, 16)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned_or_null(mean, 16) || !aligned_or_null(rstd, 16))
        return MOE_ERR_INVALID_ARG;
    LayerNormProblem p{};
    p.rows = rows; p.hidden = hidden; p.type = type; p.wtype = wtype;
    p.x = x; p.gamma = gamma; p.beta = beta; p.eps = eps;
    p.y = y; p.mean = mean; p.rstd = rstd;
    return from_cuda(launch_layernorm(p, static_cast<cudaStream_t>(stream)));
}

moe_status moe_layernorm_scratch_size(int64_t rows, int32_t hidden, size_t* bytes) {
    clear_error();
    const moe_status r = check_layernorm(rows, hidden, MOE_TYPE_BF16, MOE_TYPE_F32);
    if (r != MOE_OK) return r;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = layernorm_scratch_bytes(rows, hidden);
    return MOE_OK;
}

moe_status moe_layernorm_backward(int64_t rows, int32_t hidden, int32_t type, int32_t wtype, const void* dy,
                                  const void* x, const void* gamma, const float* mean, const float* rstd,
                                  const void* dres, void* dx, float* dgamma, float* dbeta, void* scratch,
                                  size_t scratch_bytes, void* stream) {
    clear_error();
    const moe_status r = check_layernorm(rows, hidden, type, wtype);
    if (r != MOE_OK) return r;
    if (!aligned(gamma, 16) || !aligned(dgamma, 16) || !aligned(dbeta, 16)) return MOE_ERR_INVALID_ARG;
    if (!aligned(scratch, 256) || scratch_bytes < layernorm_scratch_bytes(rows, hidden)) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!aligned(dy, 16) || !aligned(x, 16) || !aligned(mean, 16) || !aligned(rstd, 16) ||
                     !aligned(dx, 16) || !aligned_or_null(dres, 16)))
        return MOE_ERR_INVALID_ARG;
    LayerNormProblem p{};
    p.rows = rows; p.hidden = hidden; p.type = type; p.wtype = wtype;
    p.x = x; p.gamma = gamma; p.dy = dy; p.dres = dres; p.dx = dx;
    p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
    p.dgamma = dgamma; p.dbeta = dbeta; p.scratch = static_cast<float*>(scratch);
    return from_cuda(launch_layernorm_backward(p, static_cast<cudaStream_t>(stream)));
}

moe_status moe_combine_backward(const moe_shape* shape, const uint16_t* dout, const uint16_t* y_perm,
                                const int32_t* dest, const float* topk_w, uint16_t* dy_perm, float* dtopk_w, void* ws,
                                size_t ws_bytes, void* stream) {
    clear_error();
    const moe_status r = check_stage(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(dout, 16) || !aligned(dest, 16) || !aligned(topk_w, 16) || !aligned(dy_perm, 16) ||
        !aligned_or_null(dtopk_w, 16) || !aligned_or_null(y_perm, 16) || (dtopk_w && !y_perm))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_combine_grad(*shape, dout, y_perm, dest, topk_w, dy_perm, dtopk_w,
                                         static_cast<cudaStream_t>(stream)));
}

moe_status moe_dispatch_backward(const moe_shape* shape, const uint16_t* dx_perm, const int32_t* dest,
                                 const uint16_t* add, uint16_t* dx, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    const moe_status r = check_stage(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(dx_perm, 16) || !aligned(dest, 16) || !aligned_or_null(add, 16) || !aligned(dx, 16))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_combine(*shape, dx_perm, dest, nullptr, nullptr, add, dx, nullptr,
                                    static_cast<cudaStream_t>(stream)));
}

moe_status moe_route_backward(const moe_shape* shape, const int32_t* topk_ids, const float* topk_w,
                              const float* dtopk_w, float* dlogits, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    const moe_status r = check_stage(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(topk_ids, 16) || !aligned(topk_w, 16) || !aligned(dtopk_w, 16) || !aligned(dlogits, 16))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_route_grad(*shape, nullptr, topk_ids, topk_w, 1.0f, dtopk_w, dlogits, header(ws),
                                       static_cast<cudaStream_t>(stream)));
}

moe_status moe_route_sigmoid_backward(const moe_shape* shape, const float* logits, const int32_t* topk_ids,
                                      float route_scale, const float* dtopk_w, float* dlogits, void* ws,
                                      size_t ws_bytes, void* stream) {
    clear_error();
    const moe_status r = check_stage(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(logits, 16) || !aligned(topk_ids, 16) || !aligned(dtopk_w, 16) || !aligned(dlogits, 16))
        return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(route_scale)) return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_route_grad(*shape, logits, topk_ids, nullptr, route_scale, dtopk_w, dlogits, header(ws),
                                       static_cast<cudaStream_t>(stream)));
}

moe_status moe_gate_backward(const moe_shape* shape, const float* dlogits, const uint16_t* x, const uint16_t* w_gate,
                             uint16_t* dlogits_bf16, uint16_t* dx, void* dw_gate, int32_t wgrad, void* ws,
                             size_t ws_bytes, void* stream) {
    clear_error();
    moe_status r = check_stage(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(dlogits, 16) || !aligned(dlogits_bf16, 16) || (!dx && !dw_gate) || !is_wgrad(wgrad))
        return MOE_ERR_INVALID_ARG;
    if (dx && (!aligned(dx, 16) || !aligned(w_gate, 16))) return MOE_ERR_INVALID_ARG;
    if (dw_gate && (!aligned(dw_gate, 16) || !aligned(x, 16))) return MOE_ERR_INVALID_ARG;
    const moe_shape& s = *shape;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int cols = (s.experts + 7) / 8 * 8;      // TMA rows are multiples of 16 bytes
    if ((r = from_cuda(launch_round_rows(s.tokens, s.experts, cols, dlogits, dlogits_bf16, st))) != MOE_OK) return r;
    ExpertGradProblem g{};
    g.a = dlogits_bf16; g.rows = s.tokens; g.a_cols = cols;
    g.offsets = nullptr; g.groups = 1;
    g.w = w_gate; g.K = s.experts; g.N = s.hidden;
    g.out = dx; g.ldo = s.hidden;
    g.wb = x; g.wM = s.experts; g.wN = s.hidden;
    g.wout = dw_gate; g.wmode = wgrad;
    return launch_expert_grad(g, partials(s, ws), header(ws), st);
}

moe_status moe_expert_up_train(const moe_shape* shape, const uint16_t* x_perm, const int32_t* offsets,
                               const uint16_t* w13, uint16_t* pre, uint16_t* h, void* ws, size_t ws_bytes,
                               void* stream) {
    clear_error();
    moe_status r = check_ffn(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(x_perm, 16) || !aligned(offsets, 16) || !aligned(w13, 16) || !aligned(pre, 16) || !aligned(h, 16))
        return MOE_ERR_INVALID_ARG;
    const moe_shape& s = *shape;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int up = up_rows(s);
    GemmProblem g{};
    g.mode = kGemmPlain;
    g.a = x_perm; g.a_rows = (long long)s.tokens * s.top_k; g.a_cols = s.hidden;
    g.b = w13; g.b_rows = (long long)s.experts * up; g.b_cols = s.hidden;
    g.offsets = offsets; g.groups = s.experts;
    g.K = s.hidden; g.nseg = 1;
    g.N = up; g.b_group_rows = up;
    g.out = pre; g.ldo = up;
    g.max_group_rows = s.tokens;
    if ((r = launch_grouped_gemm(g, header(ws), st)) != MOE_OK) return r;
    return from_cuda(launch_act(s, offsets, pre, h, st));
}

moe_status moe_expert_down_backward(const moe_shape* shape, const uint16_t* dy_perm, const int32_t* offsets,
                                    const uint16_t* w2, const uint16_t* pre, const uint16_t* h, uint16_t* dpre,
                                    void* dw2, int32_t wgrad, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    moe_status r = check_ffn(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(dy_perm, 16) || !aligned(offsets, 16) || (!dpre && !dw2) || !is_wgrad(wgrad)) return MOE_ERR_INVALID_ARG;
    if (dpre && (!aligned(dpre, 16) || !aligned(w2, 16) || !aligned(pre, 16))) return MOE_ERR_INVALID_ARG;
    if (dw2 && (!aligned(dw2, 16) || !aligned(h, 16))) return MOE_ERR_INVALID_ARG;
    const moe_shape& s = *shape;
    ExpertGradProblem g{};
    g.a = dy_perm; g.rows = (long long)s.tokens * s.top_k; g.a_cols = s.hidden;
    g.offsets = offsets; g.groups = s.experts;
    g.w = w2; g.K = s.hidden; g.N = s.inter;
    g.out = dpre; g.ldo = up_rows(s);
    g.pre = pre; g.act = s.act;
    g.wb = h; g.wM = s.hidden; g.wN = s.inter;
    g.wout = dw2; g.wmode = wgrad;
    return launch_expert_grad(g, partials(s, ws), header(ws), static_cast<cudaStream_t>(stream));
}

moe_status moe_expert_up_backward(const moe_shape* shape, const uint16_t* dpre, const int32_t* offsets,
                                  const uint16_t* x_perm, const uint16_t* w13, uint16_t* dx_perm, void* dw13,
                                  int32_t wgrad, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    moe_status r = check_ffn(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(dpre, 16) || !aligned(offsets, 16) || (!dx_perm && !dw13) || !is_wgrad(wgrad)) return MOE_ERR_INVALID_ARG;
    if (dx_perm && (!aligned(dx_perm, 16) || !aligned(w13, 16))) return MOE_ERR_INVALID_ARG;
    if (dw13 && (!aligned(dw13, 16) || !aligned(x_perm, 16))) return MOE_ERR_INVALID_ARG;
    const moe_shape& s = *shape;
    ExpertGradProblem g{};
    g.a = dpre; g.rows = (long long)s.tokens * s.top_k; g.a_cols = up_rows(s);
    g.offsets = offsets; g.groups = s.experts;
    g.w = w13; g.K = up_rows(s); g.N = s.hidden;
    g.out = dx_perm; g.ldo = s.hidden;
    g.wb = x_perm; g.wM = up_rows(s); g.wN = s.hidden;
    g.wout = dw13; g.wmode = wgrad;
    return launch_expert_grad(g, partials(s, ws), header(ws), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
