// api_fp8.cu -- the extern "C" entry points of group-limited routing and of the expert
// path in block-scaled FP8 (fp8.cuh).  Same manner as api.cu: host-side checks that
// launch nothing on an error, then kernels on the caller's stream.
#include "fp8.cuh"

#include <cmath>

namespace moe {
namespace {

template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

bool aligned_or_null(const void* p, uintptr_t a) { return p == nullptr || aligned(p, a); }

moe_status check_stage(const moe_shape* shape, const void* ws, size_t ws_bytes, bool whole_layer = false) {
    const moe_status r = validate_shape(shape);
    return r != MOE_OK ? r : check_ws(shape, ws, ws_bytes, whole_layer);
}

moe_status check_router(const moe_shape& s, const moe_router* r) {
    if (!r) return MOE_ERR_INVALID_ARG;
    if ((r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) || (r->group_top != 1 && r->group_top != 2) ||
        (r->renorm != 0 && r->renorm != 1) || !std::isfinite(r->scale)) {
        set_error("router: score %d, group_top %d, renorm %d, scale %g", r->score, r->group_top, r->renorm,
                  (double)r->scale);
        return MOE_ERR_INVALID_ARG;
    }
    if (r->groups < 1 || r->groups > 32 || s.experts % r->groups != 0 || r->topk_groups < 1 ||
        r->topk_groups > r->groups || (long long)r->topk_groups * (s.experts / r->groups) < s.top_k) {
        set_error("router: %d of %d groups for top-%d of %d experts (1 to 32 groups that divide the experts, enough "
                  "experts in the chosen ones)", r->topk_groups, r->groups, s.top_k, s.experts);
        return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

// TMA rows are multiples of 16 bytes; routed experts only.
moe_status check_fp8(const moe_shape* shape, const void* ws, size_t ws_bytes, bool whole_layer = false) {
    const moe_status r = check_stage(shape, ws, ws_bytes, whole_layer);
    if (r != MOE_OK) return r;
    if (shape->shared > 0) {
        set_error("block-scaled FP8 experts: shared experts are not supported (shape.shared must be 0; a shared "
                  "expert is a one-expert shape over all tokens)");
        return MOE_ERR_UNSUPPORTED;
    }
    if (shape->hidden % 16 != 0 || shape->inter % 16 != 0) {
        set_error("block-scaled FP8 experts: hidden and inter must be multiples of 16 (got %d, %d)", shape->hidden,
                  shape->inter);
        return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

moe_status do_dispatch(const moe_shape& s, const uint16_t* x, const int32_t* ids, int32_t* counts, int32_t* offsets,
                       int32_t* dest, int32_t* sorted_pair, uint8_t* x_perm, float* x_scale, void* ws, cudaStream_t st) {
    const WsLayout L = ws_layout(s);
    WsHeader* hdr = at<WsHeader>(ws, 0);
    if (dispatch_fp8_small(s))
        return from_cuda(launch_dispatch_fp8_small(s, x, ids, counts, offsets, dest, sorted_pair, x_perm, x_scale, hdr, st));
    int32_t* rank = at<int32_t>(ws, L.rank);
    const cudaError_t e = launch_count(s, ids, counts, offsets, rank, at<unsigned long long>(ws, L.flags),
                                       L.count_tiles, hdr, st);
    if (e != cudaSuccess) return from_cuda(e);
    return from_cuda(launch_scatter_fp8(s, x, ids, offsets, rank, dest, sorted_pair, x_perm, x_scale, hdr, st));
}

moe_status do_up(const moe_shape& s, const uint8_t* x_perm, const float* x_scale, const int32_t* offsets,
                 const uint8_t* w13, const float* w13_scale, uint8_t* h, float* h_scale, void* ws, cudaStream_t st,
                 int gated, const int32_t* ids) {
    Fp8Problem g{};
    g.mode = s.act == MOE_ACT_SWIGLU ? kGemmSwiGLU : kGemmReLU2;
    g.a = x_perm; g.a_scale = x_scale; g.rows = (long long)s.tokens * s.top_k;
    g.offsets = offsets; g.groups = s.experts;
    g.w = w13; g.w_scale = w13_scale;
    g.K = s.hidden; g.N = s.inter;
    g.out = h; g.out_scale = h_scale;
    g.max_group_rows = s.tokens;                   // a token's experts are distinct
    g.gated = gated;
    g.early = ids != nullptr;                      // (the dispatch in front has waited for them)
    g.ids = ids; g.top_k = s.top_k;
    return launch_fp8_gemm(g, at<WsHeader>(ws, 0), st);
}

moe_status do_down(const moe_shape& s, const uint8_t* h, const float* h_scale, const int32_t* offsets,
                   const uint8_t* w2, const float* w2_scale, uint16_t* y_perm, void* ws, cudaStream_t st, int gated,
                   int early) {
    Fp8Problem g{};
    g.mode = kGemmPlain;
    g.a = h; g.a_scale = h_scale; g.rows = (long long)s.tokens * s.top_k;
    g.offsets = offsets; g.groups = s.experts;
    g.w = w2; g.w_scale = w2_scale;
    g.K = s.inter; g.N = s.hidden;
    g.out = y_perm;
    g.early = early;
    g.max_group_rows = s.tokens;                   // a token's experts are distinct
    g.gated = gated;
    return launch_fp8_gemm(g, at<WsHeader>(ws, 0), st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_grouped(const moe_shape* shape, const moe_router* router, const float* logits, const float* bias,
                             int32_t* topk_ids, float* topk_w, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    moe_status r = check_stage(shape, ws, ws_bytes);
    if (r != MOE_OK || (r = check_router(*shape, router)) != MOE_OK) return r;
    if (!aligned(logits, 16) || !aligned_or_null(bias, 4) || !aligned(topk_ids, 16) || !aligned(topk_w, 16))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_route_grouped(*shape, *router, logits, bias, topk_ids, topk_w, at<WsHeader>(ws, 0),
                                          static_cast<cudaStream_t>(stream)));
}

moe_status moe_route_grouped_backward(const moe_shape* shape, const moe_router* router, const float* logits,
                                      const int32_t* topk_ids, const float* dtopk_w, float* dlogits, void* ws,
                                      size_t ws_bytes, void* stream) {
    clear_error();
    moe_status r = check_stage(shape, ws, ws_bytes);
    if (r != MOE_OK || (r = check_router(*shape, router)) != MOE_OK) return r;
    if (!aligned(logits, 16) || !aligned(topk_ids, 16) || !aligned(dtopk_w, 16) || !aligned(dlogits, 16))
        return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_route_grouped_grad(*shape, *router, logits, topk_ids, dtopk_w, dlogits,
                                               at<WsHeader>(ws, 0), static_cast<cudaStream_t>(stream)));
}

moe_status moe_dispatch_fp8_block(const moe_shape* shape, const uint16_t* x, const int32_t* topk_ids, int32_t* counts,
                                  int32_t* offsets, int32_t* dest, int32_t* sorted_pair, uint8_t* x_perm,
                                  float* x_scale, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    const moe_status r = check_fp8(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(x, 16) || !aligned(topk_ids, 16) || !aligned(counts, 16) || !aligned(offsets, 16) ||
        !aligned(dest, 16) || !aligned(sorted_pair, 16) || !aligned(x_perm, 16) || !aligned(x_scale, 16))
        return MOE_ERR_INVALID_ARG;
    return do_dispatch(*shape, x, topk_ids, counts, offsets, dest, sorted_pair, x_perm, x_scale, ws,
                       static_cast<cudaStream_t>(stream));
}

moe_status moe_expert_up_fp8_block(const moe_shape* shape, const uint8_t* x_perm, const float* x_scale,
                                   const int32_t* offsets, const uint8_t* w13, const float* w13_scale, uint8_t* h,
                                   float* h_scale, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    const moe_status r = check_fp8(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(x_perm, 16) || !aligned(x_scale, 16) || !aligned(offsets, 16) || !aligned(w13, 16) ||
        !aligned(w13_scale, 16) || !aligned(h, 16) || !aligned(h_scale, 16))
        return MOE_ERR_INVALID_ARG;
    return do_up(*shape, x_perm, x_scale, offsets, w13, w13_scale, h, h_scale, ws, static_cast<cudaStream_t>(stream), 0,
                 nullptr);
}

moe_status moe_expert_down_fp8_block(const moe_shape* shape, const uint8_t* h, const float* h_scale,
                                     const int32_t* offsets, const uint8_t* w2, const float* w2_scale,
                                     uint16_t* y_perm, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    const moe_status r = check_fp8(shape, ws, ws_bytes);
    if (r != MOE_OK) return r;
    if (!aligned(h, 16) || !aligned(h_scale, 16) || !aligned(offsets, 16) || !aligned(w2, 16) ||
        !aligned(w2_scale, 16) || !aligned(y_perm, 16))
        return MOE_ERR_INVALID_ARG;
    return do_down(*shape, h, h_scale, offsets, w2, w2_scale, y_perm, ws, static_cast<cudaStream_t>(stream), 0, 0);
}

moe_status moe_layer_fp8_block(const moe_shape* shape, const float* logits, const int32_t* ids_in, const float* w_in,
                               const uint16_t* x, const uint8_t* w13, const float* w13_scale, const uint8_t* w2,
                               const float* w2_scale, const uint16_t* residual, uint16_t* out, void* ws,
                               size_t ws_bytes, void* stream) {
    clear_error();
    moe_status r = check_fp8(shape, ws, ws_bytes, true);
    if (r != MOE_OK) return r;
    if (logits ? !aligned(logits, 16) : (!aligned(ids_in, 16) || !aligned(w_in, 16))) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w13_scale, 16) || !aligned(w2, 16) ||
        !aligned(w2_scale, 16) || !aligned(out, 16) || !aligned_or_null(residual, 16))
        return MOE_ERR_INVALID_ARG;
    const moe_shape& s = *shape;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const WsLayout L = ws_layout(s);
    WsHeader* hdr = at<WsHeader>(ws, 0);
    const int32_t* ids = ids_in;
    const float* w = w_in;
    if (logits) {
        int32_t* ids_ws = at<int32_t>(ws, L.ids);
        float* w_ws = at<float>(ws, L.w);
        if ((r = from_cuda(launch_route(s, logits, ids_ws, w_ws, hdr, st))) != MOE_OK) return r;
        ids = ids_ws;
        w = w_ws;
    }
    // codes, then their scales, where the BF16 layer keeps x_perm and h (a row of n codes
    // and n / 128 scales takes at most the 2 n bytes of a BF16 row, n being 16 at least)
    const size_t R = (size_t)s.tokens * s.top_k;
    uint8_t* x_perm = at<uint8_t>(ws, L.x_perm);
    float* x_scale = reinterpret_cast<float*>(x_perm + R * s.hidden);
    uint8_t* h = at<uint8_t>(ws, L.h);
    float* h_scale = reinterpret_cast<float*>(h + R * s.inter);
    uint16_t* y_perm = at<uint16_t>(ws, L.y_perm);
    int32_t* offsets = at<int32_t>(ws, L.offsets);
    int32_t* dest = at<int32_t>(ws, L.dest);
    if ((r = do_dispatch(s, x, ids, at<int32_t>(ws, L.counts), offsets, dest, at<int32_t>(ws, L.sorted_pair), x_perm,
                         x_scale, ws, st)) != MOE_OK)
        return r;
    if ((r = do_up(s, x_perm, x_scale, offsets, w13, w13_scale, h, h_scale, ws, st, 1, ids)) != MOE_OK)
        return r;
    if ((r = do_down(s, h, h_scale, offsets, w2, w2_scale, y_perm, ws, st, 1, 1)) != MOE_OK) return r;
    return from_cuda(launch_combine(s, y_perm, dest, w, nullptr, residual, out, hdr, st));
}

}  // extern "C"
