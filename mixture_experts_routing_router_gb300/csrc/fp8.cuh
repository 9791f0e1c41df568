// fp8.cuh -- E4M3 activations with an FP32 scale per row and 128 columns.
//
// For the values x of a block of 128 columns of a row, with a = max(max|x|, 2^-100):
//   scale = a / 448,   code = the E4M3 value nearest 448 x / a (ties to even).
// 448 x / a is taken as (0.875 x) / (a / 512): no product here can overflow, and for
// BF16 x both sides are exact, so the quotient is a tie between two codes in FP32 only
// if it is one.  For FP32 x (the up projection's results) 0.875 x is rounded first, so a
// quotient within a few 2^-24 of a border may fall to either side.  A block with a NaN or an infinity has the scale NaN and the codes NaN.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kFp8Block = 128;
constexpr float kFp8AmaxFloor = 0x1p-100f;

inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

// max(a, |b|) that keeps a NaN.
__device__ __forceinline__ float amax_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

struct Fp8Quant {
    float scale, div, inv;      // scale of the block; a / 512 and its reciprocal
};
__device__ __forceinline__ Fp8Quant fp8_quant(float amax) {
    Fp8Quant q;
    amax = amax_nan(amax, kFp8AmaxFloor);
    const float a = amax <= 3.4028235e38f ? amax : __int_as_float(0x7fffffff);
    q.scale = a / 448.0f;
    q.div = a * (1.0f / 512.0f);
    q.inv = 1.0f / q.div;
    return q;
}
// 0.875 x / div, correctly rounded: one step of correction on the product with the
// (correctly rounded) reciprocal.
__device__ __forceinline__ float fp8_scaled(const Fp8Quant& q, float x) {
    const float a = 0.875f * x;
    const float y = a * q.inv;
    return fmaf(fmaf(-y, q.div, a), q.inv, y);
}
// Two values to E4M3 codes, `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t fp8_quant4(const Fp8Quant& q, float a, float b, float c, float d) {
    return e4m3x2(fp8_scaled(q, a), fp8_scaled(q, b)) | (e4m3x2(fp8_scaled(q, c), fp8_scaled(q, d)) << 16);
}

// Grouped product of E4M3 rows and E4M3 weights:
//   y[r, n] = sum_b a_scale[r, b] w_scale[g, n / 128, b] sum_{c in block b} a[r, c] w[g, n, c]
// over the rows r of group g, FP32 sums (the scales' product is taken first, in FP32); then plain BF16, or an activation quantized
// again (SwiGLU: the weights' gate rows, then their up rows, each with blocks of its own).
struct Fp8Problem {
    int mode;                                  // kGemmSwiGLU / kGemmReLU2 / kGemmPlain
    const uint8_t* a; const float* a_scale;    // [rows, K], [rows, ceil(K / 128)]
    long long rows;
    const int32_t* offsets; int groups;        // [groups + 1]
    const uint8_t* w; const float* w_scale;    // [groups, parts, N, K], [groups, parts, ceil(N / 128), ceil(K / 128)]
    int K, N;
    void* out; float* out_scale;               // plain: bf16 [rows, N]; else E4M3 [rows, N], [rows, ceil(N / 128)]
    int max_group_rows;                        // host bound on the rows of a group
    int gated;                                 // as GemmProblem
    int early;                                 // 1: the bucket bounds are final when the kernel starts, or
    const int32_t* ids; int top_k;             //    (not null) the experts of every token, [rows / top_k, top_k]
};
moe_status launch_fp8_gemm(const Fp8Problem& p, WsHeader* hdr, cudaStream_t st);

// The dispatch with the rows quantized on the way: in one launch for a small batch, else
// launch_count and launch_scatter_fp8.
bool dispatch_fp8_small(const moe_shape& s);
cudaError_t launch_dispatch_fp8_small(const moe_shape& s, const uint16_t* x, const int32_t* ids, int32_t* counts,
                                      int32_t* offsets, int32_t* dest, int32_t* sorted_pair, uint8_t* x_perm,
                                      float* x_scale, WsHeader* hdr, cudaStream_t st);
cudaError_t launch_scatter_fp8(const moe_shape& s, const uint16_t* x, const int32_t* ids, const int32_t* offsets,
                               const int32_t* rank, int32_t* dest, int32_t* sorted_pair, uint8_t* x_perm,
                               float* x_scale, WsHeader* hdr, cudaStream_t st);

cudaError_t launch_route_grouped(const moe_shape& s, const moe_router& r, const float* logits, const float* bias,
                                 int32_t* ids, float* w, WsHeader* hdr, cudaStream_t st);
cudaError_t launch_route_grouped_grad(const moe_shape& s, const moe_router& r, const float* logits, const int32_t* ids,
                                      const float* dw, float* dlogits, WsHeader* hdr, cudaStream_t st);

}  // namespace moe
