// layernorm.cu -- the layer norm in front of the router, forward and backward,
// with the reduction of the weight's gradient.
//
//   y = (x - mean) * rstd * gamma + beta,   rstd = 1 / sqrt(var + eps)
//   a = dy * gamma, xhat = (x - mean) * rstd
//   dx = rstd * (a - mean_c(a) - xhat * mean_c(a * xhat)) + dres
//   dgamma = sum_rows dy * xhat,  dbeta = sum_rows dy
// mean_c is the mean over a row's columns.  Every sum is held in FP32; the
// variance is the mean of the centred squares (not E[x^2] - mean^2), so a row
// with a large offset keeps its digits.  Outputs of type BF16 are rounded once.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kLnThreads = 256;

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Sum over the block, the same on every thread; `red` holds one float per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += red[w];
    return s;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLnThreads)
layernorm_kernel(long long rows, int H, const T* x, const W* __restrict__ gamma, const W* __restrict__ beta,
                 float eps, T* y,      // may alias x
                 float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float red[kLnThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + (size_t)r * H;
        T* yr = y + (size_t)r * H;
        float s = 0.f;
        for (int c = tid; c < H; c += kLnThreads) s += to_f32(xr[c]);
        const float mu = block_sum(s, red) / (float)H;
        float q = 0.f;
        for (int c = tid; c < H; c += kLnThreads) {
            const float d = to_f32(xr[c]) - mu;
            q = fmaf(d, d, q);
        }
        const float rs = 1.0f / sqrtf(block_sum(q, red) / (float)H + eps);
        for (int c = tid; c < H; c += kLnThreads)
            yr[c] = from_f32<T>(fmaf((to_f32(xr[c]) - mu) * rs, to_f32(gamma[c]), to_f32(beta[c])));
        if (tid == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLnThreads)
layernorm_dx_kernel(long long rows, int H, const T* dy, const T* x, const W* __restrict__ gamma,
                    const float* __restrict__ mean, const float* __restrict__ rstd, const T* dres,
                    T* dx) {           // may alias dy, x or dres

    __shared__ float red[kLnThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
        const size_t o = (size_t)r * H;
        const float mu = mean[r], rs = rstd[r];
        float sa = 0.f, sb = 0.f;
        for (int c = tid; c < H; c += kLnThreads) {
            const float a = to_f32(dy[o + c]) * to_f32(gamma[c]);
            sa += a;
            sb = fmaf(a, (to_f32(x[o + c]) - mu) * rs, sb);
        }
        const float ma = block_sum(sa, red) / (float)H, mb = block_sum(sb, red) / (float)H;
        for (int c = tid; c < H; c += kLnThreads) {
            const float a = to_f32(dy[o + c]) * to_f32(gamma[c]);
            const float xh = (to_f32(x[o + c]) - mu) * rs;
            float v = (a - ma - xh * mb) * rs;
            if (dres) v += to_f32(dres[o + c]);
            dx[o + c] = from_f32<T>(v);
        }
    }
}

// Partial sums of dgamma and dbeta over the rows p, p + parts, ...: one block
// per (256 columns, part), written to scratch as [part][2][H].
template <typename T>
__global__ void __launch_bounds__(kLnThreads)
layernorm_dw_partial_kernel(long long rows, int H, const T* __restrict__ dy, const T* __restrict__ x,
                            const float* __restrict__ mean, const float* __restrict__ rstd,
                            float* __restrict__ part) {
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x * kLnThreads + threadIdx.x;
    if (c >= H) return;
    float g = 0.f, b = 0.f;
    for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
        const float d = to_f32(dy[(size_t)r * H + c]);
        g = fmaf(d, (to_f32(x[(size_t)r * H + c]) - mean[r]) * rstd[r], g);
        b += d;
    }
    float* p = part + (size_t)blockIdx.y * 2 * H;
    p[c] = g;
    p[H + c] = b;
}

__global__ void __launch_bounds__(kLnThreads)
layernorm_dw_final_kernel(int parts, int H, const float* __restrict__ part, float* __restrict__ dgamma,
                          float* __restrict__ dbeta) {
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x * kLnThreads + threadIdx.x;
    if (c >= H) return;
    float g = 0.f, b = 0.f;
    for (int p = 0; p < parts; ++p) {
        g += part[(size_t)p * 2 * H + c];
        b += part[(size_t)p * 2 * H + H + c];
    }
    dgamma[c] = g;
    dbeta[c] = b;
}

unsigned row_blocks(long long rows) {
    const long long cap = (long long)device_sm_count() * 8;
    return (unsigned)(rows < cap ? rows : cap);
}

template <typename T, typename W>
cudaError_t forward(const LayerNormProblem& p, cudaStream_t st) {
    return launch_kernel(layernorm_kernel<T, W>, dim3(row_blocks(p.rows)), dim3(kLnThreads), 0, st, 1, kUsePdl,
                         p.rows, p.hidden, static_cast<const T*>(p.x), static_cast<const W*>(p.gamma),
                         static_cast<const W*>(p.beta), p.eps, static_cast<T*>(p.y), p.mean, p.rstd);
}

template <typename T, typename W>
cudaError_t backward(const LayerNormProblem& p, cudaStream_t st) {
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.dy);
    const unsigned cols = (unsigned)((p.hidden + kLnThreads - 1) / kLnThreads);
    const int parts = layernorm_parts(p.rows);
    // the weight's partial sums first: dx may overwrite dy
    cudaError_t e = launch_kernel(layernorm_dw_partial_kernel<T>, dim3(cols, (unsigned)parts), dim3(kLnThreads), 0, st,
                                  1, kUsePdl, p.rows, p.hidden, dy, x, p.mean, p.rstd, p.scratch);
    if (e == cudaSuccess)
        e = launch_kernel(layernorm_dw_final_kernel, dim3(cols), dim3(kLnThreads), 0, st, 1, kUsePdl, parts, p.hidden,
                          static_cast<const float*>(p.scratch), p.dgamma, p.dbeta);
    if (e == cudaSuccess && p.rows > 0)
        e = launch_kernel(layernorm_dx_kernel<T, W>, dim3(row_blocks(p.rows)), dim3(kLnThreads), 0, st, 1, kUsePdl,
                          p.rows, p.hidden, dy, x, static_cast<const W*>(p.gamma), p.mean, p.rstd,
                          static_cast<const T*>(p.dres), static_cast<T*>(p.dx));
    return e;
}

}  // namespace

cudaError_t launch_layernorm(const LayerNormProblem& p, cudaStream_t st) {
    if (p.rows == 0) return cudaSuccess;
    if (p.type == MOE_TYPE_BF16)
        return p.wtype == MOE_TYPE_BF16 ? forward<__nv_bfloat16, __nv_bfloat16>(p, st) : forward<__nv_bfloat16, float>(p, st);
    return p.wtype == MOE_TYPE_BF16 ? forward<float, __nv_bfloat16>(p, st) : forward<float, float>(p, st);
}

cudaError_t launch_layernorm_backward(const LayerNormProblem& p, cudaStream_t st) {
    if (p.type == MOE_TYPE_BF16)
        return p.wtype == MOE_TYPE_BF16 ? backward<__nv_bfloat16, __nv_bfloat16>(p, st) : backward<__nv_bfloat16, float>(p, st);
    return p.wtype == MOE_TYPE_BF16 ? backward<float, __nv_bfloat16>(p, st) : backward<float, float>(p, st);
}

}  // namespace moe
