// permute_grad.cu -- gradients of the weighted combine and of the router.
//
// Combine:  out[t] = sum_j w[t,j] y_perm[dest[t,j]] + ...   (p = t*k + j)
//   dy_perm[dest[p]] = bf16(w[p] * dout[t]),  dw[p] = <dout[t], y_perm[dest[p]]>
// The shared term's and the residual's gradients are dout itself.  Dispatch's
// gradient, dx[t] = sum_j dx_perm[dest[t,j]], is the combine kernel with unit
// weights (launch_combine with w == NULL).
// Router, softmax over the selection: dlogit[ids[j]] = w_j (dw_j - sum_i w_i dw_i),
// zero for the experts not selected.
// Router, sigmoid: w_j = scale p_j with p_j = s_j / sum_i s_i, s = sigmoid(l), so
// dlogit[ids[j]] = scale p_j (1 - s_j) (dw_j - sum_i p_i dw_i); the bias only
// selects and has no gradient.
#include "common.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

constexpr int kBatch = 8;      // pairs of a token whose dot products are in flight together

// One block per token; the pairs in batches of kBatch, each batch one pass over
// the row's 16-byte groups: the batch's y rows are loaded together, then each is
// dotted with dout in FP32 and the scaled dout stored over its slot.  Bound by HBM
// (k rows read and k written a token); what it takes is enough loads in flight,
// which is why the loads stand apart from the stores that might alias them.
// Measured, 16384 tokens x 7168, k = 8: 584 us, 6.9 TB/s (one pair at a time: 795).
// DOTS == false: only dy_perm.
template <bool DOTS>
__global__ void __launch_bounds__(256)
combine_grad_kernel(int T, int HV, int k, const uint4* __restrict__ dout, const uint4* y_perm,
                    const int32_t* __restrict__ dest, const float* __restrict__ w,
                    uint4* dy_perm,    // may alias y_perm: each group is read, then written, by one thread
                    float* __restrict__ dw) {
    __shared__ int dsh[32];
    __shared__ float wsh[32];
    __shared__ float red[8][kBatch];
    pdl_wait();
    pdl_trigger();
    const long long R = (long long)T * k;
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        if (tid < k) {
            const long long p = (long long)t * k + tid;
            const int d = dest[p];
            dsh[tid] = (d >= 0 && d < R) ? d : -1;
            wsh[tid] = w[p];
        }
        __syncthreads();
        for (int j0 = 0; j0 < k; j0 += kBatch) {
            const int nj = min(kBatch, k - j0);
            float acc[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) acc[u] = 0.f;
            for (int c = tid; c < HV; c += nt) {
                uint4 v[DOTS ? kBatch : 1];
                const uint4 dv = __ldg(dout + (size_t)t * HV + c);
                if (DOTS) {
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
                        if (u < nj && dsh[j0 + u] >= 0) v[DOTS ? u : 0] = __ldcs(y_perm + (size_t)dsh[j0 + u] * HV + c);
                }
                float g[8];
                unpack_bf16x8(dv, g);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    if (u >= nj || dsh[j0 + u] < 0) continue;
                    if (DOTS) {
                        float y[8];
                        unpack_bf16x8(v[DOTS ? u : 0], y);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[u] = fmaf(g[i], y[i], acc[u]);
                    }
                    const float wj = wsh[j0 + u];
                    __stcs(dy_perm + (size_t)dsh[j0 + u] * HV + c,
                           make_uint4(pack_bf16x2(wj * g[0], wj * g[1]), pack_bf16x2(wj * g[2], wj * g[3]),
                                      pack_bf16x2(wj * g[4], wj * g[5]), pack_bf16x2(wj * g[6], wj * g[7])));
                }
            }
            if (DOTS) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) acc[u] += __shfl_xor_sync(kAll, acc[u], off);
                    if (lane == 0) red[warp][u] = acc[u];
                }
                __syncthreads();
                if (tid < nj) {
                    float s = 0.f;
                    for (int v = 0; v < (nt >> 5); ++v) s += red[v][tid];
                    dw[(long long)t * k + j0 + tid] = s;       // 0 for an invalid pair
                }
                __syncthreads();
            }
        }
        __syncthreads();
    }
}

// G lanes a token (the power of two at or above k), 32 / G tokens a warp: the warp
// zeroes its tokens' rows, then lane j of a group writes the gradient of the token's
// j-th selected expert.  An id out of range or repeated inside the token (the first
// stays valid, as in the dispatch) takes no part and raises the status.  The
// differences dw_j - sum w dw cancel when one expert dominates, so the few terms of
// a token are taken in double; that unit is slow here (two results a cycle and SM),
// which is why tokens share a warp (a warp a token: 18 us for 16384 x 256, k = 8,
// where writing the rows takes 3).
template <bool SIGMOID, int G>
__global__ void __launch_bounds__(256)
route_grad_kernel(int T, int E, int k, const float* __restrict__ logits, const int32_t* __restrict__ ids,
                  const float* __restrict__ w, float scale, const float* __restrict__ dw,
                  float* __restrict__ dlogits, WsHeader* hdr) {
    constexpr int TPW = 32 / G;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, j = lane % G;
    const unsigned group = (G == 32 ? kAll : ((1u << (G & 31)) - 1u)) << (lane / G * G);
    const int gwarp = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
    const int nwarps = (int)((gridDim.x * blockDim.x) >> 5);
    const int nt = (T + TPW - 1) / TPW;
    for (int wt = gwarp; wt < nt; wt += nwarps) {
        const int t0 = wt * TPW, t = t0 + lane / G;
        const bool mine = t < T && j < k;
        const size_t p = (size_t)t * k + j;
        const int id = mine ? ids[p] : -1 - lane;
        const double g0 = mine ? (double)dw[p] : 0.0;
        const unsigned same = __match_any_sync(kAll, id) & group;
        const bool ok = mine && id >= 0 && id < E && (__ffs(same) - 1) == lane;
        if (mine && !ok) raise_status(hdr, MOE_ERR_INVALID_ROUTE);
        float* rows = dlogits + (size_t)t0 * E;
        const int n = min(TPW, T - t0) * E;
        if (E % 4 == 0) {
            for (int i = lane; i < n / 4; i += 32) reinterpret_cast<float4*>(rows)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            for (int i = lane; i < n; i += 32) rows[i] = 0.f;
        }
        const double g = ok ? g0 : 0.0;
        double pj, f;                                  // mixture weight, outer factor
        if (SIGMOID) {
            // p_j through log s_j, so a row whose scores all underflow keeps its ratios
            const double l = ok ? (double)logits[(size_t)t * E + id] : 0.0;
            const double ls = ok ? fmin(l, 0.0) - log1p(exp(-fabs(l))) : -INFINITY;
            double m = ls;
#pragma unroll
            for (int off = G / 2; off > 0; off >>= 1) m = fmax(m, __shfl_xor_sync(kAll, m, off));
            pj = ok ? exp(ls - m) : 0.0;
            double z = pj;
#pragma unroll
            for (int off = G / 2; off > 0; off >>= 1) z += __shfl_xor_sync(kAll, z, off);
            pj = ok ? pj / z : 0.0;
            f = (double)scale * pj / (1.0 + exp(l));   // 1 - s = 1 / (1 + e^l)
        } else {
            pj = ok ? (double)w[p] : 0.0;
            f = pj;
        }
        double s = pj * g;
#pragma unroll
        for (int off = G / 2; off > 0; off >>= 1) s += __shfl_xor_sync(kAll, s, off);
        __syncwarp();                                  // the zeros come before the selected entries
        if (ok) rows[(size_t)(t - t0) * E + id] = (float)(f * (g - s));
    }
}

template <bool SIGMOID, int G>
cudaError_t route_grad(const moe_shape& s, const float* logits, const int32_t* ids, const float* w, float scale,
                       const float* dw, float* dlogits, WsHeader* hdr, cudaStream_t st) {
    long long blocks = ((long long)s.tokens * G + 255) / 256;
    const long long cap = (long long)device_sm_count() * 8;
    if (blocks > cap) blocks = cap;
    return launch_kernel(route_grad_kernel<SIGMOID, G>, dim3((unsigned)blocks), dim3(256), 0, st, 1, kUsePdl, s.tokens,
                         s.experts, s.top_k, logits, ids, w, scale, dw, dlogits, hdr);
}

template <bool SIGMOID>
cudaError_t route_grad_by_k(const moe_shape& s, const float* logits, const int32_t* ids, const float* w, float scale,
                            const float* dw, float* dlogits, WsHeader* hdr, cudaStream_t st) {
    if (s.top_k <= 2) return route_grad<SIGMOID, 2>(s, logits, ids, w, scale, dw, dlogits, hdr, st);
    if (s.top_k <= 4) return route_grad<SIGMOID, 4>(s, logits, ids, w, scale, dw, dlogits, hdr, st);
    if (s.top_k <= 8) return route_grad<SIGMOID, 8>(s, logits, ids, w, scale, dw, dlogits, hdr, st);
    if (s.top_k <= 16) return route_grad<SIGMOID, 16>(s, logits, ids, w, scale, dw, dlogits, hdr, st);
    return route_grad<SIGMOID, 32>(s, logits, ids, w, scale, dw, dlogits, hdr, st);
}

}  // namespace

cudaError_t launch_combine_grad(const moe_shape& s, const uint16_t* dout, const uint16_t* y_perm, const int32_t* dest,
                                const float* w, uint16_t* dy_perm, float* dw, cudaStream_t st) {
    const int HV = s.hidden / 8;
    int threads = 32;
    while (threads < 256 && threads < HV) threads *= 2;
    // a block a token up to many waves: with resident blocks looping over tokens a
    // token's end (its reductions) left too few loads in flight (16384 x 7168, k = 8:
    // 640 against 584 us)
    long long blocks = s.tokens;
    const long long cap = (long long)device_sm_count() * 1024;
    if (blocks > cap) blocks = cap;
    return launch_kernel(dw ? combine_grad_kernel<true> : combine_grad_kernel<false>, dim3((unsigned)blocks),
                         dim3(threads), 0, st, 1, kUsePdl, s.tokens, HV, s.top_k, reinterpret_cast<const uint4*>(dout),
                         reinterpret_cast<const uint4*>(y_perm), dest, w, reinterpret_cast<uint4*>(dy_perm), dw);
}

cudaError_t launch_route_grad(const moe_shape& s, const float* logits, const int32_t* ids, const float* w, float scale,
                              const float* dw, float* dlogits, WsHeader* hdr, cudaStream_t st) {
    return logits ? route_grad_by_k<true>(s, logits, ids, w, scale, dw, dlogits, hdr, st)
                  : route_grad_by_k<false>(s, logits, ids, w, scale, dw, dlogits, hdr, st);
}

}  // namespace moe
