// dispatch_fp8.cu -- the stable scatter of dispatch.cu with the rows quantized to E4M3
// on the way (fp8.cuh): x_perm[dest[p]] = codes of x[p / k], x_scale[dest[p]] their scales.
//
// Placement as in scatter_kernel (counts and ranks come from the same count kernel).  A
// block takes a token; 16 lanes share a 128-column block of the row, 8 columns each, find
// its largest magnitude with four shuffles and write the codes to the token's k slots.
// Bound by HBM: H * 2 bytes read and k * (H + H / 32) written a token.
#include "fp8.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__global__ void __launch_bounds__(256)
scatter_fp8_kernel(int T, int H, int k, int E, const uint16_t* __restrict__ x, const int32_t* __restrict__ ids,
                   const int32_t* __restrict__ offsets, const int32_t* __restrict__ rank, int32_t* __restrict__ dest,
                   int32_t* __restrict__ sorted_pair, uint8_t* __restrict__ x_perm, float* __restrict__ x_scale,
                   const WsHeader* hdr) {
    pdl_wait();
    pdl_trigger();
    if (hdr->cap_exceeded) return;                 // over capacity: no payload moves
    __shared__ int dsh[32];
    const long long R = (long long)T * k;
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, sub = lane & 15;
    const int HV = H / 8, nb = (H + kFp8Block - 1) / kFp8Block;
    const int warps = nt >> 5, warp = tid >> 5;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        if (tid < k) {
            const long long p = (long long)t * k + tid;
            const int e = ids[p];
            const int r = rank[p];
            int d = -1;
            if (r >= 0 && e >= 0 && e < E) {
                const long long dd = (long long)offsets[e] + r;
                if (dd >= 0 && dd < R) d = (int)dd;
            }
            dest[p] = d;
            if (d >= 0) sorted_pair[d] = (int)p;
            dsh[tid] = d;
        }
        __syncthreads();
        const uint4* src = reinterpret_cast<const uint4*>(x) + (size_t)t * HV;
        // a warp takes two 128-column blocks at a time
        for (int b0 = 2 * warp; b0 < nb; b0 += 2 * warps) {
            const int c = b0 * 16 + lane;          // 8-column group of this lane
            const bool in = c < HV;
            const uint4 v = in ? __ldcs(src + c) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
            float f[8], m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
                m = amax_nan(amax_nan(m, f[2 * i]), f[2 * i + 1]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) m = amax_nan(m, __shfl_xor_sync(kAll, m, off));
            const Fp8Quant q = fp8_quant(m);
            const uint2 code = make_uint2(fp8_quant4(q, f[0], f[1], f[2], f[3]), fp8_quant4(q, f[4], f[5], f[6], f[7]));
            const int b = b0 + (lane >> 4);
            for (int j = 0; j < k; ++j) {
                const int d = dsh[j];
                if (d < 0) continue;
                if (in) *reinterpret_cast<uint2*>(x_perm + (size_t)d * H + 8 * c) = code;
                if (sub == 0 && b < nb) x_scale[(size_t)d * nb + b] = q.scale;
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_scatter_fp8(const moe_shape& s, const uint16_t* x, const int32_t* ids, const int32_t* offsets,
                               const int32_t* rank, int32_t* dest, int32_t* sorted_pair, uint8_t* x_perm,
                               float* x_scale, WsHeader* hdr, cudaStream_t st) {
    int threads = 32;
    while (threads < 256 && threads < s.hidden / 8) threads *= 2;
    long long blocks = s.tokens;
    const long long cap = (long long)device_sm_count() * (2048 / threads);
    if (blocks > cap) blocks = cap;
    return launch_kernel(scatter_fp8_kernel, dim3((unsigned)blocks), dim3(threads), 0, st, 1, kUsePdl, s.tokens,
                         s.hidden, s.top_k, s.experts, x, ids, offsets, rank, dest, sorted_pair, x_perm, x_scale,
                         static_cast<const WsHeader*>(hdr));
}

}  // namespace moe
