// dispatch_fp8.cu -- the stable scatter of dispatch.cu with the rows quantized to E4M3
// on the way (fp8.cuh): x_perm[dest[p]] = codes of x[p / k], x_scale[dest[p]] their scales.
//
// Placement as in scatter_kernel (counts and ranks come from the same count kernel; a small
// batch has a kernel of its own, below).  A block takes a token; 8 lanes share a 128-column
// block of the row, 16 columns each, find its largest magnitude with three shuffles and
// write the codes to the token's k slots.
// Bound by HBM: H * 2 bytes read and k * (H + H / 32) written a token.  16384 tokens x 7168,
// k = 8: 184 us, 6.2 TB/s, of a dispatch's 202.  A block a token over many waves: resident
// blocks that loop over tokens have too few loads in flight (a dispatch takes 225).
#include "fp8.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// Four 128-column blocks, b0 .. b0 + 3, of a row (H columns) on one warp, 16 columns a lane.
__device__ __forceinline__ void load_four_blocks(const uint16_t* src, int H, int b0, int lane, uint32_t (&u)[8]) {
    const int c = b0 * 128 + lane * 16;            // this lane's columns
    uint4 v = make_uint4(0u, 0u, 0u, 0u), w = v;
    if (c < H) {
        v = __ldcs(reinterpret_cast<const uint4*>(src + c));
        w = __ldcs(reinterpret_cast<const uint4*>(src + c) + 1);
    }
    u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
    u[4] = w.x; u[5] = w.y; u[6] = w.z; u[7] = w.w;
}
// Their codes and scales to the slots dsh[0 .. k-1] (negative ones are left out).
__device__ __forceinline__ void quantize_four_blocks(const uint32_t (&u)[8], int H, int nb, int b0, int lane, int k,
                                                     const int* dsh, uint8_t* x_perm, float* x_scale) {
    const int c = b0 * 128 + lane * 16;
    const bool in = c < H;
    float f[16], m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        m = amax_nan(amax_nan(m, f[2 * i]), f[2 * i + 1]);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) m = amax_nan(m, __shfl_xor_sync(kAll, m, off));
    const Fp8Quant q = fp8_quant(m);
    uint32_t code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) code[i] = fp8_quant4(q, f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    const int b = b0 + (lane >> 3);
    const bool lead = (lane & 7) == 0 && b < nb;
    for (int j = 0; j < k; ++j) {
        const int d = dsh[j];
        if (d < 0) continue;
        if (in) *reinterpret_cast<uint4*>(x_perm + (size_t)d * H + c) = make_uint4(code[0], code[1], code[2], code[3]);
        if (lead) x_scale[(size_t)d * nb + b] = q.scale;
    }
}

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
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
    const int nb = (H + kFp8Block - 1) / kFp8Block;
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
        for (int b0 = 4 * warp; b0 < nb; b0 += 4 * warps) {
            uint32_t u[8];
            load_four_blocks(x + (size_t)t * H, H, b0, lane, u);
            quantize_four_blocks(u, H, nb, b0, lane, k, dsh, x_perm, x_scale);
        }
        __syncthreads();
    }
}

// The whole dispatch of up to kSmallPairs pairs in one launch: every block counts all pairs
// (and those before its own tokens') in shared memory, so that none waits for another;
// then it places and quantizes its tokens.  1024 tokens x 2048, k = 6, 64 experts: 8.7
// us, against 14.2 of clearing the look-back flags, counting and scattering in turn.
// Stable, and what is valid, as count_kernel and scatter_kernel have it: the slot of pair p
// is offsets[e] + the valid pairs of e before p.
constexpr int kSmallThreads = 1024;

__global__ void __launch_bounds__(kSmallThreads)
dispatch_fp8_kernel(int T, int H, int k, int E, int capacity, const uint16_t* __restrict__ x,
                    const int32_t* __restrict__ ids, int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                    int32_t* __restrict__ dest, int32_t* __restrict__ sorted_pair, uint8_t* __restrict__ x_perm,
                    float* __restrict__ x_scale, WsHeader* hdr) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ int sm[];
    int* total = sm;                               // [E], then its exclusive scan
    int* before = total + E;                       // [E] of the pairs before this block's
    int* mine = before + E;                        // [own pairs] expert (-1: invalid), then slot
    __shared__ int wsum[kSmallThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = (int)((long long)T * blockIdx.x / gridDim.x), t1 = (int)((long long)T * (blockIdx.x + 1) / gridDim.x);
    const bool lead = blockIdx.x == 0;
    // the warp's first piece of a row is on its way while the pairs are counted
    const int nb = (H + kFp8Block - 1) / kFp8Block, items = (nb + 3) / 4;
    uint32_t u[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (warp < (t1 - t0) * items) load_four_blocks(x + (size_t)(t0 + warp / items) * H, H, 4 * (warp % items), lane, u);
    for (int e = tid; e < 2 * E; e += kSmallThreads) sm[e] = 0;
    __syncthreads();
    // whole tokens a warp: lanes of a token sit together, the first of equal ids counts
    const int tpw = 32 / k, used = tpw * k, step = (kSmallThreads / 32) * tpw, j = lane % k;
    constexpr int kAhead = 8;                      // loads under way together
    for (int tb = warp * tpw; tb < T; tb += kAhead * step) {
        int next[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int t = tb + a * step + lane / k;
            next[a] = lane < used && t < T ? __ldg(ids + (size_t)(tb + a * step) * k + lane) : -1;
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            if (tb + a * step >= T) break;
            const int t = tb + a * step + lane / k, id = next[a];
            const bool pair = lane < used && t < T;
            bool ok = pair && id >= 0 && id < E;
            for (int b = 1; b < k; ++b) {          // (a match over the warp took 60 cycles of the SM)
                const int earlier = __shfl_up_sync(kAll, id, b);
                ok = ok && !(j >= b && earlier == id);
            }
            if (ok) {
                atomicAdd(&total[id], 1);
                if (t < t0) atomicAdd(&before[id], 1);
            }
            if (pair && !ok && lead) raise_status(hdr, MOE_ERR_INVALID_ROUTE);
            if (pair && t >= t0 && t < t1) mine[(t - t0) * k + j] = ok ? id : -1;
        }
    }
    __syncthreads();
    // ---- exclusive scan of the counts; capacity
    const int per = (E + kSmallThreads - 1) / kSmallThreads, e0 = tid * per;
    int loc = 0, over = 0;
    for (int e = e0; e < min(e0 + per, E); ++e) {
        const int c = total[e];
        if (lead) counts[e] = c;
        over |= c > capacity;
        loc += c;
    }
    int inc = loc;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(kAll, inc, off);
        if (lane >= off) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    over = __syncthreads_or(over);
    int run = inc - loc + __reduce_add_sync(kAll, lane < warp ? wsum[lane] : 0);
    for (int e = e0; e < min(e0 + per, E); ++e) {
        const int c = total[e];
        total[e] = run;
        if (lead) offsets[e] = run;
        run += c;
    }
    if (lead && tid == kSmallThreads - 1) {
        offsets[E] = run;
        hdr->cap_exceeded = over;
        if (over) raise_status(hdr, MOE_ERR_CAPACITY);
    }
    if (over) return;                              // over capacity: no payload moves
    __syncthreads();
    // ---- slots of this block's pairs
    const int own = (t1 - t0) * k;                 // a thread each (dispatch_fp8_small)
    int slot = -1;
    if (tid < own) {
        const int e = mine[tid];
        if (e >= 0) {
            slot = total[e] + before[e];
            for (int j = 0; j < tid; ++j) slot += mine[j] == e;
        }
        dest[(size_t)t0 * k + tid] = slot;
        if (slot >= 0) sorted_pair[slot] = t0 * k + tid;
    }
    __syncthreads();
    if (tid < own) mine[tid] = slot;
    __syncthreads();
    // ---- rows
    for (int i = warp; i < (t1 - t0) * items; i += kSmallThreads / 32) {
        const int t = i / items, b0 = 4 * (i - t * items);
        if (i > warp) load_four_blocks(x + (size_t)(t0 + t) * H, H, b0, lane, u);
        quantize_four_blocks(u, H, nb, b0, lane, k, mine + t * k, x_perm, x_scale);
    }
}

}  // namespace

// Up to this many pairs the counting of all of them by every block (ids from L2) costs less
// than two more launches.
constexpr long long kSmallPairs = 12288;

bool dispatch_fp8_small(const moe_shape& s) {
    const int sms = device_sm_count(), grid = s.tokens < sms ? s.tokens : sms;
    return (long long)s.tokens * s.top_k <= kSmallPairs && (s.tokens + grid - 1) / grid * s.top_k <= kSmallThreads;
}

cudaError_t launch_dispatch_fp8_small(const moe_shape& s, const uint16_t* x, const int32_t* ids, int32_t* counts,
                                      int32_t* offsets, int32_t* dest, int32_t* sorted_pair, uint8_t* x_perm,
                                      float* x_scale, WsHeader* hdr, cudaStream_t st) {
    const int sms = device_sm_count(), grid = s.tokens < sms ? s.tokens : sms;
    const int own = (s.tokens + grid - 1) / grid * s.top_k;
    const size_t smem = (size_t)(2 * s.experts + own) * sizeof(int);
    return launch_kernel(dispatch_fp8_kernel, dim3((unsigned)grid), dim3(kSmallThreads), smem, st, 1, kUsePdl, s.tokens,
                         s.hidden, s.top_k, s.experts, s.capacity, x, ids, counts, offsets, dest, sorted_pair, x_perm,
                         x_scale, hdr);
}

cudaError_t launch_scatter_fp8(const moe_shape& s, const uint16_t* x, const int32_t* ids, const int32_t* offsets,
                               const int32_t* rank, int32_t* dest, int32_t* sorted_pair, uint8_t* x_perm,
                               float* x_scale, WsHeader* hdr, cudaStream_t st) {
    // four blocks of the row a warp and pass, no pass with idle warps; a block a token
    const int items = (fp8_blocks(s.hidden) + 3) / 4, passes = (items + 7) / 8, threads = 32 * ((items + passes - 1) / passes);
    long long blocks = s.tokens;
    const long long cap = (long long)device_sm_count() * 1024;
    if (blocks > cap) blocks = cap;
    return launch_kernel(scatter_fp8_kernel, dim3((unsigned)blocks), dim3(threads), 0, st, 1, kUsePdl, s.tokens,
                         s.hidden, s.top_k, s.experts, x, ids, offsets, rank, dest, sorted_pair, x_perm, x_scale,
                         static_cast<const WsHeader*>(hdr));
}

}  // namespace moe
