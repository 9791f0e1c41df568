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
//
// Both directions are bound by HBM: each input is read once and each output
// written once.  A row belongs to TPR threads (32 .. 512, by its width) with 32
// columns each (backward 16, and 32 above 8192 columns); a block of 512 threads
// holds 512 / TPR rows and walks down the batch, one block an SM.  A thread copies
// its own columns of the rows to come into its own shared-memory slots with
// cp.async -- no barrier, and the registers stay free -- so the next rows' reads
// run under this row's reductions.  gamma and beta stay in registers over all rows
// of the block: read again for each row, from L1, they were four times the row.
// The backward pass also keeps the running dgamma and dbeta of its columns in
// registers, so the weight's gradient costs no further read of x and dy, only one
// [blocks][2][H] FP32 array, summed by a second small kernel in a fixed order.
// Rows wider than 16384 columns (8192 FP32 columns backward) run the looping
// kernels, which re-read the row through L2.
// Measured, [16384, 7168] BF16: forward 76 us, 6.2 TB/s (weights from L1: 159 us;
// 16 columns a thread, the issue slots going to the reductions: 99 us); backward
// with the residual's gradient 154 us, 6.1 TB/s (three passes over x and dy: 507).
#include "common.cuh"

#include <mutex>

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

// ---- rows held by TPR threads ---------------------------------------------------
// One access of a thread is 16 bytes: VN elements.  When hidden is no multiple of VN
// the rows start at offsets inside such a chunk that repeat every VN rows at most.
// A row group then only takes rows of one offset (the number of groups is a multiple
// of VN), so a thread still has the same columns in every row; its chunks begin at
// the chunk boundary before the row, and the first and last one, which the row shares
// with its neighbours, are written element by element.  ([16384, 7167] BF16 forward:
// 153 us, backward 225; single elements throughout: 255 and 629.)
template <typename T> constexpr int kVN = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store(uint4* p, const float (&f)[8]) {
    __stcs(p, make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])));
}
__device__ __forceinline__ void store(uint4* p, const float (&f)[4]) {
    __stcs(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
}
// The VN elements from element c of row `out`, those inside [0, H) of a shared chunk.
template <int VN, typename T>
__device__ __forceinline__ void store_chunk(T* out, int c, int H, bool whole, const float (&f)[VN]) {
    if (whole) {
        store(reinterpret_cast<uint4*>(out + c), f);
    } else {
#pragma unroll
        for (int e = 0; e < VN; ++e)
            if (c + e >= 0 && c + e < H) out[c + e] = from_f32<T>(f[e]);
    }
}

// The VN weights from column c, zeros outside [0, H).
template <int VN>
__device__ __forceinline__ void load_weight(const void* w, bool bf16, int c, int H, bool whole, float (&f)[VN]) {
    if (!whole) {
#pragma unroll
        for (int e = 0; e < VN; ++e) {
            const int i = c + e;
            f[e] = i < 0 || i >= H ? 0.f
                   : bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
        }
    } else if ((c & (VN - 1)) != 0) {          // whole, but off the weights' own chunks
#pragma unroll
        for (int e = 0; e < VN; ++e)
            f[e] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c + e]) : static_cast<const float*>(w)[c + e];
    } else if (bf16) {
        const unsigned short* p = static_cast<const unsigned short*>(w) + c;
        if constexpr (VN == 8) {
            unpack(__ldg(reinterpret_cast<const uint4*>(p)), f);
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
            f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
            f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
        }
    } else {
        const float* p = static_cast<const float*>(w) + c;
#pragma unroll
        for (int i = 0; i < VN / 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
            f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
        }
    }
}

// Copy the chunk from element c of a row into this thread's slot.  A chunk shared with
// a neighbouring row is copied whole too (clear() drops what is not the row's); only
// one that reaches past the tensor's end (`inside` false) goes element by element.
template <typename T>
__device__ __forceinline__ void fetch_chunk(uint4* slot, const T* row, int c, int H, bool inside) {
    if (inside) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(slot)), "l"(row + c) : "memory");
    } else {
#pragma unroll
        for (int e = 0; e < kVN<T>; ++e)
            if (c + e >= 0 && c + e < H) reinterpret_cast<T*>(slot)[e] = row[c + e];
    }
}
template <int VN>
__device__ __forceinline__ void clear(float (&f)[VN], int c, int H) {
#pragma unroll
    for (int e = 0; e < VN; ++e)
        if (c + e < 0 || c + e >= H) f[e] = 0.f;
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

constexpr int NT = 512;                            // threads of a block

// N sums over the TPR threads of a row, the same on each: shuffles inside a warp,
// then each warp reads the row's warp sums, one a lane, and shuffles again.  `red`
// holds N floats per warp of the block, in two halves that alternate (`flip`), so
// one barrier a sum is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int group, int& flip) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int lane = threadIdx.x & 31;
        float* half = red + flip * (N * NT / 32);
        if (lane == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) half[n * (NT / 32) + (threadIdx.x >> 5)] = v[n];
        }
        asm volatile("bar.sync %0, %1;" :: "r"(1 + group), "n"(TPR) : "memory");
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = half[n * (NT / 32) + group * W + (lane & (W - 1))];
#pragma unroll
        for (int off = W / 2; off > 0; off >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], off);
        flip ^= 1;
    }
}

constexpr size_t kSlotBytes = 192 * 1024;          // shared memory for the rows to come, per SM
// Rows in flight per group: as many as fit.
template <typename T> constexpr int stages_of(int arrays, int cols) {
    return (int)(kSlotBytes / ((size_t)arrays * cols * sizeof(T) * NT));
}
constexpr int kFwdCols = 32, kBwdCols = 16;        // columns a thread (backward above 8192 columns: 32)

// What every thread of a row group knows about its columns: element `at(i)` of the
// row begins its i-th chunk; `has` it any element, are they all the row's (`whole`).
// ODD: the row is not a whole number of chunks.
template <typename T, int TPR, bool ODD>
struct Columns {
    static constexpr int VN = kVN<T>;
    int H, lane, shift;
    __device__ __forceinline__ Columns(int H_, int lane_, long long row) : H(H_), lane(lane_), shift(0) {
        if (ODD) shift = (int)((unsigned long long)row * (unsigned)H_ % VN);
    }
    __device__ __forceinline__ int at(int i) const { return (lane + i * TPR) * VN - shift; }
    __device__ __forceinline__ bool has(int i) const { return at(i) < H; }
    __device__ __forceinline__ bool whole(int i) const { return !ODD || (at(i) >= 0 && at(i) + VN <= H); }
    __device__ __forceinline__ bool inside(int i, long long row, long long rows) const {
        return !ODD || at(i) + VN <= (rows - row) * H;
    }
};

template <typename T, int TPR, bool ODD>
__global__ void __launch_bounds__(NT, 1)
layernorm_rows_kernel(long long rows, int H, const T* x, const void* __restrict__ gamma,
                      const void* __restrict__ beta, bool wbf16, float eps, T* y, float* __restrict__ mean,
                      float* __restrict__ rstd) {
    constexpr int VN = kVN<T>, RPB = NT / TPR, V = kFwdCols / VN, S = stages_of<T>(1, kFwdCols);
    static_assert(S >= 2, "stages");
    extern __shared__ __align__(16) uint8_t smem_ln[];
    uint4* slots = reinterpret_cast<uint4*>(smem_ln);             // [stage][V][NT]
    __shared__ float red[2 * NT / 32];
    const int tid = threadIdx.x, group = tid / TPR, lane = tid % TPR;
    const long long first = (long long)blockIdx.x * RPB + group, step = (long long)gridDim.x * RPB;
    const Columns<T, TPR, ODD> col(H, lane, first);
    int flip = 0;
    const float inv = 1.0f / (float)H;
    pdl_wait();
    pdl_trigger();
    long long next = first;
    auto fetch = [&](int stage) {
        if (next < rows) {
            const T* xr = x + (size_t)next * H;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (col.has(i))
                    fetch_chunk(slots + (stage * V + i) * NT + tid, xr, col.at(i), H, col.inside(i, next, rows));
        }
        copy_commit();
        next += step;
    };
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) fetch(s);
    float g[V][VN], b[V][VN];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (col.has(i)) {
            load_weight<VN>(gamma, wbf16, col.at(i), H, col.whole(i), g[i]);
            load_weight<VN>(beta, wbf16, col.at(i), H, col.whole(i), b[i]);
        }
    int stage = 0;
    for (long long r = first; r < rows; r += step) {
        fetch(stage == 0 ? S - 1 : stage - 1);
        copy_wait<S - 1>();
        float v[V][VN];
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col.has(i)) {
                unpack(slots[(stage * V + i) * NT + tid], v[i]);
                if (!col.whole(i)) clear(v[i], col.at(i), H);
#pragma unroll
                for (int e = 0; e < VN; ++e) s[0] += v[i][e];
            }
        row_sum<TPR>(s, red, group, flip);
        const float mu = s[0] * inv;
        float q[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col.has(i)) {
#pragma unroll
                for (int e = 0; e < VN; ++e) v[i][e] -= mu;
                if (!col.whole(i)) clear(v[i], col.at(i), H);
#pragma unroll
                for (int e = 0; e < VN; ++e) q[0] = fmaf(v[i][e], v[i][e], q[0]);
            }
        row_sum<TPR>(q, red, group, flip);
        const float rs = 1.0f / sqrtf(q[0] * inv + eps);
        T* yr = y + (size_t)r * H;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col.has(i)) {
#pragma unroll
                for (int e = 0; e < VN; ++e) v[i][e] = fmaf(v[i][e] * rs, g[i][e], b[i][e]);
                store_chunk<VN>(yr, col.at(i), H, col.whole(i), v[i]);
            }
        if (lane == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
}

// 16 columns a thread: the row's x and dy and the weights stay in registers
// between the two passes over it; 32: they are read again (slots, L1).
template <typename T, int TPR, int COLS, bool ODD>
__global__ void __launch_bounds__(NT, 1)
layernorm_grad_rows_kernel(long long rows, int H, const T* dy, const T* x, const void* __restrict__ gamma, bool wbf16,
                           const float* __restrict__ mean, const float* __restrict__ rstd, const T* dres, T* dx,
                           float* __restrict__ part) {
    constexpr int VN = kVN<T>, RPB = NT / TPR, V = COLS / VN, S = stages_of<T>(3, COLS);
    constexpr bool kKeep = COLS == 16;
    static_assert(S >= 2, "stages");
    extern __shared__ __align__(16) uint8_t smem_ln[];
    uint4* slots = reinterpret_cast<uint4*>(smem_ln);             // [stage][x, dy, dres][V][NT]
    __shared__ float red[2 * 2 * NT / 32];
    const int tid = threadIdx.x, group = tid / TPR, lane = tid % TPR;
    const long long first = (long long)blockIdx.x * RPB + group, step = (long long)gridDim.x * RPB;
    const Columns<T, TPR, ODD> col(H, lane, first);
    int flip = 0;
    const float inv = 1.0f / (float)H;
    float dg[V][VN], db[V][VN], gk[kKeep ? V : 1][VN];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < VN; ++e) dg[i][e] = db[i][e] = 0.f;
    pdl_wait();
    pdl_trigger();
    long long next = first;
    auto fetch = [&](int stage) {
        if (next < rows) {
            const size_t o = (size_t)next * H;
            const T* src[3] = {x + o, dy + o, dres ? dres + o : nullptr};
#pragma unroll
            for (int a = 0; a < 3; ++a) {
                if (a == 2 && !dres) break;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (col.has(i))
                        fetch_chunk(slots + ((stage * 3 + a) * V + i) * NT + tid, src[a], col.at(i), H,
                                    col.inside(i, next, rows));
            }
        }
        copy_commit();
        next += step;
    };
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) fetch(s);
    float mu_n = 0.f, rs_n = 0.f;                                 // of the next row
    if (first < rows) {
        mu_n = mean[first];
        rs_n = rstd[first];
    }
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col.has(i)) load_weight<VN>(gamma, wbf16, col.at(i), H, col.whole(i), gk[i]);
    }
    int stage = 0;
    for (long long r = first; r < rows; r += step) {
        const float mu = mu_n, rs = rs_n;
        if (r + step < rows) {
            mu_n = mean[r + step];
            rs_n = rstd[r + step];
        }
        fetch(stage == 0 ? S - 1 : stage - 1);
        copy_wait<S - 1>();
        const uint4* sx = slots + (size_t)(stage * 3) * V * NT + tid;
        const uint4* sy = sx + V * NT;
        const uint4* sr = sy + V * NT;
        uint4 rx[V], ry[V];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col.has(i)) {
                float xv[VN], dv[VN], g[VN];
                rx[i] = sx[i * NT];
                ry[i] = sy[i * NT];
                unpack(rx[i], xv);
                unpack(ry[i], dv);
                if (!col.whole(i)) {
                    clear(xv, col.at(i), H);
                    clear(dv, col.at(i), H);
                }
                if constexpr (!kKeep) load_weight<VN>(gamma, wbf16, col.at(i), H, col.whole(i), g);
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    const float xh = (xv[e] - mu) * rs, a = dv[e] * (kKeep ? gk[kKeep ? i : 0][e] : g[e]);
                    s[0] += a;
                    s[1] = fmaf(a, xh, s[1]);
                    dg[i][e] = fmaf(dv[e], xh, dg[i][e]);
                    db[i][e] += dv[e];
                }
            }
        row_sum<TPR>(s, red, group, flip);
        const float ma = s[0] * inv, mb = s[1] * inv;
        T* out = dx + (size_t)r * H;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col.has(i)) {
                float xv[VN], dv[VN], g[VN];
                unpack(kKeep ? rx[i] : sx[i * NT], xv);
                unpack(kKeep ? ry[i] : sy[i * NT], dv);
                if constexpr (!kKeep) load_weight<VN>(gamma, wbf16, col.at(i), H, col.whole(i), g);
#pragma unroll
                for (int e = 0; e < VN; ++e)
                    dv[e] = (dv[e] * (kKeep ? gk[kKeep ? i : 0][e] : g[e]) - ma - (xv[e] - mu) * rs * mb) * rs;
                if (dres) {
                    unpack(sr[i * NT], xv);
#pragma unroll
                    for (int e = 0; e < VN; ++e) dv[e] += xv[e];
                }
                store_chunk<VN>(out, col.at(i), H, col.whole(i), dv);
            }
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    // the block's partial sums, the rows of its groups added in order
    float* p = part + (size_t)blockIdx.x * 2 * H;
    float* acc = p;
    if constexpr (RPB > 1) {
        copy_wait<0>();
        __syncthreads();
        acc = reinterpret_cast<float*>(smem_ln) + (size_t)group * 2 * H;      // [group][2][H]
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < VN; ++e) {
            const int c = col.at(i) + e;
            if (c >= 0 && c < H) {
                acc[c] = dg[i][e];
                acc[H + c] = db[i][e];
            }
        }
    if constexpr (RPB > 1) {
        __syncthreads();
        const float* all = reinterpret_cast<const float*>(smem_ln);
        for (int c = tid; c < 2 * H; c += NT) {
            float t = 0.f;
#pragma unroll
            for (int g = 0; g < RPB; ++g) t += all[(size_t)g * 2 * H + c];
            p[c] = t;
        }
    }
}

// dgamma and dbeta from the [parts][2][H] partial sums: 32 columns a block, the
// parts split over 32 warps (at most 10 each), so all loads are in flight at once.
__global__ void __launch_bounds__(1024)
layernorm_dw_final_kernel(int parts, int H, const float* __restrict__ part, float* __restrict__ dgamma,
                          float* __restrict__ dbeta) {
    __shared__ float sg[32][33], sb[32][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float g = 0.f, b = 0.f;
    if (c < H) {
#pragma unroll
        for (int i = 0; i < (kLayerNormParts + 31) / 32; ++i) {
            const int p = warp + 32 * i;
            if (p < parts) {
                g += part[(size_t)p * 2 * H + c];
                b += part[(size_t)p * 2 * H + H + c];
            }
        }
    }
    sg[warp][lane] = g;
    sb[warp][lane] = b;
    __syncthreads();
    // warp w sums column w
    g = sg[lane][warp];
    b = sb[lane][warp];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        g += __shfl_xor_sync(0xffffffffu, g, off);
        b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    const int cw = blockIdx.x * 32 + warp;
    if (lane == 0 && cw < H) {
        dgamma[cw] = g;
        dbeta[cw] = b;
    }
}

unsigned row_blocks(long long rows) {
    const long long cap = (long long)device_sm_count() * 8;
    return (unsigned)(rows < cap ? rows : cap);
}

template <typename T, typename W>
cudaError_t forward_wide(const LayerNormProblem& p, cudaStream_t st) {
    return launch_kernel(layernorm_kernel<T, W>, dim3(row_blocks(p.rows)), dim3(kLnThreads), 0, st, 1, kUsePdl,
                         p.rows, p.hidden, static_cast<const T*>(p.x), static_cast<const W*>(p.gamma),
                         static_cast<const W*>(p.beta), p.eps, static_cast<T*>(p.y), p.mean, p.rstd);
}

cudaError_t finish_weights(const LayerNormProblem& p, int parts, cudaStream_t st) {
    return launch_kernel(layernorm_dw_final_kernel, dim3((unsigned)((p.hidden + 31) / 32)), dim3(1024), 0, st, 1,
                         kUsePdl, parts, p.hidden, static_cast<const float*>(p.scratch), p.dgamma, p.dbeta);
}

template <typename T, typename W>
cudaError_t backward_wide(const LayerNormProblem& p, cudaStream_t st) {
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.dy);
    const unsigned cols = (unsigned)((p.hidden + kLnThreads - 1) / kLnThreads);
    const int parts = layernorm_parts(p.rows);
    // the weight's partial sums first: dx may overwrite dy
    cudaError_t e = launch_kernel(layernorm_dw_partial_kernel<T>, dim3(cols, (unsigned)parts), dim3(kLnThreads), 0, st,
                                  1, kUsePdl, p.rows, p.hidden, dy, x, p.mean, p.rstd, p.scratch);
    if (e == cudaSuccess) e = finish_weights(p, parts, st);
    if (e == cudaSuccess)
        e = launch_kernel(layernorm_dx_kernel<T, W>, dim3(row_blocks(p.rows)), dim3(kLnThreads), 0, st, 1, kUsePdl,
                          p.rows, p.hidden, dy, x, static_cast<const W*>(p.gamma), p.mean, p.rstd,
                          static_cast<const T*>(p.dres), static_cast<T*>(p.dx));
    return e;
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::once_flag& once, cudaError_t& err) {
    std::call_once(once, [&] { err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes); });
    return err;
}

// Blocks of `rpb` row groups: a block for each SM at most; for odd rows the number of
// groups is a multiple of vn.
unsigned blocks_of(long long rows, int rpb, bool odd, int vn) {
    long long blocks = (rows + rpb - 1) / rpb;
    if (blocks > device_sm_count()) blocks = device_sm_count();
    const int unit = odd && rpb < vn ? vn / rpb : 1;
    blocks = blocks < device_sm_count() / unit * unit ? (blocks + unit - 1) / unit * unit : blocks / unit * unit;
    return (unsigned)(blocks < unit ? unit : blocks);
}

template <typename T, int TPR, bool ODD>
cudaError_t forward_rows(const LayerNormProblem& p, cudaStream_t st) {
    constexpr size_t smem = (size_t)stages_of<T>(1, kFwdCols) * kFwdCols * sizeof(T) * NT;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    if (allow_smem(layernorm_rows_kernel<T, TPR, ODD>, smem, once, err) != cudaSuccess) return err;
    return launch_kernel(layernorm_rows_kernel<T, TPR, ODD>, dim3(blocks_of(p.rows, NT / TPR, ODD, kVN<T>)), dim3(NT),
                         smem, st, 1, kUsePdl, p.rows, p.hidden, static_cast<const T*>(p.x), p.gamma, p.beta,
                         p.wtype == MOE_TYPE_BF16, p.eps, static_cast<T*>(p.y), p.mean, p.rstd);
}

template <typename T, int TPR, int COLS, bool ODD>
cudaError_t backward_rows(const LayerNormProblem& p, cudaStream_t st) {
    constexpr int RPB = NT / TPR;
    constexpr size_t smem = (size_t)stages_of<T>(3, COLS) * 3 * COLS * sizeof(T) * NT;
    // the partial sums of the block's row groups reuse the slots
    static_assert(RPB == 1 || smem >= (size_t)NT * 2 * COLS * sizeof(float), "partial sums");
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    if (allow_smem(layernorm_grad_rows_kernel<T, TPR, COLS, ODD>, smem, once, err) != cudaSuccess) return err;
    const unsigned blocks = blocks_of(p.rows, RPB, ODD, kVN<T>);
    if ((int)blocks > layernorm_parts(p.rows)) return cudaErrorInvalidConfiguration;      // the scratch is sized by it
    const cudaError_t e =
        launch_kernel(layernorm_grad_rows_kernel<T, TPR, COLS, ODD>, dim3(blocks), dim3(NT), smem, st, 1, kUsePdl,
                      p.rows, p.hidden, static_cast<const T*>(p.dy), static_cast<const T*>(p.x), p.gamma,
                      p.wtype == MOE_TYPE_BF16, static_cast<const float*>(p.mean), static_cast<const float*>(p.rstd),
                      static_cast<const T*>(p.dres), static_cast<T*>(p.dx), p.scratch);
    return e != cudaSuccess ? e : finish_weights(p, (int)blocks, st);
}

// The fewest threads whose columns cover the row, wherever it starts in a chunk
// (whole warps share a row).
template <typename T, bool ODD>
bool forward_by_width(const LayerNormProblem& p, cudaStream_t st, cudaError_t* e) {
    const int need = (p.hidden + (ODD ? kVN<T> - 1 : 0) + kFwdCols - 1) / kFwdCols;
    if (need <= 32) *e = forward_rows<T, 32, ODD>(p, st);
    else if (need <= 64) *e = forward_rows<T, 64, ODD>(p, st);
    else if (need <= 128) *e = forward_rows<T, 128, ODD>(p, st);
    else if (need <= 256) *e = forward_rows<T, 256, ODD>(p, st);
    else if (need <= 512) *e = forward_rows<T, 512, ODD>(p, st);
    else return false;
    return true;
}

template <typename T, bool ODD>
bool backward_by_width(const LayerNormProblem& p, cudaStream_t st, cudaError_t* e) {
    const int need = (p.hidden + (ODD ? kVN<T> - 1 : 0) + kBwdCols - 1) / kBwdCols;
    if (need <= 32) *e = backward_rows<T, 32, kBwdCols, ODD>(p, st);
    else if (need <= 64) *e = backward_rows<T, 64, kBwdCols, ODD>(p, st);
    else if (need <= 128) *e = backward_rows<T, 128, kBwdCols, ODD>(p, st);
    else if (need <= 256) *e = backward_rows<T, 256, kBwdCols, ODD>(p, st);
    else if (need <= 512) *e = backward_rows<T, 512, kBwdCols, ODD>(p, st);
    else if (sizeof(T) == 2 && need <= 1024) *e = backward_rows<__nv_bfloat16, 512, 32, ODD>(p, st);
    else return false;
    return true;
}

template <typename T>
cudaError_t run(const LayerNormProblem& p, bool fwd, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    const bool odd = p.hidden % kVN<T> != 0;
    if (fwd ? (odd ? forward_by_width<T, true>(p, st, &e) : forward_by_width<T, false>(p, st, &e))
            : (odd ? backward_by_width<T, true>(p, st, &e) : backward_by_width<T, false>(p, st, &e)))
        return e;
    if (p.wtype == MOE_TYPE_BF16) return fwd ? forward_wide<T, __nv_bfloat16>(p, st) : backward_wide<T, __nv_bfloat16>(p, st);
    return fwd ? forward_wide<T, float>(p, st) : backward_wide<T, float>(p, st);
}

}  // namespace

cudaError_t launch_layernorm(const LayerNormProblem& p, cudaStream_t st) {
    if (p.rows == 0) return cudaSuccess;
    return p.type == MOE_TYPE_BF16 ? run<__nv_bfloat16>(p, true, st) : run<float>(p, true, st);
}

cudaError_t launch_layernorm_backward(const LayerNormProblem& p, cudaStream_t st) {
    if (p.rows == 0) return finish_weights(p, 0, st);
    return p.type == MOE_TYPE_BF16 ? run<__nv_bfloat16>(p, false, st) : run<float>(p, false, st);
}

}  // namespace moe
