// gemm_grad.cu -- the grouped GEMMs of the expert FFN's backward pass on tcgen05.
//
// With the rows of expert e at [offsets[e], offsets[e+1]):
//   rows form     dh = dy W2[e],  dx = dpre W13[e]:  C[r, n] = sum_k A[r, k] B[e][k, n]
//   weights form  dW2[e] = dy^T h,  dW13[e] = dpre^T x:  C[e][m, n] = sum_r A[r, m] B[r, n]
// Every operand is read as it lies in memory; nothing is transposed in a pass of
// its own.  A tile that is contiguous along the output dimension instead of the
// reduction is loaded as boxes of [64 reduction rows x 64 columns] (128-byte
// swizzle) and given to the MMA as an MN-major operand.
//
// Both forms run on CTA pairs: a cluster of two CTAs owns a 256 x 256 output tile
// through tcgen05.mma.cta_group::2, each CTA loading its 128 A rows (or columns)
// and its 128 B columns per 64-deep step (32 KiB a stage, six stages) and holding
// 128 rows of two 256-column accumulators, so the epilogue of one tile runs under
// the next tile's main loop.  The rows form's epilogue applies the activation's
// derivative: dpre = act'(pre) * dh, from the saved pre-activations.
//
// The weights form reduces over a group's rows.  A last step of fewer than 64
// rows also loads rows of the next group (or past the last one); each CTA's fixer
// warp waits for that step's copies on a barrier of its own, zeroes the rows past
// the bound up to the next multiple of 16 in both operands -- zeroing one would
// leave 0 * NaN --, the peer's fixer tells the leader's, and that arrives on the
// stage barrier; the MMA issues only the 16-row slices that hold rows.  A group
// without rows writes zeros.  (An arrival of the peer on the leader's barrier in
// every step, released at cluster scope, took the step from 0.28 to 0.84 us.)
//
// Every wait is bounded; on a timeout the CTA stops issuing work, lets its copies
// land, frees TMEM, raises MOE_ERR_TIMEOUT and returns.
#include "common.cuh"

#include <climits>
#include <mutex>

namespace moe {
namespace {

enum GradKind : int { kRowsSwiGLU = 0, kRowsReLU2 = 1, kRowsPlain = 2, kWeights = 3 };

constexpr int TM = 256, TN = 256, BK = 64;        // output tile of the pair, reduction step
constexpr int HALF = 128;                         // rows / columns each CTA contributes
constexpr int OP_BYTES = HALF * BK * 2;           // 16 KiB an operand and CTA
constexpr int BOX_BYTES = 64 * BK * 2;            // one 64 x 64 box of an MN-major operand
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int STAGES = 5;
constexpr int EPI_WARPS = 4;
constexpr int EPI_BYTES = 8192;                   // staging of one epilogue warp
constexpr int THREADS = 32 * (3 + EPI_WARPS);     // producer, MMA, epilogue, fixer
constexpr uint32_t TMEM_COLS = 512;
constexpr int kBand = 8;                          // column tiles per band of the tile order
constexpr int MAX_DYN_SMEM = 216 * 1024;

struct GParams {
    const int32_t* offsets;
    int groups, a_rows;              // bucket bounds are clamped to [0, a_rows]
    int K;                           // rows form: reduction length
    int M, N;                        // weights form: output rows; output columns
    void* out;
    long long ldo;
    const __nv_bfloat16* pre;        // activation forms: [a_rows, up] pre-activations
    long long ldp;
    int up_off;                      // SwiGLU: columns from gate to up half
    int wmode;                       // weights form: moe_wgrad
    WsHeader* hdr;
};

struct Ctl {
    unsigned long long full[STAGES], empty[STAGES], part[STAGES], fixed[STAGES];
    unsigned long long tfull[2], tempty[2];
    unsigned long long drain;
    uint32_t tmem_base;
    int abort;
    int total_tiles;
};

// Instruction descriptor bits: operand A / B is MN-major.
constexpr uint32_t kMajorA = 1u << 15, kMajorB = 1u << 16;

// Shared-memory descriptor of an MN-major operand of 128-byte swizzled boxes of
// [BK reduction rows x 64 elements]: boxes BOX_BYTES apart along the operand's
// outer dimension (leading offset), 8-row groups of the reduction 1 KiB apart
// (stride offset).  A 16-deep slice starts 2 KiB after the one before.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(BOX_BYTES >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}
constexpr uint64_t kMnStep = 2048 >> 4, kKStep = 32 >> 4;   // descriptor units per 16-deep slice

__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// mbar_wait_bounded with the acquire at cluster scope: the fixer of the other
// CTA of the pair arrives on the leader's barrier.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((i & 31u) == 0u) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) { *abort = 1; return false; }
        }
    }
}
// Arrive on a barrier of the pair without releasing earlier memory accesses at
// cluster scope: it hands back an accumulator, and the stores of the tile before
// need not be waited for.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, uint32_t bar_cluster, int x, int y,
                                                 int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z) : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// max(z, 0) that keeps a NaN.
__device__ __forceinline__ float relu(float z) { return z <= 0.f ? 0.f : z; }
// d silu(g) u: dg = dh u s (1 + g (1 - s)), du = dh g s, s = sigmoid(g).
__device__ __forceinline__ void swiglu_grad(float dh, float g, float u, float& dg, float& du) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-g));
    const float gs = g * s;
    dg = dh * u * fmaf(gs, 1.0f - s, s);
    du = dh * gs;
}

// ---- epilogue -------------------------------------------------------------------
// A warp turns 32 accumulator rows into output rows through its staging slot, so
// that global memory is written in whole 64- or 128-byte row pieces: a thread holds
// one row of the accumulator, and storing from there put 32 rows into each store
// instruction (4.5 us a tile where the bytes take 1.5).  The 16-byte units of a
// staged row are XORed with its index, so that both the row-wise and the
// column-wise side are free of bank conflicts.
__device__ __forceinline__ uint4* unit128(uint8_t* slot, int row, int u) {     // 128-byte rows
    return reinterpret_cast<uint4*>(slot + row * 128 + ((u ^ (row & 7)) * 16));
}
__device__ __forceinline__ uint4* unit64(uint8_t* slot, int row, int u) {      // 64-byte rows
    return reinterpret_cast<uint4*>(slot + row * 64 + ((u ^ ((row >> 1) & 3)) * 16));
}
__device__ __forceinline__ uint4 pack8(const uint32_t* v) {
    return make_uint4(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])), pack2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                      pack2(__uint_as_float(v[4]), __uint_as_float(v[5])), pack2(__uint_as_float(v[6]), __uint_as_float(v[7])));
}

// BF16 output, 64 columns at a time.
template <typename F>
__device__ __forceinline__ void bf16_tile(uint32_t tl, bool empty, int rows, int n0, int N, __nv_bfloat16* out,
                                          long long ldo, uint8_t* slot, int lane, F&& release) {
#pragma unroll 1
    for (int c = 0; c < TN / 64; ++c) {
        uint8_t* s = slot + (c & 1) * 4096;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
            if (!empty) {
                tmem_ld_32cols(tl + c * 64 + h * 32, v);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0u;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) *unit128(s, lane, h * 4 + u) = pack8(v + 8 * u);
        }
        if (c == TN / 64 - 1 && !empty) release();
        __syncwarp();
        const int u = lane & 7, col = n0 + c * 64 + u * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            if (r < rows && col < N) *reinterpret_cast<uint4*>(out + r * ldo + col) = *unit128(s, r, u);
        }
    }
    __syncwarp();
}

// FP32 output (stored or added to), 32 columns at a time.
template <typename F>
__device__ __forceinline__ void f32_tile(const GParams& p, uint32_t tl, bool empty, int rows, int n0, float* out,
                                         uint8_t* slot, int lane, F&& release) {
#pragma unroll 1
    for (int c = 0; c < TN / 32; ++c) {
        uint8_t* s = slot + (c & 1) * 4096;
        uint32_t v[32];
        if (!empty) {
            tmem_ld_32cols(tl + c * 32, v);
            tmem_ld_wait();
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) *unit128(s, lane, u) = make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
        if (c == TN / 32 - 1 && !empty) release();
        __syncwarp();
        const int u = lane & 7, col = n0 + c * 32 + u * 4;
        const bool add = p.wmode == MOE_WGRAD_F32_ADD;
        float4 old[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            old[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (add && r < rows && col < p.N) old[i] = *reinterpret_cast<const float4*>(out + r * p.ldo + col);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            const uint4 w = *unit128(s, r, u);
            if (r < rows && col < p.N)
                *reinterpret_cast<float4*>(out + r * p.ldo + col) =
                    make_float4(old[i].x + __uint_as_float(w.x), old[i].y + __uint_as_float(w.y),
                                old[i].z + __uint_as_float(w.z), old[i].w + __uint_as_float(w.w));
        }
    }
    __syncwarp();
}

// The activation's gradient, 32 columns at a time: the pre-activations of a chunk
// come into the slot with cp.async while the chunk before is worked on (two slots
// of [gate 2 KiB | up 2 KiB]), each thread replaces its row's values by their
// gradients, and the slot is written out.
template <bool GLU>
__device__ __forceinline__ void act_fetch(const GParams& p, int c, int m0, int rows, int row0, int n0, uint8_t* slot,
                                          int lane) {
    uint8_t* s = slot + (c & 1) * 4096;
    const int u = lane & 3, col = n0 + c * 32 + u * 8;
    if (c < TN / 32 && col < p.N) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            if (r < rows) {
                const __nv_bfloat16* src = p.pre + (size_t)(row0 + m0 + r) * p.ldp + col;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(unit64(s, r, u))), "l"(src) : "memory");
                if (GLU)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                 :: "r"(smem_u32(unit64(s + 2048, r, u))), "l"(src + p.up_off) : "memory");
            }
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <bool GLU>
__device__ __forceinline__ void act_prefetch(const GParams& p, int m0, int rows, int row0, int n0, uint8_t* slot, int lane) {
    act_fetch<GLU>(p, 0, m0, rows, row0, n0, slot, lane);
    act_fetch<GLU>(p, 1, m0, rows, row0, n0, slot, lane);
}
template <bool GLU, typename F>
__device__ __forceinline__ void act_tile(const GParams& p, uint32_t tl, int m0, int rows, int row0, int n0,
                                         uint8_t* slot, int lane, F&& release) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (size_t)(row0 + m0) * p.ldo;
#pragma unroll 1
    for (int c = 0; c < TN / 32; ++c) {
        uint8_t* s = slot + (c & 1) * 4096;
        uint32_t v[32];
        tmem_ld_32cols(tl + c * 32, v);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        tmem_ld_wait();
        if (c == TN / 32 - 1) release();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint4 g4 = *unit64(s, lane, u);
            const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
            uint32_t o[4];
            if (GLU) {
                const uint4 u4 = *unit64(s + 2048, lane, u);
                const uint32_t uw[4] = {u4.x, u4.y, u4.z, u4.w};
                uint32_t ou[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float dg0, du0, dg1, du1;
                    swiglu_grad(__uint_as_float(v[8 * u + 2 * i]), bf_lo(gw[i]), bf_lo(uw[i]), dg0, du0);
                    swiglu_grad(__uint_as_float(v[8 * u + 2 * i + 1]), bf_hi(gw[i]), bf_hi(uw[i]), dg1, du1);
                    o[i] = pack2(dg0, dg1);
                    ou[i] = pack2(du0, du1);
                }
                *unit64(s + 2048, lane, u) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = pack2(__uint_as_float(v[8 * u + 2 * i]) * (2.0f * relu(bf_lo(gw[i]))),
                                 __uint_as_float(v[8 * u + 2 * i + 1]) * (2.0f * relu(bf_hi(gw[i]))));
            }
            *unit64(s, lane, u) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
        const int u = lane & 3, col = n0 + c * 32 + u * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            if (r < rows && col < p.N) {
                *reinterpret_cast<uint4*>(out + r * p.ldo + col) = *unit64(s, r, u);
                if (GLU) *reinterpret_cast<uint4*>(out + r * p.ldo + p.up_off + col) = *unit64(s + 2048, r, u);
            }
        }
        __syncwarp();
        act_fetch<GLU>(p, c + 2, m0, rows, row0, n0, slot, lane);
    }
}

struct Tile { int g, mt, nt, row0, mrows; };

template <int KIND>
__device__ __forceinline__ Tile decode_tile(int tile, const int* prefix, const int* rstart, const int* rcount,
                                            int groups, int ntm, int ntn) {
    Tile t;
    int local, mtiles;
    if (KIND == kWeights) {
        const int per = ntm * ntn;
        t.g = tile / per;
        local = tile - t.g * per;
        mtiles = ntm;
    } else {
        int lo = 0, hi = groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= tile) lo = mid; else hi = mid;
        }
        t.g = lo;
        local = tile - prefix[lo];
        mtiles = (rcount[lo] + TM - 1) / TM;
    }
    const int band = local / (mtiles * kBand);
    const int idx = local - band * mtiles * kBand;
    t.mt = idx % mtiles;
    t.nt = band * kBand + idx / mtiles;
    t.row0 = rstart[t.g];
    t.mrows = rcount[t.g];
    return t;
}

template <int KIND>
__global__ void __launch_bounds__(THREADS, 1)
grad_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const GParams p) {
    constexpr bool kW = KIND == kWeights;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
    uint8_t* epi_smem = smem + STAGES * STAGE_BYTES;
    Ctl* ctl = reinterpret_cast<Ctl*>(epi_smem + EPI_WARPS * EPI_BYTES);
    int* prefix = reinterpret_cast<int*>(ctl + 1);
    int* rstart = prefix + (p.groups + 1);
    int* rcount = rstart + p.groups;
    const uint32_t smem_base = smem_u32(smem);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();                 // 0: leader, 1: peer
    const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
    const int ntn = (p.N + TN - 1) / TN, ntm = kW ? (p.M + TM - 1) / TM : 0;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
            mbar_init(smem_u32(&ctl->part[s]), 1);
            mbar_init(smem_u32(&ctl->fixed[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&ctl->tfull[a]), 1);
            mbar_init(smem_u32(&ctl->tempty[a]), 2 * EPI_WARPS);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), TMEM_COLS);
        tmem_relinquish_pair();
    }
    pdl_wait();
    pdl_trigger();
    // each bucket is clamped to [0, a_rows], so malformed offsets stay in bounds
    for (int g = tid; g < p.groups; g += THREADS) {
        int lo = p.offsets[g], hi = p.offsets[g + 1];
        lo = lo < 0 ? 0 : (lo > p.a_rows ? p.a_rows : lo);
        hi = hi < lo ? lo : (hi > p.a_rows ? p.a_rows : hi);
        rstart[g] = lo;
        rcount[g] = hi - lo;
    }
    __syncthreads();
    if (!kW) {
        // exclusive scan of tiles per group -> prefix[0..groups]
        const int n = p.groups;
        const int per = (n + THREADS - 1) / THREADS;
        const int g0 = tid * per;
        int loc = 0;
        for (int i = 0; i < per; ++i)
            if (g0 + i < n) loc += ((rcount[g0 + i] + TM - 1) / TM) * ntn;
        int inc = loc;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        __shared__ int wtot[THREADS / 32];
        if (lane == 31) wtot[warp] = inc;
        __syncthreads();
        int run = inc - loc;
        for (int w = 0; w < warp; ++w) run += wtot[w];
        for (int i = 0; i < per; ++i) {
            if (g0 + i < n) {
                prefix[g0 + i] = run;
                run += ((rcount[g0 + i] + TM - 1) / TM) * ntn;
            }
        }
        if (tid == THREADS - 1) { prefix[n] = run; ctl->total_tiles = run; }
    } else if (tid == 0) {
        ctl->total_tiles = p.groups * ntm * ntn;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();              // both CTAs' barriers are initialised before any cross-CTA arrive
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const int total = ctl->total_tiles;
    volatile int* abort = &ctl->abort;
    const int nk_rows = (p.K + BK - 1) / BK;

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        if (lane == 0) {
            int stage = 0;
            uint32_t ph = 0;
            bool ok = true;
            long long armed = 0;
            for (int tile = pair; tile < total && ok; tile += npairs) {
                const Tile t = decode_tile<KIND>(tile, prefix, rstart, rcount, p.groups, ntm, ntn);
                const int nk = kW ? (t.mrows + BK - 1) / BK : nk_rows;
                const int a0 = t.mt * TM + (int)rank * HALF;     // A's row (rows form) or column
                const int b0 = t.nt * TN + (int)rank * HALF;
                for (int i = 0; i < nk; ++i) {
                    if (!mbar_wait_bounded(smem_u32(&ctl->empty[stage]), ph ^ 1u, abort)) { ok = false; break; }
                    const uint32_t full_local = smem_u32(&ctl->full[stage]);
                    const uint32_t full_leader = mapa_shared(full_local, 0);
                    const uint32_t sa = smem_base + stage * STAGE_BYTES, sb = sa + OP_BYTES;
                    if (kW) {
                        const int y = t.row0 + i * BK;
                        if (t.mrows - i * BK < BK) {
                            // partial step: counted on this CTA's own barrier, for its fixer
                            const uint32_t part = smem_u32(&ctl->part[stage]);
                            mbar_arrive_expect_tx(part, STAGE_BYTES);
                            tma_load_2d(sa, &tmA, part, a0, y);
                            tma_load_2d(sa + BOX_BYTES, &tmA, part, a0 + 64, y);
                            tma_load_2d(sb, &tmB, part, b0, y);
                            tma_load_2d(sb + BOX_BYTES, &tmB, part, b0 + 64, y);
                        } else {
                            if (rank == 0) mbar_arrive_expect_tx(full_local, 2 * STAGE_BYTES);
                            tma_load_2d_pair(sa, &tmA, full_leader, a0, y);
                            tma_load_2d_pair(sa + BOX_BYTES, &tmA, full_leader, a0 + 64, y);
                            tma_load_2d_pair(sb, &tmB, full_leader, b0, y);
                            tma_load_2d_pair(sb + BOX_BYTES, &tmB, full_leader, b0 + 64, y);
                        }
                    } else {
                        if (rank == 0) mbar_arrive_expect_tx(full_local, 2 * STAGE_BYTES);
                        tma_load_2d_pair(sa, &tmA, full_leader, i * BK, t.row0 + a0);
                        tma_load_3d_pair(sb, &tmB, full_leader, b0, i * BK, t.g);
                        tma_load_3d_pair(sb + BOX_BYTES, &tmB, full_leader, b0 + 64, i * BK, t.g);
                    }
                    ++armed;
                    if (++stage == STAGES) { stage = 0; ph ^= 1u; }
                }
            }
            if (!ok) {
                // as in the forward pair kernel: the leader waits for the phases it
                // armed, the peer (which cannot wait on a remote barrier) adds a delay
                if (rank != 0 || !wait_armed_stages(smem_u32(&ctl->full[0]), STAGES, armed)) settle_delay();
                raise_status(p.hdr, MOE_ERR_TIMEOUT);
                p.hdr->timeout_site = kSiteGradProducer;
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader CTA) ----------------
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(TM, TN) | kMajorB | (kW ? kMajorA : 0u);
            constexpr uint64_t astep = kW ? kMnStep : kKStep;
            int stage = 0;
            uint32_t ph = 0;
            int acc = 0;
            uint32_t aph = 0;
            bool ok = true;
            for (int tile = pair; tile < total && ok; tile += npairs) {
                const Tile t = decode_tile<KIND>(tile, prefix, rstart, rcount, p.groups, ntm, ntn);
                const int nk = kW ? (t.mrows + BK - 1) / BK : nk_rows;
                if (nk == 0) continue;
                if (!mbar_wait_bounded(smem_u32(&ctl->tempty[acc]), aph ^ 1u, abort)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(acc * TN);
                for (int i = 0; i < nk; ++i) {
                    const uint32_t full = smem_u32(&ctl->full[stage]);
                    const int left = kW ? t.mrows - i * BK : BK;
                    // a partial step: the other CTA's fixer wrote its shared memory
                    if (!(kW && left < BK ? mbar_wait_cluster(full, ph, abort) : mbar_wait_bounded(full, ph, abort))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_base + stage * STAGE_BYTES;
                    const uint64_t ad = kW ? sdesc_mn_sw128(sa) : sdesc_k_sw128(sa);
                    const uint64_t bd = sdesc_mn_sw128(sa + OP_BYTES);
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk)
                        if (!kW || kk * 16 < left)
                            tc_mma_bf16_pair(d, ad + (uint64_t)kk * astep, bd + (uint64_t)kk * kMnStep, idesc,
                                             (i > 0 || kk > 0) ? 1u : 0u);
                    tc_commit_pair_mc(smem_u32(&ctl->empty[stage]), (uint16_t)3);
                    if (++stage == STAGES) { stage = 0; ph ^= 1u; }
                }
                if (!ok) break;
                tc_commit_pair_mc(smem_u32(&ctl->tfull[acc]), (uint16_t)3);
                acc ^= 1;
                if (acc == 0) aph ^= 1u;
            }
            tc_commit_pair(smem_u32(&ctl->drain));
            volatile int never = 0;
            const bool drained = mbar_wait_bounded(smem_u32(&ctl->drain), 0, &never);
            if (!ok || !drained) {
                raise_status(p.hdr, MOE_ERR_TIMEOUT);
                p.hdr->timeout_site = kSiteGradMma;
                *abort = 1;
            }
        }
    } else if (warp < 2 + EPI_WARPS) {
        // ---------------- epilogue (both CTAs): a warp = 32 rows of the tile ----------------
        const int q = warp & 3;
        uint8_t* epi = epi_smem + q * EPI_BYTES;
        int acc = 0;
        uint32_t aph = 0;
        for (int tile = pair; tile < total; tile += npairs) {
            const Tile t = decode_tile<KIND>(tile, prefix, rstart, rcount, p.groups, ntm, ntn);
            const int m0 = t.mt * TM + (int)rank * HALF + q * 32;      // this warp's 32 rows
            const int rows = (kW ? p.M : t.mrows) - m0;                // of which below the bound
            const int n0 = t.nt * TN;
            const bool empty = kW && t.mrows == 0;
            if (KIND == kRowsSwiGLU || KIND == kRowsReLU2)
                act_prefetch<KIND == kRowsSwiGLU>(p, m0, rows, t.row0, n0, epi, lane);
            if (!empty) {
                if (!mbar_wait_bounded(smem_u32(&ctl->tfull[acc]), aph, abort)) {
                    if (lane == 0) {
                        raise_status(p.hdr, MOE_ERR_TIMEOUT);
                        p.hdr->timeout_site = kSiteGradEpilogue;
                    }
                    break;
                }
                tc_fence_after();
            }
            const uint32_t tl = tmem_base + (uint32_t)(acc * TN) + ((uint32_t)(q * 32) << 16);
            auto release = [&] {               // the accumulator is read: the next tile may overwrite it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&ctl->tempty[acc]), 0));
            };
            if (KIND == kRowsSwiGLU || KIND == kRowsReLU2) {
                act_tile<KIND == kRowsSwiGLU>(p, tl, m0, rows, t.row0, n0, epi, lane, release);
            } else if (kW && p.wmode != MOE_WGRAD_BF16) {
                if (!(empty && p.wmode == MOE_WGRAD_F32_ADD))
                    f32_tile(p, tl, empty, rows, n0, static_cast<float*>(p.out) + ((size_t)t.g * p.M + m0) * p.ldo, epi,
                             lane, release);
            } else {
                const size_t row = kW ? (size_t)t.g * p.M + m0 : (size_t)(t.row0 + m0);
                bf16_tile(tl, empty, rows, n0, p.N, static_cast<__nv_bfloat16*>(p.out) + row * p.ldo, p.ldo, epi, lane,
                          release);
            }
            if (empty) continue;
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (kW) {
        // ---------------- fixer (both CTAs): partial reduction steps ----------------
        int stage = 0;
        uint32_t pph = 0;                          // parity of part[s] and fixed[s] in bit s
        bool ok = true;
        for (int tile = pair; tile < total && ok; tile += npairs) {
            const Tile t = decode_tile<KIND>(tile, prefix, rstart, rcount, p.groups, ntm, ntn);
            const int nk = (t.mrows + BK - 1) / BK;
            const int rem = t.mrows & (BK - 1);
            if (rem) {
                const int s = (stage + nk - 1) % STAGES;
                const uint32_t parity = (pph >> s) & 1u;
                pph ^= 1u << s;
                if (!mbar_wait_bounded(smem_u32(&ctl->part[s]), parity, abort)) { ok = false; break; }
                const int end = (rem + 15) & ~15;
                // four boxes of 128-byte rows; the swizzle stays inside a row
                for (int i = lane; i < 4 * (end - rem) * 8; i += 32) {
                    const int box = i / ((end - rem) * 8), j = i - box * ((end - rem) * 8);
                    *reinterpret_cast<uint4*>(smem + s * STAGE_BYTES + box * BOX_BYTES + (rem + (j >> 3)) * 128 +
                                              (j & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (rank != 0) {
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl->fixed[s]), 0));
                } else {
                    if (!mbar_wait_cluster(smem_u32(&ctl->fixed[s]), parity, abort)) { ok = false; break; }
                    if (lane == 0) mbar_arrive_cluster(smem_u32(&ctl->full[s]));
                }
            }
            stage = (stage + nk) % STAGES;
        }
        if (!ok && lane == 0) {
            raise_status(p.hdr, MOE_ERR_TIMEOUT);
            p.hdr->timeout_site = kSiteGradMma;
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();              // the leader's MMAs have drained before either CTA frees its TMEM
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

size_t smem_bytes(int groups) {
    return 1024 + (size_t)STAGES * STAGE_BYTES + EPI_WARPS * EPI_BYTES + sizeof(Ctl) + 3 * (size_t)(groups + 1) * 4;
}

template <int KIND>
moe_status launch_kind(const CUtensorMap& ma, const CUtensorMap& mb, const GParams& gp, cudaStream_t st) {
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [] {
        attr_err = cudaFuncSetAttribute(grad_gemm_pair_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        MAX_DYN_SMEM);
    });
    if (attr_err != cudaSuccess) {
        set_error("cudaFuncSetAttribute(max dynamic smem %d): %s", MAX_DYN_SMEM, cudaGetErrorString(attr_err));
        return MOE_ERR_CUDA;
    }
    const size_t smem = smem_bytes(gp.groups);
    const cudaError_t e = launch_kernel(grad_gemm_pair_kernel<KIND>, dim3((unsigned)(device_sm_count() & ~1)),
                                        dim3(THREADS), smem, st, 2, kUsePdl, ma, mb, gp);
    if (e != cudaSuccess) {
        set_error("gradient GEMM launch (smem %zu): %s", smem, cudaGetErrorString(e));
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

// h = bf16(act(pre)) for the valid rows; eight columns a thread.
template <bool GLU>
__global__ void __launch_bounds__(256)
act_kernel(long long rows, int IV, long long ldv, const int32_t* __restrict__ offsets, int groups,
           const uint4* __restrict__ pre, uint4* __restrict__ h) {
    pdl_wait();
    pdl_trigger();
    long long valid = offsets[groups];
    valid = valid < 0 ? 0 : (valid > rows ? rows : valid);
    const long long n = valid * IV;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const long long r = i / IV;
        const int c = (int)(i - r * IV);
        const uint4 a = pre[r * ldv + c];
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
        uint32_t uw[4] = {0u, 0u, 0u, 0u}, o[4];
        if (GLU) {
            const uint4 u = pre[r * ldv + IV + c];
            uw[0] = u.x; uw[1] = u.y; uw[2] = u.z; uw[3] = u.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x0 = bf_lo(aw[j]), x1 = bf_hi(aw[j]);
            if (GLU) {
                o[j] = pack2(x0 / (1.0f + __expf(-x0)) * bf_lo(uw[j]), x1 / (1.0f + __expf(-x1)) * bf_hi(uw[j]));
            } else {
                const float z0 = relu(x0), z1 = relu(x1);
                o[j] = pack2(z0 * z0, z1 * z1);
            }
        }
        h[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

moe_status launch_rows_grad(const RowsGradProblem& g, WsHeader* hdr, cudaStream_t st) {
    const long long tiles = (g.rows / TM + g.groups) * (((long long)g.N + TN - 1) / TN);
    if (device_sm_count() < 2 || tiles > INT_MAX / 2 || smem_bytes(g.groups) > (size_t)MAX_DYN_SMEM) {
        set_error("gradient GEMM: unsupported problem (groups %d, K %d, N %d)", g.groups, g.K, g.N);
        return MOE_ERR_UNSUPPORTED;
    }
    CUtensorMap ma, mb;
    if (!make_tensor_map_bf16(&ma, g.a, g.rows, g.K, 128u)) return MOE_ERR_CUDA;
    if (!make_tensor_map_bf16_groups(&mb, g.w, g.groups, g.K, g.N, 64u)) return MOE_ERR_CUDA;
    GParams gp{};
    gp.offsets = g.offsets;
    gp.groups = g.groups;
    gp.a_rows = (int)g.rows;
    gp.K = g.K;
    gp.N = g.N;
    gp.out = g.out;
    gp.ldo = g.ldo;
    gp.pre = reinterpret_cast<const __nv_bfloat16*>(g.pre);
    gp.ldp = g.ldo;
    gp.up_off = g.N;
    gp.hdr = hdr;
    if (!g.pre) return launch_kind<kRowsPlain>(ma, mb, gp, st);
    return g.act == MOE_ACT_SWIGLU ? launch_kind<kRowsSwiGLU>(ma, mb, gp, st) : launch_kind<kRowsReLU2>(ma, mb, gp, st);
}

moe_status launch_weights_grad(const WeightsGradProblem& g, WsHeader* hdr, cudaStream_t st) {
    const long long tiles = (long long)g.groups * ((g.M + TM - 1) / TM) * ((g.N + TN - 1) / TN);
    if (device_sm_count() < 2 || tiles > INT_MAX / 2 || smem_bytes(g.groups) > (size_t)MAX_DYN_SMEM) {
        set_error("weight-gradient GEMM: unsupported problem (groups %d, M %d, N %d)", g.groups, g.M, g.N);
        return MOE_ERR_UNSUPPORTED;
    }
    CUtensorMap ma, mb;
    if (!make_tensor_map_bf16(&ma, g.a, g.rows, g.M, 64u) || !make_tensor_map_bf16(&mb, g.b, g.rows, g.N, 64u))
        return MOE_ERR_CUDA;
    GParams gp{};
    gp.offsets = g.offsets;
    gp.groups = g.groups;
    gp.a_rows = (int)g.rows;
    gp.M = g.M;
    gp.N = g.N;
    gp.out = g.out;
    gp.ldo = g.N;
    gp.wmode = g.wmode;
    gp.hdr = hdr;
    return launch_kind<kWeights>(ma, mb, gp, st);
}

cudaError_t launch_act(const moe_shape& s, const int32_t* offsets, const uint16_t* pre, uint16_t* h, cudaStream_t st) {
    const long long rows = (long long)s.tokens * s.top_k;
    const int IV = s.inter / 8;
    const bool glu = s.act == MOE_ACT_SWIGLU;
    long long blocks = (rows * IV + 255) / 256;
    const long long cap = (long long)device_sm_count() * 8;
    if (blocks > cap) blocks = cap;
    const long long ldv = (glu ? 2LL : 1LL) * IV;
    const uint4* p = reinterpret_cast<const uint4*>(pre);
    uint4* o = reinterpret_cast<uint4*>(h);
    if (glu) return launch_kernel(act_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, st, 1, kUsePdl, rows, IV, ldv, offsets, s.experts, p, o);
    return launch_kernel(act_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, st, 1, kUsePdl, rows, IV, ldv, offsets, s.experts, p, o);
}

}  // namespace moe
