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
// and its 128 B columns per 64-deep step (32 KiB a stage, five or six stages) and
// holding 128 rows of two 256-column accumulators, so the epilogue of one tile runs
// under the next tile's main loop.  The rows form's epilogue applies the
// activation's derivative: dpre = act'(pre) * dh, from the saved pre-activations.
//
// A group's last, partial row tile of the rows form runs with the operands swapped
// (C^T = W^T A^T): the pair's 256 weight columns on the MMA's M side, the tile's
// rows, padded to 16, on its N side, so that a few rows cost a few rows of tensor
// work -- under the power cap saved work is saved time.
//
// One launch does both forms of one projection (dh with dW2, dx with dW13): they
// read the same rows and need nothing of each other, a launch less costs a small
// layer 8 us less, and the short tiles of the weights form fill the last, partly
// filled round of the long tiles of the rows form.
//
// A form with few output tiles and long reductions (grad_plan) has them split: a pair
// takes one part of one tile and writes its FP32 partial result to the workspace, and
// join_kernel adds the parts in order and does what the epilogue would have done.  One
// expert of 565 rows, H 6432, I 416: 57 us in one piece, 42 split.
//
// The weights form reduces over a group's rows.  A last step of fewer than 64
// rows also loads rows of the next group (or past the last one); each CTA's fixer
// warp waits for that step's copies on a barrier of its own, zeroes the rows past
// the bound up to the next multiple of 16 in both operands -- zeroing one would
// leave 0 * NaN --, the peer's fixer tells the leader's, and that arrives on the
// stage barrier; the MMA issues only the 16-row slices that hold rows.  A group
// without rows writes zeros.
//
// dpre is rounded to BF16 between the two calls, as every tensor that a GEMM reads: the
// MMA takes BF16 operands.  With FP32 sums on both sides of it the weight and row
// gradients after it carry two independent roundings instead of one: 0.0023 to 0.0024
// relative against the formulas in 64 bits, where one rounding is 0.0017.
//
// Every wait is bounded, and a warp that waits gives up as a whole; on a timeout the
// CTA stops issuing work, lets its copies land, frees TMEM, raises MOE_ERR_TIMEOUT and
// returns.
#include "common.cuh"

#include <climits>
#include <mutex>
#include <type_traits>

namespace moe {
namespace {

enum Act : int { kSwiGLU = 0, kReLU2 = 1, kPlain = 2 };      // what the rows form's epilogue applies

constexpr int TM = kGradTile, TN = kGradTile, BK = kGradStep;   // output tile of the pair, reduction step
constexpr int HALF = 128;                         // rows / columns each CTA contributes
constexpr int OP_BYTES = HALF * BK * 2;           // 16 KiB an operand and CTA
constexpr int BOX_BYTES = 64 * BK * 2;            // one 64 x 64 box of an MN-major operand
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int MAX_STAGES = 6;                     // five where the group tables leave no room for six
constexpr int EPI_WARPS = 8;                      // two per 32 rows, 128 columns each
constexpr int EPI_COLS = TN * 4 / EPI_WARPS;
constexpr int EPI_BYTES = 4096;                   // staging of one epilogue warp
constexpr int THREADS = 32 * (3 + EPI_WARPS);     // producer, MMA, epilogue, fixer
constexpr uint32_t TMEM_COLS = 512;
constexpr int kBand = 8;                          // column tiles per band of the tile order
constexpr int MAX_DYN_SMEM = 232448 - 1024;       // the opt-in limit less the kernel's static part

struct GParams {
    const int32_t* offsets;          // NULL: one group of all rows
    int groups, a_rows;              // the bounds lie in [0, a_rows]
    int stages;                      // of the shared-memory ring
    WsHeader* hdr;
    // rows form (N == 0: not asked for)
    int K, N;
    __nv_bfloat16* out;
    long long ldo;
    const __nv_bfloat16* pre;        // [a_rows, up] pre-activations, row stride ldo
    int up_off;                      // SwiGLU: columns from gate to up half
    // weights form (wM == 0: not asked for)
    int wM, wN, wmode;               // wmode: moe_wgrad
    void* wout;
    // SPLIT: parts of each form's reduction, and their results [rsplit][a_rows][N] and
    // [wsplit][groups][wM][wN] (not used where there is one part)
    int rsplit, wsplit;
    float* rpart;
    float* wpart;
};

struct Ctl {
    unsigned long long full[MAX_STAGES], empty[MAX_STAGES], part[MAX_STAGES], fixed[MAX_STAGES];
    unsigned long long tfull[2], tempty[2];
    unsigned long long drain;
    uint32_t tmem_base;
    int abort;
    int rows_tiles;
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
// mbar_wait_bounded with the acquire at cluster scope: the other CTA of the pair
// arrives on the leader's barrier (its fixer, its epilogue warps).
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
__device__ __forceinline__ bool mbar_wait_cluster_warp(uint32_t bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort)) != 0;
}
// Relaxed arrival on a barrier of the pair: it hands back an accumulator, whose
// reads tcgen05.fence::before_thread_sync orders; a release would also wait for the
// warp's stores of the tile before.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}
// wait_armed_stages for one CTA of a pair (`rank`).  The copies of a whole step count
// on the leader's full barrier, which only the leader can wait on; those of a partial
// step (stage s last armed so: bit s of `on_part`) on a barrier of each CTA's own,
// whose uses `part_uses` counts modulo two -- the leader's full barrier then waits for
// the fixer, which may have given up as well.
__device__ __forceinline__ bool wait_armed_pair_stages(uint32_t full0, uint32_t part0, int stages, long long armed,
                                                       uint32_t on_part, uint32_t part_uses, uint32_t rank) {
    const unsigned long long end = globaltimer_ns() + kWaitLimitNs;
    bool all = true;
    for (long long j = armed > stages ? armed - stages : 0; j < armed; ++j) {
        const uint32_t s = (uint32_t)(j % stages);
        if ((on_part >> s) & 1u) {
            if (!mbar_wait_until(part0 + 8u * s, ((part_uses >> s) & 1u) ^ 1u, end)) all = false;
        } else if (rank != 0 || !mbar_wait_until(full0 + 8u * s, (uint32_t)((j / stages) & 1), end)) {
            all = false;
        }
    }
    return all;
}
// Release, at cluster scope, of this CTA's shared memory only.  (A full release
// waits for every store of the thread: it took the fixer 0.5 us and more a tile.)
__device__ __forceinline__ void fence_release_smem_cluster() {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
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
// d silu(g) u: dg = dh u s (1 + g (1 - s)), du = dh g s, s = sigmoid(g).  s and 1 - s
// come from e = exp(-|g|), so neither cancels and a saturated gate keeps its small s
// (1 / (1 + exp(-g)) drops it from |g| = 87 on).
__device__ __forceinline__ void swiglu_grad(float dh, float g, float u, float& dg, float& du) {
    const float e = __expf(-fabsf(g));
    const float r = __fdividef(1.0f, 1.0f + e), er = e * r;
    const float s = g >= 0.f ? r : er, t = g >= 0.f ? er : r;      // t = 1 - s
    const float gs = g * s;
    dg = dh * u * fmaf(gs, t, s);
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
__device__ __forceinline__ uint4* unit32(uint8_t* slot, int row, int u) {      // 32-byte rows
    return reinterpret_cast<uint4*>(slot + row * 32 + ((u ^ ((row >> 2) & 1)) * 16));
}
__device__ __forceinline__ uint4 pack8(const uint32_t* v) {
    return make_uint4(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])), pack2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                      pack2(__uint_as_float(v[4]), __uint_as_float(v[5])), pack2(__uint_as_float(v[6]), __uint_as_float(v[7])));
}

// BF16 output, 64 columns at a time.
template <typename F>
__device__ __forceinline__ void bf16_tile(uint32_t tl, bool empty, int rows, int n0, int N, __nv_bfloat16* out,
                                          long long ldo, uint8_t* s, int lane, F&& release) {
#pragma unroll 1
    for (int c = 0; c < EPI_COLS / 64; ++c) {
        uint32_t v[2][32];
        if (!empty) {
            tmem_ld_32cols(tl + c * 64, v[0]);
            tmem_ld_32cols(tl + c * 64 + 32, v[1]);
            tmem_ld_wait();
            if (c == EPI_COLS / 64 - 1) release();
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[0][i] = v[1][i] = 0u;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) *unit128(s, lane, u) = pack8(v[u >> 2] + 8 * (u & 3));
        __syncwarp();
        const int u = lane & 7, col = n0 + c * 64 + u * 8;
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = *unit128(s, i * 4 + (lane >> 3), u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            if (r < rows && col < N) *reinterpret_cast<uint4*>(out + r * ldo + col) = w[i];
        }
        __syncwarp();
    }
}

// FP32 output (stored or added to), 32 columns at a time.
template <typename F>
__device__ __forceinline__ void f32_tile(uint32_t tl, bool empty, int rows, int n0, int N, bool add, float* out,
                                         uint8_t* s, int lane, F&& release) {
#pragma unroll 1
    for (int c = 0; c < EPI_COLS / 32; ++c) {
        const int u = lane & 7, col = n0 + c * 32 + u * 4;
        float4 old[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            old[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (add && r < rows && col < N) old[i] = *reinterpret_cast<const float4*>(out + (size_t)r * N + col);
        }
        uint32_t v[32];
        if (!empty) {
            tmem_ld_32cols(tl + c * 32, v);
            tmem_ld_wait();
            if (c == EPI_COLS / 32 - 1) release();
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) *unit128(s, lane, i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            const uint4 w = *unit128(s, r, u);
            if (r < rows && col < N)
                *reinterpret_cast<float4*>(out + (size_t)r * N + col) =
                    make_float4(old[i].x + __uint_as_float(w.x), old[i].y + __uint_as_float(w.y),
                                old[i].z + __uint_as_float(w.z), old[i].w + __uint_as_float(w.w));
        }
        __syncwarp();
    }
}

// The activation's gradient, 16 columns at a time: the pre-activations of a chunk
// come into the slot with cp.async while the chunk before is worked on (two halves
// of [gate 1 KiB | up 1 KiB]), each thread replaces its row's values by their
// gradients, and the half is written out.
constexpr int ACT_COLS = 16, ACT_CHUNKS = EPI_COLS / ACT_COLS;
template <bool GLU>
__device__ __forceinline__ void act_fetch(const GParams& p, int c, int m0, int rows, int row0, int n0, uint8_t* slot,
                                          int lane) {
    uint8_t* s = slot + (c & 1) * 2048;
    const int u = lane & 1, col = n0 + c * ACT_COLS + u * 8;
    if (c < ACT_CHUNKS && col < p.N) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 16 + (lane >> 1);
            if (r < rows) {
                const __nv_bfloat16* src = p.pre + (size_t)(row0 + m0 + r) * p.ldo + col;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(unit32(s, r, u))), "l"(src) : "memory");
                if (GLU)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                 :: "r"(smem_u32(unit32(s + 1024, r, u))), "l"(src + p.up_off) : "memory");
            }
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <bool GLU>
__device__ __forceinline__ void act_prefetch(const GParams& p, int m0, int rows, int row0, int n0, uint8_t* slot, int lane) {
    act_fetch<GLU>(p, 0, m0, rows, row0, n0, slot, lane);
    act_fetch<GLU>(p, 1, m0, rows, row0, n0, slot, lane);
    // the rest of the warp's rows into L2 (64 columns a line), while the tile is multiplied
    if (lane < rows) {
        const __nv_bfloat16* src = p.pre + (size_t)(row0 + m0 + lane) * p.ldo;
#pragma unroll
        for (int c = 0; c < EPI_COLS; c += 64) {
            const int col = n0 + c;
            if (col < p.N) {
                asm volatile("prefetch.global.L2 [%0];" :: "l"(src + col));
                if (GLU) asm volatile("prefetch.global.L2 [%0];" :: "l"(src + p.up_off + col));
            }
        }
    }
}
template <bool GLU, typename F>
__device__ __forceinline__ void act_tile(const GParams& p, uint32_t tl, int m0, int rows, int row0, int n0,
                                         uint8_t* slot, int lane, F&& release) {
    __nv_bfloat16* out = p.out + (size_t)(row0 + m0) * p.ldo;
#pragma unroll 1
    for (int c = 0; c < ACT_CHUNKS; ++c) {
        uint8_t* s = slot + (c & 1) * 2048;
        uint32_t v[16];
        tmem_ld_16cols(tl + c * ACT_COLS, v);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        tmem_ld_wait();
        if (c == ACT_CHUNKS - 1) release();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint4 g4 = *unit32(s, lane, u);
            const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
            uint32_t o[4];
            if (GLU) {
                const uint4 u4 = *unit32(s + 1024, lane, u);
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
                *unit32(s + 1024, lane, u) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = pack2(__uint_as_float(v[8 * u + 2 * i]) * (2.0f * relu(bf_lo(gw[i]))),
                                 __uint_as_float(v[8 * u + 2 * i + 1]) * (2.0f * relu(bf_hi(gw[i]))));
            }
            *unit32(s, lane, u) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
        const int u = lane & 1, col = n0 + c * ACT_COLS + u * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 16 + (lane >> 1);
            if (r < rows && col < p.N) {
                *reinterpret_cast<uint4*>(out + r * p.ldo + col) = *unit32(s, r, u);
                if (GLU) *reinterpret_cast<uint4*>(out + r * p.ldo + p.up_off + col) = *unit32(s + 1024, r, u);
            }
        }
        __syncwarp();
        act_fetch<GLU>(p, c + 2, m0, rows, row0, n0, slot, lane);
    }
}

// The pre-activations a warp of a swapped tile will read, into L2.
template <bool GLU>
__device__ __forceinline__ void swapped_prefetch(const GParams& p, int rows, int row0, int n0, int first, int lane) {
    if (n0 >= p.N) return;
    for (int r = first * 32 + lane; r < rows; r += 32 * (EPI_WARPS / 4)) {
        const __nv_bfloat16* src = p.pre + (size_t)(row0 + r) * p.ldo + n0;
        asm volatile("prefetch.global.L2 [%0];" :: "l"(src));
        if (GLU) asm volatile("prefetch.global.L2 [%0];" :: "l"(src + p.up_off));
    }
}

// A swapped tile: lane = output column n0 + lane, accumulator column = row.  The two
// warps of a lane quarter take its 32-row chunks in turn, through a slot of [32 rows x
// 32 columns] (SwiGLU: gate, then up), pre-activations fetched into it first.
template <int ACT, typename F>
__device__ __forceinline__ void swapped_tile(const GParams& p, uint32_t tl, int rows, int row0, int n0, int first,
                                             uint8_t* s, int lane, F&& release) {
    constexpr int STEP = EPI_WARPS / 4;
    const int u = lane & 3, col = n0 + u * 8;
    __nv_bfloat16* mine = reinterpret_cast<__nv_bfloat16*>(s) + lane;
    int last = (rows - 1) / 32;                                   // this warp's last chunk
    last -= (last - first) & (STEP - 1);
    if (first > last) release();
#pragma unroll 1
    for (int c = first; c * 32 < rows; c += STEP) {
        const int left = rows - c * 32;
        const size_t base = (size_t)(row0 + c * 32) * p.ldo + col;
        if (ACT != kPlain) {
            if (col < p.N) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 8 + (lane >> 2);
                    if (r < left) {
                        const __nv_bfloat16* src = p.pre + base + (size_t)r * p.ldo;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(s + r * 64 + u * 16)), "l"(src) : "memory");
                        if (ACT == kSwiGLU)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                         :: "r"(smem_u32(s + 2048 + r * 64 + u * 16)), "l"(src + p.up_off) : "memory");
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        uint32_t v[32];
        tmem_ld_32cols(tl + c * 32, v);
        if (ACT != kPlain) asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        tmem_ld_wait();
        if (c == last) release();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            float f = __uint_as_float(v[j]);
            if (ACT == kSwiGLU) {
                float dg, du;
                swiglu_grad(f, __bfloat162float(mine[j * 32]), __bfloat162float(mine[1024 + j * 32]), dg, du);
                mine[1024 + j * 32] = __float2bfloat16_rn(du);
                f = dg;
            } else if (ACT == kReLU2) {
                f *= 2.0f * relu(__bfloat162float(mine[j * 32]));
            }
            mine[j * 32] = __float2bfloat16_rn(f);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            if (r < left && col < p.N) {
                __nv_bfloat16* o = p.out + base + (size_t)r * p.ldo;
                *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(s + r * 64 + u * 16);
                if (ACT == kSwiGLU)
                    *reinterpret_cast<uint4*>(o + p.up_off) = *reinterpret_cast<const uint4*>(s + 2048 + r * 64 + u * 16);
            }
        }
        __syncwarp();
    }
}

struct Tile {
    int g, m0, n0, row0, mrows;
    __device__ __forceinline__ bool partial() const { return mrows - m0 < TM; }          // rows form
    __device__ __forceinline__ int padded() const { return (mrows - m0 + 15) & ~15; }
};

// Tile `local` of a group of mtiles row tiles: bands of kBand column tiles, row
// tiles first inside a band, so the tiles in flight share their operands in L2.
__device__ __forceinline__ void place(Tile& t, int local, int mtiles) {
    if (mtiles == 1) {           // a small group: no division
        t.m0 = 0;
        t.n0 = local * TN;
        return;
    }
    const int band = local / (mtiles * kBand);
    const int idx = local - band * mtiles * kBand;
    const int nt = idx / mtiles;
    t.m0 = (idx - nt * mtiles) * TM;
    t.n0 = (band * kBand + nt) * TN;
}

__device__ __forceinline__ Tile rows_tile(int tile, const int* prefix, const int* rstart, const int* rcount, int groups) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= tile) lo = mid; else hi = mid;
    }
    Tile t;
    t.g = lo;
    t.row0 = rstart[lo];
    t.mrows = rcount[lo];
    place(t, tile - prefix[lo], (t.mrows + TM - 1) / TM);
    return t;
}

__device__ __forceinline__ Tile weights_tile(int tile, const int* rstart, const int* rcount, int ntm, int ntn) {
    Tile t;
    t.g = tile / (ntm * ntn);
    t.row0 = rstart[t.g];
    t.mrows = rcount[t.g];
    place(t, tile - t.g * ntm * ntn, ntm);
    return t;
}

// The tiles of one CTA pair, the same for every role: first the rows form's, dealt
// round; the `extra` pairs that got one more of them than the rest then sit out the
// first `skip` rounds of the (mostly shorter) weights form's tiles, as many as take
// about as long as that tile: the loop adds up their steps, five at least, which is
// what writing a tile takes.
// Split: the same with every part of a tile in its place.
template <bool SPLIT>
struct Walk {
    int nrows, total, pairs, pair, extra, skip, i, s, j;          // counts of parts
    int rsplit, wsplit, part;                                     // part: of the tile next() returned
    __device__ __forceinline__ Walk(int row_tiles, int weight_tiles, int pairs_, int pair_, int row_steps, int per_group,
                                    const int* rcount, int rsplit_, int wsplit_)
        : pairs(pairs_), pair(pair_), skip(0), i(pair_), s(0), rsplit(rsplit_), wsplit(wsplit_), part(0) {
        nrows = row_tiles * (SPLIT ? rsplit : 1);
        total = nrows + weight_tiles * (SPLIT ? wsplit : 1);
        if (SPLIT) row_steps /= rsplit;
        extra = nrows % pairs;
        if (extra)
            for (int steps = 0; nrows + skip * pairs < total; ++skip) {
                const int g = skip * pairs / per_group / (SPLIT ? wsplit : 1);
                const int mine = max((rcount[g] + BK - 1) / BK / (SPLIT ? wsplit : 1), 5);
                if (steps + mine / 2 >= row_steps) break;
                steps += mine;
            }
        j = nrows + skip * (pairs - extra) + pair;
    }
    // The tile, the rows form's first; -1: done.
    __device__ __forceinline__ int next() {
        int t;
        if (i < nrows) {
            t = i;
            i += pairs;
        } else if (s < skip && pair >= extra) {
            t = nrows + s * (pairs - extra) + pair - extra;
            ++s;
        } else {
            t = j;
            j += pairs;
        }
        if (t >= total) return -1;
        if (!SPLIT) return t;
        if (t < nrows) {
            part = t % rsplit;
            return t / rsplit;
        }
        part = (t - nrows) % wsplit;
        return nrows / rsplit + (t - nrows) / wsplit;
    }
    // The steps of this part of a reduction of nk, and whether it is one of several.
    __device__ __forceinline__ int parts(bool weights) const { return SPLIT ? (weights ? wsplit : rsplit) : 1; }
    __device__ __forceinline__ int first(int nk, bool weights) const {
        return SPLIT ? (int)((long long)nk * part / parts(weights)) : 0;
    }
    __device__ __forceinline__ int last(int nk, bool weights) const {
        return SPLIT ? (int)((long long)nk * (part + 1) / parts(weights)) : nk;
    }
};

template <int ACT, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
grad_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmWA, const __grid_constant__ CUtensorMap tmWB,
                      const GParams p) {
    const int stages = p.stages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
    uint8_t* epi_smem = smem + stages * STAGE_BYTES;
    Ctl* ctl = reinterpret_cast<Ctl*>(epi_smem + EPI_WARPS * EPI_BYTES);
    int* prefix = reinterpret_cast<int*>(ctl + 1);          // rows form: tiles before group g
    int* rstart = prefix + (p.groups + 1);
    int* rcount = rstart + p.groups;
    const uint32_t smem_base = smem_u32(smem);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();                 // 0: leader, 1: peer
    const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
    const int ntn = (p.N + TN - 1) / TN;
    const int wtm = (p.wM + TM - 1) / TM, wtn = (p.wN + TN - 1) / TN;

    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
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
        tma_prefetch_desc(&tmWA);
        tma_prefetch_desc(&tmWB);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();              // both CTAs' barriers are initialised before any cross-CTA arrive
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    // Bounds that decrease or leave [0, a_rows] are refused as a whole: with none of
    // them the buckets are disjoint, so the tile count stays below the host's bound.
    int bad = 0;
    for (int g = tid; g < p.groups; g += THREADS) {
        const int lo = p.offsets ? p.offsets[g] : 0, hi = p.offsets ? p.offsets[g + 1] : p.a_rows;
        bad |= lo < 0 || hi < lo || hi > p.a_rows;
        rstart[g] = lo;
        rcount[g] = hi - lo;
    }
    if (__syncthreads_or(bad)) {
        for (int g = tid; g < p.groups; g += THREADS) rstart[g] = rcount[g] = 0;
        if (tid == 0) raise_status(p.hdr, MOE_ERR_INVALID_ROUTE);
        __syncthreads();
    }
    // prefix[0..groups]: tiles of the rows form before each group
    if (p.groups <= 32) {        // one warp's scan
        if (warp == 0) {
            const int mine = lane < p.groups ? ((rcount[lane] + TM - 1) / TM) * ntn : 0;
            int inc = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += v;
            }
            if (lane < p.groups) prefix[lane] = inc - mine;
            if (lane == 31) { prefix[p.groups] = inc; ctl->rows_tiles = inc; }
        }
    } else {
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
        if (tid == THREADS - 1) { prefix[n] = run; ctl->rows_tiles = run; }
    }
    __syncthreads();
    const uint32_t tmem_base = ctl->tmem_base;
    volatile int* abort = &ctl->abort;
    const int nk_rows = (p.K + BK - 1) / BK;
    const int nrows = ctl->rows_tiles;
    Walk<SPLIT> walk(nrows, p.groups * wtm * wtn, npairs, pair, nk_rows, wtm * wtn, rcount, p.rsplit, p.wsplit);

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        if (lane == 0) {
            int stage = 0;
            uint32_t ph = 0;
            bool ok = true;
            long long armed = 0;
            uint32_t on_part = 0, part_uses = 0;     // for wait_armed_pair_stages
            for (int tile; ok && (tile = walk.next()) >= 0;) {
                const bool weights = tile >= nrows;
                const Tile t = weights ? weights_tile(tile - nrows, rstart, rcount, wtm, wtn)
                                       : rows_tile(tile, prefix, rstart, rcount, p.groups);
                const bool swap = !weights && t.partial() && walk.parts(false) == 1;
                // this CTA's rows (rows form) or columns of A: 128, or half of the padded rows
                const int a0 = t.m0 + (int)rank * (swap ? t.padded() / 2 : HALF);
                const int b0 = t.n0 + (int)rank * HALF;
                // one loop for each form: a step has 512 cycles, and one thread issues it
                auto load = [&](auto form) {
                    constexpr bool kW = decltype(form)::value;
                    const int nk = kW ? (t.mrows + BK - 1) / BK : nk_rows;
                    for (int i = walk.first(nk, kW), end = walk.last(nk, kW); i < end; ++i) {
                        if (!mbar_wait_bounded(smem_u32(&ctl->empty[stage]), ph ^ 1u, abort)) { ok = false; break; }
                        const uint32_t full_local = smem_u32(&ctl->full[stage]);
                        const uint32_t full_leader = mapa_shared(full_local, 0);
                        const uint32_t sa = smem_base + stage * STAGE_BYTES, sb = sa + OP_BYTES;
                        on_part &= ~(1u << stage);
                        if (kW) {
                            const int y = t.row0 + i * BK;
                            if (t.mrows - i * BK < BK) {
                                // partial step: counted on this CTA's own barrier, for its fixer
                                const uint32_t part = smem_u32(&ctl->part[stage]);
                                on_part |= 1u << stage;
                                part_uses ^= 1u << stage;
                                mbar_arrive_expect_tx(part, STAGE_BYTES);
                                tma_load_2d(sa, &tmWA, part, a0, y);
                                tma_load_2d(sa + BOX_BYTES, &tmWA, part, a0 + 64, y);
                                tma_load_2d(sb, &tmWB, part, b0, y);
                                tma_load_2d(sb + BOX_BYTES, &tmWB, part, b0 + 64, y);
                            } else {
                                if (rank == 0) mbar_arrive_expect_tx(full_local, 2 * STAGE_BYTES);
                                tma_load_2d_pair(sa, &tmWA, full_leader, a0, y);
                                tma_load_2d_pair(sa + BOX_BYTES, &tmWA, full_leader, a0 + 64, y);
                                tma_load_2d_pair(sb, &tmWB, full_leader, b0, y);
                                tma_load_2d_pair(sb + BOX_BYTES, &tmWB, full_leader, b0 + 64, y);
                            }
                        } else {
                            // swapped: weights in the MMA's A slot, rows in its B slot
                            const uint32_t s_rows = swap ? sb : sa, s_w = swap ? sa : sb;
                            if (rank == 0) mbar_arrive_expect_tx(full_local, 2 * STAGE_BYTES);
                            tma_load_2d_pair(s_rows, &tmA, full_leader, i * BK, t.row0 + a0);
                            tma_load_3d_pair(s_w, &tmB, full_leader, b0, i * BK, t.g);
                            tma_load_3d_pair(s_w + BOX_BYTES, &tmB, full_leader, b0 + 64, i * BK, t.g);
                        }
                        ++armed;
                        if (++stage == stages) { stage = 0; ph ^= 1u; }
                    }
                };
                if (weights) load(std::true_type{});
                else load(std::false_type{});
            }
            if (ok) ok = drain_ring(smem_u32(&ctl->empty[0]), stages, stage, ph, abort);
            if (!ok) {
                // the copies issued land before the CTA exits; the closing cluster barrier
                // holds the peer until the leader has seen its whole steps' too
                if (!wait_armed_pair_stages(smem_u32(&ctl->full[0]), smem_u32(&ctl->part[0]), stages, armed, on_part,
                                            part_uses, rank))
                    settle_delay();
                raise_status(p.hdr, MOE_ERR_TIMEOUT);
                p.hdr->timeout_site = kSiteGradProducer;
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader CTA) ----------------
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t ph = 0;
            int acc = 0;
            uint32_t aph = 0;
            bool ok = true;
            for (int tile; ok && (tile = walk.next()) >= 0;) {
                const bool weights = tile >= nrows;
                Tile t{};
                if (weights) t.mrows = rcount[(tile - nrows) / (wtm * wtn)];
                else t = rows_tile(tile, prefix, rstart, rcount, p.groups);
                const int nk_all = weights ? (t.mrows + BK - 1) / BK : nk_rows;
                const int i0 = walk.first(nk_all, weights), nk = walk.last(nk_all, weights);
                if (i0 == nk) continue;
                if (!mbar_wait_cluster(smem_u32(&ctl->tempty[acc]), aph ^ 1u, abort)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(acc * TN);
                // A and B: MN-major (boxes of reduction rows) or K-major
                auto multiply = [&](auto a_mn, auto b_mn, uint32_t idesc) {
                    constexpr bool kAmn = decltype(a_mn)::value, kBmn = decltype(b_mn)::value, kW = kAmn && kBmn;
                    for (int i = i0; i < nk; ++i) {
                        if (!mbar_wait_bounded(smem_u32(&ctl->full[stage]), ph, abort)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t sa = smem_base + stage * STAGE_BYTES, sb = sa + OP_BYTES;
                        const uint64_t ad = kAmn ? sdesc_mn_sw128(sa) : sdesc_k_sw128(sa);
                        const uint64_t bd = kBmn ? sdesc_mn_sw128(sb) : sdesc_k_sw128(sb);
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            if (!kW || i * BK + kk * 16 < t.mrows)        // slices that hold rows
                                tc_mma_bf16_pair(d, ad + (uint64_t)kk * (kAmn ? kMnStep : kKStep),
                                                 bd + (uint64_t)kk * (kBmn ? kMnStep : kKStep), idesc,
                                                 (i > i0 || kk > 0) ? 1u : 0u);
                        tc_commit_pair_mc(smem_u32(&ctl->empty[stage]), (uint16_t)3);
                        if (++stage == stages) { stage = 0; ph ^= 1u; }
                    }
                };
                if (weights) multiply(std::true_type{}, std::true_type{}, idesc_bf16_f32(TM, TN) | kMajorA | kMajorB);
                else if (t.partial() && walk.parts(false) == 1) multiply(std::true_type{}, std::false_type{}, idesc_bf16_f32(TM, t.padded()) | kMajorA);
                else multiply(std::false_type{}, std::true_type{}, idesc_bf16_f32(TM, TN) | kMajorB);
                if (!ok) break;
                tc_commit_pair_mc(smem_u32(&ctl->tfull[acc]), (uint16_t)3);
                acc ^= 1;
                if (acc == 0) aph ^= 1u;
            }
            // and every one that the peer's epilogue sends to the leader: after this CTA
            // they would hit the next one's memory
            for (int a = 0; ok && a < 2; ++a) {
                if (!mbar_wait_cluster(smem_u32(&ctl->tempty[acc]), aph ^ 1u, abort)) ok = false;
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
        // ---------------- epilogue (both CTAs): a warp = 32 rows x EPI_COLS columns ----------------
        const int q = warp & 3;                                      // the TMEM lanes a warp can read
        const int c0 = (warp - 2) / 4 * EPI_COLS;
        uint8_t* epi = epi_smem + (warp - 2) * EPI_BYTES;
        int acc = 0;
        uint32_t aph = 0;
        for (int tile; (tile = walk.next()) >= 0;) {
            const bool weights = tile >= nrows;
            const Tile t = weights ? weights_tile(tile - nrows, rstart, rcount, wtm, wtn)
                                   : rows_tile(tile, prefix, rstart, rcount, p.groups);
            const int m0 = t.m0 + (int)rank * HALF + q * 32;
            const int rows = (weights ? p.wM : t.mrows) - m0;            // of its 32 rows, those below the bound
            const int n0 = t.n0 + c0;
            const int nk = weights ? (t.mrows + BK - 1) / BK : nk_rows;
            const bool empty = walk.first(nk, weights) == walk.last(nk, weights);   // zeros, no accumulator
            const bool parts = walk.parts(weights) > 1;
            const bool swap = !weights && t.partial() && !parts;
            if (ACT != kPlain && !weights && !parts) {
                if (!swap)
                    act_prefetch<ACT == kSwiGLU>(p, m0, rows, t.row0, n0, epi, lane);
                else
                    swapped_prefetch<ACT == kSwiGLU>(p, t.mrows - t.m0, t.row0 + t.m0, t.n0 + (int)rank * HALF + q * 32,
                                                     (warp - 2) / 4, lane);
            }
            if (!empty) {
                if (!mbar_wait_warp(smem_u32(&ctl->tfull[acc]), aph, abort)) {
                    if (lane == 0) {
                        raise_status(p.hdr, MOE_ERR_TIMEOUT);
                        p.hdr->timeout_site = kSiteGradEpilogue;
                    }
                    break;
                }
                tc_fence_after();
            }
            const uint32_t tl = tmem_base + (uint32_t)(acc * TN + c0) + ((uint32_t)(q * 32) << 16);
            auto release = [&] {               // the accumulator is read: the next tile may overwrite it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(mapa_shared(smem_u32(&ctl->tempty[acc]), 0));
            };
            if (SPLIT && parts) {
                float* out = weights ? p.wpart + (((size_t)walk.part * p.groups + t.g) * p.wM + m0) * p.wN
                                     : p.rpart + ((size_t)walk.part * p.a_rows + t.row0 + m0) * p.N;
                f32_tile(tl, empty, rows, n0, weights ? p.wN : p.N, false, out, epi, lane, release);
            } else if (swap) {
                swapped_tile<ACT>(p, tl - c0, t.mrows - t.m0, t.row0 + t.m0, t.n0 + (int)rank * HALF + q * 32,
                                  (warp - 2) / 4, epi, lane, release);
            } else if (weights && p.wmode != MOE_WGRAD_BF16) {
                if (!(empty && p.wmode == MOE_WGRAD_F32_ADD))
                    f32_tile(tl, empty, rows, n0, p.wN, p.wmode == MOE_WGRAD_F32_ADD,
                             static_cast<float*>(p.wout) + ((size_t)t.g * p.wM + m0) * p.wN, epi, lane, release);
            } else if (ACT != kPlain && !weights) {
                act_tile<ACT == kSwiGLU>(p, tl, m0, rows, t.row0, n0, epi, lane, release);
            } else {
                const int N = weights ? p.wN : p.N;
                const long long ldo = weights ? (long long)p.wN : p.ldo;
                __nv_bfloat16* out = weights ? static_cast<__nv_bfloat16*>(p.wout) + ((size_t)t.g * p.wM + m0) * p.wN
                                             : p.out + (size_t)(t.row0 + m0) * p.ldo;
                bf16_tile(tl, empty, rows, n0, N, out, ldo, epi, lane, release);
            }
            if (empty) continue;
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
        // ---------------- fixer (both CTAs): the weights form's partial steps ----------------
        int stage = 0;
        uint32_t pph = 0;                          // parity of part[s] and fixed[s] in bit s
        bool ok = true;
        for (int tile; ok && (tile = walk.next()) >= 0;) {
            const bool weights = tile >= nrows;
            int nk = nk_rows, rem = 0;
            if (weights) {
                const int mrows = rcount[(tile - nrows) / (wtm * wtn)];
                nk = (mrows + BK - 1) / BK;
                if (walk.last(nk, true) == nk && walk.first(nk, true) < nk) rem = mrows & (BK - 1);
            }
            nk = walk.last(nk, weights) - walk.first(nk, weights);   // this part's
            if (rem) {
                const int s = (stage + nk - 1) % stages;
                const uint32_t parity = (pph >> s) & 1u;
                pph ^= 1u << s;
                if (!mbar_wait_warp(smem_u32(&ctl->part[s]), parity, abort)) { ok = false; break; }
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
                    if (lane == 0) {
                        fence_release_smem_cluster();
                        mbar_arrive_relaxed(mapa_shared(smem_u32(&ctl->fixed[s]), 0));
                    }
                } else {
                    if (!mbar_wait_cluster_warp(smem_u32(&ctl->fixed[s]), parity, abort)) { ok = false; break; }
                    if (lane == 0) mbar_arrive(smem_u32(&ctl->full[s]));
                }
            }
            stage = (stage + nk) % stages;
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

size_t smem_bytes(int groups, int stages) {
    return 1024 + (size_t)stages * STAGE_BYTES + EPI_WARPS * EPI_BYTES + sizeof(Ctl) + 3 * (size_t)(groups + 1) * 4;
}

template <int ACT, bool SPLIT>
moe_status launch_grad(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mwa, const CUtensorMap& mwb,
                       const GParams& gp, cudaStream_t st) {
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [] {
        attr_err = cudaFuncSetAttribute(grad_gemm_pair_kernel<ACT, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        MAX_DYN_SMEM);
    });
    if (attr_err != cudaSuccess) {
        set_error("cudaFuncSetAttribute(max dynamic smem %d): %s", MAX_DYN_SMEM, cudaGetErrorString(attr_err));
        return MOE_ERR_CUDA;
    }
    const size_t smem = smem_bytes(gp.groups, gp.stages);
    const cudaError_t e = launch_kernel(grad_gemm_pair_kernel<ACT, SPLIT>, dim3((unsigned)(device_sm_count() & ~1)),
                                        dim3(THREADS), smem, st, 2, kUsePdl, ma, mb, mwa, mwb, gp);
    if (e != cudaSuccess) {
        set_error("gradient GEMM launch (smem %zu): %s", smem, cudaGetErrorString(e));
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

// Eight consecutive elements of the parts, added in order.
__device__ __forceinline__ void add_parts(const float* part, size_t stride, int split, float (&f)[8]) {
    const float4* q = reinterpret_cast<const float4*>(part);
    float4 a = q[0], b = q[1];
    for (int s = 1; s < split; ++s) {
        q = reinterpret_cast<const float4*>(part + (size_t)s * stride);
        const float4 c = q[0], d = q[1];
        a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
        b.x += d.x; b.y += d.y; b.z += d.z; b.w += d.w;
    }
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ uint4 pack8f(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// The split reductions' second half: sums the parts and stores them as the epilogue of
// an unsplit one does, eight elements a thread (N and wN are multiples of 8).
__global__ void __launch_bounds__(256)
join_kernel(const GParams p, int act) {
    pdl_wait();
    pdl_trigger();
    // refused bounds, as in the GEMM: no bucket has rows, so no row is written and each
    // expert's weight gradient is that of an empty bucket (the GEMM left zeros as its parts)
    int bad = 0;
    for (int g = threadIdx.x; p.offsets && g < p.groups; g += blockDim.x)
        bad |= p.offsets[g] < 0 || p.offsets[g + 1] < p.offsets[g] || p.offsets[g + 1] > p.a_rows;
    const bool none = __syncthreads_or(bad) != 0;
    const int lo = p.offsets ? p.offsets[0] : 0, hi = p.offsets ? p.offsets[p.groups] : p.a_rows;
    const int nv = p.N / 8;
    const long long nr = p.rsplit > 1 && !none ? (long long)(hi - lo) * nv : 0;
    const long long nw = p.wsplit > 1 ? (long long)p.groups * p.wM * (p.wN / 8) : 0;
    const size_t rstride = (size_t)p.a_rows * p.N, wstride = (size_t)p.groups * p.wM * p.wN;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < nr + nw; i += (long long)gridDim.x * blockDim.x) {
        float f[8];
        if (i < nr) {
            const long long r = lo + i / nv;
            const int c = (int)(i % nv) * 8;
            add_parts(p.rpart + r * p.N + c, rstride, p.rsplit, f);
            __nv_bfloat16* o = p.out + r * p.ldo + c;
            if (act == kPlain) {
                *reinterpret_cast<uint4*>(o) = pack8f(f);
                continue;
            }
            const uint4 g4 = *reinterpret_cast<const uint4*>(p.pre + r * p.ldo + c);
            const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
            if (act == kReLU2) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] *= 2.0f * relu(bf_lo(gw[j]));
                    f[2 * j + 1] *= 2.0f * relu(bf_hi(gw[j]));
                }
                *reinterpret_cast<uint4*>(o) = pack8f(f);
                continue;
            }
            const uint4 u4 = *reinterpret_cast<const uint4*>(p.pre + r * p.ldo + p.up_off + c);
            const uint32_t uw[4] = {u4.x, u4.y, u4.z, u4.w};
            float du[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d0 = f[2 * j], d1 = f[2 * j + 1];
                swiglu_grad(d0, bf_lo(gw[j]), bf_lo(uw[j]), f[2 * j], du[2 * j]);
                swiglu_grad(d1, bf_hi(gw[j]), bf_hi(uw[j]), f[2 * j + 1], du[2 * j + 1]);
            }
            *reinterpret_cast<uint4*>(o) = pack8f(f);
            *reinterpret_cast<uint4*>(o + p.up_off) = pack8f(du);
        } else {
            const size_t e = (size_t)(i - nr) * 8;
            add_parts(p.wpart + e, wstride, p.wsplit, f);
            if (p.wmode == MOE_WGRAD_BF16) {
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.wout) + e) = pack8f(f);
                continue;
            }
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.wout) + e);
            float4 a = make_float4(f[0], f[1], f[2], f[3]), b = make_float4(f[4], f[5], f[6], f[7]);
            if (p.wmode == MOE_WGRAD_F32_ADD) {
                const int g = (int)(e / ((size_t)p.wM * p.wN));
                if (none || (p.offsets && p.offsets[g] == p.offsets[g + 1])) continue;    // no rows: left as it is
                const float4 x = o[0], y = o[1];
                a = make_float4(x.x + a.x, x.y + a.y, x.z + a.z, x.w + a.w);
                b = make_float4(y.x + b.x, y.y + b.y, y.z + b.z, y.w + b.w);
            }
            o[0] = a;
            o[1] = b;
        }
    }
}

// FP32 [rows, cols] to BF16 [rows, cols8], the columns past cols zero.
__global__ void __launch_bounds__(256)
round_rows_kernel(long long n, int cols, int cols8, const float* __restrict__ a, __nv_bfloat16* __restrict__ b) {
    pdl_wait();
    pdl_trigger();
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const long long r = i / cols8;
        const int c = (int)(i - r * cols8);
        b[i] = __float2bfloat16_rn(c < cols ? a[r * cols + c] : 0.f);
    }
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

moe_status launch_expert_grad(const ExpertGradProblem& g, float* partials, WsHeader* hdr, cudaStream_t st) {
    const long long rows_tiles = g.out ? (g.rows / TM + g.groups) * (((long long)g.N + TN - 1) / TN) : 0;
    const long long w_tiles = g.wout ? (long long)g.groups * ((g.wM + TM - 1) / TM) * ((g.wN + TN - 1) / TN) : 0;
    if (device_sm_count() < 2 || rows_tiles + w_tiles > INT_MAX / 2 ||
        smem_bytes(g.groups, MAX_STAGES - 1) > (size_t)MAX_DYN_SMEM) {
        set_error("gradient GEMM: unsupported problem (groups %d, K %d, N %d)", g.groups, g.K, g.N);
        return MOE_ERR_UNSUPPORTED;
    }
    CUtensorMap ma, mb, mwa, mwb;
    GParams gp{};
    if (g.out) {
        if (!make_tensor_map_bf16(&ma, g.a, g.rows, g.a_cols, 128u)) return MOE_ERR_CUDA;
        if (!make_tensor_map_bf16_groups(&mb, g.w, g.groups, g.K, g.N, 64u)) return MOE_ERR_CUDA;
        gp.K = g.K;
        gp.N = g.N;
        gp.out = reinterpret_cast<__nv_bfloat16*>(g.out);
        gp.ldo = g.ldo;
        gp.pre = reinterpret_cast<const __nv_bfloat16*>(g.pre);
        gp.up_off = g.N;
    }
    if (g.wout) {
        if (!make_tensor_map_bf16(&mwa, g.a, g.rows, g.a_cols, 64u) || !make_tensor_map_bf16(&mwb, g.wb, g.rows, g.wN, 64u))
            return MOE_ERR_CUDA;
        gp.wM = g.wM;
        gp.wN = g.wN;
        gp.wmode = g.wmode;
        gp.wout = g.wout;
    }
    if (!g.out) { ma = mwa; mb = mwb; }        // a form not asked for has no tiles: its maps are not used
    if (!g.wout) { mwa = ma; mwb = mb; }
    gp.offsets = g.offsets;
    gp.groups = g.groups;
    gp.a_rows = (int)g.rows;
    gp.stages = smem_bytes(g.groups, MAX_STAGES) <= (size_t)MAX_DYN_SMEM ? MAX_STAGES : MAX_STAGES - 1;
    gp.hdr = hdr;
    const GradDims dims = {g.rows, g.groups, gp.K, gp.N, gp.wM, gp.wN};
    const GradPlan n = grad_plan(dims);
    gp.rsplit = n.r;
    gp.wsplit = n.w;
    gp.rpart = partials;
    gp.wpart = partials + grad_rows_partials(dims, n);
    const int act = !g.out || !g.pre ? kPlain : g.act == MOE_ACT_SWIGLU ? kSwiGLU : kReLU2;
    if (n.r == 1 && n.w == 1) {
        if (act == kPlain) return launch_grad<kPlain, false>(ma, mb, mwa, mwb, gp, st);
        return act == kSwiGLU ? launch_grad<kSwiGLU, false>(ma, mb, mwa, mwb, gp, st)
                              : launch_grad<kReLU2, false>(ma, mb, mwa, mwb, gp, st);
    }
    // an activation is only applied here when the rows form itself is not split
    const int here = n.r > 1 ? (int)kPlain : act;
    const moe_status r = here == kPlain    ? launch_grad<kPlain, true>(ma, mb, mwa, mwb, gp, st)
                         : here == kSwiGLU ? launch_grad<kSwiGLU, true>(ma, mb, mwa, mwb, gp, st)
                                           : launch_grad<kReLU2, true>(ma, mb, mwa, mwb, gp, st);
    if (r != MOE_OK) return r;
    const long long vecs = ((n.r > 1 ? g.rows * gp.N : 0) + (n.w > 1 ? (long long)g.groups * gp.wM * gp.wN : 0)) / 8;
    long long blocks = (vecs + 255) / 256;
    if (blocks > device_sm_count() * 8LL) blocks = device_sm_count() * 8LL;
    return from_cuda(launch_kernel(join_kernel, dim3((unsigned)blocks), dim3(256), 0, st, 1, kUsePdl, gp, act));
}

cudaError_t launch_round_rows(long long rows, int cols, int cols8, const float* a, uint16_t* b, cudaStream_t st) {
    const long long n = rows * cols8;
    long long blocks = (n + 255) / 256;
    const long long cap = (long long)device_sm_count() * 8;
    if (blocks > cap) blocks = cap;
    return launch_kernel(round_rows_kernel, dim3((unsigned)blocks), dim3(256), 0, st, 1, kUsePdl, n, cols, cols8, a,
                         reinterpret_cast<__nv_bfloat16*>(b));
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
