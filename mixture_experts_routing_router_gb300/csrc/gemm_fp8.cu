// gemm_fp8.cu -- the grouped expert GEMM with both operands in E4M3 and a scale per
// block of 128 (fp8.cuh), on the FP8 tensor cores (tcgen05.mma kind::f8f6f4).
//
// The scales of a K block multiply that block's partial sum, so the accumulator cannot
// stay in tensor memory across K: each 128-wide K step (one 128-byte swizzle row of
// codes, four MMAs of K 32) writes a fresh FP32 accumulator, and eight warps add it,
// times a_scale * w_scale, to sums in registers.  A tile is 128 activation rows (MMA M,
// TMEM lanes) by NSUB blocks of 128 weight rows (MMA N): a thread then has one row, one
// activation scale per step and one weight scale per step and block, so adding a value
// is one multiply-add (two at a time: fma.rn.f32x2).  TMEM holds 512 / (128 NSUB)
// accumulators, so the MMAs of the next steps run while a step is added up.
//
// Roles: warp 0 loads by TMA, warp 1 issues the MMAs, warps 4..11 add up and store:
// warp w owns TMEM lanes 32 (w % 4) .. +31 and columns 64 h .. 64 h + 63 (h = (w - 4) / 4)
// of every block.  Those eight take the registers that the first warpgroup gives up
// (setmaxnreg): 128 sums and a piece of 64 columns.  For SwiGLU the two blocks are the
// gate and up rows of the same 128 output columns, so a thread holds both factors of its
// 64 outputs; the activation is quantized again as it is stored, and the two warps that
// share a row block exchange their largest magnitude through shared memory.
//
// What bounds it at large sizes is the round trip of an accumulator: four MMAs (512
// cycles) and 300 until the warps see them, then two reads of 64 columns (240 cycles
// each, of which 175 are latency) with their multiply-adds and 250 around them: 900 to 1000
// cycles a step.  Next comes shared memory: 48 KiB brought and 48 KiB read a step, 768 cycles
// at 128 bytes a cycle (without the weights' loads a call takes 869 us of 902).  Measured
// and not kept: CTA pairs (M 256; two thirds of the shared-memory traffic, but the round trip
// crosses SMs: 2 to 8 % slower), accumulators of one block each (up to 30 % slower), 16 or
// 32 columns a read, scales brought by warps of their own, a group's rest of at most 64
// rows with the operands swapped (three quarters of a wide tile's time, and the larger
// kernel slows those: 2048 tokens, 128 experts, up 101 -> 115 us).
//
// Persistent CTAs walk a tile list built from the bucket bounds, as in gemm.cu.  Every
// wait is bounded (MOE_ERR_TIMEOUT); the exchange goes through an mbarrier so that it is,
// too.
#include "gemm_fp8.cuh"

namespace moe {
namespace {

constexpr int F_BM = 128;                       // activation rows per tile
constexpr int F_THREADS = 384;
constexpr int F_EPI_WARPS = 8;
constexpr int F_STORE = 2048;                   // shared memory of a warp's output: 32 rows of 64 bytes

template <int NSUB>
struct FCfg {
    static constexpr int STAGE_BYTES = (1 + NSUB) * F_BOX;
    static constexpr int STAGES = NSUB == 2 ? 4 : 6;
    static constexpr int ACC_COLS = 128 * NSUB;
    static constexpr int ACCS = 512 / ACC_COLS;
};

struct FCtl {
    unsigned long long full[6], empty[6];
    unsigned long long tfull[4], tempty[4];
    unsigned long long xch[4];                  // the two warps of a lane quarter
    unsigned long long drain;
    uint32_t tmem_base;
    int abort;
    int wtot[F_THREADS / 32];
    float amax[2][2][2][F_BM];                  // [exchange parity][block][column half][row]
};

// Four steps' scales for a warp, copied while the four before are used: float [32 rows][4]
// and float [2 blocks][4].
struct FScales {
    float a[32][4];
    float w[2][4];
};
static_assert(2 * sizeof(FScales) <= F_STORE && sizeof(FScales) % 16 == 0, "two of them in a warp's output buffer");

// A warp's piece of the output, 64 bytes (u) of each of its 32 rows, a row per lane: turned
// around in shared memory so that four lanes write a row's 64 bytes (straight from the
// registers a store instruction touches 32 rows: 7000 cycles for a 128 x 256 BF16 tile).
// 16-byte piece c of row r lies at c ^ (r / 2 mod 4): no bank conflicts either way.
// `out` + row * pitch + at: the first row's piece; `rows` of the 32 exist, and columns up to `end`.
__device__ __forceinline__ void store_rows(uint8_t* stg, const uint32_t (&u)[16], int lane, uint8_t* out, long long row0,
                                           int rows, long long pitch, int at, int end) {
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
    __syncwarp();
    const int c = lane & 3;
    if (at + 16 * c >= end) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        if (r < rows)
            *reinterpret_cast<uint4*>(out + (row0 + r) * pitch + at + 16 * c) =
                *reinterpret_cast<const uint4*>(stg + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    }
}

// Rows that the TMA loads of a tile with `rows` rows bring: boxes of 8, 32 or
// 128 rows.  The rows of the slot past them keep what they hold, which reaches only
// output rows that are not stored.
__device__ __forceinline__ int f_box(int rows) { return rows <= 8 ? 8 : rows <= 96 ? 32 : 128; }
__device__ __forceinline__ int f_boxes(int rows) { return (rows + f_box(rows) - 1) / f_box(rows); }

template <int MODE, int NSUB>
__global__ void __launch_bounds__(F_THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                const __grid_constant__ CUtensorMap tmA8, const __grid_constant__ CUtensorMap tmW, const FParams p) {
    using C = FCfg<NSUB>;
    constexpr bool UP = MODE != kGemmPlain;
    constexpr int BN = MODE == kGemmSwiGLU ? 128 : 128 * NSUB;        // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
    uint8_t* store = smem + C::STAGES * C::STAGE_BYTES;              // [F_EPI_WARPS][F_STORE]
    FCtl* ctl = reinterpret_cast<FCtl*>(store + F_EPI_WARPS * F_STORE);
    int* prefix = reinterpret_cast<int*>(ctl + 1);                    // [groups + 1]
    int* start = prefix + p.groups + 1;                               // [groups] first row, [groups] rows
    const uint32_t smem_base = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < C::ACCS; ++a) {
            mbar_init(smem_u32(&ctl->tfull[a]), 1);
            mbar_init(smem_u32(&ctl->tempty[a]), F_EPI_WARPS);
        }
        for (int q = 0; q < 4; ++q) mbar_init(smem_u32(&ctl->xch[q]), 2);
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctl->tmem_base), 512);
        tmem_relinquish();
    }
    __syncthreads();                          // tensor memory is allocated before a dependent kernel may start
    pdl_wait();
    pdl_trigger();
    const int total = f_tile_list<F_THREADS, F_BM>(p, prefix, start, ctl->wtot);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int* abort = &ctl->abort;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");         // 128 x 40 + 256 x 232 = 384 x 168 registers
        if (warp == 0) {
            // ---------------- TMA producer ----------------
            if (lane == 0) {
                int stage = 0;
                uint32_t ph = 0;
                bool ok = true;
                long long armed = 0;
                int group = 0;
                for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
                    const FTile t = f_tile<UP, F_BM>(tile, group, prefix, start, p);
                    const int box = f_box(t.rows), boxes = f_boxes(t.rows);
                    const uint32_t bytes = (uint32_t)(NSUB * F_BOX + boxes * box * 128);
                    const int w0 = t.g * p.parts * p.N + t.nt * BN;
                    const int w1 = MODE == kGemmSwiGLU ? w0 + p.N : w0 + 128;
                    const CUtensorMap* m = box == 128 ? &tmA : box == 32 ? &tmA32 : &tmA8;
                    for (int kb = 0; kb < p.nkb; ++kb) {
                        if (!mbar_wait_bounded(smem_u32(&ctl->empty[stage]), ph ^ 1u, abort)) { ok = false; break; }
                        const uint32_t full = smem_u32(&ctl->full[stage]);
                        const uint32_t sa = smem_base + (uint32_t)(stage * C::STAGE_BYTES);
                        mbar_arrive_expect_tx(full, bytes);
                        tma_load_2d(sa + F_BOX, &tmW, full, kb * 128, w0);
                        if (NSUB == 2) tma_load_2d(sa + 2 * F_BOX, &tmW, full, kb * 128, w1);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_2d(sa + (uint32_t)(i * box * 128), m, full, kb * 128, t.row0 + i * box);
                        ++armed;
                        if (++stage == C::STAGES) { stage = 0; ph ^= 1u; }
                    }
                }
                if (!ok) {
                    if (!wait_armed_stages(smem_u32(&ctl->full[0]), C::STAGES, armed)) settle_delay();
                    raise_status(p.hdr, MOE_ERR_TIMEOUT);
                    p.hdr->timeout_site = kSiteGemmProducer;
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer ----------------
            // The whole warp walks the loop and one elected lane issues: descriptors and
            // barriers stay in uniform registers (in a block of lane 0 alone an instruction
            // took 65 cycles to issue, here about 30).
            constexpr uint32_t idesc = idesc_e4m3_f32(F_BM, C::ACC_COLS);
            const bool leader = elect_one();
            int stage = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (!mbar_wait_warp(smem_u32(&ctl->full[stage]), ph, abort)) { ok = false; break; }
                    if (!mbar_wait_warp(smem_u32(&ctl->tempty[acc]), aph ^ 1u, abort)) { ok = false; break; }
                    tc_fence_after();
                    if (leader) {
                        const uint32_t sa = smem_base + (uint32_t)(stage * C::STAGE_BYTES);
                        const uint64_t ad = sdesc_k_sw128(sa), bd = sdesc_k_sw128(sa + F_BOX);
                        const uint32_t d = tmem + (uint32_t)(acc * C::ACC_COLS);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_e4m3(d, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), idesc, kk > 0 ? 1u : 0u);
                        tc_commit(smem_u32(&ctl->tfull[acc]));
                        tc_commit(smem_u32(&ctl->empty[stage]));
                    }
                    __syncwarp();
                    if (++stage == C::STAGES) { stage = 0; ph ^= 1u; }
                    if (++acc == C::ACCS) { acc = 0; aph ^= 1u; }
                }
            }
            // every MMA issued has completed before TMEM is freed
            if (leader) tc_commit(smem_u32(&ctl->drain));
            __syncwarp();
            volatile int never = 0;
            const bool drained = mbar_wait_warp(smem_u32(&ctl->drain), 0, &never);
            if (lane == 0 && (!ok || !drained)) {
                raise_status(p.hdr, MOE_ERR_TIMEOUT);
                p.hdr->timeout_site = kSiteGemmMma;
                *abort = 1;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        // ---------------- adding up, activation, store (warps 4..11) ----------------
        const int q = warp & 3, hf = (warp - 4) >> 2;
        const int rl = 32 * q + lane;                                 // row of the tile
        uint8_t* stg = store + (size_t)(warp - 4) * F_STORE;
        int acc = 0, parity = 0;
        uint32_t aph = 0;
        bool ok = true;
        // The scales come through the warp's piece of the output buffer, which is idle until
        // the tile ends (a load to a register in the K loop held its warp up by 15 %): four
        // steps by cp.async while the four before are used.  A tile's first four are loaded to
        // registers ahead of the output of the tile before.
        FScales* sc = reinterpret_cast<FScales*>(stg);                // [2]
        const float *as = nullptr, *ws = nullptr;                     // of this row; of lane / 4's block of weight rows
        float a4[4] = {0.f, 0.f, 0.f, 0.f}, w1 = 0.f;
        // The next 32 tiles of this CTA, one a lane (found once in 32 tiles: a search takes
        // 1000 cycles, as much as a step of K).
        FTile mytile = {0, 0, 0, 0}, t = {0, 0, 0, 0};
        int seen = 0;
        auto open_tile = [&](int tile) {
            if ((seen & 31) == 0) {
                int group = 0;
                const long long mine_at = tile + (long long)lane * gridDim.x;
                if (mine_at < total) mytile = f_tile<UP, F_BM>((int)mine_at, group, prefix, start, p);
                __syncwarp();
            }
            t.g = __shfl_sync(0xffffffffu, mytile.g, seen & 31);
            t.nt = __shfl_sync(0xffffffffu, mytile.nt, seen & 31);
            t.row0 = __shfl_sync(0xffffffffu, mytile.row0, seen & 31);
            t.rows = __shfl_sync(0xffffffffu, mytile.rows, seen & 31);
            ++seen;
            as = p.a_scale + (size_t)(t.row0 + (rl < t.rows ? rl : 0)) * p.nkb;
            // block rows of the weights' scales: the first block's, and the second's (SwiGLU: the up rows')
            const int b0 = t.nt * (BN / 128);
            const int second = MODE == kGemmSwiGLU ? p.nnb : b0 + 1 < p.nnb ? 1 : 0;
            ws = p.w_scale + ((size_t)t.g * p.parts * p.nnb + b0 + (lane < 4 ? 0 : second)) * p.nkb;
#pragma unroll
            for (int i = 0; i < 4; ++i) a4[i] = __ldcg(as + min(i, p.nkb - 1));
            if (lane < 4 * NSUB) w1 = __ldg(ws + min(lane & 3, p.nkb - 1));
        };
        auto fetch = [&](int k0) {
            FScales* d = sc + ((k0 >> 2) & 1);
            if (p.nkb % 4 == 0) {                                     // rows of scales are 16-byte aligned
                cp_async16(smem_u32(d->a[lane]), as + k0);
            } else {
                for (int i = 0; i < 4; ++i) cp_async4(smem_u32(&d->a[lane][i]), as + min(k0 + i, p.nkb - 1));
            }
            if (lane < 4 * NSUB) cp_async4(smem_u32(&d->w[lane >> 2][lane & 3]), ws + min(k0 + (lane & 3), p.nkb - 1));
        };
        int tile = blockIdx.x;
        if (tile < total) open_tile(tile);
        while (tile < total && ok) {
            const bool mine = rl < t.rows, any = 32 * q < t.rows;     // this row; a row of the warp
            const int row = t.row0 + (mine ? rl : 0), b0 = t.nt * (BN / 128), col = t.nt * BN + 64 * hf;
            const int row_w = t.row0 + 32 * q, rows_w = t.rows - 32 * q;      // the warp's first row, and how many exist
            __syncwarp();                                             // the tile before has read its output there
            *reinterpret_cast<float4*>(sc->a[lane]) = make_float4(a4[0], a4[1], a4[2], a4[3]);
            if (lane < 4 * NSUB) sc->w[lane >> 2][lane & 3] = w1;
            unsigned long long sum[NSUB][32];
#pragma unroll
            for (int s = 0; s < NSUB; ++s)
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[s][i] = 0ull;
            for (int kb = 0; kb < p.nkb; ++kb) {
                if ((kb & 3) == 0) {
                    cp_async_wait();
                    __syncwarp();
                    if (kb + 4 < p.nkb) fetch(kb + 4);
                }
                const FScales* d = sc + ((kb >> 2) & 1);
                const float sa = d->a[lane][kb & 3];
                const float f[2] = {sa * d->w[0][kb & 3], NSUB == 2 ? sa * d->w[1][kb & 3] : 0.f};
                if (!mbar_wait_warp(smem_u32(&ctl->tfull[acc]), aph, abort)) {
                    if (lane == 0) {
                        raise_status(p.hdr, MOE_ERR_TIMEOUT);
                        p.hdr->timeout_site = kSiteGemmEpilogue;
                    }
                    ok = false;
                    break;
                }
                tc_fence_after();
                // the MMAs get the accumulator back when it is read: for the plain product ahead of the
                // last multiply-adds (2 % less time), for the activations' larger kernels after them
                // (2 % less than ahead)
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[acc]));
                };
                constexpr bool kAhead = MODE == kGemmPlain;
                if (any) {
                    const uint32_t ta = tmem + (uint32_t)(acc * C::ACC_COLS + 64 * hf) + ((uint32_t)(32 * q) << 16);
#pragma unroll
                    for (int s = 0; s < NSUB; ++s) {
                        uint32_t v[64];
                        tmem_ld_cols(ta + (uint32_t)(s * 128), v);
                        tmem_ld_wait();
                        tmem_ld_done(v);
                        if (kAhead && s == NSUB - 1) release();
                        const unsigned long long ff = pack_f32x2(f[s], f[s]);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            sum[s][i] = fma_f32x2(pack_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), ff, sum[s][i]);
                    }
                }
                if (!kAhead || !any) release();
                if (++acc == C::ACCS) { acc = 0; aph ^= 1u; }
            }
            if (!ok) break;
            tile += gridDim.x;
            if (tile < total) open_tile(tile);
            if (!any) continue;                                       // as the other warp of these rows
            if (MODE == kGemmPlain) {
#pragma unroll
                for (int s = 0; s < NSUB; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {                     // 32 columns at a time
                        uint32_t u[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float a, b;
                            unpack_f32x2(sum[s][16 * j + i], a, b);
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
                            u[i] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        store_rows(stg, u, lane, static_cast<uint8_t*>(p.out), row_w, rows_w,
                                   2 * (long long)p.N, 2 * (col + 128 * s + 32 * j), 2 * p.N);
                    }
            } else {
                constexpr int NB = MODE == kGemmSwiGLU ? 1 : NSUB;    // output blocks
                // the activation, in place in the first NB blocks' registers
#pragma unroll
                for (int s = 0; s < NB; ++s) {
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float a, b;
                        unpack_f32x2(sum[s][i], a, b);
                        if (MODE == kGemmSwiGLU) {
                            float ua, ub;
                            unpack_f32x2(sum[NSUB - 1][i], ua, ub);
                            a = a * sigmoid_approx(a) * ua;
                            b = b * sigmoid_approx(b) * ub;
                        } else {
                            a = a > 0.f || a != a ? a * a : 0.f;
                            b = b > 0.f || b != b ? b * b : 0.f;
                        }
                        if (col + 128 * s + 2 * i < p.N) m = amax_nan(amax_nan(m, a), b);
                        sum[s][i] = pack_f32x2(a, b);
                    }
                    ctl->amax[parity][s][hf][rl] = m;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->xch[q]));
                if (!mbar_wait_warp(smem_u32(&ctl->xch[q]), (uint32_t)parity, abort)) {
                    if (lane == 0) {
                        raise_status(p.hdr, MOE_ERR_TIMEOUT);
                        p.hdr->timeout_site = kSiteGemmEpilogue;
                    }
                    ok = false;
                    break;
                }
#pragma unroll
                for (int s = 0; s < NB; ++s) {
                    if (b0 + s >= p.nnb) break;
                    const Fp8Quant qq = fp8_quant(amax_nan(ctl->amax[parity][s][0][rl], ctl->amax[parity][s][1][rl]));
                    if (mine && hf == 0) p.out_scale[(size_t)row * p.nnb + b0 + s] = qq.scale;
                    uint32_t u[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x[4];
                        unpack_f32x2(sum[s][2 * i], x[0], x[1]);
                        unpack_f32x2(sum[s][2 * i + 1], x[2], x[3]);
                        u[i] = fp8_quant4(qq, x[0], x[1], x[2], x[3]);
                    }
                    store_rows(stg, u, lane, static_cast<uint8_t*>(p.out), row_w, rows_w,
                               p.N, col + 128 * s, p.N);
                }
                parity ^= 1;
            }
        }
        cp_async_wait();                      // of a tile that was given up
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int MODE, int NSUB>
moe_status launch_f(const Fp8Problem& g, FParams p, const CUtensorMap& mw, const CUtensorMap (&ma)[3], cudaStream_t st) {
    using C = FCfg<NSUB>;
    constexpr int BN = MODE == kGemmSwiGLU ? 128 : 128 * NSUB;
    p.ntn = (g.N + BN - 1) / BN;
    const size_t smem = 1024 + (size_t)C::STAGES * C::STAGE_BYTES + F_EPI_WARPS * F_STORE +
                        sizeof(FCtl) + (size_t)(3 * g.groups + 1) * sizeof(int);
    cudaError_t e = allow_smem(fp8_gemm_kernel<MODE, NSUB>);
    if (e == cudaSuccess) {
        const long long used = g.rows < g.groups ? g.rows : g.groups;
        const long long tiles = (g.rows / F_BM + used) * p.ntn;     // at most
        const int sms = device_sm_count();
        e = launch_kernel(fp8_gemm_kernel<MODE, NSUB>, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(F_THREADS), smem,
                          st, 1, kUsePdl, ma[0], ma[1], ma[2], mw, p);
    }
    if (e == cudaSuccess) return MOE_OK;
    set_error("FP8 GEMM launch (smem %zu): %s", smem, cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}

}  // namespace

moe_status launch_fp8_gemm(const Fp8Problem& g, WsHeader* hdr, cudaStream_t st) {
    FParams p{};
    p.offsets = g.offsets;
    p.groups = g.groups;
    p.rows = (int)g.rows;
    p.K = g.K;
    p.N = g.N;
    p.nkb = fp8_blocks(g.K);
    p.nnb = fp8_blocks(g.N);
    p.parts = g.mode == kGemmSwiGLU ? 2 : 1;
    p.a_scale = g.a_scale;
    p.w_scale = g.w_scale;
    p.out = g.out;
    p.out_scale = g.out_scale;
    p.hdr = hdr;
    p.gated = g.gated;
    CUtensorMap ma[3], mw;
    if (!make_tensor_map_u8_rows(&mw, g.w, (long long)g.groups * p.parts * g.N, g.K, g.K, 128u, 128u)) return MOE_ERR_CUDA;
    if (g.max_group_rows <= 64)
        return launch_fp8_rows(g, p, mw, g.max_group_rows <= 16 ? 16 : g.max_group_rows <= 32 ? 32 : 64, st);
    const unsigned box[3] = {128u, 32u, 8u};
    for (int i = 0; i < 3; ++i)
        if (!make_tensor_map_u8_rows(&ma[i], g.a, g.rows, g.K, g.K, 128u, box[i])) return MOE_ERR_CUDA;
    if (g.mode == kGemmSwiGLU) return launch_f<kGemmSwiGLU, 2>(g, p, mw, ma, st);
    // Two blocks of weight rows a tile halve the activation traffic; with fewer such tiles
    // than SMs, one block a tile spreads a weight stream over twice as many.
    const long long used = g.rows < g.groups ? g.rows : g.groups;
    const bool wide = (g.rows / F_BM + used) * ((g.N + 255) / 256) > device_sm_count();
    if (g.mode == kGemmReLU2)
        return wide ? launch_f<kGemmReLU2, 2>(g, p, mw, ma, st) : launch_f<kGemmReLU2, 1>(g, p, mw, ma, st);
    return wide ? launch_f<kGemmPlain, 2>(g, p, mw, ma, st) : launch_f<kGemmPlain, 1>(g, p, mw, ma, st);
}

}  // namespace moe
