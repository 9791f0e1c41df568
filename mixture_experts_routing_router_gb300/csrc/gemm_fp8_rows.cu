// gemm_fp8_rows.cu -- the block-scaled FP8 expert GEMM for groups of few rows (decode).
//
// With a handful of rows an expert the GEMM streams weights, and the row kernel of
// gemm_fp8.cu spends a 128-row MMA and its long accumulator round trip on them.  Here the
// operands swap: D^T = W X^T, a block of 128 weight rows on the MMA's M side and NB rows of
// the group (16, 32 or 64) on its N side.  A step of K then fills NSUB NB columns of tensor
// memory, up to eight accumulators are in flight, and adding one up is one short read.
// A thread has one weight row (output column) and NB / 2 of the rows; the rows' scales are
// read from shared memory, the block's weight scale is the same for all.  The sums run in
// the order of gemm_fp8.cu, and give its bits.
//
// Bound by HBM: 8 tokens, 64 experts, 7168 x 2048: up 179 us (6.7 TB/s), down 92 (6.6); 16
// tokens with 240 experts, 1024 x 1536: 5.4 to 5.7 TB/s, what is left being the first loads
// and the last tile's epilogue.  The row kernel takes 49 us where these two take 41.  Taken
// up to 64 tokens, the host's bound on a group's rows.  More tokens over many experts can
// have as few rows a group; the one such point that was compared (200 tokens: up 66 us with
// the row kernel, 75 with this one) went to the row kernel, others are not measured.
//
// Roles: warp 0 TMA, warp 1 MMA, warps 2..9 add up and store: warp w owns TMEM lanes
// 32 (w % 4) .. +31 and rows h NB / 2 .. of the tile (h = (w - 2) / 4).  For SwiGLU the two
// blocks are gate and up rows of the same 128 output columns.  The largest magnitude of an
// output block is a warp-wide maximum of its bits, then one over the four warps of the same
// rows through shared memory and an mbarrier.  Every wait is bounded.
//
// `early` (inside moe_layer_fp8_block): what the tile list is built from was final before the
// kernel in front of this one could start, so the list is built and the first stages' weights
// are sent for before the programmatic wait.  For the down projection that is the bucket
// bounds; for the up projection of at most R_THREADS pairs the tokens' experts, from which
// every block counts the bounds itself, while the dispatch runs.
#include "gemm_fp8.cuh"

namespace moe {
namespace {

constexpr int R_THREADS = 320;
constexpr int R_EPI_WARPS = 8;
constexpr int R_MAX_STAGES = 10;
constexpr int R_MAX_ACCS = 8;
constexpr size_t R_HALF_SMEM = 112 * 1024;      // two blocks an SM

template <int NSUB, int NB>
struct RCfg {
    static constexpr int STAGE_BYTES = NSUB * F_BOX + NB * 128;
    static constexpr int STAGES = 192 * 1024 / STAGE_BYTES < R_MAX_STAGES ? 192 * 1024 / STAGE_BYTES : R_MAX_STAGES;
    // two blocks an SM: short stages, and at most 96 registers (a warp's come in eights a
    // thread: 20 warps at 104 would take 66560), which the launch bounds hold
    static constexpr bool PAIR = NSUB == 1 && NB == 16;
    static constexpr int ACC_COLS = NSUB * NB;
    static constexpr int ACCS = 512 / ACC_COLS < R_MAX_ACCS ? 512 / ACC_COLS : R_MAX_ACCS;
    static constexpr uint32_t TMEM_COLS = ACCS * ACC_COLS;            // a power of two
};

// Four steps' scales for an adding warp: of its rows, and of the weight blocks.
struct alignas(16) RScales {
    float a[4][32];
    float w[2][4];
};

struct RCtl {
    unsigned long long full[R_MAX_STAGES], empty[R_MAX_STAGES];
    unsigned long long tfull[R_MAX_ACCS], tempty[R_MAX_ACCS];
    unsigned long long xch[2];                  // the four warps of a row half
    unsigned long long drain;
    uint32_t tmem_base;
    int abort;
    int wtot[R_THREADS / 32];
    int ids[R_THREADS];
    RScales scales[R_EPI_WARPS][2];
    alignas(16) uint32_t amax[2][2][64][4];     // [exchange parity][block][row][lane quarter] bits
};

// f_tile_list with the bounds counted from p.ids, a pair a thread: as the dispatch has them
// (ids out of range, and those repeated in a token, are in no bucket).  Over capacity, where
// the dispatch moves nothing, the rows are what the workspace holds, and no later kernel of
// the call reads the results.
template <int BM>
__device__ __forceinline__ int r_tile_list(const FParams& p, int* prefix, int* start, int* ids, int* wtot) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* count = start + p.groups;
    for (int g = tid; g < p.groups; g += R_THREADS) count[g] = 0;
    const int id = tid < p.rows ? __ldcg(p.ids + tid) : -1;
    ids[tid] = id;
    __syncthreads();
    bool ok = id >= 0 && id < p.groups;
    for (int j = tid - tid % p.top_k; ok && j < tid; ++j) ok = ids[j] != id;
    if (ok) atomicAdd(&count[id], 1);
    __syncthreads();
    const int per = (p.groups + R_THREADS - 1) / R_THREADS, g0 = tid * per;
    unsigned sum = 0;                            // rows, and tiles of 2^16 on
    auto both = [&](int n) { return (unsigned)n | (unsigned)((n + BM - 1) / BM) << 16; };
    for (int g = g0; g < min(g0 + per, p.groups); ++g) sum += both(count[g]);
    unsigned inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += v;
    }
    if (lane == 31) wtot[warp] = (int)inc;
    __syncthreads();
    unsigned run = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? (unsigned)wtot[lane] : 0u);
    for (int g = g0; g < min(g0 + per, p.groups); ++g) {
        start[g] = (int)(run & 0xffffu);
        prefix[g] = (int)(run >> 16) * p.ntn;
        run += both(count[g]);
    }
    if (tid == R_THREADS - 1) prefix[p.groups] = (int)(run >> 16) * p.ntn;
    __syncthreads();
    return prefix[p.groups];
}

template <int MODE, int NSUB, int NB>
__global__ void __launch_bounds__(R_THREADS, RCfg<NSUB, NB>::PAIR ? 2 : 1)
fp8_rows_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, const FParams p,
                const int early) {
    using C = RCfg<NSUB, NB>;
    constexpr bool UP = MODE != kGemmPlain;
    constexpr int BN = MODE == kGemmSwiGLU ? 128 : 128 * NSUB;        // output columns of a tile
    constexpr int HB = NB / 2;                                        // rows of a thread
    const int stages = p.stages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
    RCtl* ctl = reinterpret_cast<RCtl*>(smem + stages * C::STAGE_BYTES);
    int* prefix = reinterpret_cast<int*>(ctl + 1);                    // [groups + 1]
    int* start = prefix + p.groups + 1;                               // [groups] first row, [groups] rows
    const uint32_t smem_base = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < C::ACCS; ++a) {
            mbar_init(smem_u32(&ctl->tfull[a]), 1);
            mbar_init(smem_u32(&ctl->tempty[a]), R_EPI_WARPS);
        }
        mbar_init(smem_u32(&ctl->xch[0]), 4);
        mbar_init(smem_u32(&ctl->xch[1]), 4);
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctl->tmem_base), C::TMEM_COLS);
        tmem_relinquish();
    }
    __syncthreads();                          // tensor memory is allocated before a dependent kernel may start
    if (!early) {
        pdl_wait();
        pdl_trigger();
    }
    const int total = p.ids ? r_tile_list<NB>(p, prefix, start, ctl->ids, ctl->wtot)
                            : f_tile_list<R_THREADS, NB>(p, prefix, start, ctl->wtot);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int* abort = &ctl->abort;

    auto load_weights = [&](const FTile& t, int stage, int kb) {
        const uint32_t full = smem_u32(&ctl->full[stage]), sw = smem_base + (uint32_t)(stage * C::STAGE_BYTES);
        const int w0 = t.g * p.parts * p.N + t.nt * BN;
        mbar_arrive_expect_tx(full, (uint32_t)C::STAGE_BYTES);
        tma_load_2d(sw, &tmW, full, kb * 128, w0);
        if (NSUB == 2) tma_load_2d(sw + F_BOX, &tmW, full, kb * 128, MODE == kGemmSwiGLU ? w0 + p.N : w0 + 128);
    };
    // Sent before the wait: the first stages' weights (no kernel writes those); their rows
    // follow in the loop.
    int ahead = 0;
    if (early) {
        if (tid == 0 && (int)blockIdx.x < total) {
            int group = 0;
            const FTile t = f_tile<UP, NB>(blockIdx.x, group, prefix, start, p);
            for (; ahead < min(stages, p.nkb); ++ahead) load_weights(t, ahead, ahead);
        }
        pdl_wait();
        pdl_trigger();
    }

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            int stage = 0, group = 0;
            uint32_t ph = 0;
            bool ok = true;
            long long armed = 0;
            for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
                const FTile t = f_tile<UP, NB>(tile, group, prefix, start, p);
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (armed >= ahead) {
                        if (!mbar_wait_bounded(smem_u32(&ctl->empty[stage]), ph ^ 1u, abort)) { ok = false; break; }
                        load_weights(t, stage, kb);
                    }
                    tma_load_2d(smem_base + (uint32_t)(stage * C::STAGE_BYTES + NSUB * F_BOX), &tmA,
                                smem_u32(&ctl->full[stage]), kb * 128, t.row0);
                    ++armed;
                    if (++stage == stages) { stage = 0; ph ^= 1u; }
                }
            }
            if (!ok) {
                // (stages armed before the wait whose rows never went out cannot complete: their
                // wait runs out and the fixed delay follows)
                if (!wait_armed_stages(smem_u32(&ctl->full[0]), stages, max(armed, (long long)ahead))) settle_delay();
                raise_status(p.hdr, MOE_ERR_TIMEOUT);
                p.hdr->timeout_site = kSiteGemmProducer;
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (one elected lane, as in gemm_fp8.cu) ----------------
        constexpr uint32_t idesc = idesc_e4m3_f32(128, NB);
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
                    const uint32_t sw = smem_base + (uint32_t)(stage * C::STAGE_BYTES);
                    const uint64_t xd = sdesc_k_sw128(sw + NSUB * F_BOX);
                    const uint32_t d = tmem + (uint32_t)(acc * C::ACC_COLS);
#pragma unroll
                    for (int s = 0; s < NSUB; ++s) {
                        const uint64_t wd = sdesc_k_sw128(sw + (uint32_t)(s * F_BOX));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_e4m3(d + (uint32_t)(s * NB), wd + (uint64_t)(kk * 2), xd + (uint64_t)(kk * 2), idesc,
                                        kk > 0 ? 1u : 0u);
                    }
                    tc_commit(smem_u32(&ctl->tfull[acc]));
                    tc_commit(smem_u32(&ctl->empty[stage]));
                }
                __syncwarp();
                if (++stage == stages) { stage = 0; ph ^= 1u; }
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
    } else {
        // ---------------- adding up, activation, store (warps 2..9) ----------------
        const int q = warp & 3, hf = (warp - 2) >> 2;
        RScales* sc = ctl->scales[warp - 2];
        int acc = 0, parity = 0, seen = 0;
        uint32_t aph = 0;
        bool ok = true;
        // as in gemm_fp8.cu: 32 tiles are found at once, one a lane, and a tile's first scales
        // are on their way to registers before the output of the tile in front of it
        FTile mytile = {0, 0, 0, 0}, t = {0, 0, 0, 0};
        const float *as = nullptr, *ws = nullptr;                     // of row `lane` of the half; of lane / 4's weight block
        float a4[4] = {0.f, 0.f, 0.f, 0.f}, w1 = 0.f;
        auto open_tile = [&](int tile) {
            if ((seen & 31) == 0) {
                int group = 0;
                const long long mine_at = tile + (long long)lane * gridDim.x;
                if (mine_at < total) mytile = f_tile<UP, NB>((int)mine_at, group, prefix, start, p);
                __syncwarp();
            }
            t.g = __shfl_sync(0xffffffffu, mytile.g, seen & 31);
            t.nt = __shfl_sync(0xffffffffu, mytile.nt, seen & 31);
            t.row0 = __shfl_sync(0xffffffffu, mytile.row0, seen & 31);
            t.rows = __shfl_sync(0xffffffffu, mytile.rows, seen & 31);
            ++seen;
            const int b0 = t.nt * (BN / 128), second = MODE == kGemmSwiGLU ? p.nnb : b0 + 1 < p.nnb ? 1 : 0;
            as = p.a_scale + (size_t)(t.row0 + min(hf * HB + min(lane, HB - 1), t.rows - 1)) * p.nkb;
            ws = p.w_scale + ((size_t)t.g * p.parts * p.nnb + b0 + (lane < 4 ? 0 : second)) * p.nkb;
#pragma unroll
            for (int i = 0; i < 4; ++i) a4[i] = __ldcg(as + min(i, p.nkb - 1));
            if (lane < 4 * NSUB) w1 = __ldg(ws + min(lane & 3, p.nkb - 1));
        };
        auto fetch = [&](int k0) {
            RScales* d = sc + ((k0 >> 2) & 1);
            if (lane < HB)
                for (int i = 0; i < 4; ++i) cp_async4(smem_u32(&d->a[i][lane]), as + min(k0 + i, p.nkb - 1));
            if (lane < 4 * NSUB) cp_async4(smem_u32(&d->w[lane >> 2][lane & 3]), ws + min(k0 + (lane & 3), p.nkb - 1));
        };
        int tile = blockIdx.x;
        if (tile < total) open_tile(tile);
        while (tile < total && ok) {
            const int rows = t.rows - hf * HB;                        // of this warp's half of the tile
            const bool any = rows > 0;
            const int b0 = t.nt * (BN / 128), n0 = t.nt * BN + 32 * q + lane;     // its first block; this thread's column there
            const size_t row0 = (size_t)t.row0 + hf * HB;
            __syncwarp();
            if (lane < HB) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sc->a[i][lane] = a4[i];
            }
            if (lane < 4 * NSUB) sc->w[lane >> 2][lane & 3] = w1;
            unsigned long long sum[NSUB][HB / 2];
#pragma unroll
            for (int s = 0; s < NSUB; ++s)
#pragma unroll
                for (int i = 0; i < HB / 2; ++i) sum[s][i] = 0ull;
            for (int kb = 0; kb < p.nkb; ++kb) {
                if ((kb & 3) == 0) {
                    cp_async_wait();
                    __syncwarp();
                    if (kb + 4 < p.nkb) fetch(kb + 4);
                }
                if (!mbar_wait_warp(smem_u32(&ctl->tfull[acc]), aph, abort)) {
                    if (lane == 0) {
                        raise_status(p.hdr, MOE_ERR_TIMEOUT);
                        p.hdr->timeout_site = kSiteGemmEpilogue;
                    }
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (any) {
                    const uint32_t ta = tmem + (uint32_t)(acc * C::ACC_COLS + hf * HB) + ((uint32_t)(32 * q) << 16);
                    uint32_t v[NSUB][HB];
#pragma unroll
                    for (int s = 0; s < NSUB; ++s) tmem_ld_cols(ta + (uint32_t)(s * NB), v[s]);
                    const RScales* d = sc + ((kb >> 2) & 1);
                    const ulonglong2* ar = reinterpret_cast<const ulonglong2*>(d->a[kb & 3]);
                    const float w0 = d->w[0][kb & 3], w1 = NSUB == 2 ? d->w[1][kb & 3] : 0.f;
                    tmem_ld_wait();
#pragma unroll
                    for (int s = 0; s < NSUB; ++s) tmem_ld_done(v[s]);
#pragma unroll
                    for (int i = 0; i < HB / 4; ++i) {                // four rows at a time
                        const ulonglong2 a = ar[i];
#pragma unroll
                        for (int s = 0; s < NSUB; ++s) {
                            const unsigned long long w2 = s == 0 ? pack_f32x2(w0, w0) : pack_f32x2(w1, w1);
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                sum[s][2 * i + h] =
                                    fma_f32x2(pack_f32x2(__uint_as_float(v[s][4 * i + 2 * h]), __uint_as_float(v[s][4 * i + 2 * h + 1])),
                                              mul_f32x2(h == 0 ? a.x : a.y, w2), sum[s][2 * i + h]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[acc]));
                if (++acc == C::ACCS) { acc = 0; aph ^= 1u; }
            }
            if (!ok) break;
            tile += gridDim.x;
            if (tile < total) open_tile(tile);
            if (!any) continue;                                       // as the other warps of these rows
            if (MODE == kGemmPlain) {
#pragma unroll
                for (int s = 0; s < NSUB; ++s) {
                    const int n = n0 + 128 * s;
                    if (n >= p.N) break;
                    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + row0 * p.N + n;
#pragma unroll
                    for (int i = 0; i < HB / 2; ++i) {
                        float a, b;
                        unpack_f32x2(sum[s][i], a, b);
                        if (2 * i < rows) o[(size_t)(2 * i) * p.N] = __float2bfloat16_rn(a);
                        if (2 * i + 1 < rows) o[(size_t)(2 * i + 1) * p.N] = __float2bfloat16_rn(b);
                    }
                }
            } else {
                constexpr int OB = MODE == kGemmSwiGLU ? 1 : NSUB;    // output blocks
                // the activation, in place in the first OB blocks' registers, and its largest magnitude
#pragma unroll
                for (int s = 0; s < OB; ++s)
#pragma unroll
                    for (int i = 0; i < HB / 2; ++i) {
                        if (2 * i >= rows) break;
                        float x[2];
                        unpack_f32x2(sum[s][i], x[0], x[1]);
                        if (MODE == kGemmSwiGLU) {
                            float u[2];
                            unpack_f32x2(sum[NSUB - 1][i], u[0], u[1]);
                            x[0] = x[0] * sigmoid_approx(x[0]) * u[0];
                            x[1] = x[1] * sigmoid_approx(x[1]) * u[1];
                        } else {
                            x[0] = x[0] > 0.f || x[0] != x[0] ? x[0] * x[0] : 0.f;
                            x[1] = x[1] > 0.f || x[1] != x[1] ? x[1] * x[1] : 0.f;
                        }
                        sum[s][i] = pack_f32x2(x[0], x[1]);
                        // magnitudes order as their bits do, a NaN's last
                        const bool in = n0 + 128 * s < p.N;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t m = __reduce_max_sync(0xffffffffu, in ? __float_as_uint(x[h]) & 0x7fffffffu : 0u);
                            if (lane == 0) ctl->amax[parity][s][hf * HB + 2 * i + h][q] = m;
                        }
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->xch[hf]));
                if (!mbar_wait_warp(smem_u32(&ctl->xch[hf]), (uint32_t)parity, abort)) {
                    if (lane == 0) {
                        raise_status(p.hdr, MOE_ERR_TIMEOUT);
                        p.hdr->timeout_site = kSiteGemmEpilogue;
                    }
                    ok = false;
                    break;
                }
#pragma unroll
                for (int s = 0; s < OB; ++s) {
                    if (b0 + s >= p.nnb) break;
                    const int n = n0 + 128 * s;
                    uint8_t* o = static_cast<uint8_t*>(p.out) + row0 * p.N + n;
#pragma unroll
                    for (int i = 0; i < HB / 2; ++i) {
                        float x[2];
                        unpack_f32x2(sum[s][i], x[0], x[1]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = 2 * i + h;
                            if (r >= rows) break;
                            const uint4 m = *reinterpret_cast<const uint4*>(ctl->amax[parity][s][hf * HB + r]);
                            const Fp8Quant qq = fp8_quant(__uint_as_float(max(max(m.x, m.y), max(m.z, m.w))));
                            if (n < p.N) o[(size_t)r * p.N] = (uint8_t)e4m3x2(fp8_scaled(qq, x[h]), 0.f);
                            if (q == 0 && lane == 0) p.out_scale[(row0 + r) * p.nnb + b0 + s] = qq.scale;
                        }
                    }
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
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int MODE, int NSUB, int NB>
moe_status launch_r(const Fp8Problem& g, FParams p, const CUtensorMap& mw, cudaStream_t st) {
    using C = RCfg<NSUB, NB>;
    constexpr int BN = MODE == kGemmSwiGLU ? 128 : 128 * NSUB;
    p.ntn = (g.N + BN - 1) / BN;
    const bool counts = g.early && g.ids && g.rows <= R_THREADS;
    p.ids = counts ? g.ids : nullptr;
    p.top_k = g.top_k;
    CUtensorMap ma;
    if (!make_tensor_map_u8_rows(&ma, g.a, g.rows, g.K, g.K, 128u, (unsigned)NB)) return MOE_ERR_CUDA;
    const size_t rest = 1024 + sizeof(RCtl) + (size_t)(3 * g.groups + 1) * sizeof(int);
    const long long used = g.rows < g.groups ? g.rows : g.groups;
    const long long tiles = (g.rows / NB + used) * p.ntn;             // at most
    const int sms = device_sm_count();
    // With a tile an SM at most, a ring that leaves room for a block of the next kernel of the
    // layer, which then starts its weights in time (1 token, 9 experts: a layer 24.3 -> 23.1 us).
    p.stages = C::STAGES;
    if (C::PAIR && tiles <= sms) p.stages = (int)((R_HALF_SMEM - rest) / C::STAGE_BYTES);
    const size_t smem = rest + (size_t)p.stages * C::STAGE_BYTES;
    cudaError_t e = allow_smem(fp8_rows_kernel<MODE, NSUB, NB>);
    if (e == cudaSuccess)
        e = launch_kernel(fp8_rows_kernel<MODE, NSUB, NB>, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(R_THREADS), smem,
                          st, 1, kUsePdl, ma, mw, p, (int)(g.early && (counts || !g.ids)));
    if (e == cudaSuccess) return MOE_OK;
    set_error("FP8 small-row GEMM launch (smem %zu): %s", smem, cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}

template <int MODE, int NSUB>
moe_status launch_nb(const Fp8Problem& g, const FParams& p, const CUtensorMap& mw, int nb, cudaStream_t st) {
    if (nb == 16) return launch_r<MODE, NSUB, 16>(g, p, mw, st);
    if (nb == 32) return launch_r<MODE, NSUB, 32>(g, p, mw, st);
    return launch_r<MODE, MODE == kGemmSwiGLU ? 2 : 1, 64>(g, p, mw, st);
}

}  // namespace

moe_status launch_fp8_rows(const Fp8Problem& g, const FParams& p, const CUtensorMap& mw, int nb, cudaStream_t st) {
    if (g.mode == kGemmSwiGLU) return launch_nb<kGemmSwiGLU, 2>(g, p, mw, nb, st);
    // two blocks of weight rows a tile, unless half the SMs would have none (or the sums of 64
    // rows no registers)
    const long long used = g.rows < g.groups ? g.rows : g.groups;
    const bool wide = nb < 64 && (g.rows / nb + used) * ((g.N + 255) / 256) > device_sm_count();
    if (g.mode == kGemmReLU2)
        return wide ? launch_nb<kGemmReLU2, 2>(g, p, mw, nb, st) : launch_nb<kGemmReLU2, 1>(g, p, mw, nb, st);
    return wide ? launch_nb<kGemmPlain, 2>(g, p, mw, nb, st) : launch_nb<kGemmPlain, 1>(g, p, mw, nb, st);
}

}  // namespace moe
