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
// Roles: warp 0 loads by TMA, warp 1 issues the MMAs, warps 2..9 add up and store:
// warp w owns TMEM lanes 32 (w % 4) .. +31 and columns 64 h .. 64 h + 63 (h = (w - 2) / 4)
// of every block.  For SwiGLU the two blocks are the gate and up rows of the same 128
// output columns, so a thread holds both factors of its 64 outputs; the activation is
// quantized again as it is stored, and the two warps that share a row block exchange
// their largest magnitude through shared memory.
//
// Persistent CTAs walk a tile list built from the bucket bounds, as in gemm.cu.  Every
// wait is bounded (MOE_ERR_TIMEOUT); the exchange goes through an mbarrier so that it is,
// too.
#include "fp8.cuh"

namespace moe {
namespace {

constexpr int F_BM = 128;                       // activation rows per tile
constexpr int F_BOX = 128 * 128;                // 128 rows of 128 codes
constexpr int F_THREADS = 320;
constexpr int F_EPI_WARPS = 8;
constexpr int F_MAX_SMEM = 216 * 1024;
constexpr int F_RASTER = 8;                     // column tiles of a band (tile order)

template <int NSUB>
struct FCfg {
    static constexpr int STAGE_BYTES = (1 + NSUB) * F_BOX;
    static constexpr int STAGES = NSUB == 2 ? 4 : 6;
    static constexpr int ACC_COLS = 128 * NSUB;
    static constexpr int ACCS = 512 / ACC_COLS;
};

struct FParams {
    const int32_t* offsets;
    int groups, rows;
    int K, N, nkb, nnb;                         // nkb, nnb: 128-blocks of K and of N
    int parts;                                  // weight matrices per group (SwiGLU: gate and up)
    int ntn;                                    // column tiles
    const float* a_scale;
    const float* w_scale;
    void* out;
    float* out_scale;
    WsHeader* hdr;
    int gated;
};

struct FCtl {
    unsigned long long full[6], empty[6];
    unsigned long long tfull[4], tempty[4];
    unsigned long long xch[4];                  // the two warps of a lane quarter
    unsigned long long drain;
    uint32_t tmem_base;
    int abort;
    int total;
    int wtot[F_THREADS / 32];
    float amax[2][2][2][F_BM];                  // [tile parity][block][column half][row]
};

__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}
// kind::f8f6f4: E4M3 A and B (both K-major), FP32 D, M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ unsigned long long pack_f32x2(float lo, float hi) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack_f32x2(unsigned long long v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma_f32x2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// tcgen05.wait::ld that the registers loaded before it pass through, so that no use of
// them can be moved ahead of it.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
}

struct FTile { int g, nt, row0, rows; };        // first row of the tile and how many it holds

// The tile list: group g's row tiles times column tiles, in bands of F_RASTER column
// tiles.  The up projection (long rows) walks a band's column tiles first, the down
// projection its row tiles (as gemm.cu, for the same reuse in L2).
template <bool COLS_FIRST>
__device__ __forceinline__ FTile f_tile(int tile, const int* prefix, const int* start, const FParams& p) {
    int lo = 0, hi = p.groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= tile) lo = mid; else hi = mid;
    }
    const int cnt = start[p.groups + lo], local = tile - prefix[lo];
    const int mtiles = (cnt + F_BM - 1) / F_BM;
    const int band = local / (mtiles * F_RASTER), idx = local - band * mtiles * F_RASTER;
    FTile t;
    int mt;
    if (COLS_FIRST) {
        const int w = min(F_RASTER, p.ntn - band * F_RASTER);
        mt = idx / w;
        t.nt = band * F_RASTER + idx % w;
    } else {
        mt = idx % mtiles;
        t.nt = band * F_RASTER + idx / mtiles;
    }
    t.g = lo;
    t.row0 = start[lo] + mt * F_BM;
    t.rows = min(F_BM, cnt - mt * F_BM);
    return t;
}

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
    FCtl* ctl = reinterpret_cast<FCtl*>(smem + C::STAGES * C::STAGE_BYTES);
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
    pdl_wait();
    pdl_trigger();
    // ---- tile list: bounds clamped to the rows there are
    const bool skip = p.gated && p.hdr->cap_exceeded;
    const int per = (p.groups + F_THREADS - 1) / F_THREADS, g0 = tid * per;
    int sum = 0;
    for (int g = g0; g < min(g0 + per, p.groups); ++g) {
        int lo = p.offsets[g], hi = p.offsets[g + 1];
        lo = lo < 0 ? 0 : min(lo, p.rows);
        hi = hi < lo || skip ? lo : min(hi, p.rows);
        start[g] = lo;
        start[p.groups + g] = hi - lo;
        sum += ((hi - lo + F_BM - 1) / F_BM) * p.ntn;
    }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += v;
    }
    if (lane == 31) ctl->wtot[warp] = inc;
    __syncthreads();
    int run = inc - sum;
    for (int w = 0; w < warp; ++w) run += ctl->wtot[w];
    for (int g = g0; g < min(g0 + per, p.groups); ++g) {
        prefix[g] = run;
        run += ((start[p.groups + g] + F_BM - 1) / F_BM) * p.ntn;
    }
    if (tid == F_THREADS - 1) ctl->total = prefix[p.groups] = run;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const int total = ctl->total;
    volatile int* abort = &ctl->abort;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            int stage = 0;
            uint32_t ph = 0;
            bool ok = true;
            long long armed = 0;
            for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
                const FTile t = f_tile<UP>(tile, prefix, start, p);
                // rows the tile does not have are not loaded: whatever the slot holds there
                // reaches only output rows that are not stored
                const int box = t.rows <= 8 ? 8 : t.rows <= 96 ? 32 : 128;
                const int boxes = (t.rows + box - 1) / box;
                const int w0 = t.g * p.parts * p.N + t.nt * BN;
                const int w1 = MODE == kGemmSwiGLU ? w0 + p.N : w0 + 128;
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&ctl->empty[stage]), ph ^ 1u, abort)) { ok = false; break; }
                    const uint32_t full = smem_u32(&ctl->full[stage]);
                    const uint32_t sa = smem_base + (uint32_t)(stage * C::STAGE_BYTES);
                    mbar_arrive_expect_tx(full, (uint32_t)(NSUB * F_BOX + boxes * box * 128));
                    tma_load_2d(sa + F_BOX, &tmW, full, kb * 128, w0);
                    if (NSUB == 2) tma_load_2d(sa + 2 * F_BOX, &tmW, full, kb * 128, w1);
                    const CUtensorMap* m = box == 128 ? &tmA : box == 32 ? &tmA32 : &tmA8;
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
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3_f32(F_BM, C::ACC_COLS);
            int stage = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&ctl->full[stage]), ph, abort) ||
                        !mbar_wait_bounded(smem_u32(&ctl->tempty[acc]), aph ^ 1u, abort)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sa = smem_base + (uint32_t)(stage * C::STAGE_BYTES);
                    const uint64_t ad = sdesc_k_sw128(sa), bd = sdesc_k_sw128(sa + F_BOX);
                    const uint32_t d = tmem + (uint32_t)(acc * C::ACC_COLS);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_e4m3(d, ad + (uint64_t)(kk * 2), bd + (uint64_t)(kk * 2), idesc, kk > 0 ? 1u : 0u);
                    tc_commit(smem_u32(&ctl->empty[stage]));
                    tc_commit(smem_u32(&ctl->tfull[acc]));
                    if (++stage == C::STAGES) { stage = 0; ph ^= 1u; }
                    if (++acc == C::ACCS) { acc = 0; aph ^= 1u; }
                }
            }
            // every MMA this thread issued has completed before TMEM is freed
            tc_commit(smem_u32(&ctl->drain));
            volatile int never = 0;
            const bool drained = mbar_wait_bounded(smem_u32(&ctl->drain), 0, &never);
            if (!ok || !drained) {
                raise_status(p.hdr, MOE_ERR_TIMEOUT);
                p.hdr->timeout_site = kSiteGemmMma;
                *abort = 1;
            }
        }
    } else {
        // ---------------- adding up, activation, store (warps 2..9) ----------------
        const int q = warp & 3, hf = (warp - 2) >> 2;
        const int rl = 32 * q + lane;                                 // row of the tile
        int acc = 0, parity = 0;
        uint32_t aph = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x, parity ^= 1) {
            const FTile t = f_tile<UP>(tile, prefix, start, p);
            const bool mine = rl < t.rows, any = 32 * q < t.rows;     // this row; a row of the warp
            const int row = t.row0 + (mine ? rl : 0);
            const float* as = p.a_scale + (size_t)row * p.nkb;
            const int b0 = t.nt * (BN / 128);
            // the tile's weight scales: block rows b0 of the first block, and of the second
            const size_t wrow = (size_t)t.g * p.parts * p.nnb + b0;
            const float* ws0 = p.w_scale + wrow * p.nkb;
            const float* ws1 = MODE == kGemmSwiGLU ? p.w_scale + (wrow + p.nnb) * p.nkb
                                                   : ws0 + (b0 + 1 < p.nnb ? p.nkb : 0);
            unsigned long long sum[NSUB][32];
#pragma unroll
            for (int s = 0; s < NSUB; ++s)
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[s][i] = 0ull;
            float sa = __ldg(as), s0 = __ldg(ws0), s1 = NSUB == 2 ? __ldg(ws1) : 0.f;
            for (int kb = 0; kb < p.nkb; ++kb) {
                float f[2] = {sa * s0, sa * s1};
                const int nx = kb + 1 < p.nkb ? kb + 1 : kb;          // the next step's scales
                sa = __ldg(as + nx);
                s0 = __ldg(ws0 + nx);
                if (NSUB == 2) s1 = __ldg(ws1 + nx);
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
                    const uint32_t ta = tmem + (uint32_t)(acc * C::ACC_COLS + 64 * hf) + ((uint32_t)(32 * q) << 16);
                    uint32_t v[2][16];
                    tmem_ld_16cols(ta, v[0]);
#pragma unroll
                    for (int c = 0; c < 4 * NSUB; ++c) {              // 16-column pieces
                        tmem_ld_wait16(v[c & 1]);
                        if (c + 1 < 4 * NSUB)
                            tmem_ld_16cols(ta + (uint32_t)(((c + 1) >> 2) * 128 + ((c + 1) & 3) * 16), v[(c + 1) & 1]);
                        const unsigned long long ff = pack_f32x2(f[c >> 2], f[c >> 2]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const unsigned long long pv = pack_f32x2(__uint_as_float(v[c & 1][2 * i]),
                                                                     __uint_as_float(v[c & 1][2 * i + 1]));
                            sum[c >> 2][(c & 3) * 8 + i] = fma_f32x2(pv, ff, sum[c >> 2][(c & 3) * 8 + i]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[acc]));
                if (++acc == C::ACCS) { acc = 0; aph ^= 1u; }
            }
            if (!ok) break;
            const int col = t.nt * BN + 64 * hf;                      // first column of this thread's 64, block 0
            if (MODE == kGemmPlain) {
                if (mine) {
                    uint16_t* o = static_cast<uint16_t*>(p.out) + (size_t)row * p.N;
#pragma unroll
                    for (int s = 0; s < NSUB; ++s)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {                 // 8 columns at a time (N is a multiple of 16)
                            const int c = col + 128 * s + 8 * i;
                            if (c < p.N) {
                                uint32_t u[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    float a, b;
                                    unpack_f32x2(sum[s][4 * i + j], a, b);
                                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
                                    u[j] = *reinterpret_cast<const uint32_t*>(&h2);
                                }
                                *reinterpret_cast<uint4*>(o + c) = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        }
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
                            a = __fdividef(a, 1.0f + __expf(-a)) * ua;
                            b = __fdividef(b, 1.0f + __expf(-b)) * ub;
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
                if (mine) {
                    uint8_t* o = static_cast<uint8_t*>(p.out) + (size_t)row * p.N;
#pragma unroll
                    for (int s = 0; s < NB; ++s) {
                        if (b0 + s >= p.nnb) break;
                        const Fp8Quant qq = fp8_quant(amax_nan(ctl->amax[parity][s][0][rl], ctl->amax[parity][s][1][rl]));
                        if (hf == 0) p.out_scale[(size_t)row * p.nnb + b0 + s] = qq.scale;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {                 // 16 columns at a time
                            const int c = col + 128 * s + 16 * i;
                            if (c < p.N) {
                                uint32_t u[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    float x[4];
                                    unpack_f32x2(sum[s][8 * i + 2 * j], x[0], x[1]);
                                    unpack_f32x2(sum[s][8 * i + 2 * j + 1], x[2], x[3]);
                                    u[j] = fp8_quant4(qq, x[0], x[1], x[2], x[3]);
                                }
                                *reinterpret_cast<uint4*>(o + c) = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        }
                    }
                }
            }
        }
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
    constexpr int BN = MODE == kGemmSwiGLU ? 128 : 128 * NSUB;
    p.ntn = (g.N + BN - 1) / BN;
    const size_t smem = 1024 + (size_t)FCfg<NSUB>::STAGES * FCfg<NSUB>::STAGE_BYTES + sizeof(FCtl) +
                        (size_t)(3 * g.groups + 1) * sizeof(int);
    // the attribute belongs to the device that is current: set with every launch
    cudaError_t e = cudaFuncSetAttribute(fp8_gemm_kernel<MODE, NSUB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         F_MAX_SMEM);
    if (e == cudaSuccess) {
        const long long used = g.rows < g.groups ? g.rows : g.groups;
        const long long tiles = (g.rows / F_BM + used) * p.ntn;       // at most
        const int sms = device_sm_count();
        e = launch_kernel(fp8_gemm_kernel<MODE, NSUB>, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(F_THREADS),
                          smem, st, 1, kUsePdl, ma[0], ma[1], ma[2], mw, p);
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
    const unsigned box[3] = {128u, 32u, 8u};
    for (int i = 0; i < 3; ++i)
        if (!make_tensor_map_u8_rows(&ma[i], g.a, g.rows, g.K, g.K, 128u, box[i])) return MOE_ERR_CUDA;
    if (!make_tensor_map_u8_rows(&mw, g.w, (long long)g.groups * p.parts * g.N, g.K, g.K, 128u, 128u)) return MOE_ERR_CUDA;
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
