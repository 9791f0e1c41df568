// gemm_fp8.cuh -- what the two FP8 GEMM kernels (gemm_fp8.cu, gemm_fp8_rows.cu) share: the
// MMA, packed arithmetic, tensor-memory reads, their parameters and tile lists.
#pragma once

#include "fp8.cuh"

namespace moe {

constexpr int F_BOX = 128 * 128;                // 128 rows of 128 codes
constexpr int F_MAX_SMEM = 227 * 1024;
constexpr int F_RASTER = 8;                     // column tiles of a band (tile order)

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
__device__ __forceinline__ unsigned long long mul_f32x2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 8 consecutive FP32 columns of this warp's 32 TMEM lanes, under way until tmem_ld_done.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr));
}
// 16 consecutive FP32 columns of this warp's 32 TMEM lanes, under way until tmem_ld_done.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// 32 consecutive FP32 columns of this warp's 32 TMEM lanes, under way until tmem_ld_done.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// 64 consecutive FP32 columns of this warp's 32 TMEM lanes, under way until tmem_ld_done.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}
// The registers of loads waited for: they pass through the statement after the wait, so that
// no use of them can be moved ahead of it.
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 1 / (1 + e^-x): two of the approximate units' operations, 2^-21 of the value for |x| < 8
// (e^-x overflows to infinity where the result is 0 to FP32's normal range).
__device__ __forceinline__ float sigmoid_approx(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

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
    const int32_t* ids;                         // few-row kernel: null, or what the bounds are counted from
    int top_k;
    int stages;                                 // few-row kernel: of its ring
};

struct FTile { int g, nt, row0, rows; };        // first row of the tile and how many it holds

// The tile list: group g's row tiles times column tiles, in bands of F_RASTER column
// tiles.  The up projection (long rows) walks a band's column tiles first, the down
// projection its row tiles (as gemm.cu, for the same reuse in L2).
// `lo`: a group at or before the tile's (that of the role's last tile: they ascend).
template <bool COLS_FIRST, int BM>
__device__ __forceinline__ FTile f_tile(int tile, int& lo, const int* prefix, const int* start, const FParams& p) {
    int hi = p.groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= tile) lo = mid; else hi = mid;
    }
    const int cnt = start[p.groups + lo], local = tile - prefix[lo];
    const int mtiles = (cnt + BM - 1) / BM;
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
    t.row0 = start[lo] + mt * BM;
    t.rows = min(BM, cnt - mt * BM);
    return t;
}

// Lets a kernel have F_MAX_SMEM bytes of shared memory on the current device: the attribute
// belongs to the device, so it is set there with every launch.
template <typename... Args>
inline cudaError_t allow_smem(void (*kernel)(Args...)) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, F_MAX_SMEM);
}

// The tile list from the bucket bounds (clamped to the rows there are; empty after a
// capacity overflow of the same layer call): `prefix` [groups + 1] tiles before a group,
// `start` [groups] first rows and [groups] rows.  `wtot`: a word a warp.  All threads;
// returns the number of tiles to every one of them (after a __syncthreads).
template <int THREADS, int BM>
__device__ __forceinline__ int f_tile_list(const FParams& p, int* prefix, int* start, int* wtot) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool skip = p.gated && __ldcg(&p.hdr->cap_exceeded);
    const int per = (p.groups + THREADS - 1) / THREADS, g0 = tid * per;
    int sum = 0;
    for (int g = g0; g < min(g0 + per, p.groups); ++g) {
        int lo = __ldcg(p.offsets + g), hi = __ldcg(p.offsets + g + 1);
        lo = lo < 0 ? 0 : min(lo, p.rows);
        hi = hi < lo || skip ? lo : min(hi, p.rows);
        start[g] = lo;
        start[p.groups + g] = hi - lo;
        sum += ((hi - lo + BM - 1) / BM) * p.ntn;
    }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += v;
    }
    if (lane == 31) wtot[warp] = inc;
    __syncthreads();
    int run = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? wtot[lane] : 0);
    for (int g = g0; g < min(g0 + per, p.groups); ++g) {
        prefix[g] = run;
        run += ((start[p.groups + g] + BM - 1) / BM) * p.ntn;
    }
    if (tid == THREADS - 1) prefix[p.groups] = run;
    __syncthreads();
    return prefix[p.groups];
}

// Groups of few rows: the kernel with the operands swapped, nb (16, 32 or 64) rows a tile.
moe_status launch_fp8_rows(const Fp8Problem& g, const FParams& p, const CUtensorMap& mw, int nb, cudaStream_t st);

}  // namespace moe
