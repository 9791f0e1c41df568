// route_grouped.cu -- group-limited top-k routing and its gradient: a warp per token.
//
// The router of a layer of many experts (ONNX Runtime PR #33963, Description bullet 2:
// sigmoid scores, a correction bias that only selects, weights from the unbiased
// scores), with the experts in `groups` equal groups of consecutive experts, of which a
// token may use `topk_groups`.  Per token:
//   s_e   = sigmoid(l_e), or softmax over all experts, in double rounded once to FP32
//   key_e = s_e + bias_e in FP32
//   value of a group: its largest key, or the FP32 sum of its two largest
//   the topk_groups groups of the largest value, the k largest keys inside them
//   (ties to the lower index everywhere), in descending order
//   w_j   = scale * s_j, divided by the sum over the selection when `renorm`.
//
// Keys are defined through double so that every implementation selects the same
// experts, but the double unit is slow here (two results a cycle and SM).  The kernel
// therefore works on FP32 keys with a bound on their error (`eps`, below) and checks
// that every comparison the result hangs on -- chosen against other groups, each
// selected key against the next one -- is decided by more than that; a token where one
// is not (about one in a thousand with random logits) is selected again from the
// defined keys.  Two experts of equal logit and bias have equal keys either way.
#include "common.cuh"
#include "route_warp.cuh"

#include <climits>

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float route_unkey(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}
__device__ __forceinline__ float warp_max(float v) { return route_unkey(__reduce_max_sync(kAll, route_key(v))); }

// The FP32 scores' error: |s~ - s| <= s 2^-18 + 2^-24 for the softmax (exponents of up to
// 127 rounded to FP32 before the exponential, two units of its last place, a sum of up to
// 1024 terms, one division) and <= 2^-21 for the sigmoid, whose slope s (1 - s) damps the
// error of large exponents; one more FP32 rounding with the bias.  Two keys of magnitude
// `mag` at most, further apart than this, are in their defined order.
__device__ __forceinline__ float key_margin(bool softmax, float top_score, float mag) {
    return (softmax ? 0x1p-23f + 0x1p-17f * top_score : 0x1p-20f) + 0x1p-22f * mag;
}

// EPL = experts per lane (E <= 32 * EPL); lane l holds experts l, l + 32, ...
template <int EPL>
__global__ void __launch_bounds__(256)
route_grouped_kernel(int T, int E, int k, const moe_router r, const float* __restrict__ logits,
                     const float* __restrict__ bias, int32_t* __restrict__ ids, float* __restrict__ w, WsHeader* hdr) {
    extern __shared__ float sm[];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gwarp = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
    const int nwarps = (int)((gridDim.x * blockDim.x) >> 5);
    const bool softmax = r.score == MOE_SCORE_SOFTMAX;
    const int G = r.groups, n = E / G;
    // `per` lanes share a group (G rounded up to a power of two, 32 / that each); a key lies
    // in shared memory at e + per * group, which keeps those lanes on banks of their own
    const int lg = 32 - __clz(G - 1), per = G > 1 ? 32 >> lg : 32;
    const float inv_n = 1.0f / (float)n;
    float* row_keys = sm + (size_t)warp * (E + G * per);
    for (int t = gwarp; t < T; t += nwarps) {
        const float* row = logits + (size_t)t * E;
        float x[EPL], b[EPL];
        bool bad = false;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 32 * i;
            x[i] = -INFINITY;
            b[i] = 0.f;
            if (e < E) {
                x[i] = __ldg(row + e);
                if (bias) b[i] = __ldg(bias + e);
                if (!isfinite(x[i]) || !isfinite(b[i])) {
                    bad = true;
                    x[i] = -INFINITY;
                }
            }
            top = fmaxf(top, x[i]);
        }
        if (__any_sync(kAll, bad) && lane == 0) raise_status(hdr, MOE_ERR_NONFINITE);
        if (softmax) {
            top = warp_max(top);
            if (top == -INFINITY) top = 0.f;
        }
        float z = 1.f;
        int sel_e = 0;
        float sel_x = 0.f;
        for (int exact = 0; exact < 2; ++exact) {
            // ---- keys: an unused slot 0, a non-finite logit that of -inf
            uint32_t key[EPL];
            float top_s = 0.f;
            if (exact) {
                double zd = 1.0;
                if (softmax) {
                    double sum = 0.0;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) sum += x[i] == -INFINITY ? 0.0 : exp((double)x[i] - (double)top);
                    zd = warp_sum(sum);
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const double s = softmax ? exp((double)x[i] - (double)top) / zd : 1.0 / (1.0 + exp(-(double)x[i]));
                    const float kv = x[i] == -INFINITY ? -INFINITY : (float)s + b[i];
                    key[i] = lane + 32 * i < E ? route_key(kv) : 0u;
                }
            } else {
                float s[EPL];
                if (softmax) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        s[i] = __expf(x[i] - top);
                        sum += s[i];
                    }
                    z = warp_sum(sum);
                    z = z > 0.f ? z : 1.f;
                    top_s = 1.0f / z;
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    s[i] = softmax ? s[i] * top_s : __fdividef(1.0f, 1.0f + __expf(-x[i]));
                    const float kv = x[i] == -INFINITY ? -INFINITY : s[i] + b[i];
                    key[i] = lane + 32 * i < E ? route_key(kv) : 0u;
                }
            }
            bool sure = true;
            // ---- groups
            if (G > 1) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = lane + 32 * i;
                    if (e < E) row_keys[e + per * (int)(((float)e + 0.5f) * inv_n)] = route_unkey(key[i]);
                }
                __syncwarp();
                const int g = lane / per;
                float k1 = -INFINITY, k2 = -INFINITY;
                if (g < G)
                    for (int j = lane % per; j < n; j += per) {
                        const float v = row_keys[g * (n + per) + j];
                        k2 = fmaxf(k2, fminf(k1, v));
                        k1 = fmaxf(k1, v);
                    }
                for (int off = per >> 1; off > 0; off >>= 1) {
                    const float o1 = __shfl_xor_sync(kAll, k1, off), o2 = __shfl_xor_sync(kAll, k2, off);
                    k2 = fmaxf(fminf(k1, o1), fmaxf(k2, o2));
                    k1 = fmaxf(k1, o1);
                }
                const bool two = r.group_top == 2 && n > 1;
                const float value = two ? k1 + k2 : k1;
                int rank = 0;
                for (int q = 0; q < G; ++q) {
                    const float o = __shfl_sync(kAll, value, q * per);
                    rank += o > value || (o == value && q < g);
                }
                const bool held = g < G && rank < r.topk_groups;
                const unsigned mask = __ballot_sync(kAll, held);
                const uint32_t vk = route_key(value);
                const uint32_t lo = __reduce_min_sync(kAll, held ? vk : 0xffffffffu);
                const uint32_t hi = __reduce_max_sync(kAll, !held && g < G ? vk : 0u);
                if (hi != 0u) {
                    // two keys a side, and the rounding of their sum
                    const float mag = warp_max(g < G ? fabsf(k1) + (two ? fabsf(k2) : 0.f) : 0.f);
                    sure = route_unkey(lo) - route_unkey(hi) > 2.0f * key_margin(softmax, top_s, mag);
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = lane + 32 * i;
                    if (e < E && !((mask >> (per * (int)(((float)e + 0.5f) * inv_n))) & 1u)) key[i] = 0u;
                }
            }
            // ---- k rounds of argmax; one more to see that the last one was clear
            uint32_t best = 0u;
            int bi = 0;
            auto local_best = [&]() {
                best = 0u;
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (key[i] > best) { best = key[i]; bi = i; }
            };
            local_best();
            float prev = 0.f, prev_x = 0.f;
            int prev_e = 0;
            for (int j = 0; j < k + (exact ? 0 : 1); ++j) {
                const uint32_t m = __reduce_max_sync(kAll, best);
                if (m == 0u) break;                                  // every candidate is selected
                const unsigned e = __reduce_min_sync(kAll, best == m ? (unsigned)(lane + 32 * bi) : 0xffffffffu);
                const bool mine = (e & 31u) == (unsigned)lane;
                float xv = 0.f;
                if (mine) {
#pragma unroll
                    for (int i = 0; i < EPL; ++i)
                        if (i == (int)(e >> 5)) { xv = x[i]; key[i] = 0u; }
                    local_best();
                }
                xv = __shfl_sync(kAll, xv, (int)(e & 31u));
                const float kv = route_unkey(m);
                if (!exact && j > 0 && !(prev - kv > key_margin(softmax, top_s, fmaxf(fabsf(prev), fabsf(kv))))) {
                    const bool same = xv == prev_x && (!bias || __ldg(bias + e) == __ldg(bias + prev_e));
                    sure = sure && same;
                }
                prev = kv;
                prev_x = xv;
                prev_e = (int)e;
                if (lane == j && j < k) { sel_e = (int)e; sel_x = xv; }
            }
            if (sure) break;
        }
        // ---- weights, from the selected logits
        float p;
        if (softmax) {
            const float m = r.renorm ? warp_max(lane < k ? sel_x : -INFINITY) : top;
            p = lane < k ? expf(sel_x - m) : 0.f;
            if (!r.renorm) p = p / z;
        } else {
            // s = e^min(l, 0) / (1 + e^-|l|); renormalised weights do not change with a common
            // factor, so the largest min(l, 0) is taken out and small scores keep their ratios
            const float lo = fminf(sel_x, 0.f);
            const float m = r.renorm ? warp_max(lane < k ? lo : -INFINITY) : 0.f;
            p = lane < k ? expf(lo - m) / (1.0f + expf(-fabsf(sel_x))) : 0.f;
        }
        if (r.renorm) p = p / warp_sum(p);
        if (lane < k) {
            ids[(size_t)t * k + lane] = sel_e;
            w[(size_t)t * k + lane] = r.scale * p;
        }
    }
}

// The gradient, for the selection as it was made (the bias and the groups only select):
//   softmax, renorm   dl_j = scale p_j sum_i p_i (g_j - g_i)           selected experts
//   sigmoid, renorm   dl_j = scale p_j (1 - s_j) sum_i p_i (g_j - g_i)
//   sigmoid           dl_j = scale s_j (1 - s_j) g_j
//   softmax           dl_e = scale s_e ([e selected] g_e - sum_i s_i g_i)   every expert
// with p the renormalised scores.  The differences g_j - g_i stand for g_j - sum_i p_i g_i,
// which cancels when one expert dominates.  For the same reason the last form is taken as
// g_j (1 - s_j) - sum_{i != j} s_i g_i with 1 - s of the largest logit summed without it.
template <bool DENSE>
__global__ void __launch_bounds__(256)
route_grouped_grad_kernel(int T, int E, int k, const moe_router r, const float* __restrict__ logits,
                          const int32_t* __restrict__ ids, const float* __restrict__ dw, float* __restrict__ dlogits,
                          WsHeader* hdr) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int gwarp = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
    const int nwarps = (int)((gridDim.x * blockDim.x) >> 5);
    for (int t = gwarp; t < T; t += nwarps) {
        const float* row = logits + (size_t)t * E;
        float* out = dlogits + (size_t)t * E;
        const int id = lane < k ? ids[(size_t)t * k + lane] : -1 - lane;
        const unsigned same = __match_any_sync(kAll, id);
        const bool ok = lane < k && id >= 0 && id < E && (__ffs(same) - 1) == lane;
        if (lane < k && !ok) raise_status(hdr, MOE_ERR_INVALID_ROUTE);
        const float g = ok ? dw[(size_t)t * k + lane] : 0.f;
        const float l = ok ? row[id] : -INFINITY;
        float d;
        if (DENSE) {
            float m = -INFINITY;
            int at = 0;
            for (int e = lane; e < E; e += 32)
                if (row[e] > m) { m = row[e]; at = e; }
            const float top = warp_max(m);
            at = (int)__reduce_min_sync(kAll, m == top ? (unsigned)at : 0xffffffffu);
            float rest = 0.f;                                   // of the normaliser, without its largest term
            for (int e = lane; e < E; e += 32) rest += e == at ? 0.f : expf(row[e] - top);
            rest = warp_sum(rest);
            const float iz = 1.0f / (1.0f + rest);
            const float s = ok ? expf(l - top) * iz : 0.f;
            const float sg = s * g;
            const float a = warp_sum(sg);
            float others = 0.f;
            for (int i = 0; i < k; ++i) {
                const float o = __shfl_sync(kAll, sg, i);
                others += i == lane ? 0.f : o;
            }
            d = r.scale * s * (g * (id == at ? rest * iz : 1.0f - s) - others);
            const float f = -r.scale * a * iz;
            for (int e = lane; e < E; e += 32) out[e] = f * expf(row[e] - top);
        } else {
            if (E % 4 == 0) {
                for (int i = lane; i < E / 4; i += 32) reinterpret_cast<float4*>(out)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            } else {
                for (int i = lane; i < E; i += 32) out[i] = 0.f;
            }
            const bool softmax = r.score == MOE_SCORE_SOFTMAX;
            const float lo = softmax ? l : fminf(l, 0.f);
            const float em = softmax ? 0.f : expf(-fabsf(l));           // 1 - s = 1/(1+e^l)
            const float m = r.renorm ? warp_max(ok ? lo : -INFINITY) : 0.f;
            float p = ok ? expf(lo - m) / (1.0f + em) : 0.f;
            const float q = softmax ? 1.0f : (l > 0.f ? em : 1.0f) / (1.0f + em);
            if (r.renorm) {
                p = p / warp_sum(p);
                float s = 0.f;
                for (int i = 0; i < k; ++i) {
                    const float pi = __shfl_sync(kAll, p, i), gi = __shfl_sync(kAll, g, i);
                    s = fmaf(pi, g - gi, s);
                }
                d = r.scale * (p * q) * s;
            } else {
                d = r.scale * (p * q) * g;
            }
        }
        __syncwarp();                                  // the row comes before the selected entries
        if (ok) out[id] = d;
    }
}

unsigned warps_grid(int tokens) {
    long long blocks = ((long long)tokens + 7) / 8;
    const long long cap = (long long)device_sm_count() * 8;
    return (unsigned)(blocks < cap ? blocks : cap);
}

template <int EPL>
cudaError_t launch_epl(const moe_shape& s, const moe_router& r, const float* logits, const float* bias, int32_t* ids,
                       float* w, WsHeader* hdr, cudaStream_t st) {
    size_t smem = 0;
    if (r.groups > 1) {
        int pow2 = 1;
        while (pow2 < r.groups) pow2 *= 2;
        smem = (size_t)8 * (s.experts + r.groups * (32 / pow2)) * sizeof(float);
    }
    return launch_kernel(route_grouped_kernel<EPL>, dim3(warps_grid(s.tokens)), dim3(256), smem, st, 1, kUsePdl,
                         s.tokens, s.experts, s.top_k, r, logits, bias, ids, w, hdr);
}

}  // namespace

cudaError_t launch_route_grouped(const moe_shape& s, const moe_router& r, const float* logits, const float* bias,
                                 int32_t* ids, float* w, WsHeader* hdr, cudaStream_t st) {
    const int E = s.experts;
    if (E <= 32) return launch_epl<1>(s, r, logits, bias, ids, w, hdr, st);
    if (E <= 64) return launch_epl<2>(s, r, logits, bias, ids, w, hdr, st);
    if (E <= 128) return launch_epl<4>(s, r, logits, bias, ids, w, hdr, st);
    if (E <= 256) return launch_epl<8>(s, r, logits, bias, ids, w, hdr, st);
    if (E <= 512) return launch_epl<16>(s, r, logits, bias, ids, w, hdr, st);
    return launch_epl<32>(s, r, logits, bias, ids, w, hdr, st);
}

cudaError_t launch_route_grouped_grad(const moe_shape& s, const moe_router& r, const float* logits, const int32_t* ids,
                                      const float* dw, float* dlogits, WsHeader* hdr, cudaStream_t st) {
    const bool dense = r.score == MOE_SCORE_SOFTMAX && !r.renorm;
    return launch_kernel(dense ? route_grouped_grad_kernel<true> : route_grouped_grad_kernel<false>,
                         dim3(warps_grid(s.tokens)), dim3(256), 0, st, 1, kUsePdl, s.tokens, s.experts, s.top_k, r,
                         logits, ids, dw, dlogits, hdr);
}

}  // namespace moe
