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
// therefore works on FP32 keys with a bound on their error (key_margin) and checks
// that every comparison the result hangs on -- chosen against other groups, each
// selected key against the next one -- is decided by more than that; a token where one
// is not (about one in a thousand with logits of N(0, 1), more with peaked ones: the margin
// is absolute) is selected again from the defined keys: the winners next to one another
// among themselves, all experts where the groups are in doubt.  Once in a call (1023 tokens
// x 160, softmax: 4.5 us without) that adds 3 us, and 5.5 for all experts; in double,
// without the pairs of floats of route_df.cuh, 10 and more.  Batches of such tokens
// (16384 x 256, k = 8): BF16-valued softmax logits of N(0, 16) 32 us without groups and 39
// with 4 of 8 (30 for N(0, 1)); all logits equal, so that every token's groups tie, 75 us
// with sigmoid scores and 105 with softmax.
// Two experts of equal logit and bias have equal keys either way, which decides between
// two that are both chosen, and at the last place if all that is near is equal (all logits
// equal, one group: 23 us with sigmoid scores, 25 with softmax).
#include "common.cuh"
#include "route_df.cuh"
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

// How far two FP32 keys have to be apart to be in their defined order: twice the scores'
// error, and the rounding of keys of magnitude `mag` at most with the bias.
//   sigmoid: 2^-21; its slope s (1 - s) damps the error of large exponents.
//   softmax: of s = e^-d / Z with d = max - l, d rounded and the exponential (2 + d units
//   of 2^-24, and d e^-d <= 0.37), the division (2) and Z's own error: its terms', whose
//   weighted mean distance is at most ln(E / Z), and a sum of up to EPL + 5 additions.
__device__ __forceinline__ float key_margin(float score_margin, float mag) { return score_margin + 0x1p-22f * mag; }

// One defined key, of logit x with bias b (softmax: maximum `top`, normaliser z): in pairs
// of floats, with `doubt` set where their rounding is; and in double.
__device__ __forceinline__ float pair_key(float x, float b, bool softmax, float top, Df z, bool& doubt) {
    if (!isfinite(x) || !isfinite(b)) return -INFINITY;
    Df s;
    if (softmax) {
        s = df_div(df_exp(df_two_sum(x, -top)), z);
    } else {
        const Df one = {1.f, 0.f}, e = df_exp({-fabsf(x), 0.f});
        s = df_div(x >= 0.f ? one : e, df_add(one, e));
    }
    doubt = doubt || df_near_middle(s);
    return s.h + b;
}
__device__ __noinline__ float double_key(float x, float b, bool softmax, float top, double z) {
    if (!isfinite(x) || !isfinite(b)) return -INFINITY;
    return (float)(softmax ? exp((double)x - (double)top) / z : 1.0 / (1.0 + exp(-(double)x))) + b;
}
// (Functions of their own: few tokens come here, and their registers would be everyone's.)
__device__ __noinline__ Df pair_normaliser(const float* __restrict__ row, int E, float top, int lane) {
    Df z = {0.f, 0.f};
#pragma unroll 2
    for (int e = lane; e < E; e += 32) {
        const float x = row[e];
        if (isfinite(x)) z = df_add(z, df_exp(df_two_sum(x, -top)));
    }
    for (int off = 16; off > 0; off >>= 1) {
        const Df o = {__shfl_xor_sync(kAll, z.h, off), __shfl_xor_sync(kAll, z.l, off)};
        z = df_add(z, o);
    }
    return z;
}
__device__ __noinline__ double double_normaliser(const float* __restrict__ row, int E, float top, int lane) {
    double z = 0.0;
    for (int e = lane; e < E; e += 32) {
        const float x = row[e];
        z += isfinite(x) ? exp((double)x - (double)top) : 0.0;
    }
    return warp_sum(z);
}
// The whole row's keys.
__device__ __noinline__ void exact_keys(const float* __restrict__ row, const float* __restrict__ bias, int E,
                                        bool softmax, float top, float* out, int lane) {
    const Df z = softmax ? pair_normaliser(row, E, top, lane) : Df{1.f, 0.f};
    bool doubt = false;
#pragma unroll 2
    for (int e = lane; e < E; e += 32) out[e] = pair_key(row[e], bias ? bias[e] : 0.f, softmax, top, z, doubt);
    if (!__any_sync(kAll, doubt)) return;
    const double zd = softmax ? double_normaliser(row, E, top, lane) : 1.0;
    for (int e = lane; e < E; e += 32) out[e] = double_key(row[e], bias ? bias[e] : 0.f, softmax, top, zd);
}
// Lanes 0 .. n-1 hold the experts `e` of a row that may come before or after one another:
// lane r receives the one of rank r by its defined key.
__device__ __noinline__ int exact_order(const float* __restrict__ row, const float* __restrict__ bias, int E, bool softmax,
                                        float top, int e, int n, int lane) {
    const Df z = softmax ? pair_normaliser(row, E, top, lane) : Df{1.f, 0.f};
    bool doubt = false;
    const float x = row[e], b = bias ? bias[e] : 0.f;
    float key = lane < n ? pair_key(x, b, softmax, top, z, doubt) : 0.f;
    if (__any_sync(kAll, doubt)) {
        const double zd = softmax ? double_normaliser(row, E, top, lane) : 1.0;
        if (lane < n) key = double_key(x, b, softmax, top, zd);
    }
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const float ki = __shfl_sync(kAll, key, i);
        const int ei = __shfl_sync(kAll, e, i);
        rank += ki > key || (ki == key && ei < e);
    }
    int out = e;
    for (int i = 0; i < n; ++i) {
        const int ri = __shfl_sync(kAll, rank, i), ei = __shfl_sync(kAll, e, i);
        if (ri == lane) out = ei;
    }
    return out;
}

__device__ __forceinline__ float fast_sigmoid(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// EPL = experts per lane (E <= 32 * EPL; FULL: equal); lane l holds experts l, l + 32, ...
// Bound by the latency of a token's dependent steps (16384 tokens of 256 experts, 8 groups:
// 26.5 to 29 us, 1141 instructions a token at 48 % of the issue slots; selects
// instead of branches, and what a warp's tokens share kept in registers -- biases, a
// key's place in shared memory and its group -- took it there from 1500 instructions).
// A lane keeps its two best candidates, so that most rounds of warp-wide argmax need no
// pass over its keys; the comparisons are checked once, side by side, after the rounds.
template <int EPL, bool FULL>
__global__ void __launch_bounds__(256, EPL <= 8 ? 3 : 1)
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
    float* row_keys = sm + (size_t)warp * (E + G * per);
    const float inv_n = 1.0f / (float)n;
    auto in = [&](int i) { return FULL || lane + 32 * i < E; };
    float b[EPL];                                  // biases
    int first[EPL];                                // per * group: the group's first lane, and its padding
    bool bad_bias = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        b[i] = bias && in(i) ? __ldg(bias + e) : 0.f;
        bad_bias = bad_bias || !isfinite(b[i]);
        first[i] = in(i) ? per * (int)(((float)e + 0.5f) * inv_n) : 0;
    }
    bad_bias = __any_sync(kAll, bad_bias);
    for (int t = gwarp; t < T; t += nwarps) {
        const float* row = logits + (size_t)t * E;
        float x[EPL], probe = 0.f, top = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) x[i] = in(i) ? __ldg(row + lane + 32 * i) : -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) probe = fmaf(in(i) ? x[i] : 0.f, 0.f, probe);   // NaN if one is not finite
        if (__any_sync(kAll, probe != 0.f) || bad_bias) {
            if (lane == 0) raise_status(hdr, MOE_ERR_NONFINITE);
#pragma unroll
            for (int i = 0; i < EPL; ++i) x[i] = isfinite(x[i]) && isfinite(b[i]) ? x[i] : -INFINITY;
        }
        float z = 1.f;
        if (softmax) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) top = fmaxf(top, x[i]);
            top = warp_max(top);
            if (top == -INFINITY) top = 0.f;
        }
        int sel_e = 0;
        for (int exact = 0; exact < 2; ++exact) {
            // ---- keys: -inf for a lane's unused places and for a logit that is not finite
            float key[EPL], margin = 0x1p-20f;                       // the scores' part of key_margin
            if (!exact) {
                if (softmax) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        key[i] = expf(x[i] - top);
                        sum += key[i];
                    }
                    z = warp_sum(sum);
                    z = z > 0.f ? z : 1.f;
                    const float top_s = 1.0f / z;
                    margin = 0x1p-23f * top_s * (7.0f + fmaxf(__logf((float)E * top_s), 0.f) + (float)(EPL + 5));
#pragma unroll
                    for (int i = 0; i < EPL; ++i) key[i] *= top_s;
                } else {
#pragma unroll
                    for (int i = 0; i < EPL; ++i) key[i] = fast_sigmoid(x[i]);
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = x[i] == -INFINITY ? -INFINITY : key[i] + b[i];
            } else {
                __syncwarp();
                exact_keys(row, bias, E, softmax, top, row_keys, lane);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = in(i) ? row_keys[lane + 32 * i] : -INFINITY;
            }
            // ---- groups
            if (G > 1) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (in(i)) row_keys[lane + 32 * i + first[i]] = key[i];
                __syncwarp();
                const int g = lane >> (5 - lg);
                float k1 = -INFINITY, k2 = -INFINITY;
                if (g < G) {
                    const float* gk = row_keys + g * (n + per);
#pragma unroll 4
                    for (int j = lane & (per - 1); j < n; j += per) {
                        const float v = gk[j];
                        k2 = fmaxf(k2, fminf(k1, v));
                        k1 = fmaxf(k1, v);
                    }
                }
                for (int off = per >> 1; off > 0; off >>= 1) {
                    const float o1 = __shfl_xor_sync(kAll, k1, off), o2 = __shfl_xor_sync(kAll, k2, off);
                    k2 = fmaxf(fminf(k1, o1), fmaxf(k2, o2));
                    k1 = fmaxf(k1, o1);
                }
                const bool two = r.group_top == 2 && n > 1;
                const float value = two ? k1 + k2 : k1;
                int rank = 0;
#pragma unroll 4
                for (int q = 0; q < G; ++q) {
                    const float o = __shfl_sync(kAll, value, q * per);
                    rank += (o > value) | ((o == value) & (q < g));
                }
                const bool held = g < G && rank < r.topk_groups;
                const unsigned mask = __ballot_sync(kAll, held);
                if (!exact && r.topk_groups < G) {
                    // the chosen groups against the others: two keys a side, and their sum's rounding
                    const uint32_t vk = route_key(value);
                    const float lo = route_unkey(__reduce_min_sync(kAll, held ? vk : 0xffffffffu));
                    const float hi = route_unkey(__reduce_max_sync(kAll, !held && g < G ? vk : 0u));
                    const float mag = warp_max(g < G ? fabsf(k1) + (two ? fabsf(k2) : 0.f) : 0.f);
                    if (!(lo - hi > 2.0f * key_margin(margin, mag))) continue;       // again, from the defined keys
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = (mask >> first[i]) & 1u ? key[i] : -INFINITY;
            }
            // ---- rounds of argmax.  A lane holds its two best keys (of equal ones the lower
            // index first), as ordered bits; `gone`: those taken.  Lane j keeps the j-th winner.
            uint32_t u1, u2;
            int i1, i2;
            unsigned gone = 0u;
            auto two_best = [&]() {
                float b1 = -INFINITY, b2 = -INFINITY;
                i1 = i2 = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const float v = (gone >> i) & 1u ? -INFINITY : key[i];
                    const bool first_ = v > b1, second = v > b2;
                    i2 = first_ ? i1 : second ? i : i2;
                    i1 = first_ ? i : i1;
                    b2 = fmaxf(b2, fminf(b1, v));
                    b1 = fmaxf(b1, v);
                }
                u1 = route_key(b1);
                u2 = route_key(b2);
            };
            two_best();
            bool fresh = true;                                        // u2 is the second best
            uint32_t my_key = 0u;
            // The next winner, kept by lane j.  (With nothing left it is some expert's -inf: only
            // after a logit or bias that is not finite.)
            auto round = [&](int j) {
                const uint32_t m = __reduce_max_sync(kAll, u1);
                const int e = (int)__reduce_min_sync(kAll, u1 == m ? (unsigned)(lane + 32 * i1) : 0xffffffffu);
                const bool won = (e & 31) == lane;
                const bool refill = won && !fresh;
                gone |= won ? 1u << i1 : 0u;
                u1 = won ? u2 : u1;
                i1 = won ? i2 : i1;
                fresh = won ? !fresh : fresh;
                if (refill) two_best();
                sel_e = lane == j ? (FULL ? e : min(e, E - 1)) : sel_e;
                my_key = lane == j ? m : my_key;
            };
            for (int j = 0; j < k; ++j) round(j);
            if (exact) break;
            // ---- one more to see that the last one was clear, and more as long as it is not
            const int pool = G > 1 ? r.topk_groups * n : E;           // candidates there were
            int count = k;
            if (count == 32 && pool > 32) continue;                   // no lane for the one after
            if (pool > count) round(count++);
            const float mine = route_unkey(my_key);
            const float down = __shfl_down_sync(kAll, mine, 1);
            bool doubt = lane + 1 < count && !(mine - down > key_margin(margin, fmaxf(fabsf(mine), fabsf(down))));
            if (!__any_sync(kAll, doubt)) break;
            // equal logits with equal biases have equal keys: the lower index came first
            const int next_e = __shfl_down_sync(kAll, sel_e, 1);
            const bool equal = doubt && __ldg(row + sel_e) == __ldg(row + next_e) &&
                               (!bias || __ldg(bias + sel_e) == __ldg(bias + next_e));
            if (!__any_sync(kAll, doubt && !equal)) {
                // Between two that are chosen that settles it.  An equal of the last one that is not
                // chosen says nothing of those behind it: whatever else is near has to be its equal too.
                if (!((__ballot_sync(kAll, doubt) >> (k - 1)) & 1u)) break;
                const int last_e = __shfl_sync(kAll, sel_e, k - 1);
                const float last = route_unkey(__shfl_sync(kAll, my_key, k - 1));
                const float last_x = __ldg(row + last_e), last_b = bias ? __ldg(bias + last_e) : 0.f;
                bool other = false;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const bool left = !((gone >> i) & 1u) && key[i] > -INFINITY;
                    if (left && !(last - key[i] > key_margin(margin, fmaxf(fabsf(last), fabsf(key[i])))))
                        other = other || __ldg(row + lane + 32 * i) != last_x || b[i] != last_b;
                }
                if (!__any_sync(kAll, other)) break;
            }
            bool clear;                                               // the last winner is clearly below the others
            for (;;) {
                const float a = route_unkey(__shfl_sync(kAll, my_key, count - 2)), c = route_unkey(__shfl_sync(kAll, my_key, count - 1));
                clear = count > k && a - c > key_margin(margin, fmaxf(fabsf(a), fabsf(c)));
                if (clear || count >= pool || count == 32) break;
                round(count++);
            }
            if (!clear && count < pool) continue;                     // too many near one another
            sel_e = exact_order(row, bias, E, softmax, top, sel_e, clear ? count - 1 : count, lane);
            break;
        }
        // ---- weights, from the selected logits
        const float sel_x = lane < k ? __ldg(row + sel_e) : 0.f;
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
//
// The last form takes a warp a token.  The others take G lanes a token (the power of two at
// or above k): 32 / G tokens a warp zero their rows together, then lane j of a token writes
// its j-th expert's gradient.  An id out of range or repeated inside the token (the first
// stays valid, as in the dispatch) takes no part and raises the status.
// Bound by writing the rows (16384 x 256, k = 8: 5.5 us, 17 MB; a warp a token: 9.4).
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}
template <int G>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
    return v;
}

template <int G>
__global__ void __launch_bounds__(256)
route_grouped_grad_kernel(int T, int E, int k, const moe_router r, const float* __restrict__ logits,
                          const int32_t* __restrict__ ids, const float* __restrict__ dw, float* __restrict__ dlogits,
                          WsHeader* hdr) {
    constexpr int TPW = 32 / G;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, j = lane % G, first = lane - j;
    const unsigned mates = (G == 32 ? kAll : ((1u << (G & 31)) - 1u)) << first;
    const int gwarp = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
    const int nwarps = (int)((gridDim.x * blockDim.x) >> 5);
    const bool softmax = r.score == MOE_SCORE_SOFTMAX;
    const int nt = (T - 1) / TPW + 1;
    for (int wt = gwarp; wt < nt; wt += nwarps) {
        const int t0 = wt * TPW, t = t0 + lane / G;
        const bool mine = t < T && j < k;
        const size_t at = (size_t)t * k + j;
        const int id = mine ? ids[at] : -1 - lane;
        const unsigned same = __match_any_sync(kAll, id) & mates;
        const bool ok = mine && id >= 0 && id < E && (__ffs(same) - 1) == lane;
        if (mine && !ok) raise_status(hdr, MOE_ERR_INVALID_ROUTE);
        const float g = ok ? dw[at] : 0.f;
        const float l = ok ? logits[(size_t)t * E + id] : -INFINITY;
        float* rows = dlogits + (size_t)t0 * E;
        const long long n = (long long)min(TPW, T - t0) * E;
        if (E % 4 == 0) {
            for (long long i = lane; i < n / 4; i += 32) reinterpret_cast<float4*>(rows)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            for (long long i = lane; i < n; i += 32) rows[i] = 0.f;
        }
        // s = e^lo / (1 + em), 1 - s = q; the largest lo drops out of renormalised scores
        const float lo = softmax ? l : fminf(l, 0.f);
        const float em = softmax ? 0.f : expf(-fabsf(l));
        const float m = r.renorm ? lanes_max<G>(ok ? lo : -INFINITY) : 0.f;
        float p = ok ? expf(lo - m) / (1.0f + em) : 0.f;
        const float q = softmax ? 1.0f : (l > 0.f ? em : 1.0f) / (1.0f + em);
        float d = g;
        if (r.renorm) {
            p = p / lanes_sum<G>(p);
            d = 0.f;
            for (int i = 0; i < k; ++i) {
                const float pi = __shfl_sync(kAll, p, first + i), gi = __shfl_sync(kAll, g, first + i);
                d = fmaf(pi, g - gi, d);
            }
        }
        __syncwarp();                                  // the zeros come before the selected entries
        if (ok) rows[(size_t)(t - t0) * E + id] = r.scale * (p * q) * d;
    }
}

// Softmax scores as they are: the gradient of every logit.
__global__ void __launch_bounds__(256)
route_dense_grad_kernel(int T, int E, int k, const moe_router r, const float* __restrict__ logits,
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
        const float f = -r.scale * a * iz;
        for (int e = lane; e < E; e += 32) out[e] = f * expf(row[e] - top);
        __syncwarp();                                  // the row comes before the selected entries
        if (ok) out[id] = r.scale * s * (g * (id == at ? rest * iz : 1.0f - s) - others);
    }
}

unsigned warps_grid(long long warps) {
    const long long blocks = (warps + 7) / 8;
    const long long cap = (long long)device_sm_count() * 8;
    return (unsigned)(blocks < cap ? blocks : cap);
}

template <int EPL, bool FULL>
cudaError_t launch_epl(const moe_shape& s, const moe_router& r, const float* logits, const float* bias, int32_t* ids,
                       float* w, WsHeader* hdr, cudaStream_t st) {
    // a warp's keys: padded by 32 / pow2 lanes' worth per group, see the kernel
    int pow2 = 1;
    while (pow2 < r.groups) pow2 *= 2;
    const size_t smem = (size_t)8 * (s.experts + (r.groups > 1 ? r.groups * (32 / pow2) : 32)) * sizeof(float);
    // as many blocks as run at once: what a warp sets up serves all its tokens
    long long blocks = ((long long)s.tokens + 7) / 8;
    const long long cap = (long long)device_sm_count() * (EPL <= 8 ? 3 : 1);
    if (blocks > cap) blocks = cap;
    return launch_kernel(route_grouped_kernel<EPL, FULL>, dim3((unsigned)blocks), dim3(256), smem, st, 1, kUsePdl, s.tokens,
                         s.experts, s.top_k, r, logits, bias, ids, w, hdr);
}

template <int EPL>
cudaError_t launch_full(const moe_shape& s, const moe_router& r, const float* logits, const float* bias, int32_t* ids,
                        float* w, WsHeader* hdr, cudaStream_t st) {
    return s.experts == 32 * EPL ? launch_epl<EPL, true>(s, r, logits, bias, ids, w, hdr, st)
                                 : launch_epl<EPL, false>(s, r, logits, bias, ids, w, hdr, st);
}

}  // namespace

cudaError_t launch_route_grouped(const moe_shape& s, const moe_router& r, const float* logits, const float* bias,
                                 int32_t* ids, float* w, WsHeader* hdr, cudaStream_t st) {
    const int E = s.experts;
    if (E <= 32) return launch_full<1>(s, r, logits, bias, ids, w, hdr, st);
    if (E <= 64) return launch_full<2>(s, r, logits, bias, ids, w, hdr, st);
    if (E <= 128) return launch_full<4>(s, r, logits, bias, ids, w, hdr, st);
    if (E <= 256) return launch_full<8>(s, r, logits, bias, ids, w, hdr, st);
    if (E <= 512) return launch_full<16>(s, r, logits, bias, ids, w, hdr, st);
    return launch_full<32>(s, r, logits, bias, ids, w, hdr, st);
}

cudaError_t launch_route_grouped_grad(const moe_shape& s, const moe_router& r, const float* logits, const int32_t* ids,
                                      const float* dw, float* dlogits, WsHeader* hdr, cudaStream_t st) {
    auto go = [&](auto* kernel, int lanes) {
        return launch_kernel(kernel, dim3(warps_grid(((long long)s.tokens * lanes + 31) / 32)), dim3(256), 0, st, 1, kUsePdl,
                             s.tokens, s.experts, s.top_k, r, logits, ids, dw, dlogits, hdr);
    };
    if (r.score == MOE_SCORE_SOFTMAX && !r.renorm) return go(route_dense_grad_kernel, 32);
    if (s.top_k <= 2) return go(route_grouped_grad_kernel<2>, 2);
    if (s.top_k <= 4) return go(route_grouped_grad_kernel<4>, 4);
    if (s.top_k <= 8) return go(route_grouped_grad_kernel<8>, 8);
    if (s.top_k <= 16) return go(route_grouped_grad_kernel<16>, 16);
    return go(route_grouped_grad_kernel<32>, 32);
}

}  // namespace moe
