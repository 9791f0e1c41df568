// route_df.cuh -- scores of group-limited routing to about 2^-44, in pairs of floats.
//
// The scores are defined through double, whose unit is slow here (two results a cycle
// and SM: a warp's exponentials take microseconds).  Pairs hi + lo of floats, |lo| at most
// half a unit of hi, with Knuth's and Dekker's error-free sums and products (fma), give
// them to some 45 bits at FP32's rate: enough to round to FP32, except next to the middle
// of two floats, which is reported (df_near_middle) for double to decide.
#pragma once

#include <math.h>

#if defined(__CUDACC__)
#define MOE_DF __host__ __device__ __forceinline__
#else
#define MOE_DF inline
#endif

namespace moe {

struct Df { float h, l; };

// A product rounded by itself: contracted into a sum it would no longer be the number whose
// error the next line takes.
MOE_DF float df_product(float a, float b) {
#if defined(__CUDA_ARCH__)
    return __fmul_rn(a, b);
#else
    return a * b;
#endif
}
MOE_DF Df df_two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
MOE_DF Df df_fast_sum(float a, float b) {            // |a| >= |b|
    const float s = a + b;
    return {s, b - (s - a)};
}
MOE_DF Df df_add(Df a, Df b) {
    Df s = df_two_sum(a.h, b.h);
    const Df t = df_two_sum(a.l, b.l);
    s = df_fast_sum(s.h, s.l + t.h);
    return df_fast_sum(s.h, s.l + t.l);
}
MOE_DF Df df_mul(Df a, Df b) {
    const float p = df_product(a.h, b.h);
    return df_fast_sum(p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h));
}
MOE_DF Df df_div(Df a, Df b) {
    const float q1 = a.h / b.h;
    // a - q1 b, in which the leading parts cancel
    const float p = df_product(q1, b.h);
    const Df r = df_add(a, {-p, -fmaf(q1, b.l, fmaf(q1, b.h, -p))});
    const float q2 = r.h / b.h;
    const float q3 = (fmaf(-q2, b.h, r.h) + r.l - q2 * b.l) / b.h;
    const Df q = df_fast_sum(q1, q2);
    return df_fast_sum(q.h, q.l + q3);
}

// A double constant as a pair.
constexpr Df df_const(double v) { return {(float)v, (float)(v - (double)(float)v)}; }

// A sum with |a| well above |b|: no leading digits cancel, so the low parts are added plainly.
MOE_DF Df df_add_small(Df a, Df b) {
    const Df s = df_fast_sum(a.h, b.h);
    return df_fast_sum(s.h, s.l + (a.l + b.l));
}

// e^x for x <= 0; below -80 the pair is 0 (a score that small is reported as in doubt).
// x = n ln 2 + 4 r, |r| <= 0.087; Taylor's series of e^r, its terms from r^5 / 5! on in FP32
// (2^-24 of the whole, their error 2^-48); its fourth power by two squarings; 2^n.  The
// chain is half as long as the series of e^(4 r) (a token decided again: 7.3 -> 5.5 us).
MOE_DF Df df_exp(Df x) {
    if (!(x.h >= -80.0f)) return {0.f, 0.f};
    constexpr double kLn2 = 0.693147180559945309417;
    constexpr float kL1 = 0.693359375f;                               // 10 bits: n kL1 is exact
    constexpr Df kL2 = df_const(kLn2 - 0.693359375);
    const float n = rintf(x.h * 1.44269504f);
    const float p = df_product(-n, kL2.h);
    Df r = df_add({fmaf(-n, kL1, x.h), x.l}, {p, fmaf(-n, kL2.h, -p) - n * kL2.l});
    r = {0.25f * r.h, 0.25f * r.l};
    float t = 1.0f / 40320.0f;                                        // 1/8!
    t = fmaf(t, r.h, 1.0f / 5040.0f);
    t = fmaf(t, r.h, 1.0f / 720.0f);
    t = fmaf(t, r.h, 1.0f / 120.0f);
    constexpr Df c[5] = {{1.f, 0.f}, {1.f, 0.f}, {0.5f, 0.f}, df_const(1.0 / 6), df_const(1.0 / 24)};
    Df s = df_add_small(c[4], {df_product(t, r.h), 0.f});
#if defined(__CUDA_ARCH__)
#pragma unroll
#endif
    for (int i = 3; i >= 0; --i) s = df_add_small(c[i], df_mul(s, r));
    s = df_mul(s, s);
    s = df_mul(s, s);
    return {ldexpf(s.h, (int)n), ldexpf(s.l, (int)n)};
}

// Whether the pair's rounding to FP32 (its hi) is in doubt: lo within 2^-42 of the value
// from half way to the next float, or a value too small for a pair.
MOE_DF bool df_near_middle(Df v) {
    if (!(v.h >= 0x1p-75f)) return true;
    const float next = nextafterf(v.h, v.l < 0.f ? 0.f : 2.0f * v.h);
    return fabsf(fabsf(v.l) - 0.5f * fabsf(next - v.h)) <= v.h * 0x1p-42f;
}

}  // namespace moe
