"""The pairs of floats behind near ties of the group-limited route (route_df.cuh), compiled
for the CPU: their error against long double, and that a rounding not reported as in doubt
is the double's."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_routing_router_gb300", "csrc")

MAIN = r"""
#include <cstdio>
#include <cmath>
#include <random>
#include "route_df.cuh"
using namespace moe;
static double worst(double& w, Df a, double want_hi, double want_lo) {
    const double d = std::fabs((((double)a.h - want_hi) + ((double)a.l - want_lo)) / want_hi);
    if (d > w) w = d;
    return d;
}
int main() {
    std::mt19937_64 g(7);
    std::uniform_real_distribution<double> U(0, 1);
    double we = 0, wd = 0, ws = 0;
    long wrong = 0, doubt = 0, n = 0;
    for (int i = 0; i < 400000; ++i) {
        const float a = (float)(-50 * U(g) * U(g)), b = (float)(a * U(g) * 3e-8);
        const Df x = df_two_sum(a, b), e = df_exp(x);
        const double t = std::exp((double)x.h + (double)x.l);        // 2^-52: the pair's bound is 2^-43
        worst(we, e, t, 0);
        const Df d = df_add({(float)(1 + U(g)), 0.f}, {(float)(U(g) * 1e-8), 0.f});
        worst(wd, df_div(e, d), ((double)e.h + (double)e.l) / ((double)d.h + (double)d.l), 0);
        const Df one = {1.f, 0.f}, s = df_div(i & 1 ? one : e, df_add(one, e));
        const double v = i & 1 ? 1.0 / (1.0 + t) : t / (1.0 + t);
        worst(ws, s, v, 0);
        ++n;
        if (df_near_middle(s)) ++doubt;
        else if (s.h != (float)v) ++wrong;
    }
    // a value half way between two floats, one next to it, one too small for a pair
    const int middle = df_near_middle({1.f, 0x1p-24f}) + 2 * df_near_middle({1.f, -0x1p-25f}) + 4 * df_near_middle({1.f, 0x1p-25f})
                     + 8 * df_near_middle({0x1p-80f, 0.f}) + 16 * df_near_middle({0.f, 0.f});
    printf("%.2f %.2f %.2f %ld %ld %d\n", -std::log2(we), -std::log2(wd), -std::log2(ws), wrong, doubt, middle);
}
"""


@pytest.mark.parametrize("opt", ["-O0", "-O2"])
def test_pairs_of_floats(tmp_path, opt):
    src, exe = str(tmp_path / "m.cpp"), str(tmp_path / "m")
    with open(src, "w") as f:
        f.write(MAIN)
    # no contraction: the error-free sums and products are as written
    subprocess.run(["g++", "-std=c++17", opt, "-ffp-contract=off", "-I", CSRC, "-x", "c++", src, "-o", exe], check=True,
                   capture_output=True, text=True)
    e, d, s, wrong, doubt, middle = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    assert min(float(e), float(d), float(s)) >= 43.0          # near_middle allows for 2^-42
    assert int(wrong) == 0 and int(doubt) <= 10               # 2^-18 of them at most, about
    # the middle above 1 and the one below it (its floats are half as far apart), the small ones
    assert int(middle) == 1 + 2 + 8 + 16
