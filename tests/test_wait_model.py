"""The kernels' bounded waits against a model of the barriers, on the CPU.

The wait helpers are plain code over two primitives, "has this phase completed" and
"what time is it".  Their text is taken from the sources and compiled here against a
model of both, so that a wait that runs out can be tried without a GPU that hangs.
"""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_routing_router_gb300", "csrc")

MODEL = r"""
#include <cstdint>
#include <cstdio>
#include <map>
#define __device__
#define __forceinline__
static unsigned long long now = 1000000;              // the clock: a try costs 200 ns
static std::map<uint32_t, unsigned> phases;           // completed phases of a barrier
static unsigned long long globaltimer_ns() { return now += 20; }
static bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    now += 200;
    // true when the phase of this parity has completed: the current phase has the other one
    return (phases[bar] & 1u) != parity;
}
"""


def function(name, path):
    with open(os.path.join(CSRC, path)) as f:
        text = f.read()
    m = re.search(r"__device__ __forceinline__ bool " + name + r"\((?:[^(){}])*\) \{", text)
    if m is None:
        return ""
    depth, i = 1, m.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[m.start():i] + "\n"


def limit():
    with open(os.path.join(CSRC, "common.cuh")) as f:
        return int(re.search(r"kWaitLimitNs = (\d+)ull", f.read()).group(1))


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    def go(main):
        d = tmp_path_factory.mktemp("waits")
        src, exe = str(d / "m.cpp"), str(d / "m")
        code = MODEL + f"constexpr unsigned long long kWaitLimitNs = {limit()}ull;\n"
        for name in ("mbar_wait_bounded", "mbar_wait_until", "wait_armed_stages", "drain_ring"):
            code += function(name, "common.cuh")
        code += function("wait_armed_pair_stages", "gemm_grad.cu")
        with open(src, "w") as f:
            f.write(code + "int main() {" + main + "}\n")
        subprocess.run(["g++", "-std=c++17", "-O1", "-o", exe, src], check=True, capture_output=True, text=True)
        out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=300).stdout
        return [int(v) for v in out.split()]
    return go


def test_waiting_for_the_armed_stages_has_one_limit(run):
    """Six stages whose copies never land: one limit for all of them."""
    all_landed, took = run("""
        unsigned long long t0 = now;
        const bool r = wait_armed_stages(64, 6, 9);
        printf("%d %llu", (int)r, now - t0);
    """)
    assert all_landed == 0
    assert took < 1.1 * limit()


def test_armed_stages_that_have_landed_are_seen_at_once(run):
    # nine stages armed in a ring of six: slots 0..2 are in their second phase
    all_landed, took, early = run("""
        for (int s = 0; s < 6; ++s) phases[64 + 8 * s] = s < 3 ? 2 : 1;
        unsigned long long t0 = now;
        const bool r = wait_armed_stages(64, 6, 9);
        const unsigned long long t = now - t0;
        phases[64 + 8] = 1;                                   // slot 1's second copy is still out
        printf("%d %llu %d", (int)r, t, (int)wait_armed_stages(64, 6, 9));
    """)
    assert (all_landed, early) == (1, 0)
    assert took < 10_000


@pytest.mark.parametrize("rank", [0, 1])
def test_a_partial_step_is_awaited_on_its_own_barrier(run, rank):
    """Seven steps in a ring of five, the last one partial (slot 1, whose own barrier was
    used once before).  Its full barrier never completes when the fixer gave up; its copies
    are seen on its own barrier, by either CTA."""
    code = """
        const uint32_t full = 64, part = 512;
        for (int s = 0; s < 5; ++s) phases[full + 8 * s] = s < 1 ? 2 : 1;     // slot 1: fixer gave up
        phases[part + 8] = %d;
        unsigned long long t0 = now;
        // one use before, one now: an even count
        const bool r = wait_armed_pair_stages(full, part, 5, 7, 2u, 0u, %d);
        printf("%%d %%llu", (int)r, now - t0);
    """
    landed, took = run(code % (2, rank))
    # the peer cannot see the whole steps' copies, and says so
    assert landed == (rank == 0)
    assert took < 10_000
    landed, took = run(code % (1, rank))
    assert landed == 0
    assert 0.9 * limit() < took < 1.1 * limit()


@pytest.mark.parametrize("stages", [5, 6])
@pytest.mark.parametrize("steps", [0, 1, 4, 5, 6, 7, 29, 30, 31])
def test_the_ring_is_drained_to_its_last_commit(run, stages, steps):
    """Every stage filled `steps` times in turn: with all commits in, the drain passes at
    once; with any one of them outstanding it does not."""
    verdicts = run("""
        volatile int stop = 0;
        const int stages = %d, steps = %d;
        auto set = [&](int missing) {
            for (int s = 0; s < stages; ++s) {
                const int uses = steps / stages + (s < steps %% stages ? 1 : 0);
                phases[64 + 8 * s] = uses - (s == missing ? 1 : 0);
            }
        };
        const int stage = steps %% stages;
        const uint32_t ph = (steps / stages) & 1;
        set(-1);
        const unsigned long long t0 = now;
        printf("%%d %%d", (int)drain_ring(64, stages, stage, ph, &stop), (int)(now - t0 < 10000));
        for (int s = 0; s < stages && s < steps; ++s) {
            set(s);
            stop = 0;
            printf(" %%d", (int)drain_ring(64, stages, stage, ph, &stop));
        }
    """ % (stages, steps))
    assert verdicts[:2] == [1, 1]
    assert verdicts[2:] == [0] * min(steps, stages)
