"""Rules on the kernels' waits that no GPU test can show without hanging a GPU when
they are broken, checked on the sources (CPU).

A role is a brace block of a kernel; the checks look at what encloses a wait and
at which barriers a kernel's commits reach.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_routing_router_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", text)


def kernels(name):
    """(name, body) of every __global__ function of a file."""
    text, out = source(name), []
    for m in re.finditer(r"__global__[^{;]*?(\w+)\s*\((?:[^(){};]|\([^(){};]*\))*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        out.append((m.group(1), text[m.end():i - 1]))
    return out


def test_the_parser_finds_the_kernels():
    assert {n for n, _ in kernels("gemm.cu")} >= {"grouped_gemm_kernel", "grouped_gemm_pair_kernel"}
    assert "grad_gemm_pair_kernel" in {n for n, _ in kernels("gemm_grad.cu")}


@pytest.mark.parametrize("name", ["gemm.cu", "gemm_grad.cu"])
def test_multicast_commits_are_awaited_before_a_cta_exits(name):
    """A commit to a stage barrier of both CTAs of a pair arrives in the peer without
    the peer's having to wait for it; each producer drains its ring before it leaves,
    or the arrival may land in the shared memory of the next CTA on that SM."""
    seen = 0
    for kernel, body in kernels(name):
        if not re.search(r"tc_commit_pair_mc\(smem_u32\(&ctl->empty\[", body):
            continue
        seen += 1
        producer = body[body.index("if (warp == 0) {"):body.index("} else if (warp == 1) {")]
        assert "drain_ring(smem_u32(&ctl->empty[0])" in producer, kernel
        assert "rank" not in re.search(r"if \(([^\n]*)\) ok = drain_ring", producer).group(1), kernel   # both CTAs
    assert seen == 1


def enclosing(body, pos):
    """The texts before the open braces that enclose `pos`, outermost first."""
    heads, last = [], 0
    for i, c in enumerate(body[:pos]):
        if c == "{":
            heads.append(body[last:i])
        elif c == "}":
            heads.pop()
        if c in "{};":
            last = i + 1
    return heads


SINGLE = re.compile(r"\b(?:lane|tid) == 0\b")
KERNELS_THAT_WAIT = ["gemm.cu", "gemm_decode.cu", "decode_ffn.cu", "gemm_grad.cu"]


@pytest.mark.parametrize("name", KERNELS_THAT_WAIT)
def test_a_warp_gives_up_a_wait_as_a_whole(name):
    """Lanes that decide apart whether a wait ran out part for good: some reach the
    closing barrier, the rest a warp-wide instruction, and both wait for ever.  A wait
    outside a block of one thread has to be the warp's, or its verdict `landed` has to be
    voted on before anything else of the warp and before anyone leaves."""
    waits = 0
    for kernel, body in kernels(name):
        for m in re.finditer(r"\b(mbar_wait_bounded|mbar_wait_cluster|drain_ring|wait_armed_stages)\(", body):
            waits += 1
            if any(SINGLE.search(h) for h in enclosing(body, m.start())):
                continue
            statement = body[:m.start()].rsplit(";", 1)[-1].rsplit("{", 1)[-1].rsplit("}", 1)[-1]
            assert re.match(r"\s*(const )?(bool )?landed = ", statement), \
                f"{kernel}: {body[m.start():m.start() + 70]!r}"
            between, vote, _ = body[m.start():].partition("if (!__all_sync(0xffffffffu, landed)) { ok = false; break; }")
            assert vote, kernel
            assert not re.search(r"\b(break|continue|return|goto)\b|_sync\b|tmem_|__syncwarp|__syncthreads", between), kernel
    assert waits > 4


def test_a_warp_that_gave_up_still_meets_named_barriers():
    """The epilogue warps of the CTA-pair kernel meet at named barriers in a swapped
    SwiGLU tile.  A warp that gave up its wait and left would strand the others there:
    it stays in the tile loop and meets as many of them."""
    met = 0
    for kernel, body in kernels("gemm.cu"):
        at = [m.start() for m in re.finditer(r"epi_bar_sync\(\);", body)]
        if not at:
            continue
        met += 1
        dead = [i for i in at if any(h.strip() == "if (!live)" for h in enclosing(body, i))]
        assert len(dead) == len(at) - len(dead) == 2, kernel
        give_up = body.index("kSiteGemmEpilogue")
        assert body[give_up:].split("}")[1].split() == ["live", "=", "false;"], kernel
    assert met == 1
