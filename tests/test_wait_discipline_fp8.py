"""The rules of test_wait_discipline.py on the kernels of the block-scaled FP8 path and of
grouped routing, and the order of a kernel's start, checked on the sources (CPU)."""
import re

import pytest

from test_wait_discipline import SINGLE, enclosing, kernels

GEMMS = [("gemm_fp8.cu", "fp8_gemm_kernel"), ("gemm_fp8_rows.cu", "fp8_rows_kernel")]
FILES = ["gemm_fp8.cu", "gemm_fp8_rows.cu", "dispatch_fp8.cu", "route_grouped.cu"]


def body_of(name, kernel):
    return dict(kernels(name))[kernel]


@pytest.mark.parametrize("name,kernel", GEMMS)
def test_waits_are_one_threads_or_the_whole_warps(name, kernel):
    """A wait of one lane sits in a block of one thread; a warp's wait, which votes, never
    does, nor in that of the lane that issues."""
    body, warps = body_of(name, kernel), 0
    for m in re.finditer(r"\b(mbar_wait\w*|mbar_try_wait|drain_ring|wait_armed_stages)\(", body):
        heads = enclosing(body, m.start())
        if m.group(1) == "mbar_wait_warp":
            warps += 1
            assert not any(SINGLE.search(h) or re.search(r"\bif \((leader|mine|any)\b", h) for h in heads), body[m.start():m.start() + 70]
        else:
            assert m.group(1) in ("mbar_wait_bounded", "wait_armed_stages"), m.group(1)
            assert any(SINGLE.search(h) for h in heads), body[m.start():m.start() + 70]
    assert warps == 5


@pytest.mark.parametrize("name,kernel", GEMMS)
def test_every_wait_that_ran_out_is_reported(name, kernel):
    """Producer, issuer, accumulators and the exchange of magnitudes raise the status."""
    body = body_of(name, kernel)
    sites = re.findall(r"raise_status\(p\.hdr, MOE_ERR_TIMEOUT\);\s*p\.hdr->timeout_site = (\w+);", body)
    assert sorted(sites) == ["kSiteGemmEpilogue", "kSiteGemmEpilogue", "kSiteGemmMma", "kSiteGemmProducer"]


@pytest.mark.parametrize("name,kernel", GEMMS)
def test_tensor_memory_is_allocated_before_a_dependent_kernel_may_start(name, kernel):
    """The next kernel's blocks would otherwise hold the columns that this one waits for."""
    body = body_of(name, kernel)
    assert body.index("tmem_alloc(") < body.index("__syncthreads();") < body.index("pdl_trigger();")


@pytest.mark.parametrize("name", FILES)
def test_no_kernel_triggers_before_its_wait(name):
    """When a kernel passes its programmatic wait every earlier one of the stream has ended,
    because each of them made its own wait before it let the next one start."""
    found = kernels(name)
    assert found
    for kernel, body in found:
        assert body.count("pdl_wait();") == body.count("pdl_trigger();") >= 1, kernel
        for m in re.finditer(r"pdl_trigger\(\);", body):
            assert re.search(r"pdl_wait\(\);\s*$", body[:m.start()]), kernel
