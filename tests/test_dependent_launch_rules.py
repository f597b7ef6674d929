"""What programmatic dependent launches ask of the kernel sources, checked on the sources: such a kernel may be
resident while the kernel ahead of it still runs, and lets the kernel behind it become resident in turn."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_residual_gb300", "csrc")
SOURCES = {os.path.basename(f): open(f).read() for pattern in ("*.cu", "*.cuh", "*.h")
           for f in sorted(glob.glob(os.path.join(CSRC, pattern)))}


def code(text):
    """The source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", sorted(SOURCES))
def test_no_read_only_loads(name):
    """ld.global.nc and __ldg are for memory that nobody writes while the kernel lives, and a const __restrict__
    pointer lets the compiler choose them: what the kernel ahead writes is not that."""
    found = re.findall(r"ld\.global\.nc|__ldg|ld\.global\.[a-z:.]*nc|__restrict__", code(SOURCES[name]))
    assert not found, f"{name}: {found}"


def bodies(text):
    """(name, body) of each kernel."""
    text = code(text)
    for m in re.finditer(r"__global__[^;{]*?\b(\w*_kernel)\s*\([^{;]*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i]


def test_tensor_memory_is_taken_before_dependents_start():
    """tcgen05.alloc waits without a limit for free columns.  A dependent kernel let in before this one has its own could
    take them and then wait for this one to end: each CTA lets dependents go only behind its allocation and the
    barrier that publishes it."""
    met = []
    for name, text in SOURCES.items():
        for kernel, body in bodies(text):
            alloc, go = re.search(r"tmem_alloc\w*\(", body), body.find("pdl_launch_dependents")
            if alloc and go >= 0:
                met.append(kernel)
                between = body[alloc.end():go] if go > alloc.end() else ""
                assert "__syncthreads" in between, f"{name}: {kernel} lets dependents go before its TMEM columns are its own"
    assert {"pair_kernel", "small_kernel"} <= set(met)


def test_every_kernel_waits_before_it_lets_its_results_be_read():
    """A kernel that lets dependents go waits, itself, for the kernels ahead: else its dependents, which wait for it alone,
    could run beside those."""
    met = 0
    for name, text in SOURCES.items():
        for kernel, body in bodies(text):
            if "pdl_launch_dependents" in body:
                met += 1
                assert "pdl_wait()" in body, f"{name}: {kernel}"
    assert met >= 8


def test_commits_of_the_last_blocks_are_awaited():
    """gemm_fp8_block's MMA issuer commits a block's sums first and its ring slot last.  Nobody needs the last slots again,
    but a commit that arrives after its CTA (or its peer) has left would fall on another CTA's shared memory: the
    producer, behind its loop over the blocks, waits for the slots that the loop left occupied."""
    kernels = dict(bodies(SOURCES["far_gemm8.cu"]))
    for name in ("pair_kernel", "small_kernel"):
        body = kernels[name]
        assert body.count("umma_commit") == 2
        loop = body.index("mbar_arrive_expect_tx(full0")
        issuer = body.index("elect_one()")
        assert re.search(r"mbar_wait\(empty0 \+ 8 \* \(j % S::stages\), \(j / S::stages\) & 1u", body[loop:issuer]), name
