"""What the int8 product and the gated feed-forward block ask of their kernel sources, checked on the sources: the two
kernels that start beside the one ahead, and what a CTA waits for before it leaves."""
import os
import re

import pytest
from test_dependent_launch_rules import SOURCES, bodies

ALL = {kernel: body for text in SOURCES.values() for kernel, body in bodies(text)}
FILES = {name: dict(bodies(SOURCES[name])) for name in ("far_int8.cu", "far_ffn.cu", "far_pair16.cuh")}


def test_kernels_ahead_of_early_readers_wait_before_they_let_them_start():
    """pair8_kernel reads wt, and the weights' gradients start beside dx, before they wait: sound only if the kernel ahead
    (widen_kernel; dx's few_kernel, pair16_kernel or plain_product_kernel) waits before it lets dependents go."""
    for name in ("widen_kernel", "few_kernel", "plain_product_kernel"):
        body = next(f[name] for f in FILES.values() if name in f)
        assert body.index("pdl_wait()") < body.index("pdl_launch_dependents()"), name
    body = FILES["far_pair16.cuh"]["pair16_kernel"]
    beside, usual = body.split("if constexpr (E::kBeside) {")[1].split("} else {")[:2]
    assert "pdl_wait" not in beside and usual.index("pdl_wait()") < usual.index("pdl_launch_dependents()")


def test_early_readers_wait_for_the_kernel_ahead_before_they_end():
    body = FILES["far_pair16.cuh"]["pair16_kernel"]
    assert "if constexpr (E::kBeside) pdl_wait();" in body[body.rindex("cluster_sync()"):]
    body = FILES["far_int8.cu"]["pair8_kernel"]
    producer = body[body.index("warp == 2 && lane == 0"):]
    assert producer.index("pdl_wait()") < producer.index("tma_load_3d_pair")  # x is what the kernel ahead writes
    epilogue = body[body.index("setmaxnreg.inc"):]
    assert epilogue.index("pdl_wait()") < epilogue.index("p.ws[")
    assert body.index("if (p.packed) pdl_wait()") < body.index("tma_load_2d")  # wt's copy, where there is one, is too


@pytest.mark.parametrize("name,waits", [
    ("few_kernel", [r"mbar_wait\(empty0 \+ 8 \* \(j % S::stages\)", r"mbar_wait\(done"]),
    ("pair16_kernel", [r"mbar_wait\(empty0 \+ 8 \* \(j % kPair16Stages\)"]),
    ("few8_kernel", [r"mbar_wait\(wide_empty0 \+ 8 \* \(j & 1u\)"]),
    ("pair8_kernel", [r"mbar_wait\(a_empty0 \+ 8 \* \(j % w\.aslots\)", r"mbar_wait\(x_empty0 \+ 8 \* \(j % w\.xslots\)"])])
def test_commits_of_the_last_blocks_are_awaited(name, waits):
    """A commit that arrives after its CTA (or its peer) has left would fall on another CTA's shared memory."""
    body = ALL[name]
    for w in waits:
        assert re.search(w, body), (name, w)


def test_register_shares():
    """setmaxnreg moves registers between warpgroups of what the CTA was launched with: 640 threads at 96."""
    body = FILES["far_int8.cu"]["pair8_kernel"]
    shares = [int(v) for v in re.findall(r"setmaxnreg\.(?:dec|inc)\.sync\.aligned\.u32 (\d+)", body)]
    assert shares == [56, 72, 136]
    assert 128 * shares[0] + 256 * shares[1] + 256 * shares[2] <= 640 * 96
    log = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_residual_gb300", "_build", "ptxas.log")
    if os.path.exists(log):
        text = open(log).read()
        used = re.search(r"pair8_kernel.*?Used (\d+) registers", text, re.S)
        assert used and int(used.group(1)) == 96
