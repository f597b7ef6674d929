"""The limit of the gated block's waits on the device, compiled for the CPU: an epilogue waits for a whole sum, and every sum that
the sizes allow has to end before its limit does."""
import os
import re
import subprocess

from test_dependent_launch_rules import CSRC, SOURCES

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
%s
%s
int main() {
  for (int shift : {0, 7, 20, 24, 26}) printf("%%llu\n", (unsigned long long)wait_limit_ns((int64_t)1 << shift));
}
"""


def test_a_sum_of_any_length_ends_before_its_limit(tmp_path):
    constant = re.search(r"constexpr uint64_t kWaitTimeoutNs[^;]*;", SOURCES["far_params.h"])[0]
    limit = re.search(r"inline uint64_t wait_limit_ns\(.*?\n?\}", open(os.path.join(CSRC, "far_pair16.cuh")).read())[0]
    (tmp_path / "limit.cpp").write_text(PROGRAM % (constant, limit))
    subprocess.run(["g++", "-std=c++17", "-o", str(tmp_path / "limit"), str(tmp_path / "limit.cpp")], check=True)
    out = [int(v) for v in subprocess.run([str(tmp_path / "limit")], capture_output=True, text=True, check=True).stdout.split()]
    for slices, ns in zip((1, 128, 2 ** 20, 2 ** 24, 2 ** 26), out):
        assert 2e9 + 600 * slices <= ns <= 2e9 + 2000 * slices  # a slice takes 0.25 to 0.36 us; and a wait stays bounded
    calls = re.findall(r"kWaitTimeoutNs|wait_limit_ns\([^;]*?\)", SOURCES["far_ffn.cu"])
    assert calls and all(c.startswith("wait_limit_ns") for c in calls), calls
