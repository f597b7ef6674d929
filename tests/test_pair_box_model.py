"""The pair kernels' output boxes (csrc/far_pair16.cuh: pair_begin_box, pair_store_box), compiled for the CPU and run
against a copy engine that reads a box as late as it may: when the warp waits for its copies.

A warp puts each of a call's outputs together in one box of shared memory, one output after the other.  An output on
16-byte boundaries leaves by such a copy, any other by the warp itself, so whatever follows a copy has to wait for it,
however it leaves itself: the outputs of a call may differ in alignment."""
import itertools
import os
import subprocess

import pytest
from test_dependent_launch_rules import CSRC

HARNESS = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>
#define __device__
#define __forceinline__ inline
using std::min;
struct CUtensorMap { uint16_t* p; int64_t ld; int rows, cols; };
alignas(128) static unsigned char shared[4096];
struct Copy { const CUtensorMap* map; int x, y; };
static std::vector<Copy> pending;
static int taken = 0;
static uint32_t smem_addr(const void* p) { return (uint32_t)((const unsigned char*)p - shared); }
static void fence_async_shared() {}
static void __syncwarp() {}  // (the lanes run one after the other, phase by phase)
static void bulk_commit() {}
static void tma_store_2d(const CUtensorMap* map, uint32_t, int x, int y) { pending.push_back({map, x, y}); ++taken; }
static void bulk_wait_read() {
  for (const Copy& c : pending)
    for (int r = 0; r < 32; ++r)
      for (int k = 0; k < 64; ++k) {
        if (c.y + r >= c.map->rows || c.x + k >= c.map->cols) continue;
        uint16_t v;
        memcpy(&v, shared + r * 128 + (((k >> 3) ^ (r & 7)) * 16) + (k & 7) * 2, 2);
        c.map->p[(c.y + r) * c.map->ld + c.x + k] = v;
      }
  pending.clear();
}
%s
// arguments: outputs, their alignments in bytes, then 1 where an output's tiles all come before the next output's
int main(int argc, char** argv) {
  const int n = atoi(argv[1]), by_output = atoi(argv[2 + n]), tiles = 3, rows = 3 * 32 - 5, cols = 61, ld = 72;
  std::vector<std::vector<uint16_t>> mem(n, std::vector<uint16_t>(rows * ld, 0xffff));
  std::vector<PairOut> out(n);
  std::vector<CUtensorMap> map(n);
  for (int j = 0; j < n; ++j) {
    out[j] = PairOut{};
    out[j].p = mem[j].data();
    out[j].ld = ld;
    out[j].rows = rows;
    out[j].cols = cols;
    out[j].align = atoi(argv[2 + j]);
    map[j] = CUtensorMap{mem[j].data(), ld, rows, cols};
  }
  auto value = [](int j, int r, int c) { return (uint16_t)(j * 10000 + r * 64 + c); };
  for (int i = 0; i < tiles * n; ++i) {
    const int j = by_output ? i / tiles : i %% n, t = by_output ? i %% tiles : i / n;
    for (int lane = 0; lane < 32; ++lane) pair_begin_box(lane);
    for (int r = 0; r < 32; ++r)
      for (int c = 0; c < 64; ++c) {
        const uint16_t v = value(j, 32 * t + r, c);
        memcpy(shared + r * 128 + (((c >> 3) ^ (r & 7)) * 16) + (c & 7) * 2, &v, 2);
      }
    for (int lane = 0; lane < 32; ++lane) pair_store_box(out[j], &map[j], shared, lane, 32 * t, 0);
  }
  bulk_wait_read();
  for (int j = 0; j < n; ++j)
    for (int r = 0; r < rows; ++r)
      for (int c = 0; c < ld; ++c)
        if (mem[j][r * ld + c] != (c < cols ? value(j, r, c) : 0xffff)) {
          printf("output %%d, row %%d, column %%d: %%d\n", j, r, c, mem[j][r * ld + c]);
          return 1;
        }
  printf("%%d copies\n", taken);
  return 0;
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    text = open(os.path.join(CSRC, "far_pair16.cuh")).read()
    source = text[text.index("struct PairOut {"):text.index("// E: kAMn")]
    folder = tmp_path_factory.mktemp("box")
    path, program = folder / "box.cpp", folder / "box"
    path.write_text(HARNESS % source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-o", str(program), str(path)], check=True, capture_output=True)
    return str(program)


def outcome(model, aligns, by_output):
    r = subprocess.run([model, str(len(aligns)), *map(str, aligns), str(int(by_output))], capture_output=True, text=True)
    return r.returncode, r.stdout.strip()


@pytest.mark.parametrize("by_output", [False, True])
@pytest.mark.parametrize("aligns", list(itertools.product((16, 4, 2), repeat=3)) + list(itertools.product((16, 4, 2), repeat=2)))
def test_no_output_takes_anothers_values(model, aligns, by_output):
    """gated_ffn's three outputs a tile in turn, and the tiles of dw_gate and then dw_up that one pair works on."""
    status, said = outcome(model, aligns, by_output)
    assert status == 0, said
    assert said == f"{3 * aligns.count(16)} copies"
