"""The pair kernels' output boxes (csrc/far_pair16.cuh: pair_begin_box, pair_store_box), compiled for the CPU and run
against a copy engine that reads a box as late as it may: when the warp waits for its copies.

A warp puts each of a call's outputs together in one box of shared memory, one output after the other.  An output on
16-byte boundaries leaves by such a copy, any other by the warp itself, so whatever follows a copy has to wait for it,
however it leaves itself: the outputs of a call may differ in alignment.  And such a copy writes whole units of 16 bytes."""
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
enum { FAR_OK = 0, FAR_F32 = 0, FAR_BF16 = 2 };
struct CUtensorMap { uint16_t* p; int64_t ld, rows, cols; };
static int tma_type(int) { return 0; }
static int encode_box(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int, int, int) {
  *map = CUtensorMap{(uint16_t*)p, ld, rows, cols};
  return FAR_OK;
}
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
        if (c.y + r >= c.map->rows || c.x + k / 8 * 8 >= c.map->cols) continue;  // whole units of 16 bytes
        uint16_t v;
        memcpy(&v, shared + r * 128 + (((k >> 3) ^ (r & 7)) * 16) + (k & 7) * 2, 2);
        c.map->p[(c.y + r) * c.map->ld + c.x + k] = v;
      }
  pending.clear();
}
%s
// arguments: the outputs' places (values behind a 16-byte boundary), columns, 1 where an output's tiles all come before the
// next output's
int main(int argc, char** argv) {
  const int n = argc - 3, cols = atoi(argv[n + 1]), by_output = atoi(argv[n + 2]), tiles = 3, boxes = (cols + 63) / 64;
  const int rows = 3 * 32 - 5, ld = (cols + 7) / 8 * 8 + 8;
  struct Output { alignas(16) uint16_t mem[96 * 256]; };
  std::vector<Output> memory(n);
  std::vector<PairOut> out(n);
  std::vector<CUtensorMap> map(n);
  for (int j = 0; j < n; ++j) {
    std::fill(memory[j].mem, memory[j].mem + 96 * 256, 0xffff);
    if (pair_output(&out[j], &map[j], memory[j].mem + atoi(argv[1 + j]), rows, cols, ld, FAR_BF16) != FAR_OK) return 2;
  }
  auto value = [](int j, int r, int c) { return (uint16_t)(j * 20000 + r * 192 + c); };
  for (int i = 0; i < tiles * n; ++i)
    for (int b = 0; b < boxes; ++b) {
      const int j = by_output ? i / tiles : i %% n, t = by_output ? i %% tiles : i / n;
      for (int lane = 0; lane < 32; ++lane) pair_begin_box(lane);
      for (int r = 0; r < 32; ++r)
        for (int c = 0; c < 64; ++c) {
          const uint16_t v = value(j, 32 * t + r, 64 * b + c);
          memcpy(shared + r * 128 + (((c >> 3) ^ (r & 7)) * 16) + (c & 7) * 2, &v, 2);
        }
      for (int lane = 0; lane < 32; ++lane) pair_store_box(out[j], &map[j], shared, lane, 32 * t, 64 * b);
    }
  bulk_wait_read();
  for (int j = 0; j < n; ++j)
    for (int i = 0, first = atoi(argv[1 + j]); i < 96 * 256; ++i) {
      const int r = (i - first) / ld, c = (i - first) %% ld;
      const bool inside = i >= first && r < rows && c < cols;
      if (memory[j].mem[i] != (inside ? value(j, r, c) : 0xffff)) {
        printf("output %%d, row %%d, column %%d: %%d\n", j, r, c, memory[j].mem[i]);
        return 1;
      }
    }
  printf("%%d copies\n", taken);
  return 0;
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    text = open(os.path.join(CSRC, "far_pair16.cuh")).read()
    source = (text[text.index("struct PairOut {"):text.index("// E: kAMn")]
              + text[text.index("inline int pair_output("):text.index("template <class E>\ncudaError_t launch_pair16")])
    folder = tmp_path_factory.mktemp("box")
    path, program = folder / "box.cpp", folder / "box"
    path.write_text(HARNESS % source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-o", str(program), str(path)], check=True, capture_output=True)
    return str(program)


@pytest.mark.parametrize("by_output", [False, True])
@pytest.mark.parametrize("cols", [3, 56, 61, 64, 125, 192])
@pytest.mark.parametrize("places", list(itertools.product((0, 2, 1), repeat=3)) + list(itertools.product((0, 2, 1), repeat=2)))
def test_each_output_has_its_own_values(model, places, cols, by_output):
    """gated_ffn's three outputs a tile in turn, and the tiles of dw_gate and then dw_up that one pair works on: outputs
    on 16, 4 and 2 bytes, rows that end inside 16 bytes, and nothing written around them."""
    r = subprocess.run([model, *map(str, places), str(cols), str(int(by_output))], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    copied = (cols + 63) // 64 if cols % 8 == 0 else cols // 64  # boxes a row of tiles
    assert r.stdout.split() == [str(3 * copied * places.count(0)), "copies"]
