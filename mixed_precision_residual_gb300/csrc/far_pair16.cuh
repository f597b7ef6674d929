// Products of 16-bit matrices on the tensor cores of CTA pairs, with an epilogue of the caller's (what
// gated_ffn and its gradients share).
//
// pair16_kernel<E>: output tiles of 256 rows x up to 256 accumulator columns over a cluster of 2.
// Each CTA holds its 128 rows of A and half of the tile's rows of B for a slice of 64 of k; one
// thread of the even CTA issues tcgen05.mma.cta_group::2 over both, each CTA's TMEM receiving its
// 128 rows.  Persistent: pairs walk the tiles, those of the last, partial wave in halves where they fit
// one round.
//   warp 0     TMA producer (both CTAs): a ring of 6 slices running across tiles
//   warp 1     MMA issuer (even CTA); allocates TMEM: two accumulators of 256 columns
//   warps 2-9  epilogue, one accumulator behind: warp w the TMEM lanes 32 (w % 4) .. and one half of
//              the columns
// An operand may lie either way in memory, both read by 64 x 64 boxes with the 128-byte swizzle:
// k-major (rows of k values: a box is 64 rows x 128 bytes of k) or mn-major (rows of k are the
// memory's columns: a box is 64 values of k x 128 bytes of rows).  So no operand is transposed first.
// Every wait is bounded (FAR_ERR_TIMEOUT in the device error word on expiry).
// Bound by the MMA and, over a long run, the power it draws: gated_ffn of 8192 x 5120 x 13312 1214 to
// 1310 us on different GB300s (1.70 to 1.84 PFLOP/s, 91 to 98 % of the cuBLAS burst rate; in ncu the tensor
// cores are active 92 % of 4096 x 4096 x 8192, 86 % for dx and 92 % for dw there).  A half tile's slice takes 0.21 us where its MMA takes 0.13:
// 24 KB into an SM at 60 bytes a cycle.  (A producer thread for each operand: the same times.)
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "far.h"
#include "far_device.cuh"
#include "far_launch.h"
#include "far_params.h"
#include "far_tcgen05.cuh"
#include "far_tma.h"

namespace far {

cudaError_t ensure_smem_attribute(const void* func, size_t bytes);

constexpr int kPair16Stages = 6;
constexpr int kPair16Epilogue = 8;  // warps
constexpr int kPair16Threads = 64 + 32 * kPair16Epilogue;
constexpr uint32_t kPair16Slice = 128 * 64 * 2;  // bytes of a slice of A or B in a CTA
constexpr uint32_t kPair16Box = 64 * 64 * 2;
constexpr uint32_t kPair16Ring = kPair16Stages * 2 * kPair16Slice;
constexpr uint32_t kPair16Out = kPair16Epilogue * 4096;  // a box of 32 rows x 128 bytes of outputs a warp
constexpr int kPair16Bars = 2 * kPair16Stages + 4;
constexpr size_t kPair16Smem = kPair16Ring + kPair16Out + kPair16Bars * 8 + 16 + 1024;
static_assert(kPair16Smem <= kMaxDynamicSmem, "");

struct PairWalk {
  int32_t tiles_m, tiles_n, num_tiles;
  int32_t columns;  // of an output
  int32_t slices;   // of k, of one operand pair
  int32_t pairs;    // operand pairs summed (1 or 2)
  int32_t bf16;     // 0: f16
  unsigned int* status;
  uint64_t timeout_ns;
};

struct PairMaps {
  CUtensorMap a[2], b[2], out[3];
};

// The n-th item of a pair: tiles in groups of 8 tile rows, column by column inside a group, so that the
// pairs at work share panels in L2; whole tiles for the full waves, halves in the last one where they
// fit one round.  cols: 0 where nothing of a half is left.  False past the end of the pair's list.
struct PairItem {
  int tm, col0, cols;
};
template <int WIDTH, int STEP>
__device__ __forceinline__ bool pair_item(const PairWalk& p, int pair, int num_pairs, int n, PairItem& w) {
  const int waves = p.num_tiles / num_pairs, rest = p.num_tiles - waves * num_pairs;
  const bool halves = 2 * rest <= num_pairs;
  int t, first = 0, width = WIDTH;
  if (n < waves || (n == waves && !halves)) {
    t = pair + n * num_pairs;
    if (t >= p.num_tiles) return false;
  } else {
    if (n > waves || pair >= 2 * rest) return false;
    t = waves * num_pairs + (pair >> 1);
    width = WIDTH / 2;
    first = (pair & 1) * width;
  }
  const int per = 8 * p.tiles_n, g = t / per, r = t - g * per, gm = min(p.tiles_m - 8 * g, 8);
  w.tm = 8 * g + r % gm;
  w.col0 = r / gm * WIDTH + first;
  const int left = p.columns - w.col0;
  w.cols = left >= width ? width : left <= 0 ? 0 : (left + STEP - 1) / STEP * STEP;
  return true;
}

// What an epilogue works on: accumulator `acc` (0, 1) of this CTA's TMEM, its output rows and columns.
struct PairTileAt {
  PairItem item;
  int rank, quarter, part, lane;
  uint32_t tmem;           // of lane 32 quarter, column 0
  uint32_t acc_full, acc_empty_even;
  unsigned char* box;
  uint32_t uses;           // accumulators taken so far, by this warp
  // waits for the next accumulator, and gives its TMEM address; false when the wait ran out
  __device__ __forceinline__ bool next(const PairWalk& p, uint32_t& at) {
    const uint32_t acc = uses & 1u;
    if (!mbar_wait(acc_full + 8 * acc, (uses >> 1) & 1u, p.timeout_ns, p.status)) return false;
    tc_fence_after();
    at = tmem + acc * 256;
    return true;
  }
  // every value of it has been loaded
  __device__ __forceinline__ void release() {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_remote(acc_empty_even + 8 * (uses & 1u));
    ++uses;
  }
};

// A warp's outputs leave in boxes of 32 rows x 128 bytes, put together in shared memory (16-byte units of
// a row permuted by XOR with row % 8: the 128-byte swizzle): by TMA where out's rows allow, leaving out
// what lies past the edges, else by the warp, row by row.  A copy writes whole 16-byte units: in rows that end
// inside one the values behind their end became zeros (measured; rows past the last are left alone).  So the
// last box of such rows, too, is the warp's.
struct PairOut {
  uint16_t* p;
  int64_t ld;        // elements
  int32_t rows, cols;
  int32_t copied;    // boxes that start at a column below this leave by TMA
  int32_t align;     // bytes that p and its rows are multiples of: 16, 4 or 2
};
// The copy of the last box has read it, whichever output that was: the next one may leave the other way.
__device__ __forceinline__ void pair_begin_box(int lane) {
  if (lane == 0) bulk_wait_read();
  __syncwarp();
}
__device__ __forceinline__ void pair_store_box(const PairOut& o, const CUtensorMap* map, unsigned char* box, int lane,
                                               int64_t row, int64_t col) {
  if (col < o.copied) {
    fence_async_shared();
    __syncwarp();
    if (lane == 0 && row < o.rows) {
      tma_store_2d(map, smem_addr(box), (int)col, (int)row);
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  const int rows = (int)min((int64_t)32, o.rows - row);
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(box + r * 128 + (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4);
    const int64_t n = col + 2 * lane;
    uint16_t* d = o.p + (row + r) * o.ld + n;
    if (o.align >= 4 && n + 1 < o.cols) {
      *reinterpret_cast<uint32_t*>(d) = v;
    } else {
      if (n < o.cols) d[0] = (uint16_t)v;
      if (n + 1 < o.cols) d[1] = (uint16_t)(v >> 16);
    }
  }
  __syncwarp();  // before the next box
}

// E: kAMn, kBMn (the operand is mn-major), kSplit (B's halves are two operands' rows, gate and up: the
// even CTA loads b[0], the odd one b[1]), kDouble (the tile rows are those of two outputs, a[0]'s and then
// a[1]'s), kBeside (above), kWidth (output columns of a tile), kStep (to which a narrow tile is rounded), Params, and
// tile(): takes a tile's accumulator and stores it.
template <class E>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPair16Threads, 1)
    pair16_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairWalk p, const __grid_constant__ typename E::Params e) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);  // the same offset in both CTAs
  const uint32_t a_base = smem_addr(smem), b_base = a_base + kPair16Stages * kPair16Slice;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kPair16Ring + kPair16Out);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kPair16Bars);
  const uint32_t full0 = smem_addr(&bars[0]), empty0 = full0 + 8 * kPair16Stages;
  const uint32_t acc_full0 = empty0 + 8 * kPair16Stages, acc_empty0 = acc_full0 + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_cta_rank();
  const int pair = (int)(blockIdx.x >> 1), num_pairs = (int)(gridDim.x >> 1);
  const int total = p.slices * p.pairs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPair16Stages; ++s) {
      mbar_init(full0 + 8 * s, 1);   // even CTA: its producer's arrive + both CTAs' bytes
      mbar_init(empty0 + 8 * s, 1);  // one multicast commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full0 + 8 * a, 1);                     // one multicast commit
      mbar_init(acc_empty0 + 8 * a, 2 * kPair16Epilogue);  // even CTA: the epilogue warps of both CTAs
    }
    fence_barrier_init();
    tma_prefetch_map(&maps.a[0]);
    tma_prefetch_map(&maps.b[0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any remote arrive or copy
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (Dependents not before the TMEM columns are this CTA's: one that took them would wait for this grid.)
  // E::kBeside: the kernel ahead, of the same call, writes nothing that this one reads, and lets it start only
  // behind its own wait, when all work before it is done.  So this one runs beside its last CTAs, and
  // waits for it at the end, so that whoever waits for this grid has waited for both.
  if constexpr (E::kBeside) {
    pdl_launch_dependents();
  } else {
    pdl_wait();
    pdl_launch_dependents();
  }

  if (warp < 2) {
    PairItem w;
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer (both CTAs) ----------------
      uint32_t g = 0;
      bool ok = true;
      for (int n = 0; ok && pair_item<E::kWidth, E::kStep>(p, pair, num_pairs, n, w); ++n) {
        if (w.cols == 0) continue;
        const int half = E::kSplit ? w.cols : w.cols / 2;  // rows of B in this CTA
        const uint32_t b_bytes = half > 64 ? 2 * kPair16Box : kPair16Box;
        const int tiles = E::kDouble ? p.tiles_m / 2 : p.tiles_m;
        const int which = E::kDouble && w.tm >= tiles ? 1 : 0;
        const int a_row = (w.tm - which * tiles) * 256 + (int)rank * 128;
        const int b_row = E::kSplit ? w.col0 : w.col0 + (int)rank * half;
        for (int q = 0; ok && q < p.pairs; ++q) {
          const CUtensorMap* ma = &maps.a[E::kDouble ? which : q];
          const CUtensorMap* mb = &maps.b[E::kSplit ? (int)rank : q];
          for (int kb = 0; kb < p.slices; ++kb, ++g) {
            const uint32_t s = g % kPair16Stages;
            if (!mbar_wait(empty0 + 8 * s, ((g / kPair16Stages) & 1u) ^ 1u, p.timeout_ns, p.status)) {
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2 * (2 * kPair16Box + b_bytes));
            const uint32_t full_even = map_to_cta(full0 + 8 * s, 0);
            const uint32_t a = a_base + s * kPair16Slice, b = b_base + s * kPair16Slice;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if constexpr (E::kAMn) tma_load_2d_pair(a + h * kPair16Box, ma, a_row + 64 * h, kb * 64, full_even);
              else tma_load_2d_pair(a + h * kPair16Box, ma, kb * 64, a_row + 64 * h, full_even);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h * 64 >= half) break;
              if constexpr (E::kBMn) tma_load_2d_pair(b + h * kPair16Box, mb, b_row + 64 * h, kb * 64, full_even);
              else tma_load_2d_pair(b + h * kPair16Box, mb, kb * 64, b_row + 64 * h, full_even);
            }
          }
        }
      }
      // Before exit the pair's copies of the last slices must have landed, and the commits that free their
      // slots, which the MMA issuer multicasts, must have arrived in both CTAs.
      const uint32_t last = g > (uint32_t)kPair16Stages ? g - kPair16Stages : 0u;
      if (rank == 0)
        for (uint32_t j = last; j < g; ++j)
          mbar_wait(full0 + 8 * (j % kPair16Stages), (j / kPair16Stages) & 1u, p.timeout_ns, p.status);
      for (uint32_t j = last; ok && j < g; ++j)
        ok = mbar_wait(empty0 + 8 * (j % kPair16Stages), (j / kPair16Stages) & 1u, p.timeout_ns, p.status);
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA issuer (even CTA) ----------------
      const bool leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t a0 = E::kAMn ? sw128_mnmajor_desc(a_base, kPair16Box) : sw128_kmajor_desc(a_base);
      const uint64_t b0 = E::kBMn ? sw128_mnmajor_desc(b_base, kPair16Box) : sw128_kmajor_desc(b_base);
      // 16 of k further: 32 bytes along k-major rows, 16 mn-major rows of 128 bytes (16-byte units)
      constexpr uint32_t a_step = E::kAMn ? 128 : 2, b_step = E::kBMn ? 128 : 2;
      uint32_t s = 0, s_phase = 0, use = 0;
      bool ok = true;
      for (int n = 0; ok && pair_item<E::kWidth, E::kStep>(p, pair, num_pairs, n, w); ++n) {
        if (w.cols == 0) continue;
        const uint32_t idesc = umma_idesc_16(256, E::kSplit ? 2 * w.cols : w.cols, p.bf16, E::kAMn, E::kBMn);
        const uint32_t acc = use & 1u;
        if (!mbar_wait(acc_empty0 + 8 * acc, ((use >> 1) & 1u) ^ 1u, p.timeout_ns, p.status)) break;
        ++use;
        tc_fence_after();
        const uint32_t d = tm + acc * 256;
        for (int kb = 0; kb < total; ++kb) {
          if (!mbar_wait(full0 + 8 * s, s_phase, p.timeout_ns, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a = a0 + s * (kPair16Slice >> 4), b = b0 + s * (kPair16Slice >> 4);
          if (leader) {
            umma_f16_pair(d, a, b, idesc, kb != 0);
#pragma unroll
            for (int k = 1; k < 4; ++k) umma_f16_pair(d, a + k * a_step, b + k * b_step, idesc, 1);
            umma_commit_pair(empty0 + 8 * s, 0x3);  // both CTAs' slots are free once read
            if (kb == total - 1) umma_commit_pair(acc_full0 + 8 * acc, 0x3);
          }
          __syncwarp();
          if (++s == kPair16Stages) {
            s = 0;
            s_phase ^= 1;
          }
        }
      }
    }
  } else {
    // ---------------- epilogue ----------------
    PairTileAt at;
    at.rank = (int)rank;
    at.quarter = warp & 3;
    at.part = (warp - 2) >> 2;
    at.lane = lane;
    at.tmem = tmem + ((uint32_t)(at.quarter * 32) << 16);
    at.acc_full = acc_full0;
    at.acc_empty_even = map_to_cta(acc_empty0, 0);
    at.box = smem + kPair16Ring + (warp - 2) * 4096;
    at.uses = 0;
    for (int n = 0; pair_item<E::kWidth, E::kStep>(p, pair, num_pairs, n, at.item); ++n) {
      if (at.item.cols == 0) continue;
      if (!E::tile(at, maps, p, e)) break;
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal its barriers
  if constexpr (E::kBeside) pdl_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// a [rows, cols] matrix moved in boxes of box_rows x 128 bytes, 128-byte swizzled; elements out of range
// read as zero and are not written
inline int encode_box(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int elem, int box_rows,
                      CUtensorMapDataType type) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  const int st = get_encoder(&enc);
  if (st != FAR_OK) return st;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(ld * elem)};
  cuuint32_t box[2] = {(cuuint32_t)(128 / elem), (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FAR_OK : FAR_ERR_CUDA;
}
inline CUtensorMapDataType tma_type(int dt) {
  return dt == FAR_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}
// an operand [rows, cols] of 16-bit values, and whether TMA can read it
inline int encode_operand(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int dt) {
  return encode_box(map, base, rows, cols, ld, 2, 64, tma_type(dt));
}
inline bool tma_rows(const void* p, int64_t ld, int elem) { return ((uintptr_t)p & 15) == 0 && (ld * elem) % 16 == 0; }

// The limit of a kernel's waits, of which the longest is an epilogue's for a whole sum: a slice takes 0.25 us, so a sum
// over 2^30 values 4 s.
inline uint64_t wait_limit_ns(int64_t slices) { return kWaitTimeoutNs + (uint64_t)slices * 1000; }

// an output, and its tensor map where its rows allow one
inline int pair_output(PairOut* o, CUtensorMap* map, uint16_t* p, int64_t rows, int64_t cols, int64_t ld, int dt) {
  const uint64_t bits = (uint64_t)(uintptr_t)p | (uint64_t)(ld * 2);
  const int align = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
  const int64_t copied = align < 16 ? 0 : cols % 8 == 0 ? cols : cols / 64 * 64;
  *o = PairOut{p, ld, (int32_t)rows, (int32_t)cols, (int32_t)copied, align};
  return copied ? encode_box(map, p, rows, cols, ld, 2, 32, tma_type(dt)) : FAR_OK;
}

template <class E>
cudaError_t launch_pair16(const PairMaps& maps, const PairWalk& p, const typename E::Params& e, int sms, cudaStream_t s) {
  const cudaError_t st = ensure_smem_attribute(reinterpret_cast<const void*>(pair16_kernel<E>), kPair16Smem);
  if (st != cudaSuccess) return st;
  const int pairs = sms / 2;
  // a pair for each tile, or for each half where one round of halves takes them all
  const int64_t want = 2ll * p.num_tiles <= pairs ? 2ll * p.num_tiles : p.num_tiles < pairs ? p.num_tiles : pairs;
  return launch_k(pair16_kernel<E>, dim3((unsigned)(2 * want)), dim3(kPair16Threads), kPair16Smem, s, maps, p, e);
}

}  // namespace far
