// The product of two FP8 E4M3 matrices with a binary32 scale for each 128 values along k
// (gemm_fp8_block):
//   out[i, j] = RNE( sum_b xs[i, b] ws[j, b] sum_{k in b} x[i, k] wt[j, k] ).
//
// The scales are arbitrary binary32 values, so the tensor cores sum one block of 128 at a
// time (four tcgen05.mma of 32 values) into TMEM, and the block's sums are scaled and added
// to the result in registers ("promoted").  Per block a tile's every accumulator is loaded
// from TMEM and takes one or two FMA-pipe operations while the tensor cores work on the next
// block in the other half of TMEM; the register tile is what limits the tile's size.
//
// pair_kernel  -- many rows: 256 x 256 tiles over CTA pairs, x's rows on the TMEM lanes.
// small_kernel -- few rows (a decode batch): wt's rows on the lanes, 16 to 64 rows of x as the
//                 columns, k split over a cluster of CTAs that add their sums through
//                 distributed shared memory.  Bound by reading wt once.
// plain_kernel -- any shape, stride and alignment: 64 x 64 tiles in binary32.
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "far.h"
#include "far_device.cuh"
#include "far_launch.h"
#include "far_params.h"
#include "far_region.h"
#include "far_tcgen05.cuh"
#include "far_tma.h"

namespace far {

cudaError_t ensure_smem_attribute(const void* func, size_t bytes);

namespace {

struct Gemm8Params {
  const unsigned char* x;
  const unsigned char* wt;
  const float* xs;
  const float* ws;
  void* out;
  int64_t ldx, ldw, ldo;  // elements
  int32_t M, N, K, KB;    // KB: blocks of 128 along k
  int32_t tile_scales;    // ws: one a 128 rows of wt (1) or one a row (0)
  int32_t out_dtype;
  int32_t out_align;      // bytes that out and its row stride are multiples of: 16, 4 or 2
  int32_t xs_vec, ws_vec; // rows of scales start on 16-byte boundaries
  int32_t tiles_m, tiles_n, num_tiles;  // pair_kernel
  unsigned int* status;
  uint64_t timeout_ns;
};

__device__ __forceinline__ float e4m3_value(unsigned char c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__device__ __forceinline__ void store_out(const Gemm8Params& p, int64_t row, int64_t col, float v) {
  const int64_t i = row * p.ldo + col;
  if (p.out_dtype == FAR_F32) static_cast<float*>(p.out)[i] = v;
  else if (p.out_dtype == FAR_F16) static_cast<__half*>(p.out)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
}

// A block's sum is 0 or of a magnitude between 2^-18 (two of the smallest codes) and 2^25 (128 x 448 x 448), and its
// term is to be right wherever the term itself lies in binary32's range, whatever the two scales.
// Multiplied by one scale and then by the other it is, if the first is 0 or within 2^-108 .. 2^103: that
// product is then a normal number.  Multiplied by the scales' product it is, if that is a normal number,
// or 0 because a scale is.  The kernels' loops take one of these ways; scales for which it fails, which
// no quantiser makes of values that a model has, send a product through scaled().
__device__ __forceinline__ bool first_factor(float s) {
  const float m = fabsf(s);
  return m == 0.f || (m >= 0x1p-108f && m < 0x1p103f);
}
__device__ __forceinline__ bool one_factor(float a, float b) {
  const float m = fabsf(__fmul_rn(a, b));
  return (m >= 0x1p-126f && m <= 0x1.fffffep127f) || a == 0.f || b == 0.f;
}
// The factors that a sum is multiplied by one after the other: the scales' product and 1 where that is
// right; else the larger scale first.  (Product too small: the larger scale lies below 2^23, and where
// it lies below 2^-108 the term is below half of binary32's smallest number; too large: neither scale
// is below 1.  Infinite and NaN scales: the same as in any order.)
__device__ __forceinline__ float2 factors(float a, float b) {
  if (one_factor(a, b)) return make_float2(__fmul_rn(a, b), 1.f);
  return fabsf(a) > fabsf(b) ? make_float2(a, b) : make_float2(b, a);
}
__device__ __forceinline__ float scaled(float sum, float a, float b) {
  const float2 f = factors(a, b);
  return __fmul_rn(__fmul_rn(sum, f.x), f.y);
}

// 64 x 64 outputs a CTA of 256 threads, 4 x 4 a thread (16 apart), slices of 32 along k through
// shared memory as binary32.  Bound by the FMA pipe; there for the shapes TMA cannot read.
__global__ void __launch_bounds__(256) plain_kernel(const Gemm8Params p) {
  __shared__ float xs[32][65], ws[32][65];
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t tiles_n = ((int64_t)p.N + 63) / 64, tiles = tiles_n * (((int64_t)p.M + 63) / 64);
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t m0 = t / tiles_n * 64, n0 = t % tiles_n * 64;
    float acc[4][4] = {};
    for (int b = 0; b < p.KB; ++b) {
      float part[4][4] = {};
      for (int64_t k0 = (int64_t)b * kBlock; k0 < (int64_t)(b + 1) * kBlock && k0 < p.K; k0 += 32) {
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * 32; i += 256) {
          const int r = i >> 5, k = i & 31;
          const bool in = k0 + k < p.K;
          xs[k][r] = in && m0 + r < p.M ? e4m3_value(p.x[(m0 + r) * p.ldx + k0 + k]) : 0.f;
          ws[k][r] = in && n0 + r < p.N ? e4m3_value(p.wt[(n0 + r) * p.ldw + k0 + k]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float a[4], c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = xs[k][ty + 16 * i], c[i] = ws[k][tx + 16 * i];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[i][j] = __fmaf_rn(a[i], c[j], part[i][j]);
        }
      }
      float sx[4], sw[4];
      bool usual = true;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * i;
        sx[i] = m < p.M ? p.xs[m * p.KB + b] : 0.f;
        sw[i] = n < p.N ? p.ws[(p.tile_scales ? n / kBlock : n) * p.KB + b] : 0.f;
        usual = usual && first_factor(sx[i]);
      }
      if (usual) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(__fmul_rn(part[i][j], sx[i]), sw[j], acc[i][j]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = __fadd_rn(acc[i][j], scaled(part[i][j], sx[i], sw[j]));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < p.M && n < p.N) store_out(p, m, n, acc[i][j]);
      }
  }
}

__device__ __forceinline__ uint64_t pk_bits(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}

// The scales of blocks kb .. kb + 3 of one row of a [rows, KB] scale matrix (0 past the end, or
// without a row): consecutive in memory, one sector or two.
struct Scale4 {
  float v[4];
  // (volatile: the compiler would otherwise move the loads down to their use, four blocks of k
  // later, and their latency with them; plain, not ld.global.nc: the kernel ahead may write the
  // scales while this grid is already resident, so they are not read-only for its lifetime)
  __device__ __forceinline__ void load(const float* row, int kb, int KB, bool vec) {
    if (row == nullptr || kb >= KB) {
      v[0] = v[1] = v[2] = v[3] = 0.f;
    } else if (vec) {
      asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                   : "l"(row + kb));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = 0.f;
        if (kb + j < KB) asm volatile("ld.global.f32 %0, [%1];" : "=f"(v[j]) : "l"(row + kb + j));
      }
    }
  }
  __device__ __forceinline__ float at(int j) const {
    return j == 0 ? v[0] : j == 1 ? v[1] : j == 2 ? v[2] : v[3];
  }
};

// one scale, or 0 where `on` is false: without a branch, so that a lane's loads leave together (volatile
// and plain as Scale4's)
__device__ __forceinline__ float load_scale(const float* src, bool on) {
  float v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.f32 %0, [%1];\n\t}"
               : "=&f"(v)
               : "l"(src), "r"((int)on));
  return v;
}

// Words in shared memory behind a kernel's barriers: scales were met that its loop does not serve, so that its
// tiles are done once more with scaled(), after the loop and at no cost to it; and a role's wait ran out, so
// that nothing is done again.
constexpr int kRare = 0, kGaveUp = 1, kFlags = 2;

// The least (zeros aside) and the largest magnitude of scales, three operations each.
struct Extent {
  float least = 1.f, most = 0.f;
  __device__ __forceinline__ void add(float s) {
    const float m = fabsf(s);
    least = fminf(least, m == 0.f ? 1.f : m);
    most = fmaxf(most, m);
  }
  // n scales at p, a warp's lanes side by side
  __device__ __forceinline__ void add(const float* p, int64_t n, int lane) {
#pragma unroll 8
    for (int64_t i = lane; i < n; i += 32) add(p[i]);
  }
  // of all lanes (the bits of magnitudes are in their order)
  __device__ __forceinline__ void join() {
    least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(least)));
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
  }
};

// A ring of column scales in shared memory: slot kb % kScaleSlots holds the scales of block kb for
// the tile's columns.  One warp fills it four blocks at a time (their values are neighbours
// in memory), the epilogue warps read it.
constexpr int kScaleSlots = 8;
template <int COLS>
__device__ __forceinline__ bool fill_scales(float* ring, uint32_t full0, uint32_t empty0, const float* scales,
                                            int64_t first, int64_t rows, int kb0, int kb1, int KB, uint32_t g0, int lane,
                                            const Gemm8Params& p) {
  constexpr int PER = (COLS + 31) / 32;
  for (int kb = kb0; kb < kb1; kb += 4) {
    float v[PER][4];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = lane + 32 * i;
      const bool in = c < COLS && first + c < rows;
      const float* src = scales + (first + c) * KB;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = load_scale(src + kb + j, in && kb + j < kb1);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kb + j >= kb1) break;
      const uint32_t g = g0 + (uint32_t)(kb + j - kb0), slot = g % kScaleSlots;
      if (!mbar_wait(empty0 + 8 * slot, ((g / kScaleSlots) & 1u) ^ 1u, p.timeout_ns, p.status)) return false;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (lane + 32 * i < COLS) ring[slot * COLS + lane + 32 * i] = v[i][j];
      __syncwarp();
      if (lane == 0) mbar_arrive(full0 + 8 * slot);
    }
  }
  return true;
}

// A warp's outputs leave in boxes of 32 rows x 128 bytes, put together in shared memory (16-byte
// units of a row permuted by XOR with row % 8: the 128-byte swizzle).  Where out's rows allow, TMA
// copies a box out while the next tile's blocks arrive, leaving out what lies past the edges;
// else the warp stores it row by row, 32 neighbouring words (or half words) at a time.
__device__ __forceinline__ void begin_box(const Gemm8Params& p, int lane) {
  if (p.out_align >= 16) {
    if (lane == 0) bulk_wait_read();  // the copy of the last box has read it
    __syncwarp();
  }
}
__device__ __forceinline__ void store_box(const Gemm8Params& p, const CUtensorMap* map, unsigned char* box, int lane,
                                          int64_t row, int64_t col) {
  if (p.out_align >= 16) {
    fence_async_shared();
    __syncwarp();
    if (lane == 0 && col < p.N && row < p.M) {
      tma_store_2d(map, smem_addr(box), (int)col, (int)row);
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  const int rows = (int)min((int64_t)32, p.M - row);
#pragma unroll 8
  for (int r = 0; r < rows; ++r) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(box + r * 128 + (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4);
    if (p.out_dtype == FAR_F32) {
      if (col + lane < p.N) static_cast<uint32_t*>(p.out)[(row + r) * p.ldo + col + lane] = v;
    } else {
      const int64_t n = col + 2 * lane;
      uint16_t* o = static_cast<uint16_t*>(p.out) + (row + r) * p.ldo + n;
      if (p.out_align >= 4 && n + 1 < p.N) {
        *reinterpret_cast<uint32_t*>(o) = v;
      } else {
        if (n < p.N) o[0] = (uint16_t)v;
        if (n + 1 < p.N) o[1] = (uint16_t)(v >> 16);
      }
    }
  }
  __syncwarp();  // before the next box
}

// ---------------------------------------------------------------------------
// pair_kernel: 256 x 256 output tiles over a cluster of 2.  Each CTA holds its 128 rows of x
// and half of the tile's rows of wt (up to 128) per block of k; one thread of the even CTA issues
// tcgen05.mma.cta_group::2 over both, each CTA's TMEM receiving the sums of its 128 rows.
//   warp 0      TMA producer (both CTAs), a ring of 4 or 5 blocks of k running across tiles
//   warp 1      MMA issuer (even CTA); allocates TMEM: two halves of 256 columns
//   warps 2, 3  where wt is scaled by rows: column and row factors, some blocks of k ahead
//   warp 2 (wt scaled by tiles) or the odd CTA's warp 1 (by rows) looks for scales that the epilogue's loop does
//               not serve (kRare); where it finds one, the pair does its tiles once more, with scaled()
//   warps 4-    epilogue: warp w the TMEM lanes 32 (w % 4) .. and 128 or (row-scaled wt) 64 of the
//               columns, so that a thread keeps 128 or 64 outputs in registers
// The registers a thread: 384 threads are launched at 168; warps 0-3 give theirs up to 72 and
// the 8 epilogue warps take 216 (128 x 72 + 256 x 216 = 384 x 168).  With 16 epilogue warps
// 640 at 96, then 56 and 104 (128 x 56 + 512 x 104 = 60416 of 61440).
// The last column of tiles runs at the width that is left (a multiple of 32).
// Measured: 16384 x 8192 x 8192, tile-scaled wt, bf16 out 775 to 865 us with the codes' power draw
// (2.5 to 2.8 PFLOP/s; the same pipeline without promotion 3.7 on 8192^3), 5120 x 2056 x 4112
// row-scaled 84 us, 8192^3 656 us.  With a scale that sends the pairs through their second pass: 4096^3 152 us
// from 66 (tiles), 443 from 100 (rows).  ptxas spills 140 bytes of the row-scaled kernel (220 read back),
// in which role it does not say.  Bound by the MMA (750 cycles a block beside the epilogue's TMEM loads,
// 512 alone) and by the two hand-overs of a TMEM half, of which a block hides only the other half's
// MMA: two halves of 256 columns are all of TMEM.  Row-scaled also by two FMA-pipe operations
// an output and block, and TMEM loads in fragments, which run at half rate (32 cycles for 32
// columns against 16.5).
// ---------------------------------------------------------------------------
constexpr uint32_t kPairABytes = 128 * kBlock, kPairBBytes = 128 * kBlock;
// A slot of the scale ring (wt scaled by rows): the 128 rows' factors, then for each 64 columns
// 4 groups of 16 column factors, 20 apart (a fragment's thread reads one group, and the four
// groups lie on different banks).
constexpr int kRowFactors = 128, kColGroup = 20, kSlotFloats = kRowFactors + 4 * 4 * kColGroup;
template <bool COLS>
struct PairShape8 {
  static constexpr int warps = COLS ? 16 : 8;  // of the epilogue
  static constexpr int threads = 128 + 32 * warps;
  static constexpr int stages = COLS ? 4 : 5;
  static constexpr uint32_t ring = stages * (kPairABytes + kPairBBytes);
  static constexpr uint32_t out = warps * 4096;  // a box of 32 rows x 128 bytes of outputs a warp
  static constexpr uint32_t scales = COLS ? kScaleSlots * kSlotFloats * 4 : 0;
  static constexpr int bars = 2 * stages + 4 + 2 * kScaleSlots;
  static constexpr size_t smem = ring + out + scales + bars * 8 + 16 + 1024;
};
constexpr int kPairGroup = 8;  // tile rows that are walked together, so that CTAs at work share panels in L2

struct PairTile {
  int64_t row0, col0;
  int cols;  // of the tile, 32 .. 256
};
__device__ __forceinline__ PairTile pair_tile(const Gemm8Params& p, int t) {
  const int per = kPairGroup * p.tiles_n, g = t / per, first = g * kPairGroup;
  const int gm = min(p.tiles_m - first, kPairGroup), r = t - g * per;
  PairTile w;
  w.row0 = (int64_t)(first + r % gm) * 256;
  w.col0 = (int64_t)(r / gm) * 256;
  const int64_t left = p.N - w.col0;
  w.cols = left >= 256 ? 256 : (int)((left + 31) / 32 * 32);
  return w;
}

template <bool COLS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairShape8<COLS>::threads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ CUtensorMap map_out, const Gemm8Params p) {
  using S = PairShape8<COLS>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);  // the same offset in both CTAs
  const uint32_t sbase = smem_addr(smem);
  const uint32_t a_base = sbase, b_base = sbase + S::stages * kPairABytes;
  float* scales = reinterpret_cast<float*>(smem + S::ring + S::out);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::ring + S::out + S::scales);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + S::bars);
  volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t full0 = smem_addr(&bars[0]), empty0 = smem_addr(&bars[S::stages]);
  const uint32_t acc_full0 = smem_addr(&bars[2 * S::stages]), acc_empty0 = acc_full0 + 16;
  const uint32_t sc_full0 = acc_full0 + 32, sc_empty0 = sc_full0 + 8 * kScaleSlots;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_cta_rank();
  const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kFlags; ++i) flags[i] = 0;
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(full0 + 8 * s, 1);   // even CTA: its producer's arrive + both CTAs' bytes
      mbar_init(empty0 + 8 * s, 1);  // one multicast commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full0 + 8 * a, 1);    // one multicast commit
      mbar_init(acc_empty0 + 8 * a, 2 * S::warps);  // even CTA: the epilogue warps of both CTAs
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(sc_full0 + 8 * s, 2);  // the two scale warps
      mbar_init(sc_empty0 + 8 * s, S::warps);  // this CTA's epilogue warps
    }
    fence_barrier_init();
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_w);
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
  // Not before this CTA has its TMEM columns: a dependent kernel of any library that allocated them first
  // and then waited for this grid would leave the allocation here, which has no time limit, waiting for it.
  pdl_launch_dependents();
  pdl_wait();

  // a flag of both CTAs
  auto tell = [&](int flag) {
    const uint32_t at = smem_addr(const_cast<int*>(&flags[flag]));
    for (uint32_t r = 0; r < 2; ++r)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_cta(at, r)), "r"(1) : "memory");
  };
  // The end of a role's pass over the pair's tiles: all of the pair are done with theirs (no CTA leaves while
  // its peer may still signal its barriers).  Is there to be another?
  auto again = [&]() {
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    return flags[kRare] != 0 && flags[kGaveUp] == 0;
  };
  // blocks of k behind the barriers before the second pass
  const uint32_t done = pair < p.num_tiles ? (uint32_t)((p.num_tiles - pair + pairs - 1) / pairs) * (uint32_t)p.KB : 0u;

  if (warp < 4) {
    if constexpr (COLS) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    auto role = [&](auto second) {
      constexpr bool SECOND = decltype(second)::value;
      bool ok = true;
      uint32_t g = SECOND ? done : 0u;
      if (warp == 0 && lane == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        for (int t = pair; ok && t < p.num_tiles; t += pairs) {
          const PairTile w = pair_tile(p, t);
          const int x_row = (int)w.row0 + (int)rank * 128, w_row = (int)w.col0 + (int)rank * (w.cols / 2);
          for (int kb = 0; kb < p.KB; ++kb, ++g) {
            const uint32_t s = g % S::stages;
            if (!mbar_wait(empty0 + 8 * s, ((g / S::stages) & 1u) ^ 1u, p.timeout_ns, p.status)) {
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2 * (kPairABytes + kPairBBytes));
            const uint32_t full_even = map_to_cta(full0 + 8 * s, 0);
            tma_load_2d_pair(a_base + s * kPairABytes, &map_x, kb * kBlock, x_row, full_even);
            tma_load_2d_pair(b_base + s * kPairBBytes, &map_w, kb * kBlock, w_row, full_even);
          }
        }
        // Before exit the pair's copies of the last blocks must have landed, and the commits that free their
        // slots, which the MMA issuer multicasts last, must have arrived in both CTAs.
        const uint32_t last = g > (uint32_t)S::stages ? g - S::stages : 0u;
        if (rank == 0)
          for (uint32_t j = last; j < g; ++j)
            mbar_wait(full0 + 8 * (j % S::stages), (j / S::stages) & 1u, p.timeout_ns, p.status);
        for (uint32_t j = last; ok && j < g; ++j)
          ok = mbar_wait(empty0 + 8 * (j % S::stages), (j / S::stages) & 1u, p.timeout_ns, p.status);
      } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer (even CTA) ----------------
        // One warp issues everything, so what it does for a block of k is kept short: ring
        // positions by counters, descriptors by adding to those of the first slot (16-byte units)
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t a0 = sw128_kmajor_desc(a_base), b0 = sw128_kmajor_desc(b_base);
        uint32_t s = g % S::stages, s_phase = g / S::stages & 1u, acc = g & 1u, acc_phase = (g >> 1 & 1u) ^ 1u;
        for (int t = pair; ok && t < p.num_tiles; t += pairs) {
          const uint32_t idesc = umma_idesc_e4m3_f32(256, pair_tile(p, t).cols);
          for (int kb = 0; kb < p.KB; ++kb) {
            if (!mbar_wait(acc_empty0 + 8 * acc, acc_phase, p.timeout_ns, p.status) ||
                !mbar_wait(full0 + 8 * s, s_phase, p.timeout_ns, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t a = a0 + s * (kPairABytes >> 4), b = b0 + s * (kPairBBytes >> 4);
            const uint32_t d = tm + acc * 256;
            if (leader) {
              umma_e4m3_pair<false>(d, a, b, idesc);
              umma_e4m3_pair<true>(d, a + 2, b + 2, idesc);
              umma_e4m3_pair<true>(d, a + 4, b + 4, idesc);
              umma_e4m3_pair<true>(d, a + 6, b + 6, idesc);
              umma_commit_pair(acc_full0 + 8 * acc, 0x3);  // the block's sums are there
              umma_commit_pair(empty0 + 8 * s, 0x3);       // both CTAs' slots are free once read
            }
            __syncwarp();
            acc ^= 1;
            acc_phase ^= acc == 0;
            if (++s == S::stages) {
              s = 0;
              s_phase ^= 1;
            }
          }
        }
      } else if (COLS && warp == 3) {
        // ---------------- row factors ----------------
        for (int t = pair; ok && t < p.num_tiles; t += pairs) {
          const int64_t row0 = pair_tile(p, t).row0 + (int)rank * 128 + lane;
          for (int kb = 0; ok && kb < p.KB; kb += 4) {
            Scale4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i].load(row0 + 32 * i < p.M ? p.xs + (row0 + 32 * i) * p.KB : nullptr, kb, p.KB, p.xs_vec);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (kb + j >= p.KB) break;
              const uint32_t slot = g % kScaleSlots;
              if (!mbar_wait(sc_empty0 + 8 * slot, ((g / kScaleSlots) & 1u) ^ 1u, p.timeout_ns, p.status)) {
                ok = false;
                break;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) scales[slot * kSlotFloats + lane + 32 * i] = x[i].v[j];
              __syncwarp();
              if (lane == 0) mbar_arrive(sc_full0 + 8 * slot);
              ++g;
            }
          }
        }
      } else if (COLS && warp == 2) {
        // ---------------- column factors: a lane's 4 neighbouring columns of either half ----------------
        for (int t = pair; ok && t < p.num_tiles; t += pairs) {
          const int64_t col0 = pair_tile(p, t).col0 + 4 * lane;
          for (int kb = 0; ok && kb < p.KB; kb += 4) {
            Scale4 x[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int64_t c = col0 + 128 * h + i;
                x[h][i].load(c < p.N ? p.ws + c * p.KB : nullptr, kb, p.KB, p.ws_vec);
              }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (kb + j >= p.KB) break;
              const uint32_t slot = g % kScaleSlots;
              if (!mbar_wait(sc_empty0 + 8 * slot, ((g / kScaleSlots) & 1u) ^ 1u, p.timeout_ns, p.status)) {
                ok = false;
                break;
              }
              // column 4 lane + i of a half: pair (4 lane + i) % 8 / 2 of 8 columns
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float* dst = scales + slot * kSlotFloats + kRowFactors + (2 * h + (lane >> 4)) * 4 * kColGroup + 2 * ((lane & 15) >> 1);
#pragma unroll
                for (int i = 0; i < 4; i += 2)
                  *reinterpret_cast<float2*>(dst + ((lane & 1) * 2 + i / 2) * kColGroup) = make_float2(x[h][i].v[j], x[h][i + 1].v[j]);
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(sc_full0 + 8 * slot);
              ++g;
            }
          }
        }
      } else if (!SECOND && warp == 1 + !COLS) {
        // ---------------- are there scales that the epilogue's loop does not serve? ----------------
        // (The odd CTA's MMA warp looks at the column factors; where wt is scaled by tiles, warp 2 at the products.)
        for (int t = pair; t < p.num_tiles; t += pairs) {
          const PairTile w = pair_tile(p, t);
          if constexpr (COLS) {
            Extent all;
            all.add(p.ws + w.col0 * p.KB, (min((int64_t)p.N, w.col0 + 256) - w.col0) * p.KB, lane);
            if (!(all.least >= 0x1p-108f && all.most < 0x1p103f)) tell(kRare);
          } else {
            const int64_t row0 = w.row0 + (int)rank * 128, rows = min((int64_t)p.M, row0 + 128) - row0;
            const int64_t tile0 = w.col0 / kBlock, tiles = min(((int64_t)p.N + kBlock - 1) / kBlock, tile0 + 2) - tile0;
            if (rows <= 0) continue;
            Extent x, f;
            x.add(p.xs + row0 * p.KB, rows * p.KB, lane);
            f.add(p.ws + tile0 * p.KB, tiles * p.KB, lane);
            x.join();
            f.join();
            if (one_factor(x.least, f.least) && one_factor(x.most, f.most)) continue;  // and all between
            bool odd = false;
            for (int64_t h = tile0; h < tile0 + tiles; ++h)
              for (int kb = lane; kb < p.KB; kb += 32) {
                const float b = p.ws[h * p.KB + kb];
#pragma unroll 8
                for (int64_t r = row0; r < row0 + rows; ++r) odd |= !one_factor(p.xs[r * p.KB + kb], b);
              }
            if (odd) tell(kRare);
          }
        }
      }
      if (!ok) tell(kGaveUp);
    };
    role(std::false_type{});
    if (again()) {
      role(std::true_type{});
      again();
    }
  } else {
    // ---------------- epilogue ----------------
    if constexpr (COLS) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    constexpr int WIDE = COLS ? 64 : 128;  // columns a warp
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * WIDE);
    const uint32_t acc_empty_even = map_to_cta(acc_empty0, 0);
    unsigned char* box = smem + S::ring + (warp - 4) * 4096;
    auto role = [&](auto second) {
      constexpr bool SECOND = decltype(second)::value;
      uint32_t g = SECOND ? done : 0u;
      bool ok = true;
      if constexpr (COLS) {
        // A thread keeps rows t, t + 8, t + 16, t + 24 of its warp's 32 (t = lane / 4) and the columns
        // 8 i + 2 q, 8 i + 2 q + 1 (q = lane % 4) of its 64: 4 row factors and 16 column factors for its
        // 64 outputs.  (8192^3 with both sides scaled by rows: a row of 128 columns a thread, each
        // column factor read by every lane of every warp, 799 us: shared memory's bandwidth is what
        // the MMA's operands already take; fragments of 128 columns on 8 warps 730.)
        const int t4 = lane >> 2, q = lane & 3;
        const float* row_factors = scales + quarter * 32 + t4;
        const float* col_factors = scales + kRowFactors + (part * 4 + q) * kColGroup;
        for (int t = pair; ok && t < p.num_tiles; t += pairs) {
          const PairTile w = pair_tile(p, t);
          const int64_t row = w.row0 + (int)rank * 128 + quarter * 32;  // the warp's first
          const int64_t col = w.col0 + part * WIDE;
          const int mine = w.cols - part * WIDE;  // columns of this warp (may be none)
          float acc[64];
#pragma unroll
          for (int i = 0; i < 64; ++i) acc[i] = 0.f;
          if constexpr (SECOND) {
#pragma unroll 1
            for (int kb = 0; kb < p.KB; ++kb, ++g) {
              const uint32_t buf = g & 1u, slot = g % kScaleSlots;
              if (!mbar_wait(sc_full0 + 8 * slot, (g / kScaleSlots) & 1u, p.timeout_ns, p.status) ||
                  !mbar_wait(acc_full0 + 8 * buf, (g >> 1) & 1u, p.timeout_ns, p.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t r[16];
                tmem_ld_frag_sync(lanes + buf * 256 + 16 * c, r);
                const float4 f = reinterpret_cast<const float4*>(col_factors + slot * kSlotFloats)[c];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const float sr = row_factors[slot * kSlotFloats + 8 * u];
                  const int o = 8 * (u >> 1) + 2 * (u & 1);
                  float* a = &acc[16 * c + o];
                  a[0] = __fadd_rn(a[0], scaled(__uint_as_float(r[o]), f.x, sr));
                  a[1] = __fadd_rn(a[1], scaled(__uint_as_float(r[o + 1]), f.y, sr));
                  a[4] = __fadd_rn(a[4], scaled(__uint_as_float(r[o + 4]), f.z, sr));
                  a[5] = __fadd_rn(a[5], scaled(__uint_as_float(r[o + 5]), f.w, sr));
                }
              }
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive_remote(acc_empty_even + 8 * buf);
                mbar_arrive(sc_empty0 + 8 * slot);
              }
            }
          } else {
#pragma unroll 1
            for (int kb = 0; kb < p.KB; ++kb, ++g) {
              const uint32_t buf = g & 1u, slot = g % kScaleSlots;
              if (!mbar_wait(sc_full0 + 8 * slot, (g / kScaleSlots) & 1u, p.timeout_ns, p.status)) {
                ok = false;
                break;
              }
              // Every trip to shared memory takes ~300 cycles here, behind the MMA's operands: the factors
              // are read before the sums are waited for, the column factors two chunks ahead.
              const float* rf = row_factors + slot * kSlotFloats;
              const float4* cf = reinterpret_cast<const float4*>(col_factors + slot * kSlotFloats);
              float sr[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) sr[u] = rf[8 * u];
              float4 f = cf[0], f1 = cf[1];
              if (!mbar_wait(acc_full0 + 8 * buf, (g >> 1) & 1u, p.timeout_ns, p.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
              // All 64 columns always: those past a narrow tile's hold what nobody stores.  (The other
              // warps of this SM quarter add while this one loads.)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t r[16];
                tmem_ld_frag_sync(lanes + buf * 256 + 16 * c, r);
                if (c == 3) {  // all read: this warp's share of the buffer is free
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive_remote(acc_empty_even + 8 * buf);
                }
                const float4 f2 = c < 2 ? cf[c + 2] : f1;
#pragma unroll
                for (int u = 0; u < 4; ++u) {  // row t + 8 u
                  const int o = 8 * (u >> 1) + 2 * (u & 1);
                  float* a = &acc[16 * c + o];
                  a[0] = __fmaf_rn(__fmul_rn(__uint_as_float(r[o]), f.x), sr[u], a[0]);
                  a[1] = __fmaf_rn(__fmul_rn(__uint_as_float(r[o + 1]), f.y), sr[u], a[1]);
                  a[4] = __fmaf_rn(__fmul_rn(__uint_as_float(r[o + 4]), f.z), sr[u], a[4]);
                  a[5] = __fmaf_rn(__fmul_rn(__uint_as_float(r[o + 5]), f.w), sr[u], a[5]);
                }
                f = f1;
                f1 = f2;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(sc_empty0 + 8 * slot);
            }
          }
          if (!ok) break;
          const bool f32 = p.out_dtype == FAR_F32;
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 16 columns
            if (mine <= 16 * c) break;
            if (c == 0 || (f32 && c == 2)) begin_box(p, lane);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float* a = &acc[16 * c + 8 * (u >> 1) + 2 * (u & 1) + 4 * i];
                unsigned char* line = box + (t4 + 8 * u) * 128;  // row t4 + 8 u: its units are permuted by t4
                if (f32) {
                  *reinterpret_cast<float2*>(line + (((4 * (c & 1) + 2 * i + (q >> 1)) ^ t4) * 16) + (q & 1) * 8) = make_float2(a[0], a[1]);
                } else {
                  const uint32_t v = p.out_dtype == FAR_F16 ? narrow2<FAR_F16>(a[0], a[1]) : narrow2<FAR_BF16>(a[0], a[1]);
                  *reinterpret_cast<uint32_t*>(line + (((2 * c + i) ^ t4) * 16) + q * 4) = v;
                }
              }
            if (c == 3 || (f32 && c == 1) || mine <= 16 * (c + 1))
              store_box(p, &map_out, box, lane, row, col + (f32 ? 32 * (c / 2) : 0));
          }
        }
      } else {
        // Scaled by tiles: a thread keeps one row's 128 columns, its factors (xs times ws) in registers.
        for (int t = pair; ok && t < p.num_tiles; t += pairs) {
          const PairTile w = pair_tile(p, t);
          const int64_t row = w.row0 + (int)rank * 128 + quarter * 32 + lane;
          const int64_t col = w.col0 + part * WIDE;
          const int mine = w.cols - part * WIDE;  // columns of this warp (may be none)
          const float* xrow = row < p.M ? p.xs + row * p.KB : nullptr;
          const float* wrow = col < p.N ? p.ws + col / kBlock * p.KB : nullptr;
          float acc[128];
#pragma unroll
          for (int i = 0; i < 128; ++i) acc[i] = 0.f;
          if constexpr (SECOND) {
#pragma unroll 1
            for (int kb = 0; kb < p.KB; ++kb, ++g) {
              const uint32_t buf = g & 1u;
              const float2 two = factors(xrow ? xrow[kb] : 0.f, wrow ? wrow[kb] : 0.f);
              if (!mbar_wait(acc_full0 + 8 * buf, (g >> 1) & 1u, p.timeout_ns, p.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                uint32_t r[16];
                tmem_ld16(lanes + buf * 256 + 16 * c, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  acc[16 * c + i] = __fmaf_rn(__fmul_rn(__uint_as_float(r[i]), two.x), two.y, acc[16 * c + i]);
              }
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_remote(acc_empty_even + 8 * buf);
            }
          } else {
            Scale4 xn, wn;
            xn.load(xrow, 0, p.KB, p.xs_vec);
            wn.load(wrow, 0, p.KB, p.ws_vec);
            for (int kb4 = 0; ok && kb4 < p.KB; kb4 += 4) {
              Scale4 sc;
#pragma unroll
              for (int j = 0; j < 4; ++j) sc.v[j] = __fmul_rn(xn.v[j], wn.v[j]);
              xn.load(xrow, kb4 + 4, p.KB, p.xs_vec);  // the next four blocks', while these are worked on
              wn.load(wrow, kb4 + 4, p.KB, p.ws_vec);
#pragma unroll 1
              for (int j = 0; j < 4 && kb4 + j < p.KB; ++j, ++g) {
                const uint32_t buf = g & 1u;
                const float sr = sc.at(j);
                if (!mbar_wait(acc_full0 + 8 * buf, (g >> 1) & 1u, p.timeout_ns, p.status)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                // All 128 columns always: those past a narrow tile's hold what nobody stores.  (The
                // other warp of this SM quarter adds while this one loads.)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  uint32_t r[32];
                  tmem_ld32_sync(lanes + buf * 256 + 32 * c, r);
                  if (c == 3) {  // all read: this warp's share of the buffer is free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(acc_empty_even + 8 * buf);
                  }
#pragma unroll
                  for (int i = 0; i < 32; ++i) acc[32 * c + i] = __fmaf_rn(__uint_as_float(r[i]), sr, acc[32 * c + i]);
                }
              }
            }
          }
          if (!ok) break;
          const bool f32 = p.out_dtype == FAR_F32;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (mine <= 32 * c) break;
            if (f32 || (c & 1) == 0) begin_box(p, lane);
            uint32_t v[32];
            if (f32) narrow<FAR_F32, 32>(acc + 32 * c, v);
            else if (p.out_dtype == FAR_F16) narrow<FAR_F16, 32>(acc + 32 * c, v);
            else narrow<FAR_BF16, 32>(acc + 32 * c, v);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              if (u < 4 || f32) {
                const int unit = (f32 || (c & 1) == 0 ? u : u + 4) ^ (lane & 7);
                *reinterpret_cast<uint4*>(box + lane * 128 + unit * 16) = make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
              }
            }
            if (f32 || (c & 1) == 1 || mine <= 32 * (c + 1))
              store_box(p, &map_out, box, lane, row - lane, col + (f32 ? 32 * c : 64 * (c / 2)));
          }
        }
      }
      if (lane == 0) bulk_wait_all();
      if (!ok) tell(kGaveUp);
    };
    role(std::false_type{});
    if (again()) {
      role(std::true_type{});
      again();
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// small_kernel: 128 rows of wt x NT rows of x a CTA, the blocks of k shared out over a cluster
// of gridDim's x dimension (CTA rank r takes blocks KB r / S .. KB (r + 1) / S - 1).
//   warp 0 TMA producer, 1 MMA issuer (and TMEM), 2 x's scales, 4-7 epilogue: a thread keeps the NT
//   sums of one row of wt.
// Then each CTA leaves its sums in its shared memory and adds up every S-th row of x over the
// cluster's CTAs, in the order of k.
// Scales of x that the loop does not serve send the CTA through small_again (64 x 4096 x 4096 2.2 ms from 8.8 us).
// Bound by reading wt: m = 4, 8192 x 8192 13.4 us (5.0 TB/s), 28672 x 4096 20.7 us (5.7 TB/s); the
// rest is the launch, the set-up and the sum over the cluster (about 3 us).  Two CTAs an SM with
// five blocks in flight each and as many CTAs as fit: 1 CTA an SM with 6 or 11 blocks 15.5 and
// 14.9 us, 8192 x 8192 shared out over 2 or 8 CTAs instead of 4 15.6 and 17.4.
// ---------------------------------------------------------------------------
constexpr int kSmallThreads = 256;
template <int NT>
struct SmallShape {
  static constexpr int ctas = 2;  // an SM
  static constexpr int bufs = 4;  // TMEM accumulators
  static constexpr uint32_t a_bytes = 128 * kBlock, b_bytes = NT * kBlock;
  static constexpr int stages = NT == 64 ? 4 : 5;
  static constexpr uint32_t ring = stages * (a_bytes + b_bytes);
  static constexpr uint32_t tmem_cols = bufs * NT < 32 ? 32 : bufs * NT;
  static constexpr int bars = 2 * stages + 2 * bufs + 2 * kScaleSlots;
  static constexpr size_t smem = ring + kScaleSlots * NT * 4 + bars * 8 + 16 + 1024;
  static_assert(NT * 128 * 4 <= ring, "the sums that the cluster adds up lie in the ring");
};

// small_kernel's tile over the CTA's blocks of k once more, on the FMA pipe and with scaled(): into the ring, or out
// where the CTA has all of k.  (Its place comes from the special registers again: what the kernel's loop
// keeps for it costs the loop registers, 3 to 5 % with 64 rows of x.)
template <int NT>
__device__ __forceinline__ void small_again(const Gemm8Params& p, float* sums) {
  int split, rank, y, z;
  asm volatile("mov.u32 %0, %%nctaid.x;\n\tmov.u32 %1, %%ctaid.x;\n\tmov.u32 %2, %%ctaid.y;\n\tmov.u32 %3, %%ctaid.z;"
               : "=r"(split), "=r"(rank), "=r"(y), "=r"(z));
  const int64_t n0 = (int64_t)y * 128, m0 = (int64_t)z * NT;
  const int kb0 = (int)((int64_t)p.KB * rank / split), kb1 = (int)((int64_t)p.KB * (rank + 1) / split);
  const int r = threadIdx.x & 127;
  const int64_t n = n0 + r;
  if (n >= p.N) return;
  for (int c0 = 4 * (int)(threadIdx.x >> 7); c0 < NT && m0 + c0 < p.M; c0 += 8) {
    const int cols = (int)min((int64_t)4, p.M - m0 - c0);
    float acc[4] = {};
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb) {
      float part[4] = {};
      const int64_t end = min((int64_t)p.K, ((int64_t)kb + 1) * kBlock);
#pragma unroll 1
      for (int64_t k = (int64_t)kb * kBlock; k < end; ++k) {
        const float w = e4m3_value(p.wt[n * p.ldw + k]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < cols) part[c] = __fmaf_rn(w, e4m3_value(p.x[(m0 + c0 + c) * p.ldx + k]), part[c]);
      }
      const float ws = p.ws[(p.tile_scales ? n / kBlock : n) * p.KB + kb];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < cols) acc[c] = __fadd_rn(acc[c], scaled(part[c], p.xs[(m0 + c0 + c) * p.KB + kb], ws));
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c >= cols) continue;
      if (split > 1) sums[(c0 + c) * 128 + r] = acc[c];
      else store_out(p, m0 + c0 + c, n, acc[c]);
    }
  }
}

template <int NT>
__global__ void __launch_bounds__(kSmallThreads, SmallShape<NT>::ctas)
    small_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ Gemm8Params p) {
  using S = SmallShape<NT>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);  // the same offset in every CTA
  const uint32_t a_base = smem_addr(smem), b_base = a_base + S::stages * S::a_bytes;
  float* scales = reinterpret_cast<float*>(smem + S::ring);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::ring + kScaleSlots * NT * 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + S::bars);
  volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t full0 = smem_addr(&bars[0]), empty0 = full0 + 8 * S::stages;
  const uint32_t acc_full0 = empty0 + 8 * S::stages, acc_empty0 = acc_full0 + 8 * S::bufs;
  const uint32_t sc_full0 = acc_empty0 + 8 * S::bufs, sc_empty0 = sc_full0 + 8 * kScaleSlots;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = (int)gridDim.x, rank = (int)blockIdx.x;  // the cluster spans gridDim.x
  const int64_t n0 = (int64_t)blockIdx.y * 128, m0 = (int64_t)blockIdx.z * NT;
  const int kb0 = (int)((int64_t)p.KB * rank / split), kb1 = (int)((int64_t)p.KB * (rank + 1) / split);

  // The ring's first load of wt starts for L2 while the CTA is set up and the kernel ahead drains
  // (m = 4, 8192 x 8192: 13.2 us against 13.8; 2048 x 8192: 6.7 against 7.3; the CTA's whole
  // share instead: 13.6, and 24.3 against 20.7 on 28672 x 4096).
  if (warp == 3 && lane == 0)
    for (int kb = kb0; kb < kb1 && kb < kb0 + S::stages; ++kb) tma_prefetch_2d(&map_w, kb * kBlock, (int)n0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kFlags; ++i) flags[i] = 0;
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < S::bufs; ++a) {
      mbar_init(acc_full0 + 8 * a, 1);
      mbar_init(acc_empty0 + 8 * a, 4);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(sc_full0 + 8 * s, 1);
      mbar_init(sc_empty0 + 8 * s, 4);
    }
    fence_barrier_init();
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_w);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), S::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();  // (not before the TMEM columns are this CTA's, as in pair_kernel)
  pdl_wait();

  bool ok = true;
  uint64_t acc[NT / 2];
  if (warp == 0) {
    if (lane == 0) {
      uint32_t g = 0;
      bool running = true;
      for (int kb = kb0; kb < kb1; ++kb, ++g) {
        const uint32_t s = g % S::stages;
        if (!mbar_wait(empty0 + 8 * s, ((g / S::stages) & 1u) ^ 1u, p.timeout_ns, p.status)) {
          running = false;
          break;
        }
        mbar_arrive_expect_tx(full0 + 8 * s, S::a_bytes + S::b_bytes);
        tma_load_2d(a_base + s * S::a_bytes, &map_w, kb * kBlock, (int)n0, full0 + 8 * s);
        tma_load_2d(b_base + s * S::b_bytes, &map_x, kb * kBlock, (int)m0, full0 + 8 * s);
      }
      // Before anything else lies there the last blocks must have landed and their slots been freed by the
      // MMA issuer's last commits (the barriers they arrive on go with the CTA).
      const uint32_t last = g > (uint32_t)S::stages ? g - S::stages : 0u;
      for (uint32_t j = last; j < g; ++j)
        mbar_wait(full0 + 8 * (j % S::stages), (j / S::stages) & 1u, p.timeout_ns, p.status);
      for (uint32_t j = last; running && j < g; ++j)
        running = mbar_wait(empty0 + 8 * (j % S::stages), (j / S::stages) & 1u, p.timeout_ns, p.status);
    }
  } else if (warp == 1) {
    constexpr uint32_t IDESC = umma_idesc_e4m3_f32(128, NT);
    const bool leader = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t a0 = sw128_kmajor_desc(a_base), x0 = sw128_kmajor_desc(b_base);
    uint32_t s = 0, s_phase = 0, b = 0, b_phase = 1;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(acc_empty0 + 8 * b, b_phase, p.timeout_ns, p.status) ||
          !mbar_wait(full0 + 8 * s, s_phase, p.timeout_ns, p.status))
        break;
      tc_fence_after();
      const uint64_t a = a0 + s * (S::a_bytes >> 4), x = x0 + s * (S::b_bytes >> 4);
      const uint32_t d = tm + b * NT;
      if (leader) {
        umma_e4m3<false>(d, a, x, IDESC);
        umma_e4m3<true>(d, a + 2, x + 2, IDESC);
        umma_e4m3<true>(d, a + 4, x + 4, IDESC);
        umma_e4m3<true>(d, a + 6, x + 6, IDESC);
        umma_commit(acc_full0 + 8 * b);
        umma_commit(empty0 + 8 * s);
      }
      __syncwarp();
      if (++s == S::stages) {
        s = 0;
        s_phase ^= 1;
      }
      if (++b == S::bufs) {
        b = 0;
        b_phase ^= 1;
      }
    }
  } else if (warp == 2) {
    fill_scales<NT>(scales, sc_full0, sc_empty0, p.xs, m0, p.M, kb0, kb1, p.KB, 0u, lane, p);
  } else if (warp == 3) {
    // are there scales of x that are no first_factor?
    Extent all;
    const int rows = (int)min((int64_t)NT, p.M - m0);
    const unsigned per = (unsigned)(kb1 - kb0);
    const float* first = p.xs + m0 * p.KB + kb0;
#pragma unroll 8
    for (unsigned i = lane; i < rows * per; i += 32) all.add(first[(int64_t)(i / per) * p.KB + i % per]);  // (64 x 2^24 at most)
    if (!(all.least >= 0x1p-108f && all.most < 0x1p103f)) flags[kRare] = 1;
  } else if (warp >= 4) {
    const int quarter = warp & 3;
    const int64_t n = n0 + quarter * 32 + lane;
    const float* wrow = n < p.N ? p.ws + (p.tile_scales ? n / kBlock : n) * p.KB : nullptr;
    Scale4 next;
    next.load(wrow, kb0, kb1, p.ws_vec && kb0 % 4 == 0);
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) acc[i] = 0ull;
    uint32_t g = 0;
    for (int kb4 = kb0; ok && kb4 < kb1; kb4 += 4) {
      const Scale4 sc = next;
      next.load(wrow, kb4 + 4, kb1, p.ws_vec && kb0 % 4 == 0);
#pragma unroll 1
      for (int j = 0; j < 4 && kb4 + j < kb1; ++j, ++g) {
        const uint32_t b = g % S::bufs, slot = g % kScaleSlots;
        const float sr = sc.at(j);
        const uint64_t s2 = pk(sr, sr);
        if (!mbar_wait(sc_full0 + 8 * slot, (g / kScaleSlots) & 1u, p.timeout_ns, p.status) ||
            !mbar_wait(acc_full0 + 8 * b, (g / S::bufs) & 1u, p.timeout_ns, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float4* cs = reinterpret_cast<const float4*>(scales + slot * NT);
        const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + b * NT;
        constexpr int W = NT >= 32 ? 32 : 16;  // columns a load
#pragma unroll
        for (int c = 0; c < NT; c += W) {
          uint32_t r[W];
          if constexpr (W == 32) tmem_ld32(src + c, r);
          else tmem_ld16(src + c, r);
          tmem_ld_wait(r);
          if (c + W == NT) {  // all read: the accumulator is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty0 + 8 * b);
          }
#pragma unroll
          for (int i = 0; i < W / 2; i += 2) {
            const float4 q = cs[(c + 2 * i) / 4];
            const int a = c / 2 + i;
            acc[a] = fma_x2(mul_x2(pk_bits(r[2 * i], r[2 * i + 1]), pk(q.x, q.y)), s2, acc[a]);
            acc[a + 1] = fma_x2(mul_x2(pk_bits(r[2 * i + 2], r[2 * i + 3]), pk(q.z, q.w)), s2, acc[a + 1]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_empty0 + 8 * slot);
      }
    }
    if (split == 1) {
      if (ok && n < p.N) {
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
          const float2 f = unpk(acc[i]);
          if (m0 + 2 * i < p.M) store_out(p, m0 + 2 * i, n, f.x);
          if (m0 + 2 * i + 1 < p.M) store_out(p, m0 + 2 * i + 1, n, f.y);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::tmem_cols);
  }
  // every copy has landed and every MMA has read: the ring now holds this CTA's sums [NT][128]
  float* sums = reinterpret_cast<float*>(smem);
  if (split > 1 && warp >= 4) {
    const int r = (int)threadIdx.x - 128;
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) {
      const float2 f = unpk(acc[i]);
      sums[(2 * i) * 128 + r] = f.x;
      sums[(2 * i + 1) * 128 + r] = f.y;
    }
  }
  if (flags[kRare]) {
    __syncthreads();
    small_again<NT>(p, sums);
  }
  if (split > 1) {
    cluster_sync();
    const int64_t n = n0 + (threadIdx.x & 127);
    const uint32_t mine = smem_addr(sums) + (threadIdx.x & 127) * 4;
    for (int c = rank + split * (int)(threadIdx.x >> 7); c < NT && m0 + c < p.M; c += 2 * split) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < split) {
          const uint32_t a = map_to_cta(mine + c * 512, q);
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[q]) : "r"(a) : "memory");
        }
      float s = v[0];
#pragma unroll
      for (int q = 1; q < 8; ++q)
        if (q < split) s = __fadd_rn(s, v[q]);
      if (n < p.N) store_out(p, m0 + c, n, s);
    }
    cluster_sync();  // no CTA leaves while another still reads its sums
  }
}

int validate_gemm8(const Gemm8Params& p, int64_t m, int64_t n, int64_t k, int wt_block) {
  if ((p.out_dtype != FAR_F32 && p.out_dtype != FAR_F16 && p.out_dtype != FAR_BF16) ||
      (wt_block != FAR_BLOCK_ROW && wt_block != FAR_BLOCK_TILE))
    return FAR_ERR_DTYPE;
  if (m < 0 || n < 0 || k < 0 || m > INT32_MAX || n > INT32_MAX || k > INT32_MAX) return FAR_ERR_SHAPE;
  const int64_t lim = int64_t(1) << 31;
  if (p.ldx < k || p.ldw < k || p.ldo < n || p.ldx > lim || p.ldw > lim || p.ldo > lim) return FAR_ERR_SHAPE;
  if (m == 0 || n == 0) return FAR_OK;
  if (!p.out || (k > 0 && (!p.x || !p.wt || !p.xs || !p.ws))) return FAR_ERR_NULL;
  const int64_t so = p.out_dtype == FAR_F32 ? 4 : 2;
  if ((uintptr_t)p.out % so || ((uintptr_t)p.xs & 3) || ((uintptr_t)p.ws & 3)) return FAR_ERR_SHAPE;
  const Region O = region(p.out, m, n * so, p.ldo * so);
  if (k > 0) {
    const int64_t kb = (k + kBlock - 1) / kBlock;
    const Region rd[4] = {region(p.x, m, k, p.ldx), region(p.wt, n, k, p.ldw), region(p.xs, 1, m * kb * 4, 0),
                          region(p.ws, 1, (wt_block == FAR_BLOCK_TILE ? (n + kBlock - 1) / kBlock : n) * kb * 4, 0)};
    for (const Region& r : rd)
      if (regions_overlap(O, r)) return FAR_ERR_ALIAS;
  }
  return FAR_OK;
}

// a [rows, cols] matrix moved in boxes of box_rows x box_cols (128 bytes), 128-byte swizzled;
// elements out of range read as zero and are not written
int encode_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t row_bytes, int box_cols,
               int box_rows, CUtensorMapDataType type) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  const int st = get_encoder(&enc);
  if (st != FAR_OK) return st;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FAR_OK : FAR_ERR_CUDA;
}
int encode_codes(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int64_t ld, int box_rows) {
  return encode_map(map, base, rows, K, ld, kBlock, box_rows, CU_TENSOR_MAP_DATA_TYPE_UINT8);
}

struct Gemm8Plan {
  int kind;   // 0 plain, 1 pairs, 2 small
  int nt;     // small: rows of x a CTA
  int split;  // small: CTAs that share a tile's k
};

Gemm8Plan plan_gemm8(const Gemm8Params& p, int sms) {
  Gemm8Plan g{0, 0, 0};
  const bool tma = p.K > 0 && p.ldx % 16 == 0 && p.ldw % 16 == 0 && (((uintptr_t)p.x | (uintptr_t)p.wt) & 15) == 0;
  if (!tma) return g;
  const int64_t tiles_n = ((int64_t)p.N + 127) / 128;
  g.nt = p.M <= 16 ? 16 : p.M <= 32 ? 32 : 64;
  const int64_t tiles_m = ((int64_t)p.M + g.nt - 1) / g.nt, slots = 2ll * sms;
  // k is shared out while there are free places for it, not below two blocks a CTA
  g.split = 1;
  while (g.split < 8 && tiles_n * tiles_m * g.split * 2 <= slots && p.KB >= 4 * g.split) g.split *= 2;
  const int64_t pair_tiles = (((int64_t)p.M + 255) / 256) * (((int64_t)p.N + 255) / 256);
  // Estimated microseconds, fitted to both kernels on 44 shapes (4 to 768 rows, 128 x 384 to 8192 x
  // 8192): a launch, then waves of CTAs at so much a block of k.  E.g. (pair / small) 4 x 8192 x
  // 384 6.5 / 4.6; 64 x 2048 x 512 6.7 / 7.8, 64 x 8192 x 1024 8.9 / 7.7; 128 x 8192 x 8192 31.3 /
  // 27.0, 192 rows 31.4 / 44.1; 256 x 4096 x 4096 18.4 / 17.7, 384 rows 18.3 / 25.8.
  const int64_t waves = (tiles_n * tiles_m * g.split + slots - 1) / slots;
  const double depth = (double)waves * (double)((p.KB + g.split - 1) / g.split);
  const double small = g.nt == 16 ? 3.4 + 0.55 * depth : g.nt == 32 ? 4.5 + 0.6 * depth : 6.3 + 0.66 * depth;
  const int64_t pair_waves = (pair_tiles + sms / 2 - 1) / (sms / 2);
  const double pair = 4.8 + (p.tile_scales ? 0.42 : 0.8) * (double)pair_waves * p.KB;
  const bool fits = tiles_n <= 65535 && tiles_m <= 65535;
  g.kind = fits && small <= pair ? 2 : 1;
  if (g.kind == 1 && pair_tiles > INT32_MAX) g.kind = 0;
  return g;
}

template <int NT>
cudaError_t launch_small(const CUtensorMap& mx, const CUtensorMap& mw, const Gemm8Params& p, int split, cudaStream_t s) {
  const void* f = reinterpret_cast<const void*>(small_kernel<NT>);
  cudaError_t e = ensure_smem_attribute(f, SmallShape<NT>::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)split, (unsigned)((p.N + 127ll) / 128), (unsigned)(((int64_t)p.M + NT - 1) / NT));
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = SmallShape<NT>::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = far_get_programmatic_launch() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, small_kernel<NT>, mx, mw, p);
}

template <bool COLS>
cudaError_t launch_pair(const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& mo, const Gemm8Params& p, int sms,
                        cudaStream_t s) {
  cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(pair_kernel<COLS>), PairShape8<COLS>::smem);
  if (e != cudaSuccess) return e;
  const int pairs = p.num_tiles < sms / 2 ? p.num_tiles : sms / 2;
  return launch_k(pair_kernel<COLS>, dim3(2 * pairs), dim3(PairShape8<COLS>::threads), PairShape8<COLS>::smem, s, mx, mw, mo, p);
}

int run_gemm8(Gemm8Params& p, void* stream) {
  unsigned int* status = nullptr;
  int sms = 0;
  int st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.status = status;
  p.timeout_ns = kWaitTimeoutNs;
  const int64_t so = p.out_dtype == FAR_F32 ? 4 : 2;
  const uint64_t bits = (uint64_t)(uintptr_t)p.out | (uint64_t)(p.ldo * so);
  p.out_align = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
  p.xs_vec = p.KB % 4 == 0 && ((uintptr_t)p.xs & 15) == 0;
  p.ws_vec = p.KB % 4 == 0 && ((uintptr_t)p.ws & 15) == 0;
  const Gemm8Plan g = plan_gemm8(p, sms);
  cudaError_t e;
  if (g.kind == 0) {
    const int64_t tiles = (((int64_t)p.M + 63) / 64) * (((int64_t)p.N + 63) / 64), cap = (int64_t)sms * 8;
    e = launch_k(plain_kernel, dim3((unsigned)(tiles < cap ? tiles : cap)), dim3(256), 0, s, p);
  } else {
    CUtensorMap mx, mw;
    st = encode_codes(&mx, p.x, p.M, p.K, p.ldx, g.kind == 1 ? 128 : g.nt);
    if (st == FAR_OK) st = encode_codes(&mw, p.wt, p.N, p.K, p.ldw, 128);
    if (st != FAR_OK) return st;
    if (g.kind == 1) {
      p.tiles_m = (int32_t)(((int64_t)p.M + 255) / 256);
      p.tiles_n = (int32_t)(((int64_t)p.N + 255) / 256);
      p.num_tiles = p.tiles_m * p.tiles_n;
      CUtensorMap mo = mx;  // (not used where out's rows are not 16-byte aligned)
      if (p.out_align >= 16) {
        const int dt = p.out_dtype;
        st = encode_map(&mo, p.out, p.M, p.N, p.ldo * so, (int)(128 / so), 32,
                        dt == FAR_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                        : dt == FAR_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
        if (st != FAR_OK) return st;
      }
      e = p.tile_scales ? launch_pair<false>(mx, mw, mo, p, sms, s) : launch_pair<true>(mx, mw, mo, p, sms, s);
    } else {
      e = g.nt == 16   ? launch_small<16>(mx, mw, p, g.split, s)
          : g.nt == 32 ? launch_small<32>(mx, mw, p, g.split, s)
                       : launch_small<64>(mx, mw, p, g.split, s);
    }
  }
  return e == cudaSuccess ? FAR_OK : cuda_error_status(e);
}

}  // namespace

}  // namespace far

using namespace far;

extern "C" int gemm_fp8_block(const void* x, int64_t x_row_stride, const float* x_scale, const void* wt,
                              int64_t wt_row_stride, const float* wt_scale, int wt_block, void* out,
                              int64_t out_row_stride, int64_t m, int64_t n, int64_t k, int out_dtype, void* stream) {
  Gemm8Params p{};
  p.x = static_cast<const unsigned char*>(x);
  p.wt = static_cast<const unsigned char*>(wt);
  p.xs = x_scale;
  p.ws = wt_scale;
  p.out = out;
  p.ldx = x_row_stride;
  p.ldw = wt_row_stride;
  p.ldo = out_row_stride;
  p.out_dtype = out_dtype;
  p.tile_scales = wt_block == FAR_BLOCK_TILE;
  int st = validate_gemm8(p, m, n, k, wt_block);
  if (st != FAR_OK || m == 0 || n == 0) return st;
  p.M = (int32_t)m;
  p.N = (int32_t)n;
  p.K = (int32_t)k;
  p.KB = (int32_t)((k + kBlock - 1) / kBlock);
  return run_gemm8(p, stream);
}

extern "C" int far_plan_gemm_fp8_for_sms(int64_t m, int64_t n, int64_t k, int wt_block, int sms, int* out4) {
  if (!out4) return FAR_ERR_NULL;
  if (wt_block != FAR_BLOCK_ROW && wt_block != FAR_BLOCK_TILE) return FAR_ERR_DTYPE;
  if (m < 1 || n < 1 || k < 1 || m > INT32_MAX || n > INT32_MAX || k > INT32_MAX || sms < 2) return FAR_ERR_SHAPE;
  Gemm8Params p{};  // (16-byte aligned operands with rows of k codes)
  p.M = (int32_t)m;
  p.N = (int32_t)n;
  p.K = (int32_t)k;
  p.KB = (int32_t)((k + kBlock - 1) / kBlock);
  p.ldx = p.ldw = k;
  p.tile_scales = wt_block == FAR_BLOCK_TILE;
  const Gemm8Plan g = plan_gemm8(p, sms);
  int64_t ctas = 0;
  if (g.kind == 1) {
    const int64_t tiles = ((m + 255) / 256) * ((n + 255) / 256);
    ctas = 2 * (tiles < sms / 2 ? tiles : sms / 2);
  } else if (g.kind == 2) {
    ctas = g.split * ((n + 127) / 128) * ((m + g.nt - 1) / g.nt);
  } else {
    const int64_t tiles = ((m + 63) / 64) * ((n + 63) / 64);
    ctas = tiles < 8ll * sms ? tiles : 8ll * sms;
  }
  const int v[4] = {g.kind, g.kind == 2 ? g.nt : 0, g.kind == 2 ? g.split : 0, (int)(ctas < INT32_MAX ? ctas : INT32_MAX)};
  for (int i = 0; i < 4; ++i) out4[i] = v[i];
  return FAR_OK;
}
