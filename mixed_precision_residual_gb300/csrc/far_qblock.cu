// A matrix quantised to FP8 E4M3 with a scale for each 128 values of a row, or for each
// 128 x 128 tile, as it stands or transposed (quant_block_fp8).
//
// Bound by HBM: each value is read once and its code written once.  So a block's maximum has
// to be known while its values still stand in registers:
//   rows_kernel  rows as they stand: a block is one 16-byte chunk in each of 16 (16-bit) or 32
//                (binary32) neighbouring lanes, its maximum a few shuffles;
//   tile_kernel  tiles, and anything transposed: a CTA holds a 128 x 128 tile in its
//                registers; maxima over columns or the tile meet in shared memory, and a
//                transposed tile's codes turn there.
#include <cuda_runtime.h>
#include <stdint.h>

#include "far.h"
#include "far_device.cuh"
#include "far_launch.h"
#include "far_params.h"
#include "far_region.h"

namespace far {

namespace {

constexpr int kThreads = 256;

struct QbParams {
  const char* x;
  unsigned char* q;
  float* scale;
  int64_t x_stride;  // bytes between rows of x
  int32_t rows, cols;
  int32_t segs;      // rows_kernel: warp tasks a row
};

// 16 bytes, or zeros where `on` is false.  Volatile and without a branch: a thread's loads then
// all leave before the first is waited for (a bf16 weight of 8192 x 8192 by tiles: 32.5 us, 6.2
// TB/s; with each load under its branch 42.6).  Plain loads, not read-only ones (ld.global.nc): x may be
// what the kernel ahead writes while this grid is already resident, so it is not read-only for the
// grid's lifetime.
__device__ __forceinline__ void load16(uint32_t (&w)[4], const void* src, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
      "mov.b32 %3, 0;\n\t@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3])
      : "l"(src), "r"((int)on));
}

// one value's bits (zeros where `on` is false), as load16
template <int DT> __device__ __forceinline__ uint32_t load_bits(const void* base, int64_t i, bool on) {
  uint32_t v;
  if constexpr (DT == FAR_F32) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.b32 %0, [%1];\n\t}"
                 : "=&r"(v)
                 : "l"(static_cast<const float*>(base) + i), "r"((int)on));
  } else {
    uint16_t h;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t@p ld.global.b16 %0, [%1];\n\t}"
                 : "=&h"(h)
                 : "l"(static_cast<const uint16_t*>(base) + i), "r"((int)on));
    v = h;
  }
  return v;
}
template <int DT> __device__ __forceinline__ float value_of(uint32_t bits) {
  if constexpr (DT == FAR_F32) return __uint_as_float(bits);
  else return widen2<DT>(bits).x;
}

__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
  return quantise4<kQuantFp8>(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv), __fmul_rn(v[2], inv), __fmul_rn(v[3], inv));
}
__device__ __forceinline__ unsigned char code1(float v, float inv) {
  return (unsigned char)(quantise4<kQuantFp8>(__fmul_rn(v, inv), 0.f, 0.f, 0.f) & 0xffu);
}

// a warp task: U x 32 neighbouring chunks of a row (VEC), or U blocks of 128 values
template <int ACT, bool VEC>
__global__ void __launch_bounds__(kThreads) rows_kernel(const QbParams p) {
  constexpr int V = 16 / dtype_size<ACT>::value;
  constexpr int LANES = kBlock / V;
  constexpr int U = 4;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nblk = (p.cols + kBlock - 1) / kBlock;
  const int64_t tasks = (int64_t)p.rows * p.segs;
  for (int64_t t = blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5); t < tasks;
       t += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t row = t / p.segs;
    const int seg = (int)(t - row * p.segs);
    const char* xr = p.x + row * p.x_stride;
    unsigned char* qr = p.q + row * p.cols;
    float* sr = p.scale + row * nblk;
    if constexpr (VEC) {
      const int chunks = p.cols / V;
      const int c0 = seg * (32 * U) + lane;
      uint32_t raw[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u) load16(raw[u], xr + (int64_t)(c0 + 32 * u) * 16, c0 + 32 * u < chunks);
      float m[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        m[u] = 0.f;
        if constexpr (ACT == FAR_F32) {
#pragma unroll
          for (int e = 0; e < V; ++e) m[u] = max_nan(m[u], fabsf(__uint_as_float(raw[u][e])));
        } else {
          uint32_t m2 = 0u;
#pragma unroll
          for (int e = 0; e < V / 2; ++e) m2 = habs_max2<ACT>(m2, raw[u][e]);
          const float2 h = widen2<ACT>(m2);
          m[u] = max_nan(h.x, h.y);
        }
        m[u] = lanes_max(m[u], LANES);
      }
      // The divisions of the U blocks, shared out: of a block's lanes, number u < 4 takes the u-th
      // factor, number 4 + u the u-th scale (each lane all eight: 38.0 us for 8192 x 8192 bf16)
      static_assert(U == 4, "");
      const int j = lane & (LANES - 1), pick = j & 3;
      const float mine = pick == 0 ? m[0] : pick == 1 ? m[1] : pick == 2 ? m[2] : m[3];
      const bool scales = j & 4;
      const float quotient = __fdiv_rn(scales ? mine : 448.0f, scales ? 448.0f : mine);
      const float val = mine < kBlockTiny ? 0.f : quotient;
      const int first = c0 - j + 32 * pick;  // the block's first chunk
      if (j >= 4 && j < 8 && first < chunks) sr[first / LANES] = val;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float inv = __shfl_sync(0xffffffffu, val, (lane - j) + u);
        const int c = c0 + 32 * u;
        if (c < chunks) {
          float f[V];
          widen<ACT, V>(raw[u], f);
          uint32_t qw[V / 4];
#pragma unroll
          for (int e = 0; e < V / 4; ++e) qw[e] = codes4(f + 4 * e, inv);
          if constexpr (V == 8) *reinterpret_cast<uint2*>(qr + (int64_t)c * 8) = make_uint2(qw[0], qw[1]);
          else *reinterpret_cast<uint32_t*>(qr + (int64_t)c * 4) = qw[0];
        }
      }
    } else {
      uint32_t bits[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t i = (int64_t)(seg * U + u) * kBlock + e * 32 + lane;
          bits[u][e] = load_bits<ACT>(xr, i, i < p.cols);
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t b = (int64_t)seg * U + u;
        if (b >= nblk) break;
        float m = 0.f, f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e] = value_of<ACT>(bits[u][e]);
          m = max_nan(m, fabsf(f[e]));
        }
        m = warp_max_allreduce(m);
        const float inv = block_inverse(m);
        if (lane == 0) sr[b] = block_scale(m);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t i = b * kBlock + e * 32 + lane;
          if (i < p.cols) qr[i] = code1(f[e], inv);
        }
      }
    }
  }
}

// Writes n codes that lie in shared memory as 32 words, one a lane, to dst at any alignment: whole
// aligned words put together from two neighbours, the up to 3 codes before and behind them alone.
__device__ __forceinline__ void store_codes(unsigned char* dst, uint32_t word, int n, int lane) {
  const int s = (int)((4 - ((uintptr_t)dst & 3)) & 3);
  const uint32_t next = __shfl_down_sync(0xffffffffu, word, 1);
  const uint32_t first = __shfl_sync(0xffffffffu, word, 0);
  const int t = s + ((n - s) & ~3) + lane;  // (behind the last whole word; n < s: nothing whole)
  const uint32_t tail = __shfl_sync(0xffffffffu, word, (t >> 2) & 31);
  if (s + 4 * lane + 4 <= n) *reinterpret_cast<uint32_t*>(dst + s + 4 * lane) = __funnelshift_r(word, next, 8 * s);
  if (lane < s && lane < n) dst[lane] = (unsigned char)(first >> (8 * lane));
  if (lane < 3 && n > s && t < n) dst[t] = (unsigned char)(tail >> (8 * (t & 3)));
}

// One 128 x 128 tile a CTA (blockIdx.x over the columns, .y and .z over the rows).  A thread holds RPT
// neighbouring rows of one chunk of V columns: RPT * V = 64 values, so that the codes of a column
// it holds are RPT neighbouring bytes of the transposed row.
// Several CTAs an SM, so that some load while others store.
template <int ACT, bool VEC, bool TILE, bool TRANS>
__global__ void __launch_bounds__(kThreads, ACT == FAR_F32 ? 2 : (TRANS || !VEC) ? 3 : 4) tile_kernel(const QbParams p) {
  constexpr int V = 16 / dtype_size<ACT>::value;
  constexpr int CH = kBlock / V;           // chunks a tile row: 16 or 32
  constexpr int RPT = kBlock * CH / kThreads;  // rows a thread: 8 or 16
  constexpr int WARPS = kThreads / 32;
  __shared__ __align__(16) unsigned char sm[TRANS ? kBlock * kBlock : 16];
  __shared__ float part[TILE ? WARPS : WARPS * kBlock];
  __shared__ float invs[kBlock];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tr = blockIdx.y + (int64_t)blockIdx.z * 32768, tc = blockIdx.x;
  const int64_t r0 = tr * kBlock, c0 = tc * kBlock;
  if (r0 >= p.rows) return;  // the whole CTA
  const int ch = threadIdx.x % CH, rg = threadIdx.x / CH;  // rg: this thread's group of RPT rows
  // value e of a thread's chunk: neighbouring columns, or (without 16-byte loads) columns CH apart,
  // so that neighbouring lanes read neighbouring values
  auto at = [&](int e) { return VEC ? ch * V + e : ch + CH * e; };
  const int64_t col = c0 + ch * V;
  const int nr = (int)(p.rows - r0 < kBlock ? p.rows - r0 : kBlock);  // rows, columns of x in this tile
  const int nc = (int)(p.cols - c0 < kBlock ? p.cols - c0 : kBlock);

  uint32_t raw[RPT][4];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg * RPT + i;
    const char* xr = p.x + (r0 + r) * p.x_stride;
    if constexpr (VEC) {
      load16(raw[i], xr + col * (16 / V), r < nr && ch * V < nc);
    } else {
      uint32_t v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = load_bits<ACT>(xr, c0 + at(e), r < nr && at(e) < nc);
#pragma unroll
      for (int e = 0; e < 4; ++e) raw[i][e] = ACT == FAR_F32 ? v[e] : v[(2 * e) % V] | v[(2 * e + 1) % V] << 16;
    }
  }

  // the maxima: over each column of this thread, or over all it holds
  float cm[V];
  if constexpr (ACT == FAR_F32) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      cm[e] = 0.f;
#pragma unroll
      for (int i = 0; i < RPT; ++i) cm[e] = max_nan(cm[e], fabsf(__uint_as_float(raw[i][e])));
    }
  } else {  // two 16-bit values at a time (their maximum is exact)
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      uint32_t m2 = 0u;
#pragma unroll
      for (int i = 0; i < RPT; ++i) m2 = habs_max2<ACT>(m2, raw[i][e]);
      const float2 f = widen2<ACT>(m2);
      cm[2 * e] = f.x;
      cm[2 * e + 1] = f.y;
    }
  }
  if constexpr (TILE) {
    float m = cm[0];
#pragma unroll
    for (int e = 1; e < V; ++e) m = max_nan(m, cm[e]);
    m = warp_max_allreduce(m);
    if (lane == 0) part[warp] = m;
    __syncthreads();
    m = part[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) m = max_nan(m, part[w]);
    if (threadIdx.x == 0) {
      const int64_t wide = TRANS ? (p.rows + kBlock - 1) / kBlock : (p.cols + kBlock - 1) / kBlock;
      p.scale[TRANS ? tc * wide + tr : tr * wide + tc] = block_scale(m);
    }
    const float inv = block_inverse(m);
#pragma unroll
    for (int e = 0; e < V; ++e) cm[e] = inv;
  } else {
    // rows of the transposed output: a scale a column of x.  Warp, then the warps' partial maxima
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (CH == 16) cm[e] = max_nan(cm[e], __shfl_xor_sync(0xffffffffu, cm[e], 16));
      if (lane < CH) part[warp * kBlock + at(e)] = cm[e];
    }
    __syncthreads();
    if (threadIdx.x < kBlock) {
      float m = part[threadIdx.x];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) m = max_nan(m, part[w * kBlock + threadIdx.x]);
      invs[threadIdx.x] = block_inverse(m);
      if ((int)threadIdx.x < nc) p.scale[(c0 + threadIdx.x) * ((p.rows + kBlock - 1) / kBlock) + tr] = block_scale(m);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) cm[e] = invs[at(e)];
  }

  if constexpr (!TRANS) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = rg * RPT + i;
      if (r < nr) {
        float f[V];
        widen<ACT, V>(raw[i], f);
        uint32_t qw[V / 4];
#pragma unroll
        for (int e = 0; e < V / 4; ++e) qw[e] = codes4(f + 4 * e, cm[0]);
        unsigned char* q = p.q + (r0 + r) * p.cols + c0;
        if constexpr (VEC) {
          q += ch * V;
          if (ch * V >= nc) continue;
          if constexpr (V == 8) *reinterpret_cast<uint2*>(q) = make_uint2(qw[0], qw[1]);
          else *reinterpret_cast<uint32_t*>(q) = qw[0];
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (at(e) < nc) q[at(e)] = (unsigned char)(qw[e >> 2] >> (8 * (e & 3)));
        }
      }
    }
  } else {
    // Column c's codes go to shared row c, RPT bytes at a time.  The units of RPT bytes of a
    // row are permuted by XOR with the chunk's number, so that the lanes of one store (which
    // differ in the chunk) fall on different banks.
    constexpr int UNITS = kBlock / RPT;  // 16 of 8 bytes, or 8 of 16 bytes
    uint32_t qc[V][RPT / 4];
#pragma unroll
    for (int i4 = 0; i4 < RPT / 4; ++i4) {
      float f[4][V];
#pragma unroll
      for (int i = 0; i < 4; ++i) widen<ACT, V>(raw[4 * i4 + i], f[i]);
#pragma unroll
      for (int e = 0; e < V; ++e)
        qc[e][i4] = quantise4<kQuantFp8>(__fmul_rn(f[0][e], cm[e]), __fmul_rn(f[1][e], cm[e]), __fmul_rn(f[2][e], cm[e]),
                                         __fmul_rn(f[3][e], cm[e]));
    }
    auto turn = [](int c) { return (VEC ? c / V : c) & (UNITS - 1); };  // (a lane's own in either layout)
    const int unit = rg ^ turn(at(0));
#pragma unroll
    for (int e = 0; e < V; ++e) {
      unsigned char* s = sm + at(e) * kBlock + unit * RPT;
      if constexpr (RPT == 8) *reinterpret_cast<uint2*>(s) = make_uint2(qc[e][0], qc[e][1]);
      else *reinterpret_cast<uint4*>(s) = make_uint4(qc[e][0], qc[e][1], qc[e][2], qc[e][3]);
    }
    __syncthreads();
    if (p.rows % 16 == 0 && ((uintptr_t)p.q & 15) == 0) {
      // rows of q start on 16-byte boundaries: 8 lanes of 16 bytes each
#pragma unroll
      for (int j = 0; j < kBlock * 8 / kThreads; ++j) {
        const int c = j * (kThreads / 8) + threadIdx.x / 8, k = threadIdx.x % 8;
        const int swz = turn(c);
        if (c >= nc) break;
        unsigned char* q = p.q + (c0 + c) * p.rows + r0;
        uint4 v;
        if constexpr (RPT == 8) {  // the two 8-byte units of 16 rows share a 16-byte place, in either order
          v = *reinterpret_cast<const uint4*>(sm + c * kBlock + ((2 * k) ^ (swz & ~1)) * 8);
          if (swz & 1) v = make_uint4(v.z, v.w, v.x, v.y);
        } else {
          v = *reinterpret_cast<const uint4*>(sm + c * kBlock + (k ^ swz) * 16);
        }
        if (k * 16 < nr) *reinterpret_cast<uint4*>(q + k * 16) = v;  // (whole 16 bytes)
      }
    } else {
      // a warp a row of q, a word a lane
      for (int c = warp; c < nc; c += WARPS) {
        constexpr int W = RPT / 4;  // words a unit
        const uint32_t v = *reinterpret_cast<const uint32_t*>(sm + c * kBlock + ((lane / W) ^ turn(c)) * RPT + lane % W * 4);
        store_codes(p.q + (c0 + c) * p.rows + r0, v, nr, lane);
      }
    }
  }
}

template <int ACT>
cudaError_t launch_qb(const QbParams& p0, int block, int transpose, bool vec, int sms, cudaStream_t s) {
  QbParams p = p0;
  constexpr int V = 16 / dtype_size<ACT>::value;
  if (block == FAR_BLOCK_ROW && !transpose) {
    const int64_t chunks = p.cols / V, blocks128 = (p.cols + (int64_t)kBlock - 1) / kBlock;
    p.segs = (int32_t)(vec ? (chunks + 127) / 128 : (blocks128 + 3) / 4);
    const int64_t ctas = ((int64_t)p.rows * p.segs + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t cap = (int64_t)sms * 64;
    return launch_k(vec ? rows_kernel<ACT, true> : rows_kernel<ACT, false>, dim3((unsigned)(ctas < cap ? ctas : cap)),
                    dim3(kThreads), 0, s, p);
  }
  const int64_t tr = (p.rows + (int64_t)kBlock - 1) / kBlock, tc = (p.cols + (int64_t)kBlock - 1) / kBlock;
  const dim3 grid((unsigned)tc, (unsigned)(tr < 32768 ? tr : 32768), (unsigned)((tr + 32767) / 32768));
  void (*k)(QbParams);
  if (block == FAR_BLOCK_TILE)
    k = transpose ? (vec ? tile_kernel<ACT, true, true, true> : tile_kernel<ACT, false, true, true>)
                  : (vec ? tile_kernel<ACT, true, true, false> : tile_kernel<ACT, false, true, false>);
  else
    k = vec ? tile_kernel<ACT, true, false, true> : tile_kernel<ACT, false, false, true>;
  return launch_k(k, grid, dim3(kThreads), 0, s, p);
}

}  // namespace

}  // namespace far

using namespace far;

extern "C" int quant_block_fp8(const void* x, int64_t x_row_stride, void* q, float* scale, int64_t rows, int64_t cols,
                               int block, int transpose, int act, void* stream) {
  if (act != FAR_F32 && act != FAR_F16 && act != FAR_BF16) return FAR_ERR_DTYPE;
  if ((block != FAR_BLOCK_ROW && block != FAR_BLOCK_TILE) || (transpose != 0 && transpose != 1)) return FAR_ERR_DTYPE;
  if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX || x_row_stride < cols ||
      x_row_stride > (int64_t(1) << 40))
    return FAR_ERR_SHAPE;
  if (rows == 0 || cols == 0) return FAR_OK;
  if (!x || !q || !scale) return FAR_ERR_NULL;
  const int64_t es = act == FAR_F32 ? 4 : 2;
  if ((uintptr_t)x % es || ((uintptr_t)scale & 3)) return FAR_ERR_SHAPE;
  const int64_t orows = transpose ? cols : rows, ocols = transpose ? rows : cols;
  const int64_t scales = (block == FAR_BLOCK_ROW ? orows : (orows + kBlock - 1) / kBlock) * ((ocols + kBlock - 1) / kBlock);
  const Region X = region(x, rows, cols * es, x_row_stride * es), Q = region(q, 1, rows * cols, 0),
               S = region(scale, 1, scales * 4, 0);
  if (regions_overlap(Q, X) || regions_overlap(S, X) || regions_overlap(Q, S)) return FAR_ERR_ALIAS;
  unsigned int* status = nullptr;
  int sms = 0;
  const int st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  QbParams p{static_cast<const char*>(x), static_cast<unsigned char*>(q), scale, x_row_stride * es, (int32_t)rows,
             (int32_t)cols, 0};
  // 16-byte loads of x; codes of a chunk (8 or 4 bytes) or, transposed, whatever q allows
  const int V = (int)(16 / es);
  const bool vec = ((uintptr_t)x & 15) == 0 && (x_row_stride * es) % 16 == 0 && cols % V == 0 &&
                   (transpose || ((uintptr_t)q & (V - 1)) == 0);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = act == FAR_F16    ? launch_qb<FAR_F16>(p, block, transpose, vec, sms, s)
                        : act == FAR_BF16 ? launch_qb<FAR_BF16>(p, block, transpose, vec, sms, s)
                                          : launch_qb<FAR_F32>(p, block, transpose, vec, sms, s);
  return e == cudaSuccess ? FAR_OK : cuda_error_status(e);
}
