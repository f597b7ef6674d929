// The product of two FP8 E4M3 matrices with a binary32 scale for each 128 values along k
// (gemm_fp8_block):
//   out[i, j] = RNE( sum_b xs[i, b] ws[j, b] sum_{k in b} x[i, k] wt[j, k] ).
//
// plain_kernel -- any shape, stride and alignment: 64 x 64 tiles in binary32.
#include <cuda_runtime.h>
#include <stdint.h>

#include "far.h"
#include "far_device.cuh"
#include "far_launch.h"
#include "far_params.h"
#include "far_region.h"

namespace far {

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
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty + 16 * i;
        const float sx = m < p.M ? p.xs[m * p.KB + b] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t n = n0 + tx + 16 * j;
          const float sw = n < p.N ? p.ws[(p.tile_scales ? n / kBlock : n) * p.KB + b] : 0.f;
          acc[i][j] = __fmaf_rn(__fmul_rn(part[i][j], sx), sw, acc[i][j]);
        }
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
  unsigned int* status = nullptr;
  int sms = 0;
  st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t tiles = ((m + 63) / 64) * ((n + 63) / 64);
  const int64_t cap = (int64_t)sms * 8;
  const cudaError_t e = launch_k(plain_kernel, dim3((unsigned)(tiles < cap ? tiles : cap)), dim3(256), 0, s, p);
  return e == cudaSuccess ? FAR_OK : cuda_error_status(e);
}
