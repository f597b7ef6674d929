// A matrix quantised to int8 with a scale a row (quant_rows_int8), and the product of two such
// matrices (gemm_int8):
//   out[i, j] = RNE( fl32(sum_k x[i, k] wt[j, k]) (xs[i] ws[j]) + bias[j] ),  the sum an exact integer.
//
// rows_kernel   a row's 16-byte chunks in the registers of 1 to 16 warps: its maximum is known
//               before its values are needed again, so each is read once.  Bound by HBM.
// long_kernel   any length and alignment: a row read twice, the second time mostly from L2.
// plain_kernel  the product for any shape, stride and alignment: 64 x 64 tiles in int32.
#include <cuda_runtime.h>
#include <stdint.h>

#include "far.h"
#include "far_device.cuh"
#include "far_launch.h"
#include "far_params.h"
#include "far_region.h"

namespace far {

namespace {

// ---------------------------------------------------------------------------
// rows quantised
// ---------------------------------------------------------------------------

struct QrParams {
  const char* x;
  unsigned char* q;
  float* scale;
  int64_t x_stride;  // bytes between rows of x
  int32_t rows, cols;
  int32_t warps;     // rows_kernel: warps a row
};

// 127 / amax leaves binary32's range for a row below 2^-100 (long before any value matters): such
// rows count as zero, as 128-blocks of E4M3 do.
__device__ __forceinline__ float row_scale(float amax) { return amax < kBlockTiny ? 0.f : __fdiv_rn(amax, 127.0f); }
__device__ __forceinline__ float row_inverse(float amax) { return amax < kBlockTiny ? 0.f : __fdiv_rn(127.0f, amax); }

// Four codes.  With amax finite every fl32(v inv) lies within +-(127 + 2^-17), and adding 1.5 * 2^23
// in binary32 rounds it to the nearest integer, ties to even, and leaves that integer's two's
// complement in the low byte; the FMA pipe does it at four times the conversion's rate.
__device__ __forceinline__ uint32_t int8_codes4(const float* v, float inv) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__fadd_rn(__fmul_rn(v[i], inv), 12582912.0f));
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

constexpr int kRowChunks = 4;  // 16-byte chunks a thread, twice that for rows of more than 16 warps

template <int ACT, int U>
__global__ void __launch_bounds__(U > kRowChunks ? 512 : 256) rows_kernel(const QrParams p) {
  constexpr int V = 16 / dtype_size<ACT>::value;
  __shared__ float part[16];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % p.warps, group = warp / p.warps, groups = (int)(blockDim.x >> 5) / p.warps;
  const int64_t row = (int64_t)blockIdx.x * groups + group;
  const bool live = row < p.rows;
  const int chunks = p.cols / V;
  const char* xr = p.x + row * p.x_stride;
  const int c0 = sub * 32 + lane, step = p.warps * 32;
  uint32_t raw[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * step;
    raw[u][0] = raw[u][1] = raw[u][2] = raw[u][3] = 0u;
    if (live && c < chunks) load_bytes<16>(xr + (int64_t)c * 16, raw[u]);
  }
  float m = 0.f;
  if constexpr (ACT == FAR_F32) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max_nan(m, fabsf(__uint_as_float(raw[u][e])));
  } else {
    uint32_t m2 = 0u;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) m2 = habs_max2<ACT>(m2, raw[u][e]);
    const float2 h = widen2<ACT>(m2);
    m = max_nan(h.x, h.y);
  }
  m = warp_max_allreduce(m);
  if (p.warps > 1) {
    if (lane == 0) part[warp] = m;
    __syncthreads();
    m = 0.f;
    for (int w = 0; w < p.warps; ++w) m = max_nan(m, part[group * p.warps + w]);
  }
  if (!live) return;
  if (sub == 0 && lane == 0) p.scale[row] = row_scale(m);
  const float inv = row_inverse(m);
  const bool usual = isfinite(m);  // else every code is 0
  unsigned char* qr = p.q + row * p.cols;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * step;
    if (c >= chunks) break;
    float f[V];
    widen<ACT, V>(raw[u], f);
    uint32_t w[V / 4];
#pragma unroll
    for (int e = 0; e < V / 4; ++e) w[e] = usual ? int8_codes4(f + 4 * e, inv) : 0u;
    if constexpr (V == 8) *reinterpret_cast<uint2*>(qr + (int64_t)c * 8) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(qr + (int64_t)c * 4) = w[0];
  }
}

template <int ACT> __device__ __forceinline__ float element(const char* row, int64_t i) {
  if constexpr (ACT == FAR_F32) return reinterpret_cast<const float*>(row)[i];
  else return widen2<ACT>(reinterpret_cast<const uint16_t*>(row)[i]).x;
}

template <int ACT>
__global__ void __launch_bounds__(256) long_kernel(const QrParams p) {
  __shared__ float part[8];
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const char* xr = p.x + row * p.x_stride;
    float m = 0.f;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < p.cols; i += 256) m = max_nan(m, fabsf(element<ACT>(xr, i)));
    m = warp_max_allreduce(m);
    __syncthreads();  // the last row's parts have been read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0.f;
    for (int w = 0; w < 8; ++w) m = max_nan(m, part[w]);
    if (threadIdx.x == 0) p.scale[row] = row_scale(m);
    const float inv = row_inverse(m);
    const bool usual = isfinite(m);
    unsigned char* qr = p.q + row * p.cols;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < p.cols; i += 256) {
      const float v[4] = {element<ACT>(xr, i), 0.f, 0.f, 0.f};
      qr[i] = usual ? (unsigned char)(int8_codes4(v, inv) & 0xffu) : (unsigned char)0;
    }
  }
}

template <int ACT>
cudaError_t launch_rows(QrParams p, bool vec, int sms, cudaStream_t s) {
  constexpr int V = 16 / dtype_size<ACT>::value;
  const int64_t chunks = p.cols / V;
  if (vec && chunks <= 16 * 32 * 2 * kRowChunks) {
    // as few warps as hold the row in 4 chunks a thread, a power of two; 16 warps of 8 behind that
    p.warps = 1;
    while (p.warps < 16 && chunks > (int64_t)p.warps * 32 * kRowChunks) p.warps *= 2;
    const bool wide = p.warps == 16;
    const int threads = wide ? 512 : 256;
    const int64_t per = threads / 32 / p.warps;
    return launch_k(wide ? rows_kernel<ACT, 2 * kRowChunks> : rows_kernel<ACT, kRowChunks>,
                    dim3((unsigned)((p.rows + per - 1) / per)), dim3(threads), 0, s, p);
  }
  const int64_t cap = (int64_t)sms * 8;
  return launch_k(long_kernel<ACT>, dim3((unsigned)(p.rows < cap ? p.rows : cap)), dim3(256), 0, s, p);
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------

struct Int8Params {
  const int8_t* x;
  const int8_t* wt;
  const float* xs;
  const float* ws;
  const void* bias;
  void* out;
  int64_t ldx, ldw, ldo;  // elements
  int32_t M, N, K;
  int32_t out_dtype;
  unsigned int* status;
  uint64_t timeout_ns;
};

// fl32(acc) times both scales: times their product where that is a normal number or 0 because a scale
// is; else the larger scale first (a product too small: acc brings it back; too large: acc is 0
// or the result infinite).
__device__ __forceinline__ float scaled(float acc, float a, float b) {
  const float s = __fmul_rn(a, b), m = fabsf(s);
  if ((m >= 0x1p-126f && m <= 0x1.fffffep127f) || a == 0.f || b == 0.f) return __fmul_rn(acc, s);
  return fabsf(a) > fabsf(b) ? __fmul_rn(__fmul_rn(acc, a), b) : __fmul_rn(__fmul_rn(acc, b), a);
}

__device__ __forceinline__ float bias_at(const Int8Params& p, int64_t n) {
  if (p.out_dtype == FAR_F32) return static_cast<const float*>(p.bias)[n];
  const uint32_t h = static_cast<const uint16_t*>(p.bias)[n];
  return p.out_dtype == FAR_F16 ? widen2<FAR_F16>(h).x : widen2<FAR_BF16>(h).x;
}

// one output
__device__ __forceinline__ void store_one(const Int8Params& p, int64_t m, int64_t n, int acc, float xs, float ws) {
  float v = scaled(__int2float_rn(acc), xs, ws);
  if (p.bias) v = __fadd_rn(v, bias_at(p, n));
  const int64_t i = m * p.ldo + n;
  if (p.out_dtype == FAR_F32) static_cast<float*>(p.out)[i] = v;
  else if (p.out_dtype == FAR_F16) static_cast<__half*>(p.out)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
}

// 64 x 64 outputs a CTA of 256 threads, 4 x 4 a thread (16 apart), slices of 32 along k in shared memory.
__global__ void __launch_bounds__(256) plain_kernel(const Int8Params p) {
  __shared__ int xs[32][65], ws[32][65];
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t tiles_n = ((int64_t)p.N + 63) / 64, tiles = tiles_n * (((int64_t)p.M + 63) / 64);
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t m0 = t / tiles_n * 64, n0 = t % tiles_n * 64;
    int acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int r = i >> 5, k = i & 31;
        const bool in = k0 + k < p.K;
        xs[k][r] = in && m0 + r < p.M ? p.x[(m0 + r) * p.ldx + k0 + k] : 0;
        ws[k][r] = in && n0 + r < p.N ? p.wt[(n0 + r) * p.ldw + k0 + k] : 0;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        int a[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = xs[k][ty + 16 * i], c[i] = ws[k][tx + 16 * i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] += a[i] * c[j];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < p.M && n < p.N) store_one(p, m, n, acc[i][j], p.xs[m], p.ws[n]);
      }
  }
}

int validate_int8(const Int8Params& p, int64_t m, int64_t n, int64_t k) {
  if (p.out_dtype != FAR_F32 && p.out_dtype != FAR_F16 && p.out_dtype != FAR_BF16) return FAR_ERR_DTYPE;
  if (m < 0 || n < 0 || k < 0 || m > INT32_MAX || n > INT32_MAX || k > 131071) return FAR_ERR_SHAPE;
  const int64_t lim = int64_t(1) << 31;
  if (p.ldx < k || p.ldw < k || p.ldo < n || p.ldx > lim || p.ldw > lim || p.ldo > lim) return FAR_ERR_SHAPE;
  if (m == 0 || n == 0) return FAR_OK;
  if (!p.out || !p.xs || !p.ws || (k > 0 && (!p.x || !p.wt))) return FAR_ERR_NULL;
  const int64_t so = p.out_dtype == FAR_F32 ? 4 : 2;
  if ((uintptr_t)p.out % so || (uintptr_t)p.bias % so || ((uintptr_t)p.xs & 3) || ((uintptr_t)p.ws & 3)) return FAR_ERR_SHAPE;
  const Region O = region(p.out, m, n * so, p.ldo * so);
  const Region rd[5] = {region(p.x, k ? m : 0, k, p.ldx), region(p.wt, k ? n : 0, k, p.ldw), region(p.xs, 1, m * 4, 0),
                        region(p.ws, 1, n * 4, 0), region(p.bias, p.bias ? 1 : 0, n * so, 0)};
  for (const Region& r : rd)
    if (regions_overlap(O, r)) return FAR_ERR_ALIAS;
  return FAR_OK;
}

int run_int8(Int8Params& p, cudaStream_t s) {
  unsigned int* status = nullptr;
  int sms = 0;
  const int st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  p.status = status;
  p.timeout_ns = kWaitTimeoutNs;
  const int64_t tiles = (((int64_t)p.M + 63) / 64) * (((int64_t)p.N + 63) / 64), cap = (int64_t)sms * 8;
  const cudaError_t e = launch_k(plain_kernel, dim3((unsigned)(tiles < cap ? tiles : cap)), dim3(256), 0, s, p);
  return e == cudaSuccess ? FAR_OK : cuda_error_status(e);
}

}  // namespace

}  // namespace far

using namespace far;

extern "C" int quant_rows_int8(const void* x, int64_t x_row_stride, void* q, float* scale, int64_t rows, int64_t cols,
                               int act, void* stream) {
  if (act != FAR_F32 && act != FAR_F16 && act != FAR_BF16) return FAR_ERR_DTYPE;
  if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX || x_row_stride < cols ||
      x_row_stride > (int64_t(1) << 40))
    return FAR_ERR_SHAPE;
  if (rows == 0) return FAR_OK;
  if (!scale || (cols > 0 && (!x || !q))) return FAR_ERR_NULL;
  const int64_t es = act == FAR_F32 ? 4 : 2;
  if ((uintptr_t)x % es || ((uintptr_t)scale & 3)) return FAR_ERR_SHAPE;
  const Region X = region(x, rows, cols * es, x_row_stride * es), Q = region(q, 1, rows * cols, 0),
               S = region(scale, 1, rows * 4, 0);
  if (regions_overlap(Q, X) || regions_overlap(S, X) || regions_overlap(Q, S)) return FAR_ERR_ALIAS;
  unsigned int* status = nullptr;
  int sms = 0;
  const int st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  QrParams p{static_cast<const char*>(x), static_cast<unsigned char*>(q), scale, x_row_stride * es, (int32_t)rows,
             (int32_t)cols, 1};
  // 16-byte loads of x, whole chunks of it; a chunk's codes are 8 or 4 bytes
  const int V = (int)(16 / es);
  const bool vec = cols % V == 0 && ((uintptr_t)x & 15) == 0 && (x_row_stride * es) % 16 == 0 && ((uintptr_t)q & (V - 1)) == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = act == FAR_F16    ? launch_rows<FAR_F16>(p, vec, sms, s)
                        : act == FAR_BF16 ? launch_rows<FAR_BF16>(p, vec, sms, s)
                                          : launch_rows<FAR_F32>(p, vec, sms, s);
  return e == cudaSuccess ? FAR_OK : cuda_error_status(e);
}

extern "C" int64_t far_gemm_int8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0 || k < 0 || m > INT32_MAX || n > INT32_MAX || k > 131071) return -FAR_ERR_SHAPE;
  return 0;
}

extern "C" int gemm_int8(const void* x, int64_t x_row_stride, const float* x_scale, const void* wt, int64_t wt_row_stride,
                         const float* wt_scale, const void* bias, void* out, int64_t out_row_stride, void* workspace,
                         int64_t workspace_bytes, int64_t m, int64_t n, int64_t k, int out_dtype, void* stream) {
  Int8Params p{};
  p.x = static_cast<const int8_t*>(x);
  p.wt = static_cast<const int8_t*>(wt);
  p.xs = x_scale;
  p.ws = wt_scale;
  p.bias = bias;
  p.out = out;
  p.ldx = x_row_stride;
  p.ldw = wt_row_stride;
  p.ldo = out_row_stride;
  p.out_dtype = out_dtype;
  const int st = validate_int8(p, m, n, k);
  if (st != FAR_OK || m == 0 || n == 0) return st;
  p.M = (int32_t)m;
  p.N = (int32_t)n;
  p.K = (int32_t)k;
  (void)workspace;
  (void)workspace_bytes;
  return run_int8(p, static_cast<cudaStream_t>(stream));
}
