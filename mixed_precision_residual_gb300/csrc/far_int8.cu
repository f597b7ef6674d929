// A matrix quantised to int8 with a scale a row (quant_rows_int8), and the product of two such
// matrices (gemm_int8):
//   out[i, j] = RNE( fl32(sum_k x[i, k] wt[j, k]) (xs[i] ws[j]) + bias[j] ),  the sum an exact integer.
//
// rows_kernel   a row's 16-byte chunks in the registers of 1 to 16 warps: its maximum is known
//               before its values are needed again, so each is read once.  Bound by HBM: 8192 x 8192
//               bf16 31.6 us (6.4 TB/s, 94 % of the copy rate); 48 x 13312 2.9 us.
// long_kernel   any length and alignment: a row read twice, the second time mostly from L2 (2000 x 40000
//               bf16 48 us).  Off 16 bytes a value at a time: 8192 x 100 16.5, 8192 x 8191 77, 2000 x 40001 87.
//
// sm_103a's tcgen05 multiplies no integers, but f16 holds every code exactly, a product of two is at
// most 2^14 in magnitude, and the binary32 sum of 1024 of them at most 2^24: exact.  So the
// products run at the tensor cores' f16 rate, and the sums move from TMEM to int32 every 1024 of k.
//
// pair8_kernel  many rows: CTA pairs; wt's codes are widened on their way from shared memory into TMEM
//               (A), x's by widen_kernel ahead, into the workspace (B).
// few8_kernel   few rows of x (a decode batch): codes are widened on their way from shared memory to
//               the tensor cores, wt's rows into TMEM, x's into shared memory.  Bound by reading wt once.
// plain_kernel  the product for any shape, stride and alignment: 64 x 64 tiles in int32 (4 x 8192 x 8192 0.5 to 1 ms).
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "far.h"
#include "far_device.cuh"
#include "far_launch.h"
#include "far_pair16.cuh"
#include "far_params.h"
#include "far_region.h"
#include "far_tcgen05.cuh"
#include "far_tma.h"

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

// A row below 2^-100 counts as zero, as 128-blocks of E4M3 do: a chosen limit, above 2^-121, where 127 / amax
// leaves binary32's range and would turn the row's zeros into NaN.  (The norm's int8 output takes a row as
// zero at amax == 0 alone.)
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

// VEC: 16-byte chunks, four in flight a thread; else a value at a time.
template <int ACT, bool VEC>
__global__ void __launch_bounds__(512) long_kernel(const QrParams p) {
  constexpr int V = VEC ? 16 / dtype_size<ACT>::value : 1, T = 512, U = 4;
  __shared__ float part[T / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int units = VEC ? p.cols / V : p.cols;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const char* xr = p.x + row * p.x_stride;
    float f[U][V];
    auto load = [&](int64_t c0) {
      if constexpr (VEC) {
        uint32_t raw[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          raw[u][0] = raw[u][1] = raw[u][2] = raw[u][3] = 0u;
          if (c0 + u * T < units) load_bytes<16>(xr + (c0 + u * T) * 16, raw[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) widen<ACT, V>(raw[u], f[u]);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) f[u][0] = c0 + u * T < units ? element<ACT>(xr, c0 + u * T) : 0.f;
      }
    };
    float m = 0.f;
    for (int64_t c = threadIdx.x; c < units; c += U * T) {
      load(c);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < V; ++e) m = max_nan(m, fabsf(f[u][e]));
    }
    m = warp_max_allreduce(m);
    __syncthreads();  // the last row's parts have been read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0.f;
    for (int w = 0; w < T / 32; ++w) m = max_nan(m, part[w]);
    if (threadIdx.x == 0) p.scale[row] = row_scale(m);
    const float inv = row_inverse(m);
    const bool usual = isfinite(m);
    unsigned char* qr = p.q + row * p.cols;
    for (int64_t c = threadIdx.x; c < units; c += U * T) {
      load(c);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c + u * T >= units) break;
        if constexpr (VEC) {
          uint32_t w[V / 4];
#pragma unroll
          for (int e = 0; e < V / 4; ++e) w[e] = usual ? int8_codes4(f[u] + 4 * e, inv) : 0u;
          if constexpr (V == 8) *reinterpret_cast<uint2*>(qr + (c + u * T) * 8) = make_uint2(w[0], w[1]);
          else *reinterpret_cast<uint32_t*>(qr + (c + u * T) * 4) = w[0];
        } else {
          const float v[4] = {f[u][0], 0.f, 0.f, 0.f};
          qr[c + u * T] = usual ? (unsigned char)(int8_codes4(v, inv) & 0xffu) : (unsigned char)0;
        }
      }
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
  const int64_t cap = (int64_t)sms * 4;
  return launch_k(vec ? long_kernel<ACT, true> : long_kernel<ACT, false>, dim3((unsigned)(p.rows < cap ? p.rows : cap)), dim3(512),
                  0, s, p);
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
  int32_t packed;         // pair8_kernel: wt's codes lie where widen_kernel writes
  int32_t wide;           // four outputs of a row start on their size's multiple
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

__device__ __noinline__ float scaled_call(float acc, float a, float b) { return scaled(acc, a, b); }

__device__ __forceinline__ float bias_at(const Int8Params& p, int64_t n) {
  if (p.out_dtype == FAR_F32) return static_cast<const float*>(p.bias)[n];
  const uint32_t h = static_cast<const uint16_t*>(p.bias)[n];
  return p.out_dtype == FAR_F16 ? widen2<FAR_F16>(h).x : widen2<FAR_BF16>(h).x;
}

// a scale whose product with another such is a normal number or 0
__device__ __forceinline__ bool usual_scale(float s) {
  const float m = fabsf(s);
  return (m >= 0x1p-60f && m <= 0x1p60f) || m == 0.f;
}

// four neighbouring outputs of a row, in one store where the row allows it
__device__ __forceinline__ void store4(const Int8Params& p, int64_t m, int64_t n, const float (&v)[4]) {
  const int64_t i = m * p.ldo + n;
  if (p.out_dtype == FAR_F32) {
    float* o = static_cast<float*>(p.out) + i;
    if (p.wide && n + 4 <= p.N) {
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
      return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) o[e] = v[e];
    return;
  }
  uint16_t* o = static_cast<uint16_t*>(p.out) + i;
  const bool f16 = p.out_dtype == FAR_F16;
  const uint32_t lo = f16 ? narrow2<FAR_F16>(v[0], v[1]) : narrow2<FAR_BF16>(v[0], v[1]);
  const uint32_t hi = f16 ? narrow2<FAR_F16>(v[2], v[3]) : narrow2<FAR_BF16>(v[2], v[3]);
  if (p.wide && n + 4 <= p.N) {
    *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
    return;
  }
  const uint16_t h[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < p.N) o[e] = h[e];
}

template <int DT> __device__ __forceinline__ void store_value(void* at, float v) {
  if constexpr (DT == FAR_F32) *static_cast<float*>(at) = v;
  else *static_cast<uint16_t*>(at) = (uint16_t)narrow2<DT>(v, 0.f);
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

// ---------------------------------------------------------------------------
// codes as f16
// ---------------------------------------------------------------------------

// Four codes, a word, as two words of two f16: with its sign bit flipped a code c is the unsigned byte
// c + 128, and 0x6400 + that byte the f16 number 1024 + 128 + c: minus 1152, exactly c.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  const uint32_t u = w ^ 0x80808080u, base = 0x64646464u;
  uint2 r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r.x) : "r"(__byte_perm(u, base, 0x4140)), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r.y) : "r"(__byte_perm(u, base, 0x4342)), "r"(0x64806480u));
  return r;
}

struct WidenParams {
  const int8_t *x, *wt;
  __half* wide;      // x as f16, rows of ld values
  int8_t* packed;    // null, or wt with rows of ld codes, where TMA cannot read it as it stands
  int64_t ldx, ldw, rows, wt_rows, ld;  // ld: wide_ld(k)
  int32_t K;
  int32_t vec;       // whole 16-byte chunks of x's rows may be read
};

// 8 codes of a row (past k: zeros)
__device__ __forceinline__ uint2 load_codes(const int8_t* row, int k, int K, bool vec) {
  uint32_t w[2] = {0u, 0u};
  if (vec && k + 8 <= K) {
    load_bytes<8>(row + k, w);
  } else {
#pragma unroll
    for (int b = 0; b < 8; ++b)
      if (k + b < K) w[b >> 2] |= (uint32_t)(uint8_t)row[k + b] << (8 * (b & 3));
  }
  return make_uint2(w[0], w[1]);
}

// blockDim.x threads along a row, 8 codes each, blockDim.y rows a CTA; blockIdx.y 1: wt.  Bound by HBM.
__global__ void __launch_bounds__(256) widen_kernel(const WidenParams p) {
  pdl_wait();
  pdl_launch_dependents();  // (behind the wait: pair8_kernel reads wt before it waits itself)
  const bool repack = blockIdx.y != 0;
  const int64_t rows = repack ? p.wt_rows : p.rows;
  const int step = (int)blockDim.x * 8;
  constexpr int U = 4;
  for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < rows; row += (int64_t)gridDim.x * blockDim.y) {
    const int8_t* src = repack ? p.wt + row * p.ldw : p.x + row * p.ldx;
    for (int k0 = (int)threadIdx.x * 8; k0 < p.ld; k0 += U * step) {
      uint2 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k0 + u * step < p.ld) w[u] = load_codes(src, k0 + u * step, p.K, p.vec && !repack);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * step;
        if (k >= p.ld) break;
        if (repack) {
          *reinterpret_cast<uint2*>(p.packed + row * p.ld + k) = w[u];
        } else {
          const uint2 a = widen4(w[u].x), b = widen4(w[u].y);
          *reinterpret_cast<uint4*>(p.wide + row * p.ld + k) = make_uint4(a.x, a.y, b.x, b.y);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// pair8_kernel: tiles of 256 rows of wt x nt rows of x (64 .. 192) over a cluster of 2, wt's rows on the
// TMEM lanes.  Each CTA holds its 128 rows of wt and half of the tile's rows of x; one thread of the even
// CTA issues tcgen05.mma.cta_group::2 over both, A from each CTA's TMEM, B from shared memory, a block
// of 128 of k at a time.  Persistent.
//   warps 0, 2  TMA producers (both CTAs): a ring of blocks of wt's codes, one of blocks of x.  (One thread for
//               both spent 630 cycles a block, most of what a block took: 200 x 5120 x 13312 48 us.)
//   warp 1      MMA issuer (even CTA); allocates TMEM: two accumulators of nt columns, blocks of A in
//               the rest
//   warps 4-11  widen wt's codes, a row a thread: warps 4-7 and 8-11 every other block
//   warps 12-19 epilogue: warp w the TMEM lanes 32 (w % 4) .. and one half of the tile's rows of x; sums
//               to int32 every 8 blocks
// The registers a thread: 640 threads are launched at 96; warps 0-3 keep 56, 4-11 72, and the epilogue's
// take 136 for 96 sums (128 x 56 + 256 x 72 + 256 x 136 = 60416 of 61440).
// Why A in TMEM: widened codes in shared memory for both operands would be written once and read once more
// there, 160 bytes a cycle of MMA against the 128 that shared memory gives; TMEM takes wt's half of it.
// Why 192 rows at most: two accumulators of nt columns, so that sums leave while the next block's products
// arrive, and at least two blocks of A share 512 columns.
// Measured: 16384 x 8192 x 8192 with widen_kernel 1267 to 1297 us (1.70 to 1.74 PFLOP/s; both operands widened ahead
// and 256 x 256 tiles: 1361), 2048 x 4096 x 4096 50 (80), 200 x 5120 x 13312 41 (few8_kernel 79).  At 192 rows
// a block takes 841 cycles, 768 of them the MMA's; below 128 rows it stays at about 600: issuing 8 MMAs and 2
// commits takes one thread 340 of them, a look at its two barriers 100 (looked at one after the other 200: 200 x
// 5120 x 13312 42 us, 4096 x 1024 x 8192 67 against 60), the hand-overs between the widening warps and the
// issuer in two CTAs the rest.  (An arrival released at cluster scope on the other CTA's barrier instead of
// one behind tcgen05.wait alone: 0.68 us a slice of 64 against 0.29.)
// ---------------------------------------------------------------------------
constexpr int kPair8Threads = 640;
constexpr int kPair8Most = 192;  // rows of x
constexpr int kPair8Codes = 5, kPair8Slots = 8;  // ring slots: of wt, of x and of A at most
constexpr uint32_t kPair8CodeBytes = 128 * 128, kPair8XBytes = 120 * 1024;
constexpr uint32_t kPair8Ring = kPair8Codes * kPair8CodeBytes + kPair8XBytes;
constexpr int kPair8Bars = 2 * kPair8Codes + 4 * kPair8Slots + 4;
constexpr size_t kPair8Smem = kPair8Ring + kPair8Bars * 8 + 16 + 1024;
constexpr int kPair8Sum = 8;  // blocks that an accumulator sums exactly

struct Pair8Walk {
  int32_t nt, tiles_m, tiles_n, num_tiles, blocks;
  uint32_t xslots, aslots;
  uint32_t xhalf;  // bytes of a CTA's rows of x of 64 of k
};

// a place in a ring: slot, and the parity of the wait for its use
struct Place8 {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t slots) {
    if (++slot == slots) slot = 0, phase ^= 1;
  }
};

// groups of 8 tiles of wt, x's tiles one after the other inside a group: pairs at work share both in L2
__device__ __forceinline__ void pair8_tile(const Pair8Walk& w, int t, int& tm, int& tn) {
  const int per = 8 * w.tiles_m, g = t / per, r = t - g * per, gn = min(w.tiles_n - 8 * g, 8);
  tn = 8 * g + r % gn;
  tm = r / gn;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPair8Threads, 1)
    pair8_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ Int8Params p, const __grid_constant__ Pair8Walk w) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);  // the same offset in both CTAs
  const uint32_t w_base = smem_addr(smem), x_base = w_base + kPair8Codes * kPair8CodeBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kPair8Ring);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kPair8Bars);
  const uint32_t w_full0 = smem_addr(&bars[0]), w_empty0 = w_full0 + 8 * kPair8Codes;
  const uint32_t x_full0 = w_empty0 + 8 * kPair8Codes, x_empty0 = x_full0 + 8 * kPair8Slots;
  const uint32_t a_full0 = x_empty0 + 8 * kPair8Slots, a_empty0 = a_full0 + 8 * kPair8Slots;
  const uint32_t acc_full0 = a_empty0 + 8 * kPair8Slots, acc_empty0 = acc_full0 + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_cta_rank();
  const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
  const uint32_t a_col = 2u * (uint32_t)w.nt;  // TMEM: two accumulators, then A

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPair8Codes; ++s) {
      mbar_init(w_full0 + 8 * s, 1);
      mbar_init(w_empty0 + 8 * s, 4);  // the widening warps of a block
    }
    for (int s = 0; s < kPair8Slots; ++s) {
      mbar_init(x_full0 + 8 * s, 1);   // even CTA: its producer's arrive + both CTAs' bytes
      mbar_init(x_empty0 + 8 * s, 1);  // one multicast commit
      mbar_init(a_full0 + 8 * s, 8);   // even CTA: four widening warps of each CTA
      mbar_init(a_empty0 + 8 * s, 1);  // one multicast commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(acc_full0 + 8 * a, 1);    // one multicast commit
      mbar_init(acc_empty0 + 8 * a, 16);  // even CTA: the epilogue warps of both CTAs
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
  pdl_launch_dependents();  // (not before the TMEM columns are this CTA's)
  // Only what widen_kernel writes is waited for: it lets this kernel start behind its own wait, when all
  // work before it is done.  So wt's codes may be read, and widened, while it runs, unless it writes them.
  if (p.packed) pdl_wait();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // ---------------- wt's blocks (both CTAs) ----------------
      Place8 at;
      uint32_t g = 0;
      bool ok = true;
      for (int t = pair; ok && t < w.num_tiles; t += pairs) {
        int tm, tn;
        pair8_tile(w, t, tm, tn);
        const int row = tn * 256 + (int)rank * 128;
        for (int kb = 0; kb < w.blocks; ++kb, ++g) {
          if (!mbar_wait(w_empty0 + 8 * at.slot, at.phase ^ 1u, p.timeout_ns, p.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(w_full0 + 8 * at.slot, kPair8CodeBytes);
          tma_load_2d(w_base + at.slot * kPair8CodeBytes, &map_w, kb * 128, row, w_full0 + 8 * at.slot);
          at.next(kPair8Codes);
        }
      }
      // Before exit the last copies must have landed, and the commits that free A's places, which the MMA
      // issuer multicasts, must have arrived in both CTAs.
      for (uint32_t j = g > kPair8Codes ? g - kPair8Codes : 0u; j < g; ++j)
        mbar_wait(w_full0 + 8 * (j % kPair8Codes), (j / kPair8Codes) & 1u, p.timeout_ns, p.status);
      for (uint32_t j = g > w.aslots ? g - w.aslots : 0u; ok && j < g; ++j)
        ok = mbar_wait(a_empty0 + 8 * (j % w.aslots), (j / w.aslots) & 1u, p.timeout_ns, p.status);
    } else if (warp == 2 && lane == 0) {
      // ---------------- x's blocks (both CTAs) ----------------
      pdl_wait();
      Place8 at;
      uint32_t g = 0;
      bool ok = true;
      for (int t = pair; ok && t < w.num_tiles; t += pairs) {
        int tm, tn;
        pair8_tile(w, t, tm, tn);
        const int row = tm * w.nt + (int)rank * (w.nt / 2);
        for (int kb = 0; kb < w.blocks; ++kb, ++g) {
          if (!mbar_wait(x_empty0 + 8 * at.slot, at.phase ^ 1u, p.timeout_ns, p.status)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(x_full0 + 8 * at.slot, (uint32_t)w.nt * 256);
          tma_load_3d_pair(x_base + at.slot * 2 * w.xhalf, &map_x, 0, row, 2 * kb, map_to_cta(x_full0 + 8 * at.slot, 0));
          at.next(w.xslots);
        }
      }
      const uint32_t last = g > w.xslots ? g - w.xslots : 0u;
      if (rank == 0)
        for (uint32_t j = last; j < g; ++j)
          mbar_wait(x_full0 + 8 * (j % w.xslots), (j / w.xslots) & 1u, p.timeout_ns, p.status);
      for (uint32_t j = last; ok && j < g; ++j)
        ok = mbar_wait(x_empty0 + 8 * (j % w.xslots), (j / w.xslots) & 1u, p.timeout_ns, p.status);
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA issuer (even CTA) ----------------
      const bool leader = elect_one();
      const uint32_t tm_ = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t idesc = umma_idesc_16(256, w.nt, false, false, false);
      const uint64_t x0 = sw128_kmajor_desc(x_base);
      const uint32_t half = w.xhalf >> 4;
      Place8 px, pa;
      uint32_t use = 0;
      bool ok = true;
      for (int t = pair; ok && t < w.num_tiles; t += pairs) {
        for (int k0 = 0; ok && k0 < w.blocks; k0 += kPair8Sum, ++use) {
          const uint32_t acc = use & 1u;
          if (!mbar_wait(acc_empty0 + 8 * acc, ((use >> 1) & 1u) ^ 1u, p.timeout_ns, p.status)) {
            ok = false;
            break;
          }
          const uint32_t d = tm_ + acc * w.nt;
          const int k1 = min(w.blocks, k0 + kPair8Sum);
          for (int kb = k0; kb < k1; ++kb) {
            if (!mbar_wait_both(x_full0 + 8 * px.slot, px.phase, a_full0 + 8 * pa.slot, pa.phase, p.timeout_ns, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t x = x0 + px.slot * 2 * half;
            const uint32_t a = tm_ + a_col + 64 * pa.slot;
            if (leader) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                umma_f16_ts_pair(d, a + 8 * k, x + (k >> 2) * half + 2 * (k & 3), idesc, kb != k0 || k != 0);
              umma_commit_pair(a_empty0 + 8 * pa.slot, 0x3);
              umma_commit_pair(x_empty0 + 8 * px.slot, 0x3);
              if (kb == k1 - 1) umma_commit_pair(acc_full0 + 8 * acc, 0x3);
            }
            __syncwarp();
            px.next(w.xslots);
            pa.next(w.aslots);
          }
        }
      }
    }
  } else if (warp < 12) {
    // ---------------- wt's codes: a row a thread ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int row = 32 * (warp & 3) + lane;
    const uint32_t dst = tmem + a_col + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t a_full_even = map_to_cta(a_full0, 0);
    const unsigned char* line = smem + row * 128;
    int skip = (warp - 4) >> 2;  // the other warps' block is next
    Place8 pw, pa;
    bool ok = true;
    for (int t = pair; ok && t < w.num_tiles; t += pairs)
      for (int kb = 0; kb < w.blocks; ++kb, skip ^= 1, pw.next(kPair8Codes), pa.next(w.aslots)) {
        if (skip) continue;
        if (!mbar_wait(w_full0 + 8 * pw.slot, pw.phase, p.timeout_ns, p.status)) {
          ok = false;
          break;
        }
        const unsigned char* src = line + pw.slot * kPair8CodeBytes;
        uint32_t v[32];
        auto widen32 = [&](int h) {  // 64 codes: units 4 h .. of the swizzled row
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 c = *reinterpret_cast<const uint4*>(src + (((4 * h + u) ^ (row & 7)) * 16));
            const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint2 f = widen4(cw[e]);
              v[8 * u + 2 * e] = f.x;
              v[8 * u + 2 * e + 1] = f.y;
            }
          }
        };
        widen32(0);
        if (!mbar_wait(a_empty0 + 8 * pa.slot, pa.phase ^ 1u, p.timeout_ns, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_st32(dst + 64 * pa.slot, v);
        widen32(1);
        tmem_st32(dst + 64 * pa.slot + 32, v);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(w_empty0 + 8 * pw.slot);
          mbar_arrive_remote(a_full_even + 8 * pa.slot);  // (tcgen05.wait has seen the stores done)
        }
      }
  } else {
    // ---------------- epilogue ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    pdl_wait();  // the scales and the bias are read through L1
    const int quarter = warp & 3, part = (warp - 12) >> 2, half = w.nt / 2;
    const uint32_t src = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(part * half);
    const uint32_t acc_empty_even = map_to_cta(acc_empty0, 0);
    uint32_t use = 0;
    bool ok = true;
    for (int t = pair; ok && t < w.num_tiles; t += pairs) {
      int tm, tn;
      pair8_tile(w, t, tm, tn);
      int acc[kPair8Most / 2];  // (behind the last block: binary32 values)
#pragma unroll
      for (int i = 0; i < kPair8Most / 2; ++i) acc[i] = 0;
#pragma unroll 1
      for (int k0 = 0; k0 < w.blocks; k0 += kPair8Sum, ++use) {
        const uint32_t buf = use & 1u;
        if (!mbar_wait(acc_full0 + 8 * buf, (use >> 1) & 1u, p.timeout_ns, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kPair8Most / 2; c += 16) {
          if (c < half) {
            uint32_t r[16];
            tmem_ld16(src + buf * w.nt + c, r);
            tmem_ld_wait(r);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c + i] += __float2int_rn(__uint_as_float(r[i]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(acc_empty_even + 8 * buf);
      }
      if (!ok) break;
      const int64_t n = (int64_t)tn * 256 + rank * 128 + quarter * 32 + lane, m0 = (int64_t)tm * w.nt + part * half;
      const float ws = n < p.N ? p.ws[n] : 0.f, bias = p.bias && n < p.N ? bias_at(p, n) : -0.f;
      // A thread's column of up to 96 rows: scaled in place, then stored, 32 neighbouring columns a store.  (The
      // code of a tile's end runs once a tile, so what it costs is its length, in instruction fetches: with
      // the scales' rare sizes and the types' stores inlined at each value it took 12 us, as it stands 2.)
#pragma unroll
      for (int c = 0; c < kPair8Most / 2; c += 16) {
        const int64_t m = m0 + c + (lane & 15);
        if (c < half && m0 + c < p.M) {
          const float xs = m < p.M ? p.xs[m] : 0.f;
          if (__all_sync(0xffffffffu, usual_scale(xs) && usual_scale(ws))) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[c + i] = __float_as_int(__fadd_rn(__fmul_rn(__int2float_rn(acc[c + i]), __fmul_rn(__shfl_sync(0xffffffffu, xs, i), ws)), bias));
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[c + i] = __float_as_int(__fadd_rn(scaled_call(__int2float_rn(acc[c + i]), __shfl_sync(0xffffffffu, xs, i), ws), bias));
          }
        }
      }
      const int rows = n < p.N ? (int)min((int64_t)half, p.M - m0) : 0;
      auto store = [&](auto dt) {
        constexpr int DT = decltype(dt)::value, SIZE = DT == FAR_F32 ? 4 : 2;
        char* out = static_cast<char*>(p.out) + (m0 * p.ldo + n) * SIZE;
        const int64_t step = p.ldo * SIZE;
#pragma unroll
        for (int i = 0; i < kPair8Most / 2; ++i, out += step)
          if (i < rows) store_value<DT>(out, __int_as_float(acc[i]));
      };
      if (p.out_dtype == FAR_F32) store(std::integral_constant<int, FAR_F32>{});
      else if (p.out_dtype == FAR_F16) store(std::integral_constant<int, FAR_F16>{});
      else store(std::integral_constant<int, FAR_BF16>{});
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// few8_kernel: 128 rows of wt x NT rows of x a CTA, the blocks of 128 of k shared out over a cluster of
// gridDim's x dimension (CTA rank r takes blocks KB r / S .. KB (r + 1) / S - 1).
//   warps 0-3  wt's codes of one row a thread from shared memory, widened, into TMEM: A, two blocks
//   warps 4-   the sums, 4 or 8 warps: to int32 every 8 blocks
//   then       a TMA producer, an MMA issuer (and TMEM), and 2 or 4 warps that widen x's codes into
//              shared memory: B, two blocks
// Then each CTA leaves its sums in its shared memory and adds up every S-th row of x over the
// cluster's CTAs (integers: in any order the same), scales and stores.
// Bound by reading wt: 4 x 8192 x 8192 14.6 us (4.6 TB/s), 4 x 32768 x 4096 24.2 (5.5); about 3 us is the launch,
// the set-up and the sum over the cluster, and a CTA alone on its SM has 80 KB in flight, which takes
// 3 us to arrive under load.  Two sets of widening warps and three places for A and B: the same
// (14.9 and 24.2).
// ---------------------------------------------------------------------------
template <int NT> struct Few8Shape {
  static constexpr int ctas = NT <= 32 ? 2 : 1;  // an SM
  static constexpr int xwarps = NT <= 32 ? 2 : 4;
  static constexpr int swarps = NT <= 32 ? 4 : 8;  // so that a thread keeps at most 64 sums
  static constexpr int threads = 32 * (6 + swarps + xwarps);
  static constexpr uint32_t a_bytes = 128 * 128, b_bytes = NT * 128;  // codes of a block
  static constexpr int stages = NT == 16 ? 5 : NT == 32 ? 4 : NT == 64 ? 6 : 4;
  static constexpr uint32_t ring = stages * (a_bytes + b_bytes);
  static constexpr uint32_t wide = NT * 256;  // a block of x as f16: two tiles of 64 of k
  static constexpr uint32_t tmem_a = 2 * NT;  // behind two accumulators
  static constexpr uint32_t tmem_cols = 2 * NT + 128 <= 256 ? 256 : 512;
  static constexpr int bars = 2 * stages + 8;
  static constexpr size_t smem = ring + 2 * wide + bars * 8 + 16 + 1024;
  static_assert(NT * 128 * 4 <= ring, "the sums that the cluster adds up lie in the ring");
  static_assert((smem + 1024) * ctas <= 228 * 1024 && ctas * tmem_cols <= 512, "");
};

template <int NT>
__global__ void __launch_bounds__(Few8Shape<NT>::threads, Few8Shape<NT>::ctas)
    few8_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ Int8Params p) {
  using S = Few8Shape<NT>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);  // the same offset in every CTA
  const uint32_t a_base = smem_addr(smem), b_base = a_base + S::stages * S::a_bytes;
  unsigned char* wide = smem + S::ring;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::ring + 2 * S::wide);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + S::bars);
  const uint32_t full0 = smem_addr(&bars[0]), empty0 = full0 + 8 * S::stages;
  const uint32_t wide_full0 = empty0 + 8 * S::stages, wide_empty0 = wide_full0 + 16;
  const uint32_t acc_full0 = wide_empty0 + 16, acc_empty0 = acc_full0 + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = (int)gridDim.x, rank = (int)blockIdx.x;  // the cluster spans gridDim.x
  const int64_t n0 = (int64_t)blockIdx.y * 128, m0 = (int64_t)blockIdx.z * NT;
  const int KB = (p.K + 127) / 128;
  const int kb0 = (int)((int64_t)KB * rank / split), kb1 = (int)((int64_t)KB * (rank + 1) / split);
  constexpr int kSum = 8;  // blocks that an accumulator sums exactly
  constexpr int kProducer = 4 + S::swarps, kIssuer = kProducer + 1;

  // the ring's first load of wt starts for L2 while the CTA is set up and the kernel ahead drains
  if (warp == kProducer && lane == 0)
    for (int kb = kb0; kb < kb1 && kb < kb0 + S::stages; ++kb) tma_prefetch_2d(&map_w, kb * 128, (int)n0);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 4 + S::xwarps);  // the widening warps
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(wide_full0 + 8 * b, 4 + S::xwarps);
      mbar_init(wide_empty0 + 8 * b, 1);  // a commit
      mbar_init(acc_full0 + 8 * b, 1);    // a commit
      mbar_init(acc_empty0 + 8 * b, S::swarps);
    }
    fence_barrier_init();
    tma_prefetch_map(&map_x);
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_addr(tmem_slot), S::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();  // (not before the TMEM columns are this CTA's)
  pdl_wait();

  int* sums = reinterpret_cast<int*>(smem);
  if (warp < 4) {
    // ---------------- wt: a row a thread ----------------
    const int row = 32 * warp + lane;
    const uint32_t dst = tmem + S::tmem_a + ((uint32_t)(32 * warp) << 16);
    uint32_t g = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++g) {
      const uint32_t s = g % S::stages, b = g & 1u;
      if (!mbar_wait(full0 + 8 * s, (g / S::stages) & 1u, p.timeout_ns, p.status) ||
          !mbar_wait(wide_empty0 + 8 * b, ((g >> 1) & 1u) ^ 1u, p.timeout_ns, p.status))
        break;
      tc_fence_after();
      const unsigned char* src = smem + s * S::a_bytes + row * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // 16 codes: unit 4 h + u of the swizzled row
          const uint4 c = *reinterpret_cast<const uint4*>(src + (((4 * h + u) ^ (row & 7)) * 16));
          const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint2 t = widen4(cw[e]);
            v[8 * u + 2 * e] = t.x;
            v[8 * u + 2 * e + 1] = t.y;
          }
        }
        tmem_st32(dst + b * 64 + 32 * h, v);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(empty0 + 8 * s);
        mbar_arrive(wide_full0 + 8 * b);
      }
    }
  } else if (warp < kProducer) {
    // ---------------- sums ----------------
    constexpr int MINE = NT * 4 / S::swarps;  // columns of a warp
    const int first = (warp - 4) / 4 * MINE;
    const uint32_t src = tmem + ((uint32_t)((warp & 3) * 32) << 16) + first;
    int acc[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) acc[i] = 0;
    uint32_t use = 0;
#pragma unroll 1
    for (int kb = kb0; kb < kb1; kb += kSum, ++use) {
      const uint32_t b = use & 1u;
      if (!mbar_wait(acc_full0 + 8 * b, (use >> 1) & 1u, p.timeout_ns, p.status)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < MINE; c += 16) {
        uint32_t r[16];
        tmem_ld16(src + b * NT + c, r);
        tmem_ld_wait(r);
        if (c + 16 == MINE) {  // all read: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty0 + 8 * b);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c + i] += __float2int_rn(__uint_as_float(r[i]));
      }
    }
    // every MMA has read its operands, so every copy has landed and been widened: the ring takes the sums [NT][128]
#pragma unroll
    for (int i = 0; i < MINE; ++i) sums[(first + i) * 128 + 32 * (warp & 3) + lane] = acc[i];
  } else if (warp == kProducer) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      uint32_t g = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++g) {
        const uint32_t s = g % S::stages;
        if (!mbar_wait(empty0 + 8 * s, ((g / S::stages) & 1u) ^ 1u, p.timeout_ns, p.status)) break;
        mbar_arrive_expect_tx(full0 + 8 * s, S::a_bytes + S::b_bytes);
        tma_load_2d(a_base + s * S::a_bytes, &map_w, kb * 128, (int)n0, full0 + 8 * s);
        tma_load_2d(b_base + s * S::b_bytes, &map_x, kb * 128, (int)m0, full0 + 8 * s);
      }
      // before the CTA may leave the last blocks must have landed
      for (uint32_t j = g > (uint32_t)S::stages ? g - S::stages : 0u; j < g; ++j)
        mbar_wait(full0 + 8 * (j % S::stages), (j / S::stages) & 1u, p.timeout_ns, p.status);
    }
  } else if (warp == kIssuer) {
    // ---------------- MMA issuer ----------------
    constexpr uint32_t IDESC = umma_idesc_16(128, NT, false, false, false);
    const bool leader = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t x0 = sw128_kmajor_desc(smem_addr(wide));
    uint32_t g = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++g) {
      const uint32_t b = g & 1u, use = g / kSum, acc = use & 1u;
      const bool begins = g % kSum == 0, ends = g % kSum == kSum - 1 || kb == kb1 - 1;
      if (begins && !mbar_wait(acc_empty0 + 8 * acc, ((use >> 1) & 1u) ^ 1u, p.timeout_ns, p.status)) break;
      if (!mbar_wait(wide_full0 + 8 * b, (g >> 1) & 1u, p.timeout_ns, p.status)) break;
      tc_fence_after();
      const uint64_t x = x0 + b * (S::wide >> 4);
      const uint32_t a = tm + S::tmem_a + b * 64, d = tm + acc * NT;
      if (leader) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_f16_ts(d, a + 8 * k, x + (k >> 2) * (NT * 128 >> 4) + 2 * (k & 3), IDESC, !begins || k != 0);
        umma_commit(wide_empty0 + 8 * b);
        if (ends) umma_commit(acc_full0 + 8 * acc);
      }
      __syncwarp();
    }
    // the commits that free the last two blocks' places must have arrived before the CTA may leave
    for (uint32_t j = g > 2 ? g - 2 : 0u; j < g; ++j) mbar_wait(wide_empty0 + 8 * (j & 1u), (j >> 1) & 1u, p.timeout_ns, p.status);
  } else {
    // ---------------- x: 16 codes of a row at a time ----------------
    const int t = (int)threadIdx.x - 32 * (kIssuer + 1);
    uint32_t g = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++g) {
      const uint32_t s = g % S::stages, b = g & 1u;
      if (!mbar_wait(full0 + 8 * s, (g / S::stages) & 1u, p.timeout_ns, p.status) ||
          !mbar_wait(wide_empty0 + 8 * b, ((g >> 1) & 1u) ^ 1u, p.timeout_ns, p.status))
        break;
      const unsigned char* src = smem + S::stages * S::a_bytes + s * S::b_bytes;
      unsigned char* dst = wide + b * S::wide;
#pragma unroll
      for (int i = 0; i < NT * 8 / (32 * S::xwarps); ++i) {
        const int unit = t + i * 32 * S::xwarps, row = unit >> 3, u = unit & 7;
        const uint4 c = *reinterpret_cast<const uint4*>(src + row * 128 + ((u ^ (row & 7)) * 16));
        const uint2 a0 = widen4(c.x), a1 = widen4(c.y), a2 = widen4(c.z), a3 = widen4(c.w);
        unsigned char* line = dst + (u >> 2) * (NT * 128) + row * 128;
        const int j = 2 * (u & 3);
        *reinterpret_cast<uint4*>(line + ((j ^ (row & 7)) * 16)) = make_uint4(a0.x, a0.y, a1.x, a1.y);
        *reinterpret_cast<uint4*>(line + (((j + 1) ^ (row & 7)) * 16)) = make_uint4(a2.x, a2.y, a3.x, a3.y);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(empty0 + 8 * s);
        mbar_arrive(wide_full0 + 8 * b);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, S::tmem_cols);
  }
  if (split > 1) cluster_sync();
  // a thread takes four neighbouring columns of a row of x at a time, over the cluster's CTAs
  const int f = 4 * lane;
  const int64_t n = n0 + f;
  const int rows = (int)min((int64_t)NT, p.M - m0);
  float ws[4], bias[4];
  bool usual = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ws[i] = n + i < p.N ? p.ws[n + i] : 0.f;
    bias[i] = p.bias && n + i < p.N ? bias_at(p, n + i) : -0.f;
    usual = usual && usual_scale(ws[i]);
  }
  for (int c = rank + split * warp; c < rows; c += split * (S::threads / 32)) {
    const uint32_t at = smem_addr(sums) + (c * 128 + f) * 4;
    const float xs = p.xs[m0 + c];
    int v[8][4];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < split)
        asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[q][0]), "=r"(v[q][1]), "=r"(v[q][2]), "=r"(v[q][3])
                     : "r"(map_to_cta(at, q))
                     : "memory");
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int sum = v[0][i];
#pragma unroll
      for (int q = 1; q < 8; ++q)
        if (q < split) sum += v[q][i];
      y[i] = __int2float_rn(sum);
    }
    if (usual && usual_scale(xs)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(y[i], __fmul_rn(xs, ws[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = scaled_call(y[i], xs, ws[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __fadd_rn(y[i], bias[i]);
    store4(p, m0 + c, n, y);
  }
  if (split > 1) cluster_sync();  // no CTA leaves while another still reads its sums
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

struct Int8Plan {
  int kind;   // 0 plain, 1 CTA pairs, 2 few
  int nt;     // rows of x a tile
  int split;  // few: CTAs that share a tile's k
};

int64_t wide_ld(int64_t k) { return (k + 127) / 128 * 128; }  // a row in the workspace: whole blocks, zeros behind k

// By the sizes alone, so that the workspace's size goes by them too (a GB300's 152 SMs).
Int8Plan plan_int8(int64_t m, int64_t n, int64_t k) {
  if (k == 0) return Int8Plan{0, 0, 0};
  const int64_t blocks = (k + 127) / 128;
  Int8Plan few{0, m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128, 0};
  const int64_t few_n = (n + 127) / 128, few_m = (m + few.nt - 1) / few.nt;
  double few_us = 1e30;
  if (k % 16 != 0) {
    // few8_kernel cannot step over such rows: the plain kernel (3 us a step of 32 of k: 400 x 1000 x 3000 298 us), or
    // pairs, whose widening repacks wt
    few_us = 5 + 3 * (double)((((m + 63) / 64) * ((n + 63) / 64) + 1215) / 1216) * (double)((k + 31) / 32);
  } else if (few_n <= 65535 && few_m <= 65535) {
    const ClusterPlan c = plan_clusters(few_n * few_m, blocks, few.nt <= 32 ? 2 : 1, 6);
    few.kind = 2;
    few.split = c.split;
    few_us = 5.5 + 0.75 * (double)(c.waves * ((blocks + c.split - 1) / c.split));
    if (m <= 128) return few;  // (128 x 8192 x 8192 29.9 us, pairs 35.0; 64 x 5120 x 2048 9.4 and 15.3)
  }
  // Above: estimated microseconds, fitted to both kernels on 40 shapes (17 to 16384 rows).  A block takes a
  // pair 0.2 us of issuing and hand-overs and 1.6 ns a row of x.  E.g. (few / pairs) 200 x 512 x 4096 9.9 / 21.0,
  // 777 x 512 x 8192 17.0 / 36.1, 200 x 5120 x 13312 79 / 40, 256 x 8192 x 8192 52 / 30.
  Int8Plan pairs{0, 0, 0};
  double pairs_us = 1e30;
  // (Tiles of 32 rows would take as long a block as 64.)
  for (int nt = 64; nt <= kPair8Most; nt += 32) {
    const int64_t tiles = ((n + 255) / 256) * ((m + nt - 1) / nt), waves = (tiles + 75) / 76;
    const double block = 0.2 + 0.0016 * nt, us = 7 + (double)(waves * blocks) * (block < 0.34 ? 0.34 : block);
    if (tiles <= INT32_MAX && us <= pairs_us) {
      pairs_us = us;
      pairs = Int8Plan{1, nt, 0};
    }
  }
  if (k % 16 != 0) pairs_us += 3 + (double)n * (double)k * 4e-7;  // (repacking)
  return few_us <= pairs_us ? few : pairs;
}

// Rows of f16, whole blocks of 128, as [row][64 of k][which 64]: a box of two is a block of `rows` rows, one half behind
// the other.  (One copy instead of two a block: its thread spent 470 cycles a block on them.)
int encode_wide(CUtensorMap* map, const void* base, int64_t m, int64_t ld, int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  const int st = get_encoder(&enc);
  if (st != FAR_OK) return st;
  cuuint64_t dims[3] = {64, (cuuint64_t)m, (cuuint64_t)(ld / 64)}, strides[2] = {(cuuint64_t)ld * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)rows, 2}, estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FAR_OK : FAR_ERR_CUDA;
}

template <int NT> cudaError_t launch_few8(const CUtensorMap& mx, const CUtensorMap& mw, const Int8Params& p, int split, cudaStream_t s) {
  const cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(few8_kernel<NT>), Few8Shape<NT>::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)split, (unsigned)((p.N + 127ll) / 128), (unsigned)(((int64_t)p.M + NT - 1) / NT));
  cfg.blockDim = dim3(Few8Shape<NT>::threads);
  cfg.dynamicSmemBytes = Few8Shape<NT>::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = far_get_programmatic_launch() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, few8_kernel<NT>, mx, mw, p);
}

int run_int8(Int8Params& p, void* workspace, cudaStream_t s) {
  unsigned int* status = nullptr;
  int sms = 0;
  int st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  p.status = status;
  p.timeout_ns = kWaitTimeoutNs;
  const int64_t so = p.out_dtype == FAR_F32 ? 4 : 2;
  p.wide = (uintptr_t)p.out % (4 * so) == 0 && p.ldo % 4 == 0;
  Int8Plan g = plan_int8(p.M, p.N, p.K);
  if (g.kind == 2 && (!tma_rows(p.x, p.ldx, 1) || !tma_rows(p.wt, p.ldw, 1))) g.kind = 0;
  cudaError_t e;
  if (g.kind == 0) {
    const int64_t tiles = (((int64_t)p.M + 63) / 64) * (((int64_t)p.N + 63) / 64), cap = (int64_t)sms * 8;
    e = launch_k(plain_kernel, dim3((unsigned)(tiles < cap ? tiles : cap)), dim3(256), 0, s, p);
  } else if (g.kind == 2) {
    CUtensorMap mx, mw;
    st = encode_box(&mx, p.x, p.M, p.K, p.ldx, 1, g.nt, CU_TENSOR_MAP_DATA_TYPE_UINT8);
    if (st == FAR_OK) st = encode_box(&mw, p.wt, p.N, p.K, p.ldw, 1, 128, CU_TENSOR_MAP_DATA_TYPE_UINT8);
    if (st != FAR_OK) return st;
    e = g.nt == 16   ? launch_few8<16>(mx, mw, p, g.split, s)
        : g.nt == 32 ? launch_few8<32>(mx, mw, p, g.split, s)
        : g.nt == 64 ? launch_few8<64>(mx, mw, p, g.split, s)
                     : launch_few8<128>(mx, mw, p, g.split, s);
  } else {
    const int64_t ld = wide_ld(p.K);
    __half* wide = static_cast<__half*>(workspace);
    int8_t* packed = tma_rows(p.wt, p.ldw, 1) ? nullptr : reinterpret_cast<int8_t*>(wide + p.M * ld);
    p.packed = packed != nullptr;
    const WidenParams q{p.x, p.wt, wide, packed, p.ldx, p.ldw, p.M, p.N, ld, p.K, tma_rows(p.x, p.ldx, 1)};
    unsigned along = 16;  // threads: a row of one block of k has 16 units of 8 codes
    while (along < 256 && (int64_t)along * 8 < ld) along *= 2;
    const int64_t most = packed && p.N > p.M ? p.N : p.M, per = 256 / along, groups = (most + per - 1) / per, cap = (int64_t)sms * 64;
    e = launch_k(widen_kernel, dim3((unsigned)(groups < cap ? groups : cap), packed ? 2 : 1), dim3(along, (unsigned)per), 0, s, q);
    if (e != cudaSuccess) return cuda_error_status(e);
    Pair8Walk w{};
    w.nt = g.nt;
    w.tiles_m = (int32_t)(((int64_t)p.M + g.nt - 1) / g.nt);
    w.tiles_n = (int32_t)(((int64_t)p.N + 255) / 256);
    w.num_tiles = w.tiles_m * w.tiles_n;
    w.blocks = (p.K + 127) / 128;
    w.xhalf = (uint32_t)g.nt * 64;
    const uint32_t xslots = kPair8XBytes / (2 * w.xhalf), aslots = (uint32_t)(512 - 2 * g.nt) / 64;
    w.xslots = xslots < kPair8Slots ? xslots : kPair8Slots;
    w.aslots = aslots < kPair8Slots ? aslots : kPair8Slots;
    CUtensorMap mx, mw;
    st = encode_wide(&mx, wide, p.M, ld, g.nt / 2);
    if (st == FAR_OK) st = encode_box(&mw, packed ? packed : p.wt, p.N, p.K, packed ? ld : p.ldw, 1, 128, CU_TENSOR_MAP_DATA_TYPE_UINT8);
    if (st != FAR_OK) return st;
    e = ensure_smem_attribute(reinterpret_cast<const void*>(pair8_kernel), kPair8Smem);
    const int pairs = w.num_tiles < sms / 2 ? w.num_tiles : sms / 2;
    if (e == cudaSuccess) e = launch_k(pair8_kernel, dim3(2 * pairs), dim3(kPair8Threads), kPair8Smem, s, mx, mw, p, w);
  }
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
  return m && n && plan_int8(m, n, k).kind == 1 ? (2 * m + n) * wide_ld(k) : 0;  // x as f16, and wt's codes in case TMA cannot read them as they stand
}

extern "C" int far_plan_gemm_int8(int64_t m, int64_t n, int64_t k, int* out3) {
  if (!out3) return FAR_ERR_NULL;
  if (m < 1 || n < 1 || k < 1 || m > INT32_MAX || n > INT32_MAX || k > 131071) return FAR_ERR_SHAPE;
  const Int8Plan g = plan_int8(m, n, k);
  out3[0] = g.kind;
  out3[1] = g.kind ? g.nt : 0;
  out3[2] = g.split;
  return FAR_OK;
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
  const int64_t bytes = far_gemm_int8_workspace_bytes(m, n, k);
  if (bytes > 0) {
    if (!workspace || workspace_bytes < bytes || ((uintptr_t)workspace & 15)) return FAR_ERR_WORKSPACE;
    const int64_t so = out_dtype == FAR_F32 ? 4 : 2;
    const Region W = region(workspace, 1, bytes, 0);
    const Region rest[6] = {region(x, m, k, p.ldx), region(wt, n, k, p.ldw), region(x_scale, 1, m * 4, 0), region(wt_scale, 1, n * 4, 0),
                            region(bias, bias ? 1 : 0, n * so, 0), region(out, m, n * so, p.ldo * so)};
    for (const Region& r : rest)
      if (regions_overlap(W, r)) return FAR_ERR_ALIAS;
  }
  return run_int8(p, workspace, static_cast<cudaStream_t>(stream));
}
