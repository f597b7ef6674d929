// A matrix quantised to int8 with a scale a row (quant_rows_int8), and the product of two such
// matrices (gemm_int8):
//   out[i, j] = RNE( fl32(sum_k x[i, k] wt[j, k]) (xs[i] ws[j]) + bias[j] ),  the sum an exact integer.
//
// rows_kernel   a row's 16-byte chunks in the registers of 1 to 16 warps: its maximum is known
//               before its values are needed again, so each is read once.  Bound by HBM.
// long_kernel   any length and alignment: a row read twice, the second time mostly from L2.
//
// sm_103a's tcgen05 multiplies no integers, but f16 holds every code exactly, a product of two is at
// most 2^14 in magnitude, and the binary32 sum of 1024 of them at most 2^24: exact.  So the
// products run at the tensor cores' f16 rate, and the sums move from TMEM to int32 every 1024 of k.
//
// widen_kernel  both operands as f16, into the workspace, for
// pair16_kernel the product of many rows, on the tensor cores of CTA pairs.
// few8_kernel   few rows of x (a decode batch): codes are widened on their way from shared memory to
//               the tensor cores, wt's rows into TMEM, x's into shared memory.  Bound by reading wt once.
// plain_kernel  the product for any shape, stride and alignment: 64 x 64 tiles in int32.
#include <cuda_runtime.h>
#include <stdint.h>

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
  const int8_t* src[2];  // x, wt
  __half* dst[2];        // rows of `ld` values
  int64_t ldsrc[2], rows[2], ld;
  int32_t K;
  int32_t vec[2];        // whole 16-byte chunks of the source's rows may be read
};

// A thread takes 16 codes of a row (past k: zeros); neighbouring threads neighbouring chunks.
__global__ void __launch_bounds__(256) widen_kernel(const WidenParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t per = p.ld / 16, first = per * p.rows[0], total = first + per * p.rows[1];
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int which = i >= first;
    const int64_t j = which ? i - first : i, row = j / per;
    const int k = (int)(j - row * per) * 16;
    const int8_t* src = (which ? p.src[1] : p.src[0]) + row * (which ? p.ldsrc[1] : p.ldsrc[0]) + k;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if ((which ? p.vec[1] : p.vec[0]) && k + 16 <= p.K) {
      load_bytes<16>(src, w);
    } else {
#pragma unroll
      for (int b = 0; b < 16; ++b)
        if (k + b < p.K) w[b >> 2] |= (uint32_t)(uint8_t)src[b] << (8 * (b & 3));
    }
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint2 v = widen4(w[e]);
      h[2 * e] = v.x;
      h[2 * e + 1] = v.y;
    }
    __half* dst = (which ? p.dst[1] : p.dst[0]) + row * p.ld + k;
    store_bytes<16>(dst, h);
    store_bytes<16>(dst + 8, h + 4);
  }
}

// ---------------------------------------------------------------------------
// many rows: tensor cores over CTA pairs
// ---------------------------------------------------------------------------

struct Int8Out {
  PairOut out;
  Int8Params p;
};

struct Int8Epilogue {
  static constexpr bool kAMn = false, kBMn = false, kSplit = false, kDouble = false;
  static constexpr int kWidth = 256, kStep = 32, kFlush = 16;  // 1024 of k
  using Params = Int8Out;
  static __device__ __forceinline__ bool tile(PairTileAt& at, const PairMaps& maps, const PairWalk& w, const Params& e) {
    const int first = at.part * 128, mine = at.item.cols - first;
    const int64_t row0 = (int64_t)at.item.tm * 256 + at.rank * 128 + at.quarter * 32, row = row0 + at.lane;
    const int64_t col0 = at.item.col0 + first;
    const int chunks = (w.slices + kFlush - 1) / kFlush;
    int acc[128];
#pragma unroll
    for (int i = 0; i < 128; ++i) acc[i] = 0;
    // (all 128 columns always: those past a narrow tile's hold what nobody stores)
#pragma unroll 1
    for (int k = 0; k < chunks; ++k) {
      uint32_t t;
      if (!at.next(w, t)) return false;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tmem_ld32_sync(t + first + 32 * c, r);
        if (c == 3) at.release();
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[32 * c + i] += __float2int_rn(__uint_as_float(r[i]));
      }
    }
    if (mine <= 0) return true;
    const Int8Params& p = e.p;
    const float xs = row < p.M ? p.xs[row] : 0.f;
    const bool f32 = p.out_dtype == FAR_F32;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (32 * c >= mine) break;
      const int64_t mycol = col0 + 32 * c + at.lane;  // a lane holds one column's scale and bias
      const float ws = mycol < p.N ? p.ws[mycol] : 0.f;
      const float bias = p.bias && mycol < p.N ? bias_at(p, mycol) : 0.f;
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        v[i] = scaled(__int2float_rn(acc[32 * c + i]), xs, __shfl_sync(0xffffffffu, ws, i));
        if (p.bias) v[i] = __fadd_rn(v[i], __shfl_sync(0xffffffffu, bias, i));
      }
      if (f32 || (c & 1) == 0) pair_begin_box(e.out, at.lane);
      uint32_t o[32];
      if (f32) narrow<FAR_F32, 32>(v, o);
      else if (p.out_dtype == FAR_F16) narrow<FAR_F16, 32>(v, o);
      else narrow<FAR_BF16, 32>(v, o);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (u < 4 || f32) {
          const int unit = (f32 || (c & 1) == 0 ? u : u + 4) ^ (at.lane & 7);
          *reinterpret_cast<uint4*>(at.box + at.lane * 128 + unit * 16) = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
      }
      if (f32 || (c & 1) == 1 || mine <= 32 * (c + 1))
        pair_store_box(e.out, &maps.out[0], at.box, at.lane, row0, col0 + (f32 ? 32 * c : 64 * (c / 2)));
    }
    return true;
  }
};

// ---------------------------------------------------------------------------
// few8_kernel: 128 rows of wt x NT rows of x a CTA, the blocks of 128 of k shared out over a cluster of
// gridDim's x dimension (CTA rank r takes blocks KB r / S .. KB (r + 1) / S - 1).
//   warps 0-3  wt's codes of one row a thread from shared memory, widened, into TMEM: A, two blocks
//   warps 4-   the sums, 4 or 8 warps: to int32 every 8 blocks
//   then       a TMA producer, an MMA issuer (and TMEM), and 2 or 4 warps that widen x's codes into
//              shared memory: B, two blocks
// Then each CTA leaves its sums in its shared memory and adds up every S-th row of x over the
// cluster's CTAs (integers: in any order the same), scales and stores.
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
  const int64_t n = n0 + (threadIdx.x & 127);
  const uint32_t mine = smem_addr(sums) + (threadIdx.x & 127) * 4;
  const float ws = n < p.N ? p.ws[n] : 0.f;
  constexpr int GROUPS = S::threads / 128;
  if ((int)(threadIdx.x >> 7) < GROUPS)
    for (int c = rank + split * (int)(threadIdx.x >> 7); c < NT && m0 + c < p.M; c += GROUPS * split) {
      int v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < split) {
          const uint32_t a = map_to_cta(mine + c * 512, q);
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[q]) : "r"(a) : "memory");
        }
      int s = v[0];
#pragma unroll
      for (int q = 1; q < 8; ++q)
        if (q < split) s += v[q];
      if (n < p.N) store_one(p, m0 + c, n, s, p.xs[m0 + c], ws);
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
  int kind;   // 0 plain, 1 widened, over CTA pairs, 2 few
  int nt;     // few: rows of x a CTA
  int split;  // few: CTAs that share a tile's k
};

// What does not go by alignment, so that the workspace's size does not.
constexpr int kFewRows = 256;
bool many_rows(int64_t m, int64_t n, int64_t k) {
  return k > 0 && m > kFewRows && ((m + 255) / 256) * ((n + 255) / 256) <= INT32_MAX;
}
int64_t wide_ld(int64_t k) { return (k + 15) / 16 * 16; }

Int8Plan plan_int8(const Int8Params& p, int sms) {
  Int8Plan g{0, 0, 0};
  if (many_rows(p.M, p.N, p.K)) {
    g.kind = 1;
    return g;
  }
  const int64_t tiles_n = ((int64_t)p.N + 127) / 128, KB = (p.K + 127) / 128;
  g.nt = p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
  const int64_t tiles_m = ((int64_t)p.M + g.nt - 1) / g.nt, slots = (g.nt <= 32 ? 2ll : 1ll) * sms;
  if (p.K == 0 || !tma_rows(p.x, p.ldx, 1) || !tma_rows(p.wt, p.ldw, 1) || tiles_n > 65535 || tiles_m > 65535) return g;
  // k is shared out while there are free places for it, not below two blocks a CTA
  g.split = 1;
  while (g.split < 8 && tiles_n * tiles_m * g.split * 2 <= slots && KB >= 4 * g.split) g.split *= 2;
  g.kind = 2;
  return g;
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
  const Int8Plan g = plan_int8(p, sms);
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
    __half* wx = static_cast<__half*>(workspace);
    WidenParams q{{p.x, p.wt}, {wx, wx + p.M * ld}, {p.ldx, p.ldw}, {p.M, p.N}, ld, p.K, {tma_rows(p.x, p.ldx, 1), tma_rows(p.wt, p.ldw, 1)}};
    const int64_t blocks = (((int64_t)p.M + p.N) * (ld / 16) + 255) / 256, cap = (int64_t)sms * 32;
    e = launch_k(widen_kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, s, q);
    if (e != cudaSuccess) return cuda_error_status(e);
    PairMaps maps{};
    Int8Out out{};
    out.p = p;
    st = encode_operand(&maps.a[0], q.dst[0], p.M, p.K, ld, FAR_F16);
    if (st == FAR_OK) st = encode_operand(&maps.b[0], q.dst[1], p.N, p.K, ld, FAR_F16);
    if (st == FAR_OK) st = pair_output(&out.out, &maps.out[0], p.out, p.M, p.N, p.ldo, p.out_dtype);
    if (st != FAR_OK) return st;
    PairWalk w{};
    w.tiles_m = (int32_t)(((int64_t)p.M + 255) / 256);
    w.tiles_n = (int32_t)(((int64_t)p.N + 255) / 256);
    w.num_tiles = w.tiles_m * w.tiles_n;
    w.columns = p.N;
    w.slices = (p.K + 63) / 64;
    w.pairs = 1;
    w.status = status;
    w.timeout_ns = kWaitTimeoutNs;
    e = launch_pair16<Int8Epilogue>(maps, w, out, sms, s);
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
  return many_rows(m, n, k) ? (m + n) * wide_ld(k) * 2 : 0;  // both operands as f16
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
