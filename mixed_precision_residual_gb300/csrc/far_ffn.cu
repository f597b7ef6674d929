// The gated feed-forward block's way in and its gradients, on 16-bit tensors (gated_ffn,
// gated_ffn_backward):
//   gate = x wg^T, up = x wu^T (binary32),  h = RNE(act(gate) up)
//   dgate = RNE(dh up act'(gate)), dup = RNE(dh act(gate)),
//   dx = RNE(dgate wg + dup wu),  dwg = RNE(dgate^T x),  dwu = RNE(dup^T x).
//
// pair16_kernel  many tokens and every product of the way back: tensor cores over CTA pairs.  The way in
//                gives a pair 128 columns of both weights at once, gate in one half of the accumulator
//                and up in the other, so that act(gate) up is formed where they meet.
// few_kernel     few tokens (a decode batch): the weights' rows on the TMEM lanes, 64 of each a CTA, 16 to
//                128 tokens as the columns, k split over a cluster.  Bound by reading the weights once.
// slope_kernel   dgate and dup, into the workspace.  Bound by HBM.
// plain_gate_kernel, plain_product_kernel  any shape, stride and alignment: 64 x 64 tiles in binary32.
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

namespace far {

namespace {

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------

// sigma(z) and sigma(z) (1 - sigma(z)), from e = exp(-|z|) <= 1, so that nothing overflows and both
// keep their relative precision at either end.  (ex2.approx's argument z log2(e) carries |z| 2^-24
// of error: 2^-17 of the value at |z| = 88, where binary32 ends.)
struct Sigma {
  float s, slope;
};
__device__ __forceinline__ Sigma sigma(float z) {
  const float e = __expf(-fabsf(z)), r = __fdividef(1.0f, __fadd_rn(1.0f, e));
  return Sigma{z < 0.f ? __fmul_rn(e, r) : r, __fmul_rn(__fmul_rn(e, r), r)};
}

constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi): (1 + tanh(y)) / 2 = sigma(2 y)
constexpr float kTanhCube = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// The cubic's argument saturates sigma long before |g| = 32; held there, so that g^2 stays finite.
// (A comparison, not fminf, so that NaN stays.)
__device__ __forceinline__ float held(float g) { return fabsf(g) > 32.f ? copysignf(32.f, g) : g; }
__device__ __forceinline__ float tanh_argument(float g) {
  return __fmul_rn(kTanhScale * g, __fmaf_rn(kTanhCube, __fmul_rn(g, g), 1.0f));
}

template <int ACT> __device__ __forceinline__ float activation(float g) {
  if constexpr (ACT == FAR_ACT_SILU) return __fmul_rn(g, sigma(g).s);
  else if constexpr (ACT == FAR_ACT_GELU) return __fmul_rn(g, normcdff(g));
  else return __fmul_rn(g, sigma(tanh_argument(held(g))).s);
}

// (act(g), act'(g))
template <int ACT> __device__ __forceinline__ float2 activation_slope(float g) {
  if constexpr (ACT == FAR_ACT_SILU) {
    const Sigma s = sigma(g);
    return make_float2(__fmul_rn(g, s.s), __fmaf_rn(g, s.slope, s.s));
  } else if constexpr (ACT == FAR_ACT_GELU) {
    const float c = normcdff(g), h = held(g);
    return make_float2(__fmul_rn(g, c), __fmaf_rn(h, __fmul_rn(kInvSqrt2Pi, __expf(__fmul_rn(-0.5f * h, h))), c));
  } else {
    const float h = held(g);
    const Sigma s = sigma(tanh_argument(h));
    const float inner = __fmul_rn(kTanhScale, __fmaf_rn(3.0f * kTanhCube, __fmul_rn(h, h), 1.0f));
    return make_float2(__fmul_rn(g, s.s), __fmaf_rn(__fmul_rn(h, s.slope), inner, s.s));
  }
}

template <int DT> __device__ __forceinline__ float value16(const uint16_t* p, int64_t i) { return widen2<DT>(p[i]).x; }
template <int DT> __device__ __forceinline__ uint16_t round16(float v) { return (uint16_t)narrow2<DT>(v, 0.f); }

// f(std::integral_constant<DT>, std::integral_constant<ACT>) of a call's dtype and activation
template <class F> auto with_types(int dtype, int act, const F& f) {
  auto typed = [&](auto dt) {
    switch (act) {
      case FAR_ACT_SILU: return f(dt, std::integral_constant<int, FAR_ACT_SILU>{});
      case FAR_ACT_GELU: return f(dt, std::integral_constant<int, FAR_ACT_GELU>{});
      default: return f(dt, std::integral_constant<int, FAR_ACT_GELU_TANH>{});
    }
  };
  return dtype == FAR_F16 ? typed(std::integral_constant<int, FAR_F16>{}) : typed(std::integral_constant<int, FAR_BF16>{});
}

// ---------------------------------------------------------------------------
// tensor cores over CTA pairs
// ---------------------------------------------------------------------------

// 32 columns of a row, 16 words, into the warp's box: 16-byte units 4 half .. 4 half + 3
__device__ __forceinline__ void box_words(unsigned char* box, int lane, int half, const uint32_t (&v)[16]) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    *reinterpret_cast<uint4*>(box + lane * 128 + (((4 * half + u) ^ (lane & 7)) * 16)) = make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
}

struct PairOuts {
  PairOut out[3];
};

// The way in: gate in columns 0 .. cols - 1, up in cols .. 2 cols - 1.  SAVE: out, gate and up one after
// the other, each from the accumulator again.
template <int DT, int ACT, bool SAVE> struct GateEpilogue {
  static constexpr bool kAMn = false, kBMn = false, kSplit = true, kDouble = false, kBeside = false;
  static constexpr int kWidth = 128, kStep = 16;
  using Params = PairOuts;
  static __device__ __forceinline__ bool tile(PairTileAt& at, const PairMaps& maps, const PairWalk& p, const Params& e) {
    uint32_t t;
    if (!at.next(p, t)) return false;
    const int cols = at.item.cols, first = at.part * 64, mine = cols - first;
    const int64_t row = (int64_t)at.item.tm * 256 + at.rank * 128 + at.quarter * 32, col = at.item.col0 + first;
    if (mine <= 0) {
      at.release();
      return true;
    }
    constexpr int OUTS = SAVE ? 3 : 1;
#pragma unroll 1
    for (int j = 0; j < OUTS; ++j) {
      pair_begin_box(at.lane);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (32 * c >= mine) break;
        uint32_t g[32], u[32], v[16];
        tmem_ld32x2_sync(t + first + 32 * c, t + cols + first + 32 * c, g, u);
        if (j == OUTS - 1 && (c == 1 || mine <= 32)) at.release();
        if (SAVE && j > 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = j == 1 ? narrow2<DT>(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]))
                          : narrow2<DT>(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = narrow2<DT>(__fmul_rn(activation<ACT>(__uint_as_float(g[2 * i])), __uint_as_float(u[2 * i])),
                               __fmul_rn(activation<ACT>(__uint_as_float(g[2 * i + 1])), __uint_as_float(u[2 * i + 1])));
        }
        box_words(at.box, at.lane, c, v);
      }
      pair_store_box(e.out[j], &maps.out[j], at.box, at.lane, row, col);
    }
    return true;
  }
};

// The products of the way back, rounded.  dx: rows of dgate and dup, both summed; the weights' rows are k.
// WEIGHTS: dgate and dup give the rows of one output each, tokens are k; launched behind dx, which lets it start
// beside itself (as every kernel of dx does).
template <int DT, bool WEIGHTS> struct ProductEpilogue {
  static constexpr bool kAMn = WEIGHTS, kBMn = true, kSplit = false, kDouble = WEIGHTS, kBeside = WEIGHTS;
  static constexpr int kWidth = 256, kStep = 32;
  using Params = PairOuts;
  static __device__ __forceinline__ bool tile(PairTileAt& at, const PairMaps& maps, const PairWalk& p, const Params& e) {
    uint32_t t;
    if (!at.next(p, t)) return false;
    const int first = at.part * 128, mine = at.item.cols - first;
    const int tiles = WEIGHTS ? p.tiles_m / 2 : p.tiles_m, which = WEIGHTS && at.item.tm >= tiles ? 1 : 0;
    const int64_t row = (int64_t)(at.item.tm - which * tiles) * 256 + at.rank * 128 + at.quarter * 32;
    if (mine <= 0) {
      at.release();
      return true;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (32 * c >= mine) break;
      uint32_t r[32], v[16];
      tmem_ld32_sync(t + first + 32 * c, r);
      const bool last = c == 3 || mine <= 32 * (c + 1);
      if (last) at.release();
      if ((c & 1) == 0) pair_begin_box(at.lane);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = narrow2<DT>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      box_words(at.box, at.lane, c & 1, v);
      if ((c & 1) == 1 || last)
        pair_store_box(e.out[which], &maps.out[which], at.box, at.lane, row, at.item.col0 + first + 64 * (c >> 1));
    }
    return true;
  }
};

// ---------------------------------------------------------------------------
// plain kernels
// ---------------------------------------------------------------------------

struct GateParams {
  const uint16_t *x, *wg, *wu;
  uint16_t *out, *gate, *up;                    // gate and up may be null
  int64_t ldx, ldwg, ldwu, ldo, ldgate, ldup;   // elements
  int32_t M, F, K;                              // tokens, ffn, hidden
};

// 64 x 64 outputs a CTA of 256 threads, 4 x 4 a thread (16 apart), both projections at once.
template <int DT, int ACT> __global__ void __launch_bounds__(256) plain_gate_kernel(const GateParams p) {
  __shared__ float xs[16][65], gs[16][65], us[16][65];
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t tiles_n = ((int64_t)p.F + 63) / 64, tiles = tiles_n * (((int64_t)p.M + 63) / 64);
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t m0 = t / tiles_n * 64, n0 = t % tiles_n * 64;
    float g[4][4] = {}, u[4][4] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += 16) {
      __syncthreads();
      for (int i = threadIdx.x; i < 64 * 16; i += 256) {
        const int r = i >> 4, k = i & 15;
        const bool in = k0 + k < p.K;
        xs[k][r] = in && m0 + r < p.M ? value16<DT>(p.x, (m0 + r) * p.ldx + k0 + k) : 0.f;
        gs[k][r] = in && n0 + r < p.F ? value16<DT>(p.wg, (n0 + r) * p.ldwg + k0 + k) : 0.f;
        us[k][r] = in && n0 + r < p.F ? value16<DT>(p.wu, (n0 + r) * p.ldwu + k0 + k) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float a[4], b[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = xs[k][ty + 16 * i], b[i] = gs[k][tx + 16 * i], c[i] = us[k][tx + 16 * i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            g[i][j] = __fmaf_rn(a[i], b[j], g[i][j]);
            u[i][j] = __fmaf_rn(a[i], c[j], u[i][j]);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m >= p.M || n >= p.F) continue;
        p.out[m * p.ldo + n] = round16<DT>(__fmul_rn(activation<ACT>(g[i][j]), u[i][j]));
        if (p.gate) {
          p.gate[m * p.ldgate + n] = round16<DT>(g[i][j]);
          p.up[m * p.ldup + n] = round16<DT>(u[i][j]);
        }
      }
  }
}

// out[i, j] = RNE( sum over `pairs` operand pairs and k of a[i sai + k sak] b[j sbj + k sbk] )
struct ProductParams {
  const uint16_t *a[2], *b[2];
  uint16_t* out;
  int64_t sai[2], sak[2], sbj[2], sbk[2], ldo;
  int32_t M, N, K, pairs;
};
template <int DT> __global__ void __launch_bounds__(256) plain_product_kernel(const ProductParams p) {
  __shared__ float as[32][65], bs[32][65];
  pdl_wait();
  pdl_launch_dependents();  // (behind the wait for what runs beside dx)
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t tiles_n = ((int64_t)p.N + 63) / 64, tiles = tiles_n * (((int64_t)p.M + 63) / 64);
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t m0 = t / tiles_n * 64, n0 = t % tiles_n * 64;
    float acc[4][4] = {};
    for (int q = 0; q < p.pairs; ++q) {
      const bool ak = p.sak[q] == 1, bk = p.sbk[q] == 1;  // neighbours in memory: along k, or along the rows
      for (int64_t k0 = 0; k0 < p.K; k0 += 32) {
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * 32; i += 256) {
          const int ra = ak ? i >> 5 : i & 63, ka = ak ? i & 31 : i >> 6;
          const int rb = bk ? i >> 5 : i & 63, kb = bk ? i & 31 : i >> 6;
          as[ka][ra] = k0 + ka < p.K && m0 + ra < p.M ? value16<DT>(p.a[q], (m0 + ra) * p.sai[q] + (k0 + ka) * p.sak[q]) : 0.f;
          bs[kb][rb] = k0 + kb < p.K && n0 + rb < p.N ? value16<DT>(p.b[q], (n0 + rb) * p.sbj[q] + (k0 + kb) * p.sbk[q]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float a[4], b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = as[k][ty + 16 * i], b[i] = bs[k][tx + 16 * i];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(a[i], b[j], acc[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < p.M && n < p.N) p.out[m * p.ldo + n] = round16<DT>(acc[i][j]);
      }
  }
}

// ---------------------------------------------------------------------------
// few_kernel: 128 rows of weights x NT tokens a CTA, the slices of 64 of k shared out over a cluster of
// gridDim's x dimension (CTA rank r takes slices KB r / S .. KB (r + 1) / S - 1).
//   warp 0 TMA producer, 1 MMA issuer (and TMEM), 4-7 read the sums
// Each CTA leaves its sums in its shared memory; the cluster's CTAs add up every S-th token over all of
// them, in the order of k, and form the outputs.
// Bound by reading the weights: 1 x 5120 x 13312 43.7 us (6.2 TB/s), 1 x 2048 x 5632 10.4 (4.4), 1 x 1024 x 1024 4.0; what
// is not bytes is the launch, the set-up and the sum over the cluster, 3 to 4 us (7 with 128 tokens, whose
// sums are eight times as many).  Rows off 128 bytes cost two: 60 x 2056 x 5640 14.0 us, 48 x 2048 x 5632
// 11.9.  (Sums read a value at a time from the other CTAs, not four: 100 x 5120 x 13312 54.6 us against 49.5.)
//   GATE  64 rows of either weight: gate in lanes 0 .. 63, up in 64 .. 127
//   else  dx: 128 columns of the weights (mn-major), k all rows of w_gate and then all of w_up
// ---------------------------------------------------------------------------
struct FewParams {
  uint16_t *out, *gate, *up;     // gate and up may be null
  int64_t ldo, ldgate, ldup;     // elements
  int32_t M, N;                  // tokens, columns of an output
  int32_t slices, half;          // of k; dx: of which the first `half` are w_gate's
  int32_t wide;                  // bits: out's, gate's, up's rows start on 8 bytes
  unsigned int* status;
  uint64_t timeout_ns;
};
struct FewMaps {
  CUtensorMap w[2], x[2];  // GATE: x[0] alone
};

constexpr int kFewThreads = 256;
template <int NT> struct FewShape {
  static constexpr int ctas = 2;  // an SM
  static constexpr uint32_t a_bytes = 2 * kPair16Box, b_bytes = NT * 128;
  static constexpr int stages = NT == 16 ? 6 : NT == 32 ? 5 : NT == 64 ? 4 : 3;
  static constexpr uint32_t ring = stages * (a_bytes + b_bytes);
  static constexpr uint32_t tmem_cols = NT < 32 ? 32 : NT;
  static constexpr int bars = 2 * stages + 1;
  static constexpr size_t smem = ring + bars * 8 + 16 + 1024;
  static_assert(NT * 128 * 4 <= ring, "the sums that the cluster adds up lie in the ring");
};

// four neighbouring rows' sums over the cluster's CTAs, in their order
__device__ __forceinline__ void cluster_sums4(uint32_t at, int split, float (&sum)[4]) {
  float v[8][4];
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < split)
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[q][0]), "=f"(v[q][1]), "=f"(v[q][2]), "=f"(v[q][3])
                   : "r"(map_to_cta(at, q))
                   : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = v[0][i];
#pragma unroll
  for (int q = 1; q < 8; ++q)
    if (q < split) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = __fadd_rn(sum[i], v[q][i]);
    }
}

// four neighbouring values of an output row, in one store where the row allows it
template <int DT> __device__ __forceinline__ void store4(uint16_t* row, int64_t n, int64_t N, bool wide, const float (&v)[4]) {
  const uint32_t lo = narrow2<DT>(v[0], v[1]), hi = narrow2<DT>(v[2], v[3]);
  if (wide && n + 4 <= N) {
    *reinterpret_cast<uint2*>(row + n) = make_uint2(lo, hi);
    return;
  }
  const uint16_t h[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < N) row[n + i] = h[i];
}

template <int NT, int DT, int ACT, bool GATE>
__global__ void __launch_bounds__(kFewThreads, FewShape<NT>::ctas)
    few_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewParams p) {
  using S = FewShape<NT>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);  // the same offset in every CTA
  const uint32_t a_base = smem_addr(smem), b_base = a_base + S::stages * S::a_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::ring);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + S::bars);
  const uint32_t full0 = smem_addr(&bars[0]), empty0 = full0 + 8 * S::stages, done = empty0 + 8 * S::stages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = (int)gridDim.x, rank = (int)blockIdx.x;  // the cluster spans gridDim.x
  constexpr int ROWS = GATE ? 64 : 128;  // of the output's columns
  const int64_t n0 = (int64_t)blockIdx.y * ROWS, m0 = (int64_t)blockIdx.z * NT;
  const int kb0 = (int)((int64_t)p.slices * rank / split), kb1 = (int)((int64_t)p.slices * (rank + 1) / split);

  // the ring's first load of the weights starts for L2 while the CTA is set up and the kernel ahead drains
  if (warp == 3 && lane == 0)
    for (int kb = kb0; kb < kb1 && kb < kb0 + S::stages; ++kb) {
      if constexpr (GATE) {
        tma_prefetch_2d(&maps.w[0], kb * 64, (int)n0);
        tma_prefetch_2d(&maps.w[1], kb * 64, (int)n0);
      } else {
        const int q = kb >= p.half, k = (kb - (q ? p.half : 0)) * 64;
        tma_prefetch_2d(&maps.w[q], (int)n0, k);
        tma_prefetch_2d(&maps.w[q], (int)n0 + 64, k);
      }
    }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done, 1);
    fence_barrier_init();
    tma_prefetch_map(&maps.x[0]);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), S::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();  // (not before the TMEM columns are this CTA's; behind the wait for what runs beside dx)

  float* sums = reinterpret_cast<float*>(smem);
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
        const uint32_t a = a_base + s * S::a_bytes, b = b_base + s * S::b_bytes;
        if constexpr (GATE) {
          tma_load_2d(a, &maps.w[0], kb * 64, (int)n0, full0 + 8 * s);
          tma_load_2d(a + kPair16Box, &maps.w[1], kb * 64, (int)n0, full0 + 8 * s);
          tma_load_2d(b, &maps.x[0], kb * 64, (int)m0, full0 + 8 * s);
        } else {
          const int q = kb >= p.half, k = (kb - (q ? p.half : 0)) * 64;
          tma_load_2d(a, &maps.w[q], (int)n0, k, full0 + 8 * s);
          tma_load_2d(a + kPair16Box, &maps.w[q], (int)n0 + 64, k, full0 + 8 * s);
          tma_load_2d(b, &maps.x[q], k, (int)m0, full0 + 8 * s);
        }
      }
      // Before the CTA may leave the last slices must have landed and their slots been freed by the MMA
      // issuer's last commits (the barriers they arrive on go with the CTA).
      const uint32_t last = g > (uint32_t)S::stages ? g - S::stages : 0u;
      for (uint32_t j = last; j < g; ++j)
        mbar_wait(full0 + 8 * (j % S::stages), (j / S::stages) & 1u, p.timeout_ns, p.status);
      for (uint32_t j = last; running && j < g; ++j)
        running = mbar_wait(empty0 + 8 * (j % S::stages), (j / S::stages) & 1u, p.timeout_ns, p.status);
    }
  } else if (warp == 1) {
    constexpr uint32_t IDESC = umma_idesc_16(128, NT, DT == FAR_BF16, !GATE, false);
    constexpr uint32_t a_step = GATE ? 2 : 128;
    const bool leader = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t a0 = GATE ? sw128_kmajor_desc(a_base) : sw128_mnmajor_desc(a_base, kPair16Box), x0 = sw128_kmajor_desc(b_base);
    uint32_t s = 0, s_phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(full0 + 8 * s, s_phase, p.timeout_ns, p.status)) break;
      tc_fence_after();
      const uint64_t a = a0 + s * (S::a_bytes >> 4), x = x0 + s * (S::b_bytes >> 4);
      if (leader) {
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f16(tm, a + k * a_step, x + 2 * k, IDESC, (kb != kb0) | (k != 0));
        umma_commit(empty0 + 8 * s);
        if (kb == kb1 - 1) umma_commit(done);
      }
      __syncwarp();
      if (++s == S::stages) {
        s = 0;
        s_phase ^= 1;
      }
    }
  } else if (warp >= 4) {
    // (a wait that runs out leaves the error word set and the outputs undefined)
    mbar_wait(done, 0u, p.timeout_ns, p.status);
    tc_fence_after();
    // every MMA has read its operands, so every copy has landed: the ring now takes this CTA's sums [NT][128]
    const uint32_t src = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    constexpr int W = NT == 16 ? 16 : 32;  // columns a load
#pragma unroll
    for (int c = 0; c < NT; c += W) {
      uint32_t r[W];
      if constexpr (W == 32) tmem_ld32(src + c, r);
      else tmem_ld16(src + c, r);
      tmem_ld_wait(r);
#pragma unroll
      for (int i = 0; i < W; ++i) sums[(c + i) * 128 + (int)threadIdx.x - 128] = __uint_as_float(r[i]);
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::tmem_cols);
  }
  if (split > 1) cluster_sync();
  // A thread takes four neighbouring columns of a token: a trip to another CTA's shared memory costs most
  // of a microsecond, so few and wide ones.
  constexpr int QUADS = ROWS / 4, SETS = kFewThreads / QUADS;
  const int f = 4 * (int)(threadIdx.x % QUADS);
  const int64_t n = n0 + f;
  const int tokens = (int)min((int64_t)NT, p.M - m0);
  for (int c = rank + split * (int)(threadIdx.x / QUADS); c < tokens; c += SETS * split) {
    const uint32_t at = smem_addr(sums) + (c * 128 + f) * 4;
    const int64_t m = m0 + c;
    float a[4];
    cluster_sums4(at, split, a);
    if constexpr (GATE) {
      float b[4], h[4];
      cluster_sums4(at + 256, split, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __fmul_rn(activation<ACT>(a[i]), b[i]);
      store4<DT>(p.out + m * p.ldo, n, p.N, p.wide & 1, h);
      if (p.gate) {
        store4<DT>(p.gate + m * p.ldgate, n, p.N, p.wide & 2, a);
        store4<DT>(p.up + m * p.ldup, n, p.N, p.wide & 4, b);
      }
    } else {
      store4<DT>(p.out + m * p.ldo, n, p.N, p.wide & 1, a);
    }
  }
  if (split > 1) cluster_sync();  // no CTA leaves while another still reads its sums
}

// ---------------------------------------------------------------------------
// dgate and dup: rows of `ld` elements, a multiple of 8, in the workspace, rounded to 16 bits: kind::f16 is the
// tensor cores' rate of 1.9 PFLOP/s and takes nothing wider (tf32 halves it and doubles the bytes).  It costs
// as much error as the result's own rounding (8192 x 4096 x 8192 in bf16: 2.34e-3 of a gradient's size, with
// binary32 operands 1.65e-3), and in f16 the range: 65520 and more is infinite.  Written once, because every column of
// dx's tiles and both weights' gradients read them again as the tensor cores' operands.  Bound by HBM, five
// tensors: 4096 x 8192 48 us (7.0 TB/s); 7 % of the way back of 8192 x 4096 x 8192.
// ---------------------------------------------------------------------------

struct SlopeParams {
  const uint16_t *dh, *gate, *up;
  uint16_t *dgate, *dup;
  int64_t lddh, ldgate, ldup, ld;  // elements
  int32_t M, F;
};
template <int DT, int ACT, bool VEC> __global__ void __launch_bounds__(256) slope_kernel(const SlopeParams p) {
  constexpr int V = VEC ? 8 : 1;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t per = ((int64_t)p.F + V - 1) / V, total = per * p.M;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t m = i / per, c = (i - m * per) * V;
    if constexpr (VEC) {
      uint32_t h[4], g[4], u[4], a[4], b[4];
      load_bytes<16>(p.dh + m * p.lddh + c, h);
      load_bytes<16>(p.gate + m * p.ldgate + c, g);
      load_bytes<16>(p.up + m * p.ldup + c, u);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 hv = widen2<DT>(h[e]), gv = widen2<DT>(g[e]), uv = widen2<DT>(u[e]);
        const float2 s0 = activation_slope<ACT>(gv.x), s1 = activation_slope<ACT>(gv.y);
        a[e] = narrow2<DT>(__fmul_rn(__fmul_rn(hv.x, uv.x), s0.y), __fmul_rn(__fmul_rn(hv.y, uv.y), s1.y));
        b[e] = narrow2<DT>(__fmul_rn(hv.x, s0.x), __fmul_rn(hv.y, s1.x));
      }
      store_bytes<16>(p.dgate + m * p.ld + c, a);
      store_bytes<16>(p.dup + m * p.ld + c, b);
    } else {
      const float hv = value16<DT>(p.dh, m * p.lddh + c), uv = value16<DT>(p.up, m * p.ldup + c);
      const float2 s = activation_slope<ACT>(value16<DT>(p.gate, m * p.ldgate + c));
      p.dgate[m * p.ld + c] = round16<DT>(__fmul_rn(__fmul_rn(hv, uv), s.y));
      p.dup[m * p.ld + c] = round16<DT>(__fmul_rn(hv, s.x));
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

bool known(int dtype, int act) {
  return (dtype == FAR_F16 || dtype == FAR_BF16) && (act == FAR_ACT_SILU || act == FAR_ACT_GELU || act == FAR_ACT_GELU_TANH);
}

// a [rows, cols] 16-bit matrix of a call
struct Matrix {
  const void* p;
  int64_t ld, rows, cols;
  Region at() const { return region(p, rows && cols ? rows : 0, cols * 2, ld * 2); }
};

// sizes, strides, pointers and aliasing of a call's inputs and outputs
int check_matrices(const Matrix* in, int n_in, const Matrix* out, int n_out) {
  const int64_t lim = int64_t(1) << 31;
  auto sizes = [&](const Matrix& m) {
    if (m.rows < 0 || m.cols < 0 || m.rows > INT32_MAX || m.cols > INT32_MAX) return (int)FAR_ERR_SHAPE;
    if (m.ld < m.cols || m.ld > lim) return (int)FAR_ERR_SHAPE;
    return FAR_OK;
  };
  auto pointer = [&](const Matrix& m) {
    if (m.rows == 0 || m.cols == 0) return FAR_OK;
    return !m.p ? (int)FAR_ERR_NULL : (uintptr_t)m.p % 2 ? (int)FAR_ERR_SHAPE : FAR_OK;
  };
  for (int i = 0; i < n_in; ++i)
    if (const int st = sizes(in[i])) return st;
  for (int i = 0; i < n_out; ++i)
    if (const int st = sizes(out[i])) return st;
  for (int i = 0; i < n_in; ++i)
    if (const int st = pointer(in[i])) return st;
  for (int i = 0; i < n_out; ++i)
    if (const int st = pointer(out[i])) return st;
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (regions_overlap(out[i].at(), in[j].at())) return FAR_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (regions_overlap(out[i].at(), out[j].at())) return FAR_ERR_ALIAS;
  }
  return FAR_OK;
}

unsigned plain_grid(int64_t m, int64_t n, int sms) {
  const int64_t tiles = ((m + 63) / 64) * ((n + 63) / 64), cap = (int64_t)sms * 8;
  return (unsigned)(tiles < cap ? tiles : cap);
}

struct FewPlan {
  int nt;     // tokens a CTA; 0: too many tiles for the grid
  int split;  // CTAs that share a tile's k
  double us;  // estimated, where tokens fill more than one kind of CTA (nt 128)
};
// `rows` output columns a CTA.  A CTA's set-up and its part of the cluster's sum take about the time of
// ten slices.
FewPlan plan_few(int64_t tokens, int64_t columns, int rows, int64_t slices) {
  const int nt = tokens <= 16 ? 16 : tokens <= 32 ? 32 : tokens <= 64 ? 64 : 128;
  const int64_t tiles_n = (columns + rows - 1) / rows, tiles_m = (tokens + nt - 1) / nt;
  if (tiles_n > 65535 || tiles_m > 65535) return FewPlan{0, 0, 0};
  const ClusterPlan c = plan_clusters(tiles_n * tiles_m, slices, 2, 10);
  const double ctas = (double)(tiles_n * tiles_m * c.split) / 152;
  return FewPlan{nt, c.split, 5 + 0.55 * (double)(c.waves * ((slices + c.split - 1) / c.split)) + 1.5 * (ctas < 2 ? ctas : 2)};
}

// Does few_kernel pay, against pairs with `pair_tiles` tiles in `tiles_m` rows of tiles?  Up to 64 tokens always
// (17 x 1024 x 1024 4.7 us, pairs 7.4; 60 x 2056 x 5640 14.0 and 16.1); above by both estimates, fitted to 35
// shapes: a slice takes a pair 0.245 us, or what HBM gives of weights that no tile row above has read, a
// half tile 0.21 (an SM's intake).  E.g. (few / pairs) 200 x 5120 x 512 12.5 / 19.8, 200 x 2048 x 5632
// 19.5 / 15.5; dx of 777 x 512 x 8192 43 / 73 with the rest of the way back.
bool few_pays(int64_t tokens, const FewPlan& g, int64_t pair_tiles, int64_t slices) {
  if (g.nt == 0) return false;
  if (tokens <= 64) return true;
  const int64_t waves = pair_tiles / 76, rest = pair_tiles % 76;
  const double fresh = 256.0 / (double)(tokens > 256 ? (tokens + 255) / 256 * 256 : 256);
  const double whole = 0.36 * fresh > 0.245 ? 0.36 * fresh : 0.245, half = 0.18 * fresh > 0.21 ? 0.18 * fresh : 0.21;
  return g.us < 3.9 + (double)slices * ((double)waves * whole + (rest == 0 ? 0 : 2 * rest <= 76 ? half : whole));
}

template <int NT, int DT, int ACT, bool GATE>
cudaError_t launch_few_nt(const FewMaps& maps, const FewParams& p, int split, cudaStream_t s) {
  const void* f = reinterpret_cast<const void*>(few_kernel<NT, DT, ACT, GATE>);
  const cudaError_t e = ensure_smem_attribute(f, FewShape<NT>::smem);
  if (e != cudaSuccess) return e;
  constexpr int64_t ROWS = GATE ? 64 : 128;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)split, (unsigned)((p.N + ROWS - 1) / ROWS), (unsigned)(((int64_t)p.M + NT - 1) / NT));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = FewShape<NT>::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = far_get_programmatic_launch() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<NT, DT, ACT, GATE>, maps, p);
}
template <int DT, int ACT, bool GATE>
cudaError_t launch_few(const FewMaps& maps, const FewParams& p, const FewPlan& g, cudaStream_t s) {
  return g.nt == 16   ? launch_few_nt<16, DT, ACT, GATE>(maps, p, g.split, s)
         : g.nt == 32 ? launch_few_nt<32, DT, ACT, GATE>(maps, p, g.split, s)
         : g.nt == 64 ? launch_few_nt<64, DT, ACT, GATE>(maps, p, g.split, s)
                      : launch_few_nt<128, DT, ACT, GATE>(maps, p, g.split, s);
}

struct GatePlan {
  int kind;  // 0 plain, 1 pairs, 2 few
  FewPlan few;
};
int64_t slices_of(int64_t k) { return (k + 63) / 64; }
int wide_rows(const void* p, int64_t ld) { return ((uintptr_t)p & 7) == 0 && ld % 4 == 0; }

GatePlan plan_gate(const GateParams& p) {
  GatePlan g{0, {0, 0, 0}};
  if (p.K == 0 || !tma_rows(p.x, p.ldx, 2) || !tma_rows(p.wg, p.ldwg, 2) || !tma_rows(p.wu, p.ldwu, 2)) return g;
  g.few = plan_few(p.M, p.F, 64, slices_of(p.K));
  const int64_t pair_tiles = (((int64_t)p.M + 255) / 256) * (((int64_t)p.F + 127) / 128);
  g.kind = few_pays(p.M, g.few, pair_tiles, slices_of(p.K)) ? 2 : 1;
  if (g.kind == 1 && pair_tiles > INT32_MAX) g.kind = 0;
  return g;
}

int run_gate(GateParams& p, int dtype, int act, cudaStream_t s) {
  unsigned int* status = nullptr;
  int sms = 0;
  int st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  const GatePlan g = plan_gate(p);
  cudaError_t e;
  if (g.kind == 0) {
    e = with_types(dtype, act, [&](auto dt, auto a) {
      return launch_k(plain_gate_kernel<decltype(dt)::value, decltype(a)::value>, dim3(plain_grid(p.M, p.F, sms)), dim3(256), 0, s, p);
    });
  } else if (g.kind == 2) {
    FewMaps maps{};
    st = encode_box(&maps.x[0], p.x, p.M, p.K, p.ldx, 2, g.few.nt, tma_type(dtype));
    if (st == FAR_OK) st = encode_operand(&maps.w[0], p.wg, p.F, p.K, p.ldwg, dtype);
    if (st == FAR_OK) st = encode_operand(&maps.w[1], p.wu, p.F, p.K, p.ldwu, dtype);
    if (st != FAR_OK) return st;
    const FewParams q{p.out, p.gate, p.up, p.ldo, p.ldgate, p.ldup, p.M, p.F, (int32_t)slices_of(p.K), 0,
                      wide_rows(p.out, p.ldo) | wide_rows(p.gate, p.ldgate) << 1 | wide_rows(p.up, p.ldup) << 2, status,
                      wait_limit_ns(slices_of(p.K))};
    e = with_types(dtype, act, [&](auto dt, auto a) { return launch_few<decltype(dt)::value, decltype(a)::value, true>(maps, q, g.few, s); });
  } else {
    PairMaps maps{};
    PairOuts outs{};
    st = encode_operand(&maps.a[0], p.x, p.M, p.K, p.ldx, dtype);
    if (st == FAR_OK) st = encode_operand(&maps.b[0], p.wg, p.F, p.K, p.ldwg, dtype);
    if (st == FAR_OK) st = encode_operand(&maps.b[1], p.wu, p.F, p.K, p.ldwu, dtype);
    if (st == FAR_OK) st = pair_output(&outs.out[0], &maps.out[0], p.out, p.M, p.F, p.ldo, dtype);
    if (st == FAR_OK && p.gate) st = pair_output(&outs.out[1], &maps.out[1], p.gate, p.M, p.F, p.ldgate, dtype);
    if (st == FAR_OK && p.gate) st = pair_output(&outs.out[2], &maps.out[2], p.up, p.M, p.F, p.ldup, dtype);
    if (st != FAR_OK) return st;
    PairWalk w{};
    w.tiles_m = (int32_t)(((int64_t)p.M + 255) / 256);
    w.tiles_n = (int32_t)(((int64_t)p.F + 127) / 128);
    w.num_tiles = w.tiles_m * w.tiles_n;
    w.columns = p.F;
    w.slices = (int32_t)(((int64_t)p.K + 63) / 64);
    w.pairs = 1;
    w.bf16 = dtype == FAR_BF16;
    w.status = status;
    w.timeout_ns = wait_limit_ns(w.slices);
    e = with_types(dtype, act, [&](auto dt, auto a) {
      constexpr int DT = decltype(dt)::value, ACT = decltype(a)::value;
      return p.gate ? launch_pair16<GateEpilogue<DT, ACT, true>>(maps, w, outs, sms, s)
                    : launch_pair16<GateEpilogue<DT, ACT, false>>(maps, w, outs, sms, s);
    });
  }
  return e == cudaSuccess ? FAR_OK : cuda_error_status(e);
}

int64_t padded(int64_t ffn) { return (ffn + 7) / 8 * 8; }

struct BackCall {
  const uint16_t *dh, *gate, *up, *x, *wg, *wu;
  uint16_t *dx, *dwg, *dwu, *ws;
  int64_t lddh, ldgate, ldup, ldx, ldwg, ldwu, lddx, lddwg, lddwu;
  int32_t M, K, F;  // tokens, hidden, ffn
};

int run_back(const BackCall& c, int dtype, int act, cudaStream_t s) {
  unsigned int* status = nullptr;
  int sms = 0;
  int st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  const int64_t ld = padded(c.F);
  uint16_t *dg = c.ws, *du = c.ws + c.M * ld;
  cudaError_t e = cudaSuccess;
  if (c.M && c.F) {
    const SlopeParams p{c.dh, c.gate, c.up, dg, du, c.lddh, c.ldgate, c.ldup, ld, c.M, c.F};
    auto al = [](const void* q, int64_t stride) { return ((uintptr_t)q & 15) == 0 && stride % 8 == 0; };
    const bool vec = c.F % 8 == 0 && al(c.dh, c.lddh) && al(c.gate, c.ldgate) && al(c.up, c.ldup);
    const int64_t units = c.M * (vec ? (int64_t)c.F / 8 : c.F), blocks = (units + 255) / 256, cap = (int64_t)sms * 32;
    e = with_types(dtype, act, [&](auto dt, auto a) {
      constexpr int DT = decltype(dt)::value, ACT = decltype(a)::value;
      return launch_k(vec ? slope_kernel<DT, ACT, true> : slope_kernel<DT, ACT, false>, dim3((unsigned)(blocks < cap ? blocks : cap)),
                      dim3(256), 0, s, p);
    });
  }
  auto product = [&](const ProductParams& p) {
    if (e != cudaSuccess || !p.M || !p.N) return;
    e = launch_k(dtype == FAR_F16 ? plain_product_kernel<FAR_F16> : plain_product_kernel<FAR_BF16>, dim3(plain_grid(p.M, p.N, sms)),
                 dim3(256), 0, s, p);
  };
  auto tiles = [](int64_t n) { return (n + 255) / 256; };
  const int64_t dx_tiles = tiles(c.M) * tiles(c.K), dw_tiles = 2 * tiles(c.F) * tiles(c.K);
  const bool dx_tma = c.M && c.F && tma_rows(c.wg, c.ldwg, 2) && tma_rows(c.wu, c.ldwu, 2) && dx_tiles <= INT32_MAX;
  const bool dw_tma = c.M && c.F && tma_rows(c.x, c.ldx, 2) && dw_tiles <= INT32_MAX;
  PairWalk w{};
  w.columns = c.K;
  w.tiles_n = (int32_t)tiles(c.K);
  w.bf16 = dtype == FAR_BF16;
  w.status = status;
  PairMaps maps{};
  PairOuts outs{};
  if (dx_tma || dw_tma) {
    st = encode_operand(&maps.a[0], dg, c.M, c.F, ld, dtype);
    if (st == FAR_OK) st = encode_operand(&maps.a[1], du, c.M, c.F, ld, dtype);
    if (st != FAR_OK) return st;
  }
  const int64_t f_slices = slices_of(c.F);
  const FewPlan few = plan_few(c.M, c.K, 128, 2 * f_slices);
  if (dx_tma && few_pays(c.M, few, dx_tiles, 2 * f_slices)) {
    FewMaps fm{};
    st = encode_box(&fm.x[0], dg, c.M, c.F, ld, 2, few.nt, tma_type(dtype));
    if (st == FAR_OK) st = encode_box(&fm.x[1], du, c.M, c.F, ld, 2, few.nt, tma_type(dtype));
    if (st == FAR_OK) st = encode_operand(&fm.w[0], c.wg, c.F, c.K, c.ldwg, dtype);
    if (st == FAR_OK) st = encode_operand(&fm.w[1], c.wu, c.F, c.K, c.ldwu, dtype);
    if (st != FAR_OK) return st;
    const FewParams q{c.dx, nullptr, nullptr, c.lddx, 0, 0, c.M, c.K, (int32_t)(2 * f_slices), (int32_t)f_slices,
                      wide_rows(c.dx, c.lddx), status, wait_limit_ns(2 * f_slices)};
    if (e == cudaSuccess)
      e = dtype == FAR_F16 ? launch_few<FAR_F16, FAR_ACT_SILU, false>(fm, q, few, s) : launch_few<FAR_BF16, FAR_ACT_SILU, false>(fm, q, few, s);
  } else if (dx_tma) {
    st = encode_operand(&maps.b[0], c.wg, c.F, c.K, c.ldwg, dtype);
    if (st == FAR_OK) st = encode_operand(&maps.b[1], c.wu, c.F, c.K, c.ldwu, dtype);
    if (st == FAR_OK) st = pair_output(&outs.out[0], &maps.out[0], c.dx, c.M, c.K, c.lddx, dtype);
    if (st != FAR_OK) return st;
    w.tiles_m = (int32_t)tiles(c.M);
    w.num_tiles = (int32_t)dx_tiles;
    w.slices = (int32_t)f_slices;
    w.pairs = 2;
    w.timeout_ns = wait_limit_ns(2 * f_slices);
    if (e == cudaSuccess)
      e = dtype == FAR_F16 ? launch_pair16<ProductEpilogue<FAR_F16, false>>(maps, w, outs, sms, s)
                           : launch_pair16<ProductEpilogue<FAR_BF16, false>>(maps, w, outs, sms, s);
  } else {
    product(ProductParams{{dg, du}, {c.wg, c.wu}, c.dx, {ld, ld}, {1, 1}, {1, 1}, {c.ldwg, c.ldwu}, c.lddx, c.M, c.K, c.F, 2});
  }
  if (dw_tma) {
    st = encode_operand(&maps.b[0], c.x, c.M, c.K, c.ldx, dtype);
    if (st == FAR_OK) st = pair_output(&outs.out[0], &maps.out[0], c.dwg, c.F, c.K, c.lddwg, dtype);
    if (st == FAR_OK) st = pair_output(&outs.out[1], &maps.out[1], c.dwu, c.F, c.K, c.lddwu, dtype);
    if (st != FAR_OK) return st;
    w.tiles_m = (int32_t)(2 * tiles(c.F));
    w.num_tiles = (int32_t)dw_tiles;
    w.slices = (int32_t)(((int64_t)c.M + 63) / 64);
    w.pairs = 1;
    w.timeout_ns = wait_limit_ns(w.slices);
    if (e == cudaSuccess)
      e = dtype == FAR_F16 ? launch_pair16<ProductEpilogue<FAR_F16, true>>(maps, w, outs, sms, s)
                           : launch_pair16<ProductEpilogue<FAR_BF16, true>>(maps, w, outs, sms, s);
  } else {
    product(ProductParams{{dg, dg}, {c.x, c.x}, c.dwg, {1, 1}, {ld, ld}, {1, 1}, {c.ldx, c.ldx}, c.lddwg, c.F, c.K, c.M, 1});
    product(ProductParams{{du, du}, {c.x, c.x}, c.dwu, {1, 1}, {ld, ld}, {1, 1}, {c.ldx, c.ldx}, c.lddwu, c.F, c.K, c.M, 1});
  }
  return e == cudaSuccess ? FAR_OK : cuda_error_status(e);
}

}  // namespace

}  // namespace far

using namespace far;

extern "C" int gated_ffn(const void* x, int64_t x_row_stride, const void* w_gate, int64_t w_gate_row_stride, const void* w_up,
                         int64_t w_up_row_stride, void* out, int64_t out_row_stride, void* gate_out,
                         int64_t gate_out_row_stride, void* up_out, int64_t up_out_row_stride, int64_t tokens,
                         int64_t hidden, int64_t ffn, int activation, int dtype, void* stream) {
  if (!known(dtype, activation)) return FAR_ERR_DTYPE;
  if ((gate_out == nullptr) != (up_out == nullptr)) return FAR_ERR_NULL;
  const Matrix in[3] = {{x, x_row_stride, tokens, hidden}, {w_gate, w_gate_row_stride, ffn, hidden}, {w_up, w_up_row_stride, ffn, hidden}};
  const Matrix out3[3] = {{out, out_row_stride, tokens, ffn}, {gate_out, gate_out_row_stride, tokens, ffn}, {up_out, up_out_row_stride, tokens, ffn}};
  const int st = check_matrices(in, 3, out3, gate_out ? 3 : 1);
  if (st != FAR_OK || tokens == 0 || ffn == 0) return st;
  GateParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.wg = static_cast<const uint16_t*>(w_gate);
  p.wu = static_cast<const uint16_t*>(w_up);
  p.out = static_cast<uint16_t*>(out);
  p.gate = static_cast<uint16_t*>(gate_out);
  p.up = static_cast<uint16_t*>(up_out);
  p.ldx = x_row_stride;
  p.ldwg = w_gate_row_stride;
  p.ldwu = w_up_row_stride;
  p.ldo = out_row_stride;
  p.ldgate = gate_out_row_stride;
  p.ldup = up_out_row_stride;
  p.M = (int32_t)tokens;
  p.F = (int32_t)ffn;
  p.K = (int32_t)hidden;
  return run_gate(p, dtype, activation, static_cast<cudaStream_t>(stream));
}

extern "C" int far_plan_gated_ffn(int64_t tokens, int64_t hidden, int64_t ffn, int* out3) {
  if (!out3) return FAR_ERR_NULL;
  if (tokens < 1 || hidden < 1 || ffn < 1 || tokens > INT32_MAX || hidden > INT32_MAX || ffn > INT32_MAX) return FAR_ERR_SHAPE;
  GateParams p{};  // (16-byte aligned operands)
  p.M = (int32_t)tokens;
  p.F = (int32_t)ffn;
  p.K = (int32_t)hidden;
  p.ldx = p.ldwg = p.ldwu = 8;
  const GatePlan g = plan_gate(p);
  out3[0] = g.kind;
  out3[1] = g.kind == 2 ? g.few.nt : 0;
  out3[2] = g.kind == 2 ? g.few.split : 0;
  return FAR_OK;
}

extern "C" int64_t far_gated_ffn_backward_workspace_bytes(int64_t tokens, int64_t ffn) {
  if (tokens < 0 || ffn < 0 || tokens > INT32_MAX || ffn > INT32_MAX) return -FAR_ERR_SHAPE;
  if (ffn && tokens > (INT64_MAX / 8) / padded(ffn)) return -FAR_ERR_SHAPE;
  return 2 * tokens * padded(ffn) * 2;
}

extern "C" int gated_ffn_backward(const void* dout, int64_t dout_row_stride, const void* gate, int64_t gate_row_stride,
                                  const void* up, int64_t up_row_stride, const void* x, int64_t x_row_stride,
                                  const void* w_gate, int64_t w_gate_row_stride, const void* w_up, int64_t w_up_row_stride,
                                  void* dx, int64_t dx_row_stride, void* dw_gate, int64_t dw_gate_row_stride, void* dw_up,
                                  int64_t dw_up_row_stride, void* workspace, int64_t workspace_bytes, int64_t tokens,
                                  int64_t hidden, int64_t ffn, int activation, int dtype, void* stream) {
  if (!known(dtype, activation)) return FAR_ERR_DTYPE;
  const Matrix in[6] = {{dout, dout_row_stride, tokens, ffn}, {gate, gate_row_stride, tokens, ffn}, {up, up_row_stride, tokens, ffn},
                        {x, x_row_stride, tokens, hidden}, {w_gate, w_gate_row_stride, ffn, hidden}, {w_up, w_up_row_stride, ffn, hidden}};
  const int64_t bytes = far_gated_ffn_backward_workspace_bytes(tokens, ffn);
  if (bytes < 0) return (int)-bytes;
  const Matrix out[3] = {{dx, dx_row_stride, tokens, hidden}, {dw_gate, dw_gate_row_stride, ffn, hidden}, {dw_up, dw_up_row_stride, ffn, hidden}};
  const int st = check_matrices(in, 6, out, 3);
  if (st != FAR_OK) return st;
  if (bytes > 0) {
    if (!workspace || workspace_bytes < bytes || ((uintptr_t)workspace & 15)) return FAR_ERR_WORKSPACE;
    const Region W = region(workspace, 1, bytes, 0);
    for (const Matrix& m : in)
      if (regions_overlap(W, m.at())) return FAR_ERR_ALIAS;
    for (int i = 0; i < 3; ++i)
      if (regions_overlap(W, out[i].at())) return FAR_ERR_ALIAS;
  }
  if (hidden == 0 || (tokens == 0 && ffn == 0)) return FAR_OK;
  auto c16 = [](const void* p) { return static_cast<const uint16_t*>(p); };
  auto m16 = [](void* p) { return static_cast<uint16_t*>(p); };
  const BackCall c{c16(dout), c16(gate), c16(up), c16(x), c16(w_gate), c16(w_up), m16(dx), m16(dw_gate), m16(dw_up), m16(workspace),
                   dout_row_stride, gate_row_stride, up_row_stride, x_row_stride, w_gate_row_stride, w_up_row_stride,
                   dx_row_stride, dw_gate_row_stride, dw_up_row_stride, (int32_t)tokens, (int32_t)hidden, (int32_t)ffn};
  return run_back(c, dtype, activation, static_cast<cudaStream_t>(stream));
}
