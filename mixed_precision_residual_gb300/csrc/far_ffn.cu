// The gated feed-forward block's way in and its gradients, on 16-bit tensors (gated_ffn,
// gated_ffn_backward):
//   gate = x wg^T, up = x wu^T (binary32),  h = RNE(act(gate) up)
//   dgate = RNE(dh up act'(gate)), dup = RNE(dh act(gate)),
//   dx = RNE(dgate wg + dup wu),  dwg = RNE(dgate^T x),  dwu = RNE(dup^T x).
//
// plain_gate_kernel, plain_product_kernel  any shape, stride and alignment: 64 x 64 tiles in binary32.
// slope_kernel                             dgate and dup, into the workspace.  Bound by HBM.
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "far.h"
#include "far_device.cuh"
#include "far_launch.h"
#include "far_params.h"
#include "far_region.h"

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
// plain kernels
// ---------------------------------------------------------------------------

struct GateParams {
  const uint16_t *x, *wg, *wu;
  uint16_t *out, *gate, *up;                    // gate and up may be null
  int64_t ldx, ldwg, ldwu, ldo, ldgate, ldup;   // elements
  int32_t M, F, K;                              // tokens, ffn, hidden
  unsigned int* status;
  uint64_t timeout_ns;
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
  pdl_launch_dependents();
  pdl_wait();
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
// dgate and dup: rows of `ld` elements, a multiple of 8, in the workspace
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

int run_gate(GateParams& p, int dtype, int act, cudaStream_t s) {
  unsigned int* status = nullptr;
  int sms = 0;
  const int st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  p.status = status;
  p.timeout_ns = kWaitTimeoutNs;
  const cudaError_t e = with_types(dtype, act, [&](auto dt, auto a) {
    return launch_k(plain_gate_kernel<decltype(dt)::value, decltype(a)::value>, dim3(plain_grid(p.M, p.F, sms)), dim3(256), 0, s, p);
  });
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
  const int st = device_info(&status, &sms);
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
  product(ProductParams{{dg, du}, {c.wg, c.wu}, c.dx, {ld, ld}, {1, 1}, {1, 1}, {c.ldwg, c.ldwu}, c.lddx, c.M, c.K, c.F, 2});
  product(ProductParams{{dg, dg}, {c.x, c.x}, c.dwg, {1, 1}, {ld, ld}, {1, 1}, {c.ldx, c.ldx}, c.lddwg, c.F, c.K, c.M, 1});
  product(ProductParams{{du, du}, {c.x, c.x}, c.dwu, {1, 1}, {ld, ld}, {1, 1}, {c.ldx, c.ldx}, c.lddwu, c.F, c.K, c.M, 1});
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
