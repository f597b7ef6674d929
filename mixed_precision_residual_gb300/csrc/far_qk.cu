// Per-head RMSNorm of queries and keys with the rotation by position in the same pass, the
// rotation alone, their gradients, and the table of cosines and sines they read.
//
// Per (token, head) vector x of D values: r = 1 / sqrt(sum(x^2) / D + eps), n = x r w, and
// the first `rot` values of n turned in pairs by the token's row of the table.  Backward,
// with g the transposed rotation of dy and u = x r:  dw = sum g u,
// dx = r (h - u mean(h u)),  h = g w.
//
// Bound by HBM: a value is read once and written once (backward: two reads, one write), and
// a table row once a token.  So a head lives in the registers of L lanes (L a power of two),
// two 16-byte chunks a lane, and its sums are log2(L) shuffles:
//   half pairs:  lane p holds chunk p of the rotated part's first half and the chunk it is
//                turned with, so a rotation needs no exchange between lanes;
//   interleaved: both values of a pair lie in one chunk; the second chunk is the one half a
//                head further, so that each load instruction reads whole sectors.
// A warp keeps one token's cosines and sines, and one weight vector, in registers for all
// the heads it takes of that token (blockIdx.y picks the heads: queries' or keys').
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "far.h"
#include "far_device.cuh"
#include "far_launch.h"
#include "far_params.h"
#include "far_region.h"

namespace far {

namespace {

constexpr int kQkThreads = 256;
constexpr int kQkMaxDim = 2048;
constexpr int kQkParts = 1024;  // partial rows of the weights' gradients a backward call may write

struct QkSeg {  // the queries' or the keys' half of a call; strides in bytes
  const char* x;
  const char* g;  // backward: the output's gradient
  char* y;        // forward: the output; backward: the input's gradient
  const void* w;
  int64_t xt, xh, gt, gh, yt, yh;
  int32_t heads;
};

struct QkParams {
  QkSeg seg[2];
  const float* table;
  const void* pos;
  float* parts;  // backward: [gridDim.y * gridDim.x][D] partial sums of the weights' gradients
  int64_t table_rows, tokens;
  unsigned int* status;
  float eps, dim_f, sign;  // sign: -1 turns the other way
  int32_t D, rot;
  int32_t pos64, w32;
  int32_t log_l;    // vector kernels: log2 of the lanes a head takes
  int32_t units_q;  // blockIdx.y below this: queries, else keys
  int32_t hb;       // heads a unit takes
};

__device__ __forceinline__ int64_t load_pos(const QkParams& p, int64_t t) {
  return p.pos64 ? static_cast<const int64_t*>(p.pos)[t] : (int64_t) static_cast<const int32_t*>(p.pos)[t];
}

template <int DT> __device__ __forceinline__ float load_one(const void* base, int64_t i) {
  if constexpr (DT == FAR_F16) return __half2float(static_cast<const __half*>(base)[i]);
  else if constexpr (DT == FAR_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
  else return static_cast<const float*>(base)[i];
}
template <int DT> __device__ __forceinline__ void store_one(void* base, int64_t i, float v) {
  if constexpr (DT == FAR_F16) static_cast<__half*>(base)[i] = __float2half_rn(v);
  else if constexpr (DT == FAR_BF16) static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(base)[i] = v;
}
// a weight: binary32, or the 16-bit type; for binary32 activations p.w32 tells fp16 (2) from bf16 (3)
template <int ACT> __device__ __forceinline__ float load_w(const void* w, int w32, int i) {
  if (w32 == 1) return static_cast<const float*>(w)[i];
  if constexpr (ACT == FAR_F32) return w32 == 2 ? load_one<FAR_F16>(w, i) : load_one<FAR_BF16>(w, i);
  else return load_one<ACT>(w, i);
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int off = lanes >> 1; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// ---------------------------------------------------------------------------
// vector kernels
// ---------------------------------------------------------------------------

// A lane's two chunks of a head (-1: none) and, for half pairs, whether they are turned.
struct Slot {
  int ca, cb;
  bool ra, rb;
};
template <bool INTER>
__device__ __forceinline__ Slot slot_of(int s, int C, int RC) {
  Slot r;
  if constexpr (INTER) {
    const int h = (C + 1) >> 1;
    r.ca = s < h ? s : -1;
    r.cb = s < h && h + s < C ? h + s : -1;
    r.ra = r.ca >= 0 && r.ca < RC;
    r.rb = r.cb >= 0 && r.cb < RC;
  } else {
    const int np = RC >> 1;
    if (s < np) {
      r.ca = s;
      r.cb = s + np;
      r.ra = r.rb = true;
    } else {
      const int i = s - np, h = (C - RC + 1) >> 1;
      r.ca = i < h ? RC + i : -1;
      r.cb = i < h && RC + h + i < C ? RC + h + i : -1;
      r.ra = r.rb = false;
    }
  }
  return r;
}

// The cosines and sines a lane needs: for half pairs V of each (c, s), shared by its two
// chunks; for interleaved pairs V/2 of each for either chunk.
template <bool INTER, int V>
struct Turn {
  float c[V], s[V];
  __device__ __forceinline__ void load(const float* row, const Slot& k, int half, float sign) {
    if constexpr (INTER) {
      constexpr int P = V / 2;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        c[e] = k.ra ? row[k.ca * P + e] : 1.f;
        s[e] = k.ra ? sign * row[half + k.ca * P + e] : 0.f;
        c[P + e] = k.rb ? row[k.cb * P + e] : 1.f;
        s[P + e] = k.rb ? sign * row[half + k.cb * P + e] : 0.f;
      }
    } else if (k.ra) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const float4 a = reinterpret_cast<const float4*>(row + k.ca * V)[q];
        const float4 b = reinterpret_cast<const float4*>(row + half + k.ca * V)[q];
        c[4 * q] = a.x; c[4 * q + 1] = a.y; c[4 * q + 2] = a.z; c[4 * q + 3] = a.w;
        s[4 * q] = sign * b.x; s[4 * q + 1] = sign * b.y; s[4 * q + 2] = sign * b.z; s[4 * q + 3] = sign * b.w;
      }
    }
  }
  // turns the lane's two chunks in place (values outside the rotated part are left alone)
  __device__ __forceinline__ void apply(float (&a)[V], float (&b)[V], const Slot& k) const {
    if constexpr (INTER) {
      constexpr int P = V / 2;
      if (k.ra) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float x = a[2 * e], y = a[2 * e + 1];
          a[2 * e] = __fmaf_rn(x, c[e], -__fmul_rn(y, s[e]));
          a[2 * e + 1] = __fmaf_rn(y, c[e], __fmul_rn(x, s[e]));
        }
      }
      if (k.rb) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float x = b[2 * e], y = b[2 * e + 1];
          b[2 * e] = __fmaf_rn(x, c[P + e], -__fmul_rn(y, s[P + e]));
          b[2 * e + 1] = __fmaf_rn(y, c[P + e], __fmul_rn(x, s[P + e]));
        }
      }
    } else if (k.ra) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float x = a[e], y = b[e];
        a[e] = __fmaf_rn(x, c[e], -__fmul_rn(y, s[e]));
        b[e] = __fmaf_rn(y, c[e], __fmul_rn(x, s[e]));
      }
    }
  }
};

template <int ACT, int V>
__device__ __forceinline__ void load_weights(const void* w, int w32, int chunk, float (&f)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = chunk >= 0 ? load_w<ACT>(w, w32, chunk * V + e) : 0.f;
}

__device__ __forceinline__ uint4 load_chunk(const char* p, int chunk) {
  return chunk >= 0 ? *reinterpret_cast<const uint4*>(p + 16 * chunk) : make_uint4(0u, 0u, 0u, 0u);
}
template <int ACT, int V> __device__ __forceinline__ void widen_chunk(const uint4& r, float (&f)[V]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  widen<ACT, V>(w, f);
}
template <int ACT, int V> __device__ __forceinline__ void store_chunk(char* p, int chunk, const float (&f)[V]) {
  if (chunk < 0) return;
  uint32_t w[4];
  narrow<ACT, V>(f, w);
  store_bytes<16>(p + 16 * chunk, w);
}

template <int ACT, bool INTER, bool NORM>
__global__ void __launch_bounds__(kQkThreads, 2) qk_kernel(const QkParams p) {
  constexpr int V = 16 / dtype_size<ACT>::value;
  constexpr int U = 4;  // heads a lane holds at a time: 128 bytes of loads in flight a lane
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int L = 1 << p.log_l, groups = 32 >> p.log_l, grp = lane >> p.log_l;
  const bool is_k = (int)blockIdx.y >= p.units_q;
  const QkSeg& S = p.seg[is_k];
  const int h0 = (is_k ? (int)blockIdx.y - p.units_q : (int)blockIdx.y) * p.hb;
  const int h1 = min(S.heads, h0 + p.hb);
  const Slot k = slot_of<INTER>(lane & (L - 1), p.D / V, p.rot / V);
  float wa[V], wb[V];
  if constexpr (NORM) {
    load_weights<ACT, V>(S.w, p.w32, k.ca, wa);
    load_weights<ACT, V>(S.w, p.w32, k.cb, wb);
  }
  const int64_t step = (int64_t)gridDim.x * warps;
  for (int64_t t = (int64_t)blockIdx.x * warps + warp; t < p.tokens; t += step) {
    const int64_t pos = load_pos(p, t);
    const bool ok = pos >= 0 && pos < p.table_rows;
    if (pos >= p.table_rows && lane == 0) atomicOr(p.status, 1u << FAR_ERR_POSITION);
    Turn<INTER, V> turn;
    const char* xt = S.x + t * S.xt;
    char* yt = S.y + t * S.yt;
    bool first = true;
    for (int hb = h0; hb < h1; hb += U * groups) {
      uint4 xa[U], xb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * groups + grp;
        const char* x = xt + h * S.xh;
        xa[u] = load_chunk(x, h < h1 ? k.ca : -1);
        xb[u] = load_chunk(x, h < h1 ? k.cb : -1);
      }
      if (first) {
        turn.load(p.table + (ok ? pos : 0) * p.rot, k, p.rot >> 1, p.sign);
        first = false;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * groups + grp;
        if (hb + u * groups >= h1) break;  // uniform over the warp
        float a[V], b[V];
        widen_chunk<ACT, V>(xa[u], a);
        widen_chunk<ACT, V>(xb[u], b);
        if constexpr (NORM) {
          float ss = 0.f, st = 0.f;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ss = __fmaf_rn(a[e], a[e], ss);
            st = __fmaf_rn(b[e], b[e], st);
          }
          const float r = row_rstd(lanes_sum(__fadd_rn(ss, st), L), p.dim_f, p.eps);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            a[e] = __fmul_rn(__fmul_rn(a[e], r), wa[e]);
            b[e] = __fmul_rn(__fmul_rn(b[e], r), wb[e]);
          }
        }
        turn.apply(a, b, k);
        if (!ok) {
          const float v = pos < 0 ? 0.f : __uint_as_float(0x7fffffffu);
#pragma unroll
          for (int e = 0; e < V; ++e) a[e] = b[e] = v;
        }
        if (h < h1) {
          char* y = yt + h * S.yh;
          store_chunk<ACT, V>(y, k.ca, a);
          store_chunk<ACT, V>(y, k.cb, b);
        }
      }
    }
  }
}

// One partial row of the weights' gradient a block: the warps' sums, added in their order.
template <int V>
__device__ __forceinline__ void write_part(float* part, float* sm, const Slot& k, float (&da)[V], float (&db)[V],
                                           int L, int lane, int warp, int warps, int D) {
#pragma unroll
  for (int e = 0; e < V; ++e)
    for (int off = L; off < 32; off <<= 1) {
      da[e] = __fadd_rn(da[e], __shfl_xor_sync(0xffffffffu, da[e], off));
      db[e] = __fadd_rn(db[e], __shfl_xor_sync(0xffffffffu, db[e], off));
    }
  if (lane < L) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (k.ca >= 0) sm[warp * D + k.ca * V + e] = da[e];
      if (k.cb >= 0) sm[warp * D + k.cb * V + e] = db[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v = __fadd_rn(v, sm[w * D + i]);
    part[i] = v;
  }
}

template <int ACT, bool INTER>
__global__ void __launch_bounds__(kQkThreads, 2) qk_back_kernel(const QkParams p) {
  constexpr int V = 16 / dtype_size<ACT>::value;
  constexpr int U = 2;  // heads a lane holds at a time: x and dy of two, 128 bytes a lane
  extern __shared__ float sm_dw[];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int L = 1 << p.log_l, groups = 32 >> p.log_l, grp = lane >> p.log_l;
  const bool is_k = (int)blockIdx.y >= p.units_q;
  const QkSeg& S = p.seg[is_k];
  const int h0 = (is_k ? (int)blockIdx.y - p.units_q : (int)blockIdx.y) * p.hb;
  const int h1 = min(S.heads, h0 + p.hb);
  const Slot k = slot_of<INTER>(lane & (L - 1), p.D / V, p.rot / V);
  float wa[V], wb[V], da[V], db[V];
  load_weights<ACT, V>(S.w, p.w32, k.ca, wa);
  load_weights<ACT, V>(S.w, p.w32, k.cb, wb);
#pragma unroll
  for (int e = 0; e < V; ++e) da[e] = db[e] = 0.f;
  const int64_t step = (int64_t)gridDim.x * warps;
  for (int64_t t = (int64_t)blockIdx.x * warps + warp; t < p.tokens; t += step) {
    const int64_t pos = load_pos(p, t);
    const bool ok = pos >= 0 && pos < p.table_rows;
    if (pos >= p.table_rows && lane == 0) atomicOr(p.status, 1u << FAR_ERR_POSITION);
    Turn<INTER, V> turn;
    bool first = true;
    for (int hb = h0; hb < h1; hb += U * groups) {
      uint4 xa[U], xb[U], ga[U], gb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * groups + grp;
        const char* x = S.x + t * S.xt + h * S.xh;
        const char* g = S.g + t * S.gt + h * S.gh;
        xa[u] = load_chunk(x, h < h1 ? k.ca : -1);
        xb[u] = load_chunk(x, h < h1 ? k.cb : -1);
        ga[u] = load_chunk(g, h < h1 ? k.ca : -1);
        gb[u] = load_chunk(g, h < h1 ? k.cb : -1);
      }
      if (first) {
        turn.load(p.table + (ok ? pos : 0) * p.rot, k, p.rot >> 1, p.sign);
        first = false;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * groups + grp;
        if (hb + u * groups >= h1) break;  // uniform over the warp
        float a[V], b[V], c[V], d[V];
        widen_chunk<ACT, V>(xa[u], a);
        widen_chunk<ACT, V>(xb[u], b);
        widen_chunk<ACT, V>(ga[u], c);
        widen_chunk<ACT, V>(gb[u], d);
        float ss = 0.f, st = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          ss = __fmaf_rn(a[e], a[e], ss);
          st = __fmaf_rn(b[e], b[e], st);
        }
        const float r = row_rstd(lanes_sum(__fadd_rn(ss, st), L), p.dim_f, p.eps);
        turn.apply(c, d, k);
        float da1 = 0.f, db1 = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          a[e] = __fmul_rn(a[e], r);  // u = x r
          b[e] = __fmul_rn(b[e], r);
          if (ok && h < h1) {
            da[e] = __fmaf_rn(c[e], a[e], da[e]);
            db[e] = __fmaf_rn(d[e], b[e], db[e]);
          }
          c[e] = __fmul_rn(c[e], wa[e]);  // h = g w
          d[e] = __fmul_rn(d[e], wb[e]);
          da1 = __fmaf_rn(c[e], a[e], da1);
          db1 = __fmaf_rn(d[e], b[e], db1);
        }
        const float m = __fdiv_rn(lanes_sum(__fadd_rn(da1, db1), L), p.dim_f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          a[e] = __fmul_rn(r, __fmaf_rn(-a[e], m, c[e]));
          b[e] = __fmul_rn(r, __fmaf_rn(-b[e], m, d[e]));
        }
        if (!ok) {
          const float v = pos < 0 ? 0.f : __uint_as_float(0x7fffffffu);
#pragma unroll
          for (int e = 0; e < V; ++e) a[e] = b[e] = v;
        }
        if (h < h1) {
          char* y = S.y + t * S.yt + h * S.yh;
          store_chunk<ACT, V>(y, k.ca, a);
          store_chunk<ACT, V>(y, k.cb, b);
        }
      }
    }
  }
  write_part<V>(p.parts + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.D, sm_dw, k, da, db, L, lane, warp, warps,
                p.D);
}

// ---------------------------------------------------------------------------
// scalar kernels: any head size, stride, alignment and pair: a warp a head, a pair (or an
// unturned value) a lane at a time; blockIdx.y = 0 queries, 1 keys (p.units_q tells)
// ---------------------------------------------------------------------------

// item i of a head: pairs first (two values), then the values behind the rotated part
struct Item {
  int a, b;  // b = -1: a single value
};
__device__ __forceinline__ Item item_of(int i, int rot, bool inter) {
  const int np = rot >> 1;
  if (i >= np) return Item{rot + (i - np), -1};
  return inter ? Item{2 * i, 2 * i + 1} : Item{i, i + np};
}

template <int ACT, bool BACK>
__global__ void __launch_bounds__(kQkThreads) qk_any_kernel(const QkParams p, int inter, int norm) {
  extern __shared__ float sm_dw[];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const QkSeg& S = p.seg[(int)blockIdx.y >= p.units_q];
  const int items = (p.rot >> 1) + (p.D - p.rot);
  float* dw = sm_dw + warp * p.D;  // backward: this warp's sums; each value belongs to one lane
  if constexpr (BACK) {
    for (int i = lane; i < items; i += 32) {
      const Item it = item_of(i, p.rot, inter);
      dw[it.a] = 0.f;
      if (it.b >= 0) dw[it.b] = 0.f;
    }
  }
  const int64_t total = p.tokens * S.heads;
  for (int64_t n = (int64_t)blockIdx.x * warps + warp; n < total; n += (int64_t)gridDim.x * warps) {
    const int64_t t = n / S.heads;
    const int64_t h = n - t * S.heads;
    const int64_t pos = load_pos(p, t);
    const bool ok = pos >= 0 && pos < p.table_rows;
    if (pos >= p.table_rows && lane == 0) atomicOr(p.status, 1u << FAR_ERR_POSITION);
    const float* row = p.table + (ok ? pos : 0) * p.rot;
    const float bad = pos < 0 ? 0.f : __uint_as_float(0x7fffffffu);
    const char* x = S.x + t * S.xt + h * S.xh;
    char* y = S.y + t * S.yt + h * S.yh;
    float r = 1.f;
    if (norm) {
      float ss = 0.f;
      for (int i = lane; i < p.D; i += 32) {
        const float v = load_one<ACT>(x, i);
        ss = __fmaf_rn(v, v, ss);
      }
      r = row_rstd(lanes_sum(ss, 32), p.dim_f, p.eps);
    }
    if constexpr (!BACK) {
      for (int i = lane; i < items; i += 32) {
        const Item it = item_of(i, p.rot, inter);
        float a = load_one<ACT>(x, it.a), b = it.b >= 0 ? load_one<ACT>(x, it.b) : 0.f;
        if (norm) {
          a = __fmul_rn(__fmul_rn(a, r), load_w<ACT>(S.w, p.w32, it.a));
          if (it.b >= 0) b = __fmul_rn(__fmul_rn(b, r), load_w<ACT>(S.w, p.w32, it.b));
        }
        if (it.b >= 0) {
          const float c = row[i], s = p.sign * row[(p.rot >> 1) + i];
          const float a1 = __fmaf_rn(a, c, -__fmul_rn(b, s));
          b = __fmaf_rn(b, c, __fmul_rn(a, s));
          a = a1;
          store_one<ACT>(y, it.b, ok ? b : bad);
        }
        store_one<ACT>(y, it.a, ok ? a : bad);
      }
    } else {
      const char* g = S.g + t * S.gt + h * S.gh;
      float dot = 0.f;
      // two sweeps over the head: the mean of h u (and the weights' sums), then dx
      for (int sweep = 0; sweep < 2; ++sweep) {
        const float m = sweep ? __fdiv_rn(lanes_sum(dot, 32), p.dim_f) : 0.f;
        for (int i = lane; i < items; i += 32) {
          const Item it = item_of(i, p.rot, inter);
          float a = load_one<ACT>(g, it.a), b = 0.f;
          if (it.b >= 0) {
            b = load_one<ACT>(g, it.b);
            const float c = row[i], s = p.sign * row[(p.rot >> 1) + i];
            const float a1 = __fmaf_rn(a, c, -__fmul_rn(b, s));
            b = __fmaf_rn(b, c, __fmul_rn(a, s));
            a = a1;
          }
          const float ua = __fmul_rn(load_one<ACT>(x, it.a), r);
          const float ub = it.b >= 0 ? __fmul_rn(load_one<ACT>(x, it.b), r) : 0.f;
          const float ha = __fmul_rn(a, load_w<ACT>(S.w, p.w32, it.a));
          const float hb = it.b >= 0 ? __fmul_rn(b, load_w<ACT>(S.w, p.w32, it.b)) : 0.f;
          if (sweep == 0) {
            if (ok) {
              dw[it.a] = __fmaf_rn(a, ua, dw[it.a]);
              if (it.b >= 0) dw[it.b] = __fmaf_rn(b, ub, dw[it.b]);
            }
            dot = __fmaf_rn(ha, ua, dot);
            if (it.b >= 0) dot = __fmaf_rn(hb, ub, dot);
          } else {
            store_one<ACT>(y, it.a, ok ? __fmul_rn(r, __fmaf_rn(-ua, m, ha)) : bad);
            if (it.b >= 0) store_one<ACT>(y, it.b, ok ? __fmul_rn(r, __fmaf_rn(-ub, m, hb)) : bad);
          }
        }
      }
    }
  }
  if constexpr (BACK) {
    __syncthreads();
    float* part = p.parts + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.D;
    for (int i = threadIdx.x; i < p.D; i += blockDim.x) {
      float v = 0.f;
      for (int w = 0; w < warps; ++w) v = __fadd_rn(v, sm_dw[w * p.D + i]);
      part[i] = v;
    }
  }
}

// The partial rows summed in a fixed order, in binary64: block (32 columns x 32 row lanes),
// blockIdx.y = 0 the queries' weight, 1 the keys'.
__global__ void __launch_bounds__(1024)
    qk_weight_grad_kernel(const float* parts, int D, int rows_q, int rows_k, float* dq_weight, float* dk_weight) {
  __shared__ double sm[32][33];
  pdl_launch_dependents();
  pdl_wait();
  const int col = blockIdx.x * 32 + threadIdx.x;
  const int rows = blockIdx.y ? rows_k : rows_q;
  const float* base = parts + (blockIdx.y ? (int64_t)rows_q * D : 0);
  float* out = blockIdx.y ? dk_weight : dq_weight;
  double v = 0.0;
  if (col < D) {
#pragma unroll 8
    for (int r = threadIdx.y; r < rows; r += 32) v += (double)base[(int64_t)r * D + col];
  }
  sm[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && col < D && out) {
    double t = 0.0;
    for (int i = 0; i < 32; ++i) t += sm[i][threadIdx.x];
    out[col] = (float)t;
  }
}

struct Freqs {
  double f[kQkMaxDim / 2];
};

// binary64 throughout: an angle of 10^6 in binary32 would be 0.06 off
__global__ void __launch_bounds__(256)
    rope_table_kernel(float* table, int64_t rows, int half, int64_t first, double factor, const __grid_constant__ Freqs q) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t total = rows * half;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / half;
    const int j = (int)(i - t * half);
    double s, c;
    sincos((double)(first + t) * q.f[j], &s, &c);
    table[t * 2 * half + j] = (float)(factor * c);
    table[t * 2 * half + half + j] = (float)(factor * s);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct Heads {  // a [tokens, heads, D] tensor; strides in elements
  const void* p;
  int64_t ts, hs;
};

struct QkCall {
  Heads x[2], g[2], y[2];
  const void* w[2];
  int64_t heads[2];
  float eps;
  const float* table;
  int64_t table_rows;
  const void* pos;
  int pos_bytes;
  int64_t tokens, D, rot;
  int pairs, act, wd;
  bool norm, back, transpose;
  float* dw[2];
  void* ws;
  int64_t ws_bytes;
};

int esize(int dt) { return dt == FAR_F32 ? 4 : 2; }

// the bytes a tensor spans, as rows of an even pitch where its layout is one (token-major or
// head-major), else as one run
Region heads_region(const Heads& t, int64_t tokens, int64_t heads, int64_t D, int64_t es) {
  const int64_t in = (heads - 1) * t.hs + D, out = (tokens - 1) * t.ts + D;
  if (tokens == 1 || t.ts >= in) return region(t.p, tokens, in * es, t.ts * es);
  if (heads == 1 || t.hs >= out) return region(t.p, heads, out * es, t.hs * es);
  return region(t.p, 1, ((tokens - 1) * t.ts + (heads - 1) * t.hs + D) * es, 0);
}

// every (token, head) of an output has bytes of its own
bool distinct(const Heads& t, int64_t tokens, int64_t heads, int64_t D) {
  const bool th = (heads == 1 || t.hs >= D) && (tokens == 1 || t.ts >= (heads - 1) * t.hs + D);
  const bool ht = (tokens == 1 || t.ts >= D) && (heads == 1 || t.hs >= (tokens - 1) * t.ts + D);
  return th || ht;
}

bool same_heads(const Heads& a, const Heads& b, int64_t tokens, int64_t heads) {
  return a.p == b.p && (tokens == 1 || a.ts == b.ts) && (heads == 1 || a.hs == b.hs);
}

constexpr int64_t kQkLimit = int64_t(1) << 40;  // strides and sizes: byte offsets stay far inside int64

int validate_qk(const QkCall& c) {
  auto known = [](int d) { return d == FAR_F32 || d == FAR_F16 || d == FAR_BF16; };
  if (!known(c.act) || !known(c.wd)) return FAR_ERR_DTYPE;
  if ((c.act == FAR_F16 && c.wd == FAR_BF16) || (c.act == FAR_BF16 && c.wd == FAR_F16)) return FAR_ERR_DTYPE_MIX;
  if (c.pos_bytes != 4 && c.pos_bytes != 8) return FAR_ERR_DTYPE;
  if (c.pairs != FAR_PAIRS_HALF && c.pairs != FAR_PAIRS_INTERLEAVED) return FAR_ERR_DTYPE;
  if (c.norm && !(c.eps >= 0.f && isfinite(c.eps))) return FAR_ERR_EPS;
  if (c.tokens < 0 || c.heads[0] < 0 || c.heads[1] < 0 || c.D < 1 || c.D > kQkMaxDim || c.rot < 2 || c.rot > c.D ||
      c.rot % 2 != 0 || c.table_rows < 0)
    return FAR_ERR_SHAPE;
  if (c.tokens > INT32_MAX || c.heads[0] > INT32_MAX || c.heads[1] > INT32_MAX || c.table_rows > kQkLimit)
    return FAR_ERR_SHAPE;
  const int64_t es = esize(c.act);
  bool any = false;
  for (int i = 0; i < 2; ++i) {
    if (!c.heads[i]) continue;
    for (const Heads* t : {&c.x[i], &c.g[i], &c.y[i]}) {
      if (t == &c.g[i] && !c.back) continue;
      if (t->ts < 0 || t->hs < 0 || t->ts > kQkLimit || t->hs > kQkLimit) return FAR_ERR_SHAPE;
      // spans within 2^60 bytes
      if ((c.tokens > 1 && t->ts > (int64_t(1) << 57) / c.tokens) || (c.heads[i] > 1 && t->hs > (int64_t(1) << 57) / c.heads[i]))
        return FAR_ERR_SHAPE;
    }
    if (c.back && !c.dw[i]) return FAR_ERR_NULL;
    if (c.tokens == 0) continue;
    any = true;
    if (!c.x[i].p || !c.y[i].p || (c.back && !c.g[i].p) || (c.norm && !c.w[i])) return FAR_ERR_NULL;
    if (!distinct(c.y[i], c.tokens, c.heads[i], c.D)) return FAR_ERR_SHAPE;
  }
  if (!any) return FAR_OK;
  if (!c.pos || (!c.table && c.table_rows > 0)) return FAR_ERR_NULL;
  if (c.table_rows == 0) return FAR_ERR_SHAPE;
  // element alignment of every pointer
  for (int i = 0; i < 2; ++i)
    if (c.heads[i])
      for (const void* q : {c.x[i].p, (const void*)c.y[i].p, c.back ? c.g[i].p : nullptr})
        if ((uintptr_t)q % es) return FAR_ERR_SHAPE;
  if ((uintptr_t)c.table % 4 || (uintptr_t)c.pos % c.pos_bytes) return FAR_ERR_SHAPE;
  if (c.back && (!c.ws || c.ws_bytes < far_qk_backward_workspace_bytes(c.D) || ((uintptr_t)c.ws & 15)))
    return FAR_ERR_WORKSPACE;
  // overlaps: the written regions against everything else
  Region wr[5], rd[10];
  int nw = 0, nr = 0;
  for (int i = 0; i < 2; ++i)
    if (c.heads[i]) wr[nw++] = heads_region(c.y[i], c.tokens, c.heads[i], c.D, es);
  const int ny = nw;
  if (c.back) {
    for (int i = 0; i < 2; ++i)
      if (c.heads[i]) wr[nw++] = region(c.dw[i], 1, c.D * 4, 0);
    wr[nw++] = region(c.ws, 1, far_qk_backward_workspace_bytes(c.D), 0);
  }
  for (int i = 0; i < 2; ++i)
    if (c.heads[i] && c.norm) rd[nr++] = region(c.w[i], 1, c.D * esize(c.wd), 0);
  rd[nr++] = region(c.table, 1, c.table_rows * c.rot * 4, 0);
  rd[nr++] = region(c.pos, 1, c.tokens * c.pos_bytes, 0);
  for (int a = 0; a < nw; ++a) {
    for (int b = a + 1; b < nw; ++b)
      if (regions_overlap(wr[a], wr[b])) return FAR_ERR_ALIAS;
    for (int b = 0; b < nr; ++b)
      if (regions_overlap(wr[a], rd[b])) return FAR_ERR_ALIAS;
  }
  for (int i = 0, a = 0; i < 2; ++i) {
    if (!c.heads[i]) continue;
    for (int j = 0; j < 2; ++j) {
      if (!c.heads[j]) continue;
      for (const Heads* t : {&c.x[j], &c.g[j]}) {
        if (t == &c.g[j] && !c.back) continue;
        const Region R = heads_region(*t, c.tokens, c.heads[j], c.D, es);
        if (regions_overlap(wr[a], R) && !(i == j && same_heads(c.y[i], *t, c.tokens, c.heads[i]))) return FAR_ERR_ALIAS;
        for (int b = ny; b < nw; ++b)
          if (regions_overlap(wr[b], R)) return FAR_ERR_ALIAS;
      }
    }
    ++a;
  }
  return FAR_OK;
}

struct QkPlan {
  bool vec;
  int log_l, hb, units_q, units_k;
  dim3 grid, block;
  size_t smem;
};

bool heads_al16(const Heads& t, int64_t es) {
  return ((uintptr_t)t.p & 15) == 0 && (t.ts * es) % 16 == 0 && (t.hs * es) % 16 == 0;
}

QkPlan plan_qk(const QkCall& c, int sms) {
  QkPlan g{};
  const int64_t es = esize(c.act);
  const int V = (int)(16 / es), D = (int)c.D, rot = (int)c.rot;
  const bool inter = c.pairs == FAR_PAIRS_INTERLEAVED;
  g.vec = D % V == 0 && rot % (inter ? V : 2 * V) == 0 && ((uintptr_t)c.table & 15) == 0;
  for (int i = 0; i < 2; ++i)
    if (c.heads[i])
      g.vec = g.vec && heads_al16(c.x[i], es) && heads_al16(c.y[i], es) && (!c.back || heads_al16(c.g[i], es));
  const int C = D / V, RC = rot / V;
  const int slots = inter ? (C + 1) / 2 : RC / 2 + (C - RC + 1) / 2;
  g.vec = g.vec && slots <= 32;
  const int64_t hmax = c.heads[0] > c.heads[1] ? c.heads[0] : c.heads[1];
  if (!g.vec) {
    g.units_q = c.heads[0] > 0;
    g.units_k = c.heads[1] > 0;
    const int warps = c.back ? 4 : 8;
    const int64_t blocks = (c.tokens * hmax + warps - 1) / warps;
    const int64_t cap = c.back ? (2 * sms < kQkParts / 2 ? 2 * sms : kQkParts / 2) : 16 * sms;
    g.grid = dim3((unsigned)(blocks < cap ? blocks : cap), g.units_q + g.units_k);
    g.block = dim3(32 * warps);
    g.smem = c.back ? (size_t)warps * D * 4 : 0;
    return g;
  }
  while ((1 << g.log_l) < slots) ++g.log_l;
  const int groups = 32 >> g.log_l;
  // Heads a warp takes of a token: as many as two sweeps hold, fewer (down to one a group of
  // lanes) while that leaves SMs without 16 warps of work.
  const int U = c.back ? 2 : 4;
  int64_t hb = 2 * U * groups;
  auto units = [&](int64_t h) { return (c.heads[0] + h - 1) / h + (c.heads[1] + h - 1) / h; };
  while (hb > groups && c.tokens * units(hb) < (int64_t)sms * 16) hb /= 2;
  while (units(hb) > (c.back ? 64 : 32768)) hb *= 2;  // gridDim.y's limit; backward: the partial rows'
  g.hb = (int)(hb < INT32_MAX / 2 ? hb : INT32_MAX / 2);
  g.units_q = (int)((c.heads[0] + hb - 1) / hb);
  g.units_k = (int)((c.heads[1] + hb - 1) / hb);
  const int u = g.units_q + g.units_k;
  int warps = 8;
  while (warps > 1 && (c.tokens + warps - 1) / warps * u < sms) warps /= 2;
  const int64_t blocks = (c.tokens + warps - 1) / warps;
  int64_t cap;
  if (c.back) {
    cap = (2 * sms + u - 1) / u;  // two blocks an SM, one partial row each
    if (cap * u > kQkParts) cap = kQkParts / u;
  } else {
    cap = (8 * sms + u - 1) / u;
  }
  if (cap < 1) cap = 1;
  g.grid = dim3((unsigned)(blocks < cap ? blocks : cap), u);
  g.block = dim3(32 * warps);
  g.smem = c.back ? (size_t)warps * D * 4 : 0;
  return g;
}

template <int ACT>
cudaError_t launch_qk(const QkCall& c, const QkPlan& g, const QkParams& p, cudaStream_t s) {
  const int inter = c.pairs == FAR_PAIRS_INTERLEAVED, norm = c.norm;
  if (!g.vec) {
    if (c.back) {
      if (g.smem > 48 * 1024) return cudaErrorInvalidValue;
      return launch_k(qk_any_kernel<ACT, true>, g.grid, g.block, g.smem, s, p, inter, 1);
    }
    return launch_k(qk_any_kernel<ACT, false>, g.grid, g.block, g.smem, s, p, inter, norm);
  }
  void (*k)(QkParams);
  if (c.back) k = inter ? qk_back_kernel<ACT, true> : qk_back_kernel<ACT, false>;
  else if (c.norm) k = inter ? qk_kernel<ACT, true, true> : qk_kernel<ACT, false, true>;
  else k = inter ? qk_kernel<ACT, true, false> : qk_kernel<ACT, false, false>;
  return launch_k(k, g.grid, g.block, g.smem, s, p);
}

int run_qk(const QkCall& c, void* stream) {
  int st = validate_qk(c);
  if (st != FAR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.tokens == 0 || (c.heads[0] == 0 && c.heads[1] == 0)) {
    for (int i = 0; i < 2; ++i)
      if (c.back && c.heads[i]) {
        cudaError_t e = cudaMemsetAsync(c.dw[i], 0, c.D * 4, s);
        if (e != cudaSuccess) return cuda_error_status(e);
      }
    return FAR_OK;
  }
  unsigned int* status = nullptr;
  int sms = 0;
  st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  const QkPlan g = plan_qk(c, sms);
  const int64_t es = esize(c.act);
  QkParams p{};
  for (int i = 0; i < 2; ++i) {
    QkSeg& S = p.seg[i];
    S.x = static_cast<const char*>(c.x[i].p);
    S.g = static_cast<const char*>(c.g[i].p);
    S.y = static_cast<char*>(const_cast<void*>(c.y[i].p));
    S.w = c.w[i];
    S.xt = c.x[i].ts * es;
    S.xh = c.x[i].hs * es;
    S.gt = c.g[i].ts * es;
    S.gh = c.g[i].hs * es;
    S.yt = c.y[i].ts * es;
    S.yh = c.y[i].hs * es;
    S.heads = (int32_t)c.heads[i];
  }
  p.table = c.table;
  p.pos = c.pos;
  p.parts = static_cast<float*>(c.ws);
  p.table_rows = c.table_rows;
  p.tokens = c.tokens;
  p.status = status;
  p.eps = c.eps;
  p.dim_f = (float)c.D;
  p.sign = (c.back || c.transpose) ? -1.f : 1.f;
  p.D = (int32_t)c.D;
  p.rot = (int32_t)c.rot;
  p.pos64 = c.pos_bytes == 8;
  p.w32 = c.wd == FAR_F32 ? 1 : c.wd == FAR_F16 ? 2 : 3;
  p.log_l = g.log_l;
  p.units_q = g.units_q;
  p.hb = g.hb;
  cudaError_t e = c.act == FAR_F16    ? launch_qk<FAR_F16>(c, g, p, s)
                  : c.act == FAR_BF16 ? launch_qk<FAR_BF16>(c, g, p, s)
                                      : launch_qk<FAR_F32>(c, g, p, s);
  if (e == cudaSuccess && c.back) {
    const int rows = (int)g.grid.x;
    e = launch_k(qk_weight_grad_kernel, dim3((unsigned)((c.D + 31) / 32), 2), dim3(32, 32), 0, s,
                 (const float*)p.parts, (int)c.D, rows * g.units_q, rows * g.units_k, c.heads[0] ? c.dw[0] : nullptr,
                 c.heads[1] ? c.dw[1] : nullptr);
  }
  return e == cudaSuccess ? FAR_OK : cuda_error_status(e);
}

}  // namespace

}  // namespace far

using namespace far;

extern "C" {

int qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_token_stride,
                 int64_t k_head_stride, const void* q_weight, const void* k_weight, float eps, const float* table,
                 int64_t table_rows, const void* positions, int position_bytes, void* q_out,
                 int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out, int64_t k_out_token_stride,
                 int64_t k_out_head_stride, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                 int64_t rot_dim, int pairs, int dtype, void* stream) {
  if (dtype < 0 || (dtype >> 8) != 0) return FAR_ERR_DTYPE;
  QkCall c{{{q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride}},
           {},
           {{q_out, q_out_token_stride, q_out_head_stride}, {k_out, k_out_token_stride, k_out_head_stride}},
           {q_weight, k_weight},
           {q_heads, k_heads},
           eps,
           table,
           table_rows,
           positions,
           position_bytes,
           tokens,
           head_dim,
           rot_dim,
           pairs,
           dtype & 0xf,
           (dtype >> 4) & 0xf,
           true,
           false,
           false,
           {},
           nullptr,
           0};
  return run_qk(c, stream);
}

int rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_token_stride,
         int64_t k_head_stride, const float* table, int64_t table_rows, const void* positions, int position_bytes,
         void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out, int64_t k_out_token_stride,
         int64_t k_out_head_stride, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
         int64_t rot_dim, int pairs, int transpose, int act, void* stream) {
  if (transpose != 0 && transpose != 1) return FAR_ERR_DTYPE;
  QkCall c{{{q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride}},
           {},
           {{q_out, q_out_token_stride, q_out_head_stride}, {k_out, k_out_token_stride, k_out_head_stride}},
           {},
           {q_heads, k_heads},
           0.f,
           table,
           table_rows,
           positions,
           position_bytes,
           tokens,
           head_dim,
           rot_dim,
           pairs,
           act,
           act,
           false,
           false,
           transpose == 1,
           {},
           nullptr,
           0};
  return run_qk(c, stream);
}

int64_t far_qk_backward_workspace_bytes(int64_t head_dim) {
  if (head_dim < 1 || head_dim > kQkMaxDim) return -FAR_ERR_SHAPE;
  return (int64_t)kQkParts * head_dim * 4;
}

int qk_norm_rope_backward(const void* dq_out, int64_t dq_out_token_stride, int64_t dq_out_head_stride,
                          const void* dk_out, int64_t dk_out_token_stride, int64_t dk_out_head_stride, const void* q,
                          int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_token_stride,
                          int64_t k_head_stride, const void* q_weight, const void* k_weight, float eps,
                          const float* table, int64_t table_rows, const void* positions, int position_bytes, void* dq,
                          int64_t dq_token_stride, int64_t dq_head_stride, void* dk, int64_t dk_token_stride,
                          int64_t dk_head_stride, float* dq_weight, float* dk_weight, void* workspace,
                          int64_t workspace_bytes, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                          int64_t rot_dim, int pairs, int dtype, void* stream) {
  if (dtype < 0 || (dtype >> 8) != 0) return FAR_ERR_DTYPE;
  QkCall c{{{q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride}},
           {{dq_out, dq_out_token_stride, dq_out_head_stride}, {dk_out, dk_out_token_stride, dk_out_head_stride}},
           {{dq, dq_token_stride, dq_head_stride}, {dk, dk_token_stride, dk_head_stride}},
           {q_weight, k_weight},
           {q_heads, k_heads},
           eps,
           table,
           table_rows,
           positions,
           position_bytes,
           tokens,
           head_dim,
           rot_dim,
           pairs,
           dtype & 0xf,
           (dtype >> 4) & 0xf,
           true,
           true,
           false,
           {dq_weight, dk_weight},
           workspace,
           workspace_bytes};
  return run_qk(c, stream);
}

int far_rope_frequencies(int64_t rot_dim, double base, int scaling, const double* params, double* freq,
                         double* attention_factor) {
  if (rot_dim < 2 || rot_dim > kQkMaxDim || rot_dim % 2 != 0) return FAR_ERR_SHAPE;
  if (scaling < FAR_ROPE_PLAIN || scaling > FAR_ROPE_BANDS) return FAR_ERR_DTYPE;
  if (!freq || !attention_factor || (scaling != FAR_ROPE_PLAIN && !params)) return FAR_ERR_NULL;
  if (!(base > 1.0) || !isfinite(base)) return FAR_ERR_EPS;
  const int np = scaling == FAR_ROPE_PLAIN ? 0 : scaling == FAR_ROPE_YARN ? 5 : scaling == FAR_ROPE_BANDS ? 4 : 1;
  for (int i = 0; i < np; ++i)
    if (!isfinite(params[i]) || params[i] < 0.0 || (params[i] == 0.0 && !(scaling == FAR_ROPE_YARN && i == 4)))
      return FAR_ERR_EPS;
  if (scaling == FAR_ROPE_NTK && rot_dim == 2) return FAR_ERR_SHAPE;
  if (scaling == FAR_ROPE_BANDS && params[3] <= params[2]) return FAR_ERR_EPS;
  const double pi = 3.14159265358979323846, R = (double)rot_dim, a = np ? params[0] : 1.0;
  double b = base, low = 0.0, high = 1.0;
  *attention_factor = 1.0;
  if (scaling == FAR_ROPE_NTK) b = base * pow(a, R / (R - 2.0));
  if (!(b > 1.0) || !isfinite(b)) return FAR_ERR_EPS;
  if (scaling == FAR_ROPE_YARN) {
    auto d = [&](double turns) { return R * log(params[1] / (2.0 * pi * turns)) / (2.0 * log(base)); };
    low = fmin(fmax(floor(d(params[2])), 0.0), R - 1.0);
    high = fmin(fmax(ceil(d(params[3])), 0.0), R - 1.0);
    if (high < low + 0.001) high = low + 0.001;
    *attention_factor = params[4] > 0.0 ? params[4] : a > 1.0 ? 0.1 * log(a) + 1.0 : 1.0;
  }
  for (int j = 0; j < rot_dim / 2; ++j) {
    const double f = pow(b, -2.0 * j / R);
    double v = f;
    if (scaling == FAR_ROPE_LINEAR) v = f / a;
    if (scaling == FAR_ROPE_YARN) {
      const double m = fmin(fmax((j - low) / (high - low), 0.0), 1.0);
      v = f * (1.0 - m) + f / a * m;
    }
    if (scaling == FAR_ROPE_BANDS) {
      const double t = params[1] * f / (2.0 * pi);
      const double m = (t - params[2]) / (params[3] - params[2]);
      v = t > params[3] ? f : t < params[2] ? f / a : f * (m + (1.0 - m) / a);
    }
    freq[j] = v;
  }
  return FAR_OK;
}

int rope_table(float* table, int64_t rows, int64_t rot_dim, int64_t first_position, const double* freq, double factor,
               void* stream) {
  if (rot_dim < 2 || rot_dim > kQkMaxDim || rot_dim % 2 != 0 || rows < 0 || rows > (int64_t(1) << 40) / rot_dim ||
      first_position < 0 || first_position > (int64_t(1) << 40))
    return FAR_ERR_SHAPE;
  if (!isfinite(factor)) return FAR_ERR_EPS;
  if (!freq || (rows > 0 && !table)) return FAR_ERR_NULL;
  if ((uintptr_t)table & 3) return FAR_ERR_SHAPE;
  Freqs q;
  for (int j = 0; j < rot_dim / 2; ++j) {
    if (!isfinite(freq[j])) return FAR_ERR_EPS;
    q.f[j] = freq[j];
  }
  if (rows == 0) return FAR_OK;
  unsigned int* status = nullptr;
  int sms = 0;
  int st = device_info(&status, &sms);
  if (st != FAR_OK) return st;
  const int64_t blocks = (rows * (rot_dim / 2) + 255) / 256;
  cudaError_t e = launch_k(rope_table_kernel, dim3((unsigned)(blocks < 32 * sms ? blocks : 32 * sms)), dim3(256), 0,
                           static_cast<cudaStream_t>(stream), table, rows, (int)(rot_dim / 2), first_position, factor,
                           (const Freqs)q);
  return e == cudaSuccess ? FAR_OK : cuda_error_status(e);
}

}  // extern "C"
