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
// the heads it takes of that token (a block takes queries or keys).  Its heads
// arrive through a ring in shared memory (cp.async, each lane its own chunks, so no lane
// waits for another), several steps ahead: the registers hold one step's values, and what is
// in flight does not depend on how many warps they leave room for.  With loads into
// registers instead, 128 bytes a lane and 16 warps an SM, the forward pass over 16384 tokens
// of 32 + 8 heads of 128 bf16 values took 70.4 us and the backward pass over 8192 77.9; now 63.7 us
// (5.4 TB/s, 81 % of a copy's rate) and 48.8 us (5.2 TB/s).  About 210 and 400 instructions a step
// of four heads keep the schedulers 60 % busy beside DRAM at 61 %; three CTAs an SM, or the
// table's rows fetched ahead through the ring too, took longer (66.0; 64.4 and 52.1 us).
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
constexpr int kQkCtas = 2;       // CTAs an SM that the vector kernels' registers leave room for
constexpr int kQkSteps = 6;      // ring slots of 1 KB a warp: 48 KB a CTA
constexpr int kQkBackSteps = 3;  // ... of 2 KB
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
  float eps, inv_dim, sign;  // inv_dim: 1 / D rounded; sign: -1 turns the other way
  int32_t D, rot;
  int32_t pos64, w32;
  int32_t log_l;    // vector kernels: log2 of the lanes a head takes
  // vector kernels: blocks below blocks_q take queries, the others keys.  A warp's item is
  // nb steps of neighbouring heads of one token; parts_a_token items a token.
  int32_t blocks_q, nb, parts_a_token[2];
  int32_t units_q;  // scalar kernels: blockIdx.y below this: queries, else keys
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

// 1 / sqrt(S / D + eps), given S within 5.5 * 2^-24: S times the rounded 1 / D and the sum with eps (three roundings,
// halved by the root), and CUDA's rsqrtf (two units in the last place, 4 * 2^-24).  With each step rounded by
// itself (division, sum, root, reciprocal) it would be 3 * 2^-24, and four times the instructions on every step's path.
__device__ __forceinline__ float head_rstd(float S, const QkParams& p) {
  return rsqrtf(__fadd_rn(__fmul_rn(S, p.inv_dim), p.eps));
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    if (off < lanes) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));  // (the whole warp alike)
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

// Two neighbouring values, in two registers.  (In one 64-bit register, for the packed binary32
// instructions, the backward pass of 8192 tokens took 55.5 us against 55.0: what the packed
// forms saved went into moves.)
struct X2 {
  float x, y;
};
__device__ __forceinline__ X2 x2(float x, float y) { return X2{x, y}; }
__device__ __forceinline__ float2 un2(X2 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ X2 vfma(X2 a, X2 b, X2 c) { return X2{__fmaf_rn(a.x, b.x, c.x), __fmaf_rn(a.y, b.y, c.y)}; }
// c - a b
__device__ __forceinline__ X2 vnfma(X2 a, X2 b, X2 c) { return X2{__fmaf_rn(-a.x, b.x, c.x), __fmaf_rn(-a.y, b.y, c.y)}; }
__device__ __forceinline__ X2 vmul(X2 a, X2 b) { return X2{__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y)}; }
__device__ __forceinline__ X2 vadd(X2 a, X2 b) { return X2{__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)}; }

// Two chunks of V values each, in pairs.
template <int V>
struct Pair2 {
  X2 a[V / 2], b[V / 2];
};
template <int ACT, int V> __device__ __forceinline__ void widen2x(const uint4& r, X2 (&p)[V / 2]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  float f[V];
  widen<ACT, V>(w, f);
#pragma unroll
  for (int e = 0; e < V / 2; ++e) p[e] = x2(f[2 * e], f[2 * e + 1]);
}
template <int ACT, int V> __device__ __forceinline__ void store_chunk(char* dst, int chunk, const X2 (&p)[V / 2]) {
  if (chunk < 0) return;
  float f[V];
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    const float2 t = un2(p[e]);
    f[2 * e] = t.x;
    f[2 * e + 1] = t.y;
  }
  uint32_t w[4];
  narrow<ACT, V>(f, w);
  store_bytes<16>(dst + 16 * chunk, w);
}

__device__ __forceinline__ X2 swap_x2(X2 v) { return X2{v.y, v.x}; }

// The cosines and sines a lane needs.  Half pairs: V of each, shared by its two chunks, packed
// two neighbours a word: c and s.  Interleaved pairs: V/2 of each for either chunk, each
// cosine twice in a word and the sine as (-s, s), so that a pair (x, y) turns to
// (x, y) (c, c) + (y, x) (-s, s).
template <bool INTER, int V>
struct Turn {
  X2 c[V / 2 * (INTER ? 2 : 1)], s[V / 2 * (INTER ? 2 : 1)];
  __device__ __forceinline__ void load(const float* row, const Slot& k, int half, float sign) {
    if constexpr (INTER) {
      constexpr int P = V / 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool on = h ? k.rb : k.ra;
        const int chunk = h ? k.cb : k.ca;
        float cc[P], ss[P];
#pragma unroll
        for (int e = 0; e < P; e += 2) {
          float2 u = make_float2(1.f, 1.f), v = make_float2(0.f, 0.f);
          if (on) {
            u = *reinterpret_cast<const float2*>(row + chunk * P + e);
            v = *reinterpret_cast<const float2*>(row + half + chunk * P + e);
          }
          cc[e] = u.x; cc[e + 1] = u.y; ss[e] = sign * v.x; ss[e + 1] = sign * v.y;
        }
#pragma unroll
        for (int e = 0; e < P; ++e) {
          c[h * P + e] = x2(cc[e], cc[e]);
          s[h * P + e] = x2(-ss[e], ss[e]);
        }
      }
    } else if (k.ra) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const float4 u = reinterpret_cast<const float4*>(row + k.ca * V)[q];
        const float4 v = reinterpret_cast<const float4*>(row + half + k.ca * V)[q];
        c[2 * q] = x2(u.x, u.y);
        c[2 * q + 1] = x2(u.z, u.w);
        s[2 * q] = x2(v.x, v.y);
        s[2 * q + 1] = x2(v.z, v.w);
      }
    }
  }
  // turns the lane's two chunks in place (values outside the rotated part are left alone);
  // BACK: the other way (interleaved pairs: the sines' sign says which)
  template <bool BACK>
  __device__ __forceinline__ void apply(Pair2<V>& x, const Slot& k) const {
    if constexpr (INTER) {
      constexpr int P = V / 2;
      if (k.ra) {
#pragma unroll
        for (int e = 0; e < P; ++e) x.a[e] = vfma(x.a[e], c[e], vmul(swap_x2(x.a[e]), s[e]));
      }
      if (k.rb) {
#pragma unroll
        for (int e = 0; e < P; ++e) x.b[e] = vfma(x.b[e], c[P + e], vmul(swap_x2(x.b[e]), s[P + e]));
      }
    } else if (k.ra) {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const X2 u = x.a[e], v = x.b[e];
        if constexpr (BACK) {
          x.a[e] = vfma(u, c[e], vmul(v, s[e]));
          x.b[e] = vnfma(u, s[e], vmul(v, c[e]));
        } else {
          x.a[e] = vnfma(v, s[e], vmul(u, c[e]));
          x.b[e] = vfma(v, c[e], vmul(u, s[e]));
        }
      }
    }
  }
};

// the weight's values of a lane's two chunks (zeros where there is none: the lane adds nothing)
template <int ACT, int V>
__device__ __forceinline__ void load_weights(const void* w, int w32, const Slot& k, Pair2<V>& f) {
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    const int a = k.ca * V + 2 * e, b = k.cb * V + 2 * e;
    f.a[e] = k.ca >= 0 ? x2(load_w<ACT>(w, w32, a), load_w<ACT>(w, w32, a + 1)) : X2{0.f, 0.f};
    f.b[e] = k.cb >= 0 ? x2(load_w<ACT>(w, w32, b), load_w<ACT>(w, w32, b + 1)) : X2{0.f, 0.f};
  }
}

// 16 bytes into this lane's place of the ring, without waiting
__device__ __forceinline__ void async_chunk(uint32_t dst, const char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 take_chunk(uint32_t src) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(src) : "memory");
  return r;
}
__device__ __forceinline__ void clear_chunk(uint32_t dst) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// the sum over a head's lanes of what each lane holds in packed pairs
__device__ __forceinline__ float head_sum(X2 v, int lanes) {
  const float2 f = un2(v);
  return lanes_sum(__fadd_rn(f.x, f.y), lanes);
}

// What a token without a place in the table gets: zeros for padding, NaN past its end.
__device__ __forceinline__ void store_bad(char* y, const Slot& k, int64_t pos) {
  const uint32_t v = pos < 0 ? 0u : 0xffffffffu;  // all ones is a NaN in every type
  const uint32_t w[4] = {v, v, v, v};
  if (k.ca >= 0) store_bytes<16>(y + 16 * k.ca, w);
  if (k.cb >= 0) store_bytes<16>(y + 16 * k.cb, w);
}

// A warp's walk over its items: `groups` neighbouring heads a step (one for each group of
// lanes), nb steps an item.  What it points to moves along by additions.
struct Walk {
  int64_t item, t;
  int h, end;  // this step's first head; the item's heads end
  __device__ __forceinline__ bool done(int64_t items) const { return item >= items; }
  __device__ __forceinline__ void start(int parts, int span, int heads) {
    int part = 0;
    t = item;
    if (parts > 1) {
      t = item / parts;
      part = (int)(item - t * parts);
    }
    h = part * span;
    end = min(heads, h + span);
  }
};

template <int ACT, bool INTER, bool NORM, int LOGL>
__global__ void __launch_bounds__(kQkThreads, kQkCtas) qk_kernel(const QkParams p) {
  constexpr int V = 16 / dtype_size<ACT>::value;
  extern __shared__ __align__(16) unsigned char ring[];  // [warps][kQkSteps][2][32 lanes] chunks
  pdl_launch_dependents();
  pdl_wait();
  // (broadcast, so that the compiler keeps the warp's walk in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int log_l = LOGL >= 0 ? LOGL : p.log_l;
  const int L = 1 << log_l, groups = 32 >> log_l, grp = lane >> log_l;
  const bool is_k = (int)blockIdx.x >= p.blocks_q;
  const QkSeg S = is_k ? p.seg[1] : p.seg[0];
  const int parts = p.parts_a_token[is_k], span = p.nb * groups, heads = S.heads;
  const int64_t items = p.tokens * parts;
  const int64_t stride = (int64_t)(is_k ? gridDim.x - p.blocks_q : p.blocks_q) * warps;
  const Slot k = slot_of<INTER>(lane & (L - 1), p.D / V, p.rot / V);
  const uint32_t mine = smem_addr(ring) + warp * (kQkSteps * 1024) + lane * 16;
  const int64_t oa = grp * S.xh + 16 * max(k.ca, 0), ob = grp * S.xh + 16 * max(k.cb, 0);  // this lane's places
  if (k.ca < 0 || k.cb < 0)  // chunks that never arrive add nothing to their head
    for (int i = 0; i < 2 * kQkSteps; ++i) clear_chunk(mine + 512 * i);
  Walk in{(int64_t)(is_k ? (int)blockIdx.x - p.blocks_q : (int)blockIdx.x) * warps + warp, 0, 0, 0};
  Walk at = in;
  const char* src = nullptr;
  auto aim = [&]() {
    in.start(parts, span, heads);
    src = S.x + in.t * S.xt + (int64_t)in.h * S.xh;
  };
  if (!in.done(items)) aim();
  const int64_t xh = groups * S.xh, yh = groups * S.yh;
  // one step's chunks of this lane on their way
  auto fetch = [&](int slot) {
    if (!in.done(items)) {
      if (in.h + grp < in.end) {
        if (k.ca >= 0) async_chunk(mine + slot * 1024, src + oa);
        if (k.cb >= 0) async_chunk(mine + slot * 1024 + 512, src + ob);
      }
      src += xh;
      in.h += groups;
      if (in.h >= in.end) {
        in.item += stride;
        if (!in.done(items)) aim();
      }
    }
    async_commit();
  };
#pragma unroll
  for (int i = 0; i < kQkSteps - 1; ++i) fetch(i);
  Pair2<V> w;
  if constexpr (NORM) load_weights<ACT, V>(S.w, p.w32, k, w);
  Turn<INTER, V> turn;
  int slot = 0;
  for (; !at.done(items); at.item += stride) {
    at.start(parts, span, heads);
    const int64_t pos = load_pos(p, at.t);
    const bool ok = pos >= 0 && pos < p.table_rows;
    if (pos >= p.table_rows && lane == 0) atomicOr(p.status, 1u << FAR_ERR_POSITION);
    turn.load(p.table + (ok ? pos : 0) * p.rot, k, p.rot >> 1, p.sign);
    char* y = S.y + at.t * S.yt + (int64_t)(at.h + grp) * S.yh;
    for (; at.h < at.end; at.h += groups, y += yh) {
      fetch(slot == 0 ? kQkSteps - 1 : slot - 1);
      async_wait<kQkSteps - 1>();
      const bool here = at.h + grp < at.end;
      if (!ok) {  // (the whole warp)
        if (here) store_bad(y, k, pos);
        if (++slot == kQkSteps) slot = 0;
        continue;
      }
      Pair2<V> x;
      widen2x<ACT, V>(take_chunk(mine + slot * 1024), x.a);
      widen2x<ACT, V>(take_chunk(mine + slot * 1024 + 512), x.b);
      if constexpr (NORM) {
        X2 ss = X2{0.f, 0.f}, st = X2{0.f, 0.f};
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          ss = vfma(x.a[e], x.a[e], ss);
          st = vfma(x.b[e], x.b[e], st);
        }
        const float r = head_rstd(head_sum(vadd(ss, st), L), p);
        const X2 r2 = x2(r, r);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          x.a[e] = vmul(vmul(x.a[e], r2), w.a[e]);
          x.b[e] = vmul(vmul(x.b[e], r2), w.b[e]);
        }
      }
      if (!NORM && p.sign < 0.f) turn.template apply<true>(x, k);
      else turn.template apply<false>(x, k);
      if (here) {
        store_chunk<ACT, V>(y, k.ca, x.a);
        store_chunk<ACT, V>(y, k.cb, x.b);
      }
      if (++slot == kQkSteps) slot = 0;
    }
  }
}

// One partial row of the weights' gradient a block: the warps' sums, added in their order.
template <int V>
__device__ __forceinline__ void write_part(float* part, float* sm, const Slot& k, const Pair2<V>& d, int L, int lane,
                                           int warp, int warps, int D) {
  float da[V], db[V];
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    const float2 u = un2(d.a[e]), v = un2(d.b[e]);
    da[2 * e] = u.x;
    da[2 * e + 1] = u.y;
    db[2 * e] = v.x;
    db[2 * e + 1] = v.y;
  }
#pragma unroll
  for (int e = 0; e < V; ++e)
    for (int off = L; off < 32; off <<= 1) {
      da[e] = __fadd_rn(da[e], __shfl_xor_sync(0xffffffffu, da[e], off));
      db[e] = __fadd_rn(db[e], __shfl_xor_sync(0xffffffffu, db[e], off));
    }
  __syncthreads();  // every warp is done with the ring, where the sums go
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

template <int ACT, bool INTER, int LOGL>
__global__ void __launch_bounds__(kQkThreads, kQkCtas) qk_back_kernel(const QkParams p) {
  constexpr int V = 16 / dtype_size<ACT>::value;
  extern __shared__ __align__(16) unsigned char ring[];  // [warps][kQkBackSteps][x, x, dy, dy][32 lanes] chunks
  pdl_launch_dependents();
  pdl_wait();
  // (broadcast, so that the compiler keeps the warp's walk in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int log_l = LOGL >= 0 ? LOGL : p.log_l;
  const int L = 1 << log_l, groups = 32 >> log_l, grp = lane >> log_l;
  const bool is_k = (int)blockIdx.x >= p.blocks_q;
  const QkSeg S = is_k ? p.seg[1] : p.seg[0];
  const int parts = p.parts_a_token[is_k], span = p.nb * groups, heads = S.heads;
  const int64_t items = p.tokens * parts;
  const int64_t stride = (int64_t)(is_k ? gridDim.x - p.blocks_q : p.blocks_q) * warps;
  const Slot k = slot_of<INTER>(lane & (L - 1), p.D / V, p.rot / V);
  const uint32_t mine = smem_addr(ring) + warp * (kQkBackSteps * 2048) + lane * 16;
  const int64_t oa = grp * S.xh + 16 * max(k.ca, 0), ob = grp * S.xh + 16 * max(k.cb, 0);
  const int64_t ga = grp * S.gh + 16 * max(k.ca, 0), gb = grp * S.gh + 16 * max(k.cb, 0);
  if (k.ca < 0 || k.cb < 0)
    for (int i = 0; i < 4 * kQkBackSteps; ++i) clear_chunk(mine + 512 * i);
  Walk in{(int64_t)(is_k ? (int)blockIdx.x - p.blocks_q : (int)blockIdx.x) * warps + warp, 0, 0, 0};
  Walk at = in;
  const char *src = nullptr, *grad = nullptr;
  auto aim = [&]() {
    in.start(parts, span, heads);
    src = S.x + in.t * S.xt + (int64_t)in.h * S.xh;
    grad = S.g + in.t * S.gt + (int64_t)in.h * S.gh;
  };
  if (!in.done(items)) aim();
  const int64_t xh = groups * S.xh, gh = groups * S.gh, yh = groups * S.yh;
  auto fetch = [&](int slot) {
    if (!in.done(items)) {
      if (in.h + grp < in.end) {
        if (k.ca >= 0) {
          async_chunk(mine + slot * 2048, src + oa);
          async_chunk(mine + slot * 2048 + 1024, grad + ga);
        }
        if (k.cb >= 0) {
          async_chunk(mine + slot * 2048 + 512, src + ob);
          async_chunk(mine + slot * 2048 + 1536, grad + gb);
        }
      }
      src += xh;
      grad += gh;
      in.h += groups;
      if (in.h >= in.end) {
        in.item += stride;
        if (!in.done(items)) aim();
      }
    }
    async_commit();
  };
#pragma unroll
  for (int i = 0; i < kQkBackSteps - 1; ++i) fetch(i);
  Pair2<V> w, dw;
  load_weights<ACT, V>(S.w, p.w32, k, w);
#pragma unroll
  for (int e = 0; e < V / 2; ++e) dw.a[e] = dw.b[e] = X2{0.f, 0.f};
  Turn<INTER, V> turn;
  int slot = 0;
  for (; !at.done(items); at.item += stride) {
    at.start(parts, span, heads);
    const int64_t pos = load_pos(p, at.t);
    const bool ok = pos >= 0 && pos < p.table_rows;
    if (pos >= p.table_rows && lane == 0) atomicOr(p.status, 1u << FAR_ERR_POSITION);
    turn.load(p.table + (ok ? pos : 0) * p.rot, k, p.rot >> 1, p.sign);
    char* y = S.y + at.t * S.yt + (int64_t)(at.h + grp) * S.yh;
    for (; at.h < at.end; at.h += groups, y += yh) {
      fetch(slot == 0 ? kQkBackSteps - 1 : slot - 1);
      async_wait<kQkBackSteps - 1>();
      const bool here = at.h + grp < at.end;
      if (!ok) {
        if (here) store_bad(y, k, pos);
        if (++slot == kQkBackSteps) slot = 0;
        continue;
      }
      Pair2<V> x, g;
      widen2x<ACT, V>(take_chunk(mine + slot * 2048), x.a);
      widen2x<ACT, V>(take_chunk(mine + slot * 2048 + 512), x.b);
      widen2x<ACT, V>(take_chunk(mine + slot * 2048 + 1024), g.a);
      widen2x<ACT, V>(take_chunk(mine + slot * 2048 + 1536), g.b);
      X2 ss = X2{0.f, 0.f}, st = X2{0.f, 0.f};
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        ss = vfma(x.a[e], x.a[e], ss);
        st = vfma(x.b[e], x.b[e], st);
      }
      const float r = head_rstd(head_sum(vadd(ss, st), L), p);
      const X2 r2 = x2(r, r);
      turn.template apply<true>(g, k);
      ss = st = X2{0.f, 0.f};
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        x.a[e] = vmul(x.a[e], r2);  // u = x r
        x.b[e] = vmul(x.b[e], r2);
        if (here) {
          dw.a[e] = vfma(g.a[e], x.a[e], dw.a[e]);
          dw.b[e] = vfma(g.b[e], x.b[e], dw.b[e]);
        }
        g.a[e] = vmul(g.a[e], w.a[e]);  // h = g w
        g.b[e] = vmul(g.b[e], w.b[e]);
        ss = vfma(g.a[e], x.a[e], ss);
        st = vfma(g.b[e], x.b[e], st);
      }
      const float m = -__fmul_rn(head_sum(vadd(ss, st), L), p.inv_dim);
      const X2 m2 = x2(m, m);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        x.a[e] = vmul(r2, vfma(x.a[e], m2, g.a[e]));
        x.b[e] = vmul(r2, vfma(x.b[e], m2, g.b[e]));
      }
      if (here) {
        store_chunk<ACT, V>(y, k.ca, x.a);
        store_chunk<ACT, V>(y, k.cb, x.b);
      }
      if (++slot == kQkBackSteps) slot = 0;
    }
  }
  async_wait<0>();
  write_part<V>(p.parts + (int64_t)blockIdx.x * p.D, reinterpret_cast<float*>(ring), k, dw, L,
                lane, warp, warps, p.D);
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
      r = head_rstd(lanes_sum(ss, 32), p);
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
        const float m = sweep ? __fmul_rn(lanes_sum(dot, 32), p.inv_dim) : 0.f;
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

// A sum in two binary32 numbers: what each addition rounds off (exact, Knuth 1969) is added up beside it.
struct Two {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
  }
  __device__ __forceinline__ void add(const Two& x) {
    add(x.hi);
    lo = __fadd_rn(lo, x.lo);
  }
  __device__ __forceinline__ float value() const { return isfinite(hi) ? __fadd_rn(hi, lo) : hi; }
};

// The partial rows summed in a fixed order (every 32nd row by a lane of rows, then the lanes by halves), each sum in two
// binary32 numbers (Two): in binary64 it took some 2 us longer of the backward pass's 53 (8192 tokens of 32 + 8 heads).
// So what the gradients err is what the lanes that made the rows add up, one head after another: block (32 columns x 32 row lanes), blockIdx.y = 0 the queries' weight, 1 the keys'.
__global__ void __launch_bounds__(1024)
    qk_weight_grad_kernel(const float* parts, int D, int rows_q, int rows_k, float* dq_weight, float* dk_weight) {
  __shared__ float2 sm[32][33];
  pdl_launch_dependents();
  pdl_wait();
  const int col = blockIdx.x * 32 + threadIdx.x;
  const int rows = blockIdx.y ? rows_k : rows_q;
  const float* base = parts + (blockIdx.y ? (int64_t)rows_q * D : 0);
  float* out = blockIdx.y ? dk_weight : dq_weight;
  Two v;
  if (col < D) {
#pragma unroll 8
    for (int r = threadIdx.y; r < rows; r += 32) v.add(base[(int64_t)r * D + col]);
  }
  sm[threadIdx.y][threadIdx.x] = make_float2(v.hi, v.lo);
  __syncthreads();
  // turned: a warp adds the 32 row lanes of one column
  const float2 mine = sm[threadIdx.x][threadIdx.y];
  Two t{mine.x, mine.y};
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    t.add(Two{__shfl_xor_sync(0xffffffffu, t.hi, off), __shfl_xor_sync(0xffffffffu, t.lo, off)});
  const int c = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && c < D && out) out[c] = t.value();
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

// Do two [tokens, heads, D] tensors share a byte?  Exact for equal strides (queries and keys
// interleaved in one buffer in whatever way), else whether the bytes they span meet.
bool heads_meet(const Heads& a, int64_t ha, const Heads& b, int64_t hb, int64_t tokens, int64_t D, int64_t es) {
  const bool same = (tokens == 1 || a.ts == b.ts) && (a.hs == b.hs || (ha == 1 && hb == 1));
  if (!regions_overlap(heads_region(a, tokens, ha, D, es), heads_region(b, tokens, hb, D, es))) return false;
  if (!same || ha + hb > 8192) return true;
  // head i of token t of a and head j of token u of b meet iff |d + (u - t) ts + (j - i) hs| < D, in
  // elements where the bases differ by whole ones, in bytes to be exact
  const int64_t d = (int64_t)((uint64_t)(uintptr_t)b.p - (uint64_t)(uintptr_t)a.p), w = D * es, ts = tokens == 1 ? 0 : a.ts * es;
  for (int64_t dh = -(ha - 1); dh <= hb - 1; ++dh) {
    const int64_t at = d + dh * a.hs * es;
    if (ts == 0) {
      if (at > -w && at < w) return true;
      continue;
    }
    const int64_t lo = floor_div(-w - at, ts) + 1, hi = -floor_div(at - w, ts) - 1;  // -w < at + k ts < w
    if (lo <= hi && lo <= tokens - 1 && hi >= -(tokens - 1)) return true;
  }
  return false;
}

bool same_heads(const Heads& a, const Heads& b, int64_t tokens, int64_t heads) {
  return a.p == b.p && (tokens == 1 || a.ts == b.ts) && (heads == 1 || a.hs == b.hs);
}

constexpr int64_t kQkMaxHeads = int64_t(1) << 30;  // (a head's number, and the next steps', in 32 bits)
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
  if (c.tokens > INT32_MAX || c.heads[0] > kQkMaxHeads || c.heads[1] > kQkMaxHeads || c.table_rows > kQkLimit)
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
    if (c.heads[i]) {
      for (const void* q : {c.x[i].p, (const void*)c.y[i].p, c.back ? c.g[i].p : nullptr})
        if ((uintptr_t)q % es) return FAR_ERR_SHAPE;
      if ((c.norm && (uintptr_t)c.w[i] % esize(c.wd)) || (c.back && (uintptr_t)c.dw[i] % 4)) return FAR_ERR_SHAPE;
    }
  if ((uintptr_t)c.table % 4 || (uintptr_t)c.pos % c.pos_bytes) return FAR_ERR_SHAPE;
  if (c.back && (!c.ws || c.ws_bytes < far_qk_backward_workspace_bytes(c.D) || ((uintptr_t)c.ws & 15)))
    return FAR_ERR_WORKSPACE;
  // overlaps: every written buffer against every other
  Region wr[3], rd[4];
  int nw = 0, nr = 0;
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
  for (int i = 0; i < 2; ++i) {
    if (!c.heads[i]) continue;
    const Region Y = heads_region(c.y[i], c.tokens, c.heads[i], c.D, es);
    for (int b = 0; b < nr; ++b)
      if (regions_overlap(Y, rd[b])) return FAR_ERR_ALIAS;
    for (int b = 0; b < nw; ++b)
      if (regions_overlap(Y, wr[b])) return FAR_ERR_ALIAS;
    if (i == 0 && c.heads[1] && heads_meet(c.y[0], c.heads[0], c.y[1], c.heads[1], c.tokens, c.D, es)) return FAR_ERR_ALIAS;
    for (int j = 0; j < 2; ++j) {
      if (!c.heads[j]) continue;
      for (const Heads* t : {&c.x[j], &c.g[j]}) {
        if (t == &c.g[j] && !c.back) continue;
        if (!(i == j && same_heads(c.y[i], *t, c.tokens, c.heads[i])) &&
            heads_meet(c.y[i], c.heads[i], *t, c.heads[j], c.tokens, c.D, es))
          return FAR_ERR_ALIAS;
        const Region X = heads_region(*t, c.tokens, c.heads[j], c.D, es);
        for (int b = 0; b < nw; ++b)
          if (regions_overlap(wr[b], X)) return FAR_ERR_ALIAS;
      }
    }
  }
  return FAR_OK;
}

struct QkPlan {
  bool vec;
  int log_l, nb, parts[2], blocks[2];
  int units_q, units_k;
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
  // Steps (of `groups` heads) a warp takes of a token at a time, with that token's cosines and
  // sines in its registers: up to 8, fewer (down to one) while that leaves SMs without 16 warps
  // of work.
  const int64_t steps[2] = {(c.heads[0] + groups - 1) / groups, (c.heads[1] + groups - 1) / groups};
  g.nb = 8;
  auto items = [&](int i) { return c.tokens * ((steps[i] + g.nb - 1) / g.nb); };
  while (g.nb > 1 && items(0) + items(1) < (int64_t)sms * 16) g.nb /= 2;
  int warps = 8;
  while (warps > 1 && (items(0) + items(1)) / warps < sms) warps /= 2;
  // one wave of blocks, shared between queries and keys as their steps are
  const int64_t all = kQkCtas * sms < kQkParts ? kQkCtas * sms : kQkParts;
  int64_t blocks[2];
  for (int i = 0; i < 2; ++i) {
    g.parts[i] = (int)((steps[i] + g.nb - 1) / g.nb);
    const int64_t need = (items(i) + warps - 1) / warps;
    int64_t share = (all * steps[i] + (steps[0] + steps[1]) / 2) / (steps[0] + steps[1]);
    if (share < 1) share = 1;
    if (share > all - 1) share = all - 1;  // (the other has at least one)
    if (c.heads[1 - i] == 0) share = all;
    blocks[i] = c.heads[i] == 0 ? 0 : need < share ? need : share;
  }
  g.blocks[0] = (int)blocks[0];
  g.blocks[1] = (int)blocks[1];
  g.grid = dim3((unsigned)(blocks[0] + blocks[1]));
  g.block = dim3(32 * warps);
  g.smem = (size_t)warps * (c.back ? kQkBackSteps * 2048 : kQkSteps * 1024);  // (the weights' sums fit: D <= 512)
  return g;
}

template <int ACT, int LOGL>
auto pick_qk(const QkCall& c) -> void (*)(QkParams) {
  const bool inter = c.pairs == FAR_PAIRS_INTERLEAVED;
  if (c.back) return inter ? qk_back_kernel<ACT, true, LOGL> : qk_back_kernel<ACT, false, LOGL>;
  if (c.norm) return inter ? qk_kernel<ACT, true, true, LOGL> : qk_kernel<ACT, false, true, LOGL>;
  return inter ? qk_kernel<ACT, true, false, LOGL> : qk_kernel<ACT, false, false, LOGL>;
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
  // the sums over a head's lanes are unrolled for the usual head sizes (64, 128 and 256 in 16 bits)
  void (*k)(QkParams) = g.log_l == 2   ? pick_qk<ACT, 2>(c)
                        : g.log_l == 3 ? pick_qk<ACT, 3>(c)
                        : g.log_l == 4 ? pick_qk<ACT, 4>(c)
                                       : pick_qk<ACT, -1>(c);
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
  p.inv_dim = 1.0f / (float)c.D;
  p.sign = (c.back || c.transpose) ? -1.f : 1.f;
  p.D = (int32_t)c.D;
  p.rot = (int32_t)c.rot;
  p.pos64 = c.pos_bytes == 8;
  p.w32 = c.wd == FAR_F32 ? 1 : c.wd == FAR_F16 ? 2 : 3;
  p.log_l = g.log_l;
  p.units_q = g.units_q;
  p.blocks_q = g.blocks[0];
  p.nb = g.nb;
  p.parts_a_token[0] = g.parts[0];
  p.parts_a_token[1] = g.parts[1];
  cudaError_t e = c.act == FAR_F16    ? launch_qk<FAR_F16>(c, g, p, s)
                  : c.act == FAR_BF16 ? launch_qk<FAR_BF16>(c, g, p, s)
                                      : launch_qk<FAR_F32>(c, g, p, s);
  if (e == cudaSuccess && c.back) {
    const int rows = (int)g.grid.x;  // scalar kernels: of either half
    const int rows_q = g.vec ? g.blocks[0] : rows * g.units_q, rows_k = g.vec ? g.blocks[1] : rows * g.units_k;
    e = launch_k(qk_weight_grad_kernel, dim3((unsigned)((c.D + 31) / 32), 2), dim3(32, 32), 0, s,
                 (const float*)p.parts, (int)c.D, rows_q, rows_k, c.heads[0] ? c.dw[0] : nullptr,
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
