// gdr_norm.cu -- root-mean-square norm with the residual's addition, an 8-bit
// output with scales, and the backward.
//
//   s = round(x + r);  y = s rho w,  rho = 1 / sqrt(mean(s^2) + eps)
//   backward, with p = w dy:  dL/ds = ds + rho (p - s rho^2 mean(p s)),  dw = sum over rows of dy s rho
//
// One pass over memory: a row is read once, held in fp32 registers while its
// sum is formed, and written once.  The bound is HBM: 16384 x 4096 with a bf16
// residual to e4m3 take 84 us, 84 % of the copy rate; the backward with an fp32
// stream 187 us, 86 %.
#include <algorithm>

#include "gdr_layer.cuh"

namespace gdr {
namespace {

constexpr float kFp8Max = 448.f;

struct NormArgs {
  gdr_norm_desc d;
  const void *x, *res, *weight, *ds;  // backward: x is dy, res is s
  void *y, *s;                        // backward: dx, dres
  float *scale;                       // backward: dweight partials
  int64_t ngroups;
};

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {  // a in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

template <int VEC>
__device__ __forceinline__ void store_fp8(uint8_t *p, const float (&v)[VEC], float inv) {
  if constexpr (VEC == 8) {
    const uint32_t lo = pack_e4m3(v[0] * inv, v[1] * inv) | (pack_e4m3(v[2] * inv, v[3] * inv) << 16);
    const uint32_t hi = pack_e4m3(v[4] * inv, v[5] * inv) | (pack_e4m3(v[6] * inv, v[7] * inv) << 16);
    *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint32_t *>(p) =
        pack_e4m3(v[0] * inv, v[1] * inv) | (pack_e4m3(v[2] * inv, v[3] * inv) << 16);
  } else {
    p[0] = (uint8_t)(pack_e4m3(v[0] * inv, 0.f) & 0xffu);
  }
}

// The multiplier 448 / amax passes fp32's range below 1.32e-36, and an infinite one
// makes NaN of the zeros beside such values.  Smaller groups take the scale of this
// least amax, so that multiplier and scale agree: their bytes are below 448.
constexpr float kLeastAmax = 0x1.c00002p-120f;
static_assert(kFp8Max / kLeastAmax <= 3.402823466e38f, "448 / kLeastAmax is an fp32 number");
__device__ __forceinline__ float group_inv(float amax) {
  return amax == 0.f ? 1.f : kFp8Max / max_nan(amax, kLeastAmax);
}
__device__ __forceinline__ float group_scale(float amax) {
  return amax == 0.f ? 1.f : max_nan(amax, kLeastAmax) / kFp8Max;
}

// Sums (or maxima) over the NT threads of a row.  NT == 32: a warp, no barrier.
template <int NT, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, u) : v + u;
  }
  if constexpr (NT > 32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();  // the previous reduction's readers are done
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = 0.f;  // below every absolute value
#pragma unroll
    for (int i = 0; i < NT / 128; ++i) {  // four warps in each 16-byte load
      const float4 q = reinterpret_cast<const float4 *>(red)[i];
      v = MAX ? max_nan(max_nan(v, max_nan(q.x, q.y)), max_nan(q.z, q.w)) : v + ((q.x + q.y) + (q.z + q.w));
    }
  }
  return v;
}

// Column of this thread's k-th vector.  VEC 8 (all bf16) or 4 (fp32 among the
// types): 16 bytes of the widest, vectors of neighbouring threads follow one
// another.  VEC 1: a warp owns NV * 32 columns in a run,
// so that a scale group of 128 columns is four steps of one warp.
template <int NT, int VEC, int NV>
__device__ __forceinline__ int64_t col_of(int tid, int k) {
  if constexpr (VEC > 1) return ((int64_t)k * NT + tid) * VEC;
  else return (int64_t)(tid >> 5) * (NV * 32) + k * 32 + (tid & 31);
}

// One row per NT threads; blocks of 256 threads take 256 / NT rows when NT is a warp.
template <typename T, typename R, int NT, int VEC, int NV, int QUANT, bool RES>
__global__ void __launch_bounds__(NT == 32 ? 256 : NT) norm_fwd_kernel(NormArgs a) {
  __shared__ __align__(16) float red[32];
  const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t m = NT == 32 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (m >= a.d.M) return;  // whole warps, and only where no barrier follows (NT == 32)
  const int64_t E = a.d.E;
  const T *x = static_cast<const T *>(a.x) + m * a.d.ld_x;
  const R *res = static_cast<const R *>(a.res) + (RES ? m * a.d.ld_res : 0);
  const bool wf32 = a.d.weight_dtype == GDR_F32;
  float v[NV][VEC];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int64_t c = col_of<NT, VEC, NV>(tid, k);
    if (c < E) {
      load_vec<VEC>(x + c, v[k]);
      if constexpr (RES) {
        float r[VEC];
        load_vec<VEC>(res + c, r);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[k][i] = to_f32(from_f32<R>(v[k][i] + r[i]));  // s as stored
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[k][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) ss = fmaf(v[k][i], v[k][i], ss);
  }
  if constexpr (RES) {
    R *s = static_cast<R *>(a.s) + m * E;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = col_of<NT, VEC, NV>(tid, k);
      if (c < E) store_vec<VEC>(s + c, v[k]);
    }
  }
  float w[NV][VEC];  // the weights' loads overlap the sum's exchange
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int64_t c = col_of<NT, VEC, NV>(tid, k);
    if (c < E) {
      if (wf32) load_vec<VEC>(static_cast<const float *>(a.weight) + c, w[k]);
      else load_vec<VEC>(static_cast<const T *>(a.weight) + c, w[k]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[k][i] = 0.f;
    }
  }
  const float rho = rsqrtf(row_reduce<NT, false>(ss, red) / (float)E + a.d.eps);
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      v[k][i] = v[k][i] * rho * w[k][i];
      if (QUANT == GDR_QUANT_ROW) amax = max_nan(amax, col_of<NT, VEC, NV>(tid, k) < E ? fabsf(v[k][i]) : 0.f);
    }
  if constexpr (QUANT == GDR_QUANT_NONE) {
    T *y = static_cast<T *>(a.y) + m * E;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = col_of<NT, VEC, NV>(tid, k);
      if (c < E) store_vec<VEC>(y + c, v[k]);
    }
  } else if constexpr (QUANT == GDR_QUANT_ROW) {
    amax = row_reduce<NT, true>(amax, red);
    const float inv = group_inv(amax);
    uint8_t *y = static_cast<uint8_t *>(a.y) + m * E;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = col_of<NT, VEC, NV>(tid, k);
      if (c < E) store_fp8<VEC>(y + c, v[k], inv);
    }
    if (tid == 0) a.scale[m] = group_scale(amax);
  } else {
    uint8_t *y = static_cast<uint8_t *>(a.y) + m * E;
    float *scale = a.scale + m * a.ngroups;
    if constexpr (VEC > 1) {  // a group is 16 or 32 neighbouring lanes
      constexpr int kLanes = GDR_QUANT_GROUP_SIZE / VEC;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int64_t c = col_of<NT, VEC, NV>(tid, k);
        float g = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) g = max_nan(g, c < E ? fabsf(v[k][i]) : 0.f);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) g = max_nan(g, __shfl_xor_sync(0xffffffffu, g, o));
        if (c < E) {
          store_fp8<VEC>(y + c, v[k], group_inv(g));
          if ((tid & (kLanes - 1)) == 0) scale[c / GDR_QUANT_GROUP_SIZE] = group_scale(g);
        }
      }
    } else {  // a group is four steps of the warp
      static_assert(NV % 4 == 0, "a warp's run of columns is whole groups");
#pragma unroll
      for (int k = 0; k < NV; k += 4) {
        float g = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          g = max_nan(g, col_of<NT, VEC, NV>(tid, k + q) < E ? fabsf(v[k + q][0]) : 0.f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) g = max_nan(g, __shfl_xor_sync(0xffffffffu, g, o));
        const float inv = group_inv(g);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t c = col_of<NT, VEC, NV>(tid, k + q);
          if (c < E) store_fp8<VEC>(y + c, v[k + q], inv);
        }
        const int64_t c0 = col_of<NT, VEC, NV>(tid, k);
        if ((tid & 31) == 0 && c0 < E) scale[c0 / GDR_QUANT_GROUP_SIZE] = group_scale(g);
      }
    }
  }
}

// Rows too long for registers: the row is read again (from L2) for the output.
// One block of 256 threads per row; scale groups are taken a warp at a time.
template <typename T, typename R, bool RES>
__global__ void __launch_bounds__(256) norm_fwd_long_kernel(NormArgs a) {
  __shared__ __align__(16) float red[32];
  const int64_t m = blockIdx.x, E = a.d.E;
  const T *x = static_cast<const T *>(a.x) + m * a.d.ld_x;
  const R *res = static_cast<const R *>(a.res) + (RES ? m * a.d.ld_res : 0);
  R *s = static_cast<R *>(a.s) + (RES ? m * E : 0);
  const bool wf32 = a.d.weight_dtype == GDR_F32;
  auto value = [&](int64_t c) {
    float v = to_f32(x[c]);
    if constexpr (RES) v = to_f32(from_f32<R>(v + to_f32(res[c])));
    return v;
  };
  float ss = 0.f;
  for (int64_t c = threadIdx.x; c < E; c += 256) {
    const float v = value(c);
    if constexpr (RES) s[c] = from_f32<R>(v);
    ss = fmaf(v, v, ss);
  }
  const float rho = rsqrtf(row_reduce<256, false>(ss, red) / (float)E + a.d.eps);
  auto out = [&](int64_t c) { return value(c) * rho * param<T>(a.weight, wf32, c); };
  if (a.d.quant == GDR_QUANT_NONE) {
    T *y = static_cast<T *>(a.y) + m * E;
    for (int64_t c = threadIdx.x; c < E; c += 256) y[c] = from_f32<T>(out(c));
    return;
  }
  uint8_t *y = static_cast<uint8_t *>(a.y) + m * E;
  if (a.d.quant == GDR_QUANT_ROW) {
    float amax = 0.f;
    for (int64_t c = threadIdx.x; c < E; c += 256) amax = max_nan(amax, fabsf(out(c)));
    amax = row_reduce<256, true>(amax, red);
    for (int64_t c = threadIdx.x; c < E; c += 256) {
      const float v[1] = {out(c)};
      store_fp8<1>(y + c, v, group_inv(amax));
    }
    if (threadIdx.x == 0) a.scale[m] = group_scale(amax);
    return;
  }
  const int lane = threadIdx.x & 31;
  for (int64_t g = threadIdx.x >> 5; g < a.ngroups; g += 8) {
    float v[4], amax = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t c = g * GDR_QUANT_GROUP_SIZE + q * 32 + lane;
      v[q] = c < E ? out(c) : 0.f;
      amax = max_nan(amax, fabsf(v[q]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t c = g * GDR_QUANT_GROUP_SIZE + q * 32 + lane;
      const float u[1] = {v[q]};
      if (c < E) store_fp8<1>(y + c, u, group_inv(amax));
    }
    if (lane == 0) a.scale[m * a.ngroups + g] = group_scale(amax);
  }
}

// Backward.  A block takes rows b, b + grid, ...  Each thread owns two runs of
// four columns, 4 NT apart so that a warp's accesses are whole lines in either
// type, and copies its own part of the next row into its own shared memory while
// it works on this one: asynchronous copies that cost no registers and, as no
// other thread reads them, no barrier.  Held in registers instead, the next row
// took the kernel from two blocks of 512 threads per multiprocessor to one, or
// spilled.  The weight gradient of the thread's columns stays in registers over
// all its rows and ends in row b of the partials, which col_sum_kernel adds in
// order.
// A thread's part of a row in shared memory.
template <typename T, int NT>
struct Slot {
  T v[2][NT][4];
  __device__ __forceinline__ void fetch(const T *row, int tid, const bool (&in)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (in[i]) copy_async<4 * sizeof(T)>(v[i][tid], row + (i * NT + tid) * 4);
  }
  __device__ __forceinline__ void get(int i, int tid, float (&o)[4]) const { load4(v[i][tid], o); }
};
template <typename T, typename R, int NT>
struct __align__(16) BwdShared {
  Slot<float, NT> w;
  struct Row {
    Slot<R, NT> s, ds;
    Slot<T, NT> dy;
  } row[2];
  float2 red[2][32];
};

template <typename T, typename R, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) norm_bwd_kernel(NormArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdShared<T, R, NT> &sm = *reinterpret_cast<BwdShared<T, R, NT> *>(smem_raw);
  const int tid = threadIdx.x;
  const int64_t E = a.d.E;
  const bool in[2] = {tid * 4 < E, (NT + tid) * 4 < E};
  float dw[2][4] = {};
  auto fetch = [&](int64_t m, int buf) {
    auto &row = sm.row[buf];
    row.dy.fetch(static_cast<const T *>(a.x) + m * a.d.ld_x, tid, in);
    row.s.fetch(static_cast<const R *>(a.res) + m * a.d.ld_res, tid, in);
    if (a.ds) row.ds.fetch(static_cast<const R *>(a.ds) + m * a.d.ld_ds, tid, in);
  };
  if (blockIdx.x < a.d.M) fetch(blockIdx.x, 0);
  copy_commit();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float w[4] = {};
    const int c = (i * NT + tid) * 4;
    if (in[i]) {
      if (a.d.weight_dtype == GDR_F32) load4(static_cast<const float *>(a.weight) + c, w);
      else load4(static_cast<const T *>(a.weight) + c, w);
    }
    store4(sm.w.v[i][tid], w);
  }
  int buf = 0;
  for (int64_t m = blockIdx.x; m < a.d.M; m += gridDim.x) {
    if (m + gridDim.x < a.d.M) fetch(m + gridDim.x, buf ^ 1);
    copy_commit();
    copy_wait<1>();  // this row is here, the next one on its way
    const auto &row = sm.row[buf];
    float ss = 0.f, ps = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!in[i]) continue;
      float v[4], g[4], w[4];
      row.s.get(i, tid, v);
      row.dy.get(i, tid, g);
      sm.w.get(i, tid, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ss = fmaf(v[k], v[k], ss);
        ps = fmaf(v[k] * w[k], g[k], ps);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      ps += __shfl_xor_sync(0xffffffffu, ps, o);
    }
    if constexpr (NT > 32) {  // two buffers: one barrier a row
      constexpr int NW = NT / 32;
      if ((tid & 31) == 0) sm.red[buf][tid >> 5] = make_float2(ss, ps);
      __syncthreads();
      const float2 q = sm.red[buf][tid & (NW - 1)];
      ss = q.x;
      ps = q.y;
#pragma unroll
      for (int o = NW / 2; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        ps += __shfl_xor_sync(0xffffffffu, ps, o);
      }
    }
    const float rho = rsqrtf(ss / (float)E + a.d.eps);
    const float mix = rho * rho * (ps / (float)E);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!in[i]) continue;
      float v[4], g[4], w[4], o[4] = {};
      row.s.get(i, tid, v);
      row.dy.get(i, tid, g);
      sm.w.get(i, tid, w);
      if (a.ds) row.ds.get(i, tid, o);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dw[i][k] = fmaf(g[k] * rho, v[k], dw[i][k]);
        o[k] = fmaf(rho, fmaf(w[k], g[k], -v[k] * mix), o[k]);
      }
      const int64_t at = m * E + (i * NT + tid) * 4;
      if (a.y) store4(static_cast<T *>(a.y) + at, o);
      if (a.s) store4(static_cast<R *>(a.s) + at, o);
    }
    buf ^= 1;
  }
  if (a.scale) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (in[i]) store4(a.scale + (int64_t)blockIdx.x * E + (i * NT + tid) * 4, dw[i]);
  }
}

// The same for rows that allow no accesses of four columns: NV single columns of a thread.
template <typename T, typename R, int NT, int NV>
__global__ void __launch_bounds__(NT, 1024 / NT) norm_bwd_scalar_kernel(NormArgs a) {
  __shared__ __align__(16) float red[2][32];
  const int tid = threadIdx.x;
  const int64_t E = a.d.E;
  float w[NV], dw[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int64_t c = k * NT + tid;
    dw[k] = 0.f;
    w[k] = c < E ? param<T>(a.weight, a.d.weight_dtype == GDR_F32, c) : 0.f;
  }
  for (int64_t m = blockIdx.x; m < a.d.M; m += gridDim.x) {
    const T *dy = static_cast<const T *>(a.x) + m * a.d.ld_x;
    const R *s = static_cast<const R *>(a.res) + m * a.d.ld_res;
    const R *ds = static_cast<const R *>(a.ds) + (a.ds ? m * a.d.ld_ds : 0);
    float v[NV], g[NV], up[NV];
    float ss = 0.f, ps = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = k * NT + tid;
      v[k] = c < E ? to_f32(s[c]) : 0.f;
      g[k] = c < E ? to_f32(dy[c]) : 0.f;
      up[k] = c < E && a.ds ? to_f32(ds[c]) : 0.f;
      ss = fmaf(v[k], v[k], ss);
      ps = fmaf(v[k] * w[k], g[k], ps);
    }
    ss = row_reduce<NT, false>(ss, red[0]);
    ps = row_reduce<NT, false>(ps, red[1]);
    const float rho = rsqrtf(ss / (float)E + a.d.eps), mix = rho * rho * (ps / (float)E);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = k * NT + tid;
      dw[k] = fmaf(g[k] * rho, v[k], dw[k]);
      const float o = fmaf(rho, fmaf(w[k], g[k], -v[k] * mix), up[k]);
      if (c < E && a.y) static_cast<T *>(a.y)[m * E + c] = from_f32<T>(o);
      if (c < E && a.s) static_cast<R *>(a.s)[m * E + c] = from_f32<R>(o);
    }
  }
  if (a.scale) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = k * NT + tid;
      if (c < E) a.scale[(int64_t)blockIdx.x * E + c] = dw[k];
    }
  }
}

// Backward for rows too long for registers: the weight gradient's partials are
// kept in this block's own row of global scratch.
template <typename T, typename R>
__global__ void __launch_bounds__(256) norm_bwd_long_kernel(NormArgs a) {
  __shared__ __align__(16) float red[32];
  const int64_t E = a.d.E;
  const bool wf32 = a.d.weight_dtype == GDR_F32;
  float *dw = a.scale ? a.scale + (int64_t)blockIdx.x * E : nullptr;
  if (dw)
    for (int64_t c = threadIdx.x; c < E; c += 256) dw[c] = 0.f;
  for (int64_t m = blockIdx.x; m < a.d.M; m += gridDim.x) {
    const T *dy = static_cast<const T *>(a.x) + m * a.d.ld_x;
    const R *s = static_cast<const R *>(a.res) + m * a.d.ld_res;
    const R *ds = static_cast<const R *>(a.ds) + (a.ds ? m * a.d.ld_ds : 0);
    float ss = 0.f, ps = 0.f;
    for (int64_t c = threadIdx.x; c < E; c += 256) {
      const float v = to_f32(s[c]);
      ss = fmaf(v, v, ss);
      ps = fmaf(v * param<T>(a.weight, wf32, c), to_f32(dy[c]), ps);
    }
    ss = row_reduce<256, false>(ss, red);
    ps = row_reduce<256, false>(ps, red);
    const float rho = rsqrtf(ss / (float)E + a.d.eps), mix = rho * rho * (ps / (float)E);
    for (int64_t c = threadIdx.x; c < E; c += 256) {
      const float v = to_f32(s[c]), g = to_f32(dy[c]);
      if (dw) dw[c] = fmaf(g * rho, v, dw[c]);
      const float o = fmaf(rho, fmaf(param<T>(a.weight, wf32, c), g, -v * mix), a.ds ? to_f32(ds[c]) : 0.f);
      if (a.y) static_cast<T *>(a.y)[m * E + c] = from_f32<T>(o);
      if (a.s) static_cast<R *>(a.s)[m * E + c] = from_f32<R>(o);
    }
  }
}

template <typename T, typename R, int NT, int VEC, int NV, bool RES>
void launch_fwd_q(const NormArgs &a, cudaStream_t st) {
  const unsigned grid = (unsigned)(NT == 32 ? cdiv(a.d.M, 8) : a.d.M), block = NT == 32 ? 256 : NT;
  if (a.d.quant == GDR_QUANT_NONE) norm_fwd_kernel<T, R, NT, VEC, NV, 0, RES><<<grid, block, 0, st>>>(a);
  else if (a.d.quant == GDR_QUANT_ROW) norm_fwd_kernel<T, R, NT, VEC, NV, 1, RES><<<grid, block, 0, st>>>(a);
  else norm_fwd_kernel<T, R, NT, VEC, NV, 2, RES><<<grid, block, 0, st>>>(a);
}

template <typename T, typename R, bool RES>
int launch_fwd(const NormArgs &a, cudaStream_t st) {
  const int64_t E = a.d.E;
  const bool vec = E % 8 == 0 && a.d.ld_x % 8 == 0 && (!RES || a.d.ld_res % 8 == 0) && is_aligned16(a.x) &&
                   is_aligned16(a.res) && is_aligned16(a.weight) && is_aligned16(a.y) && is_aligned16(a.s);
  if (vec) {
    constexpr int V = sizeof(T) == 4 || (RES && sizeof(R) == 4) ? 4 : 8, K = 8 / V;
    if (E <= 512) launch_fwd_q<T, R, 32, V, 2 * K, RES>(a, st);
    else if (E <= 1024) launch_fwd_q<T, R, 128, V, K, RES>(a, st);
    else if (E <= 2048) launch_fwd_q<T, R, 256, V, K, RES>(a, st);
    else if (E <= 4096) launch_fwd_q<T, R, 512, V, K, RES>(a, st);
    else if (E <= 8192) launch_fwd_q<T, R, 512, V, 2 * K, RES>(a, st);
    else if (E <= 16384) launch_fwd_q<T, R, 1024, V, 2 * K, RES>(a, st);
    else norm_fwd_long_kernel<T, R, RES><<<(unsigned)a.d.M, 256, 0, st>>>(a);
  } else {
    if (E <= 256) launch_fwd_q<T, R, 32, 1, 8, RES>(a, st);
    else if (E <= 2048) launch_fwd_q<T, R, 256, 1, 8, RES>(a, st);
    else if (E <= 4096) launch_fwd_q<T, R, 256, 1, 16, RES>(a, st);
    else norm_fwd_long_kernel<T, R, RES><<<(unsigned)a.d.M, 256, 0, st>>>(a);
  }
  return launched("norm_fwd_kernel");
}

template <int SETS>
__global__ void __launch_bounds__(32 * SETS) col_sum_kernel(ColSum q) {
  __shared__ float sm[SETS][33];
  col_sum_block<SETS>(q, blockIdx.x, sm);
}

// Many columns fill the GPU with small blocks; few need their rows apart (64 rows
// of 32768 columns: 6 us against 12, 304 of 4096: 11 against 6).
int launch_col_sum(const ColSum &q, cudaStream_t stream) {
  const unsigned grid = (unsigned)cdiv(q.cols, 32);
  if (grid >= 4 * kSMs) col_sum_kernel<8><<<grid, 256, 0, stream>>>(q);
  else col_sum_kernel<32><<<grid, 1024, 0, stream>>>(q);
  return launched("col_sum_kernel");
}

template <typename T, typename R>
int launch_bwd(NormArgs a, float *dweight, cudaStream_t st) {
  const int64_t E = a.d.E;
  const bool vec = E % 4 == 0 && a.d.ld_x % 4 == 0 && a.d.ld_res % 4 == 0 && (!a.ds || a.d.ld_ds % 4 == 0) &&
                   is_aligned16(a.x) && is_aligned16(a.res) && is_aligned16(a.ds) && is_aligned16(a.weight) && is_aligned16(a.y) &&
                   is_aligned16(a.s);
  // blocks, and rows of partials: 1024 threads of them on each multiprocessor, 512 where a block is one warp
  const int64_t most = kSMs * (E <= 256 ? 16 : E <= 1024 ? 8 : E <= 2048 ? 4 : E <= 4096 ? 2 : vec && E <= 8192 ? 1 : 4);
  const unsigned grid = (unsigned)std::min<int64_t>(a.d.M, most);
  char *base = nullptr;
  int rc;
  if (dweight) {
    if ((rc = scratch_begin(sizeof(float) * (size_t)(grid * E), st, "norm backward scratch", &base)) != GDR_OK)
      return rc;
    a.scale = (float *)base;
  }
  if (vec && E <= 8192) {
    auto go = [&](auto nt) {
      constexpr int NT = decltype(nt)::value, smem = sizeof(BwdShared<T, R, NT>);
      const cudaError_t e =
          cudaFuncSetAttribute(norm_bwd_kernel<T, R, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e == cudaSuccess) norm_bwd_kernel<T, R, NT><<<grid, NT, smem, st>>>(a);
    };
    if (E <= 256) go(std::integral_constant<int, 32>{});
    else if (E <= 1024) go(std::integral_constant<int, 128>{});
    else if (E <= 2048) go(std::integral_constant<int, 256>{});
    else if (E <= 4096) go(std::integral_constant<int, 512>{});
    else go(std::integral_constant<int, 1024>{});
  } else {
    if (E <= 256) norm_bwd_scalar_kernel<T, R, 32, 8><<<grid, 32, 0, st>>>(a);
    else if (E <= 2048) norm_bwd_scalar_kernel<T, R, 256, 8><<<grid, 256, 0, st>>>(a);
    else if (E <= 4096) norm_bwd_scalar_kernel<T, R, 512, 8><<<grid, 512, 0, st>>>(a);
    else norm_bwd_long_kernel<T, R><<<grid, 256, 0, st>>>(a);
  }
  rc = launched("norm_bwd_kernel");
  if (dweight) {
    if (rc == GDR_OK) rc = launch_col_sum(ColSum{(const float *)base, grid, E, E, E, E, dweight, E, nullptr}, st);
    rc = scratch_end(base, st, "norm backward scratch", rc);
  }
  return rc;
}

int validate(const gdr_norm_desc *d) {
  if (!d) return set_error(GDR_ERR_NULLPTR, "desc is NULL");
  if (d->dtype != GDR_F32 && d->dtype != GDR_BF16) return set_error(GDR_ERR_DTYPE, "dtype must be GDR_F32 or GDR_BF16");
  if (d->res_dtype != d->dtype && d->res_dtype != GDR_F32)
    return set_error(GDR_ERR_DTYPE, "the residual must be of the input dtype or fp32");
  if (d->weight_dtype != d->dtype && d->weight_dtype != GDR_F32)
    return set_error(GDR_ERR_DTYPE, "weight must be of the input dtype or fp32");
  if (d->quant < GDR_QUANT_NONE || d->quant > GDR_QUANT_GROUP) return set_error(GDR_ERR_DTYPE, "unknown quant");
  if (d->flags) return set_error(GDR_ERR_DTYPE, "unknown bits in flags");
  if (d->M < 0 || d->M > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "M must be in [0, 2^31)");
  if (d->E < 1 || d->E > (1 << 24)) return set_error(GDR_ERR_SHAPE, "E must be in [1, 2^24]");
  if (d->ld_x < d->E || d->ld_res < d->E || d->ld_ds < d->E)
    return set_error(GDR_ERR_SHAPE, "leading dimensions must be at least E");
  if (!(d->eps >= 0.f)) return set_error(GDR_ERR_SHAPE, "eps must be >= 0");
  return GDR_OK;
}

}  // namespace

}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_norm_fwd(const gdr_norm_desc *desc, const void *x, const void *residual, const void *weight, void *y,
                 float *scale, void *s, void *stream) {
  int rc = validate(desc);
  if (rc != GDR_OK) return rc;
  if (desc->M == 0) return GDR_OK;
  if (!x || !weight || !y) return set_error(GDR_ERR_NULLPTR, "x, weight and y must be non-NULL");
  if (residual && !s) return set_error(GDR_ERR_NULLPTR, "with a residual, s must be non-NULL");
  if (desc->quant != GDR_QUANT_NONE && !scale) return set_error(GDR_ERR_NULLPTR, "an 8-bit output needs scale");
  NormArgs a{};
  a.d = *desc;
  a.x = x; a.res = residual; a.weight = weight; a.y = y; a.s = residual ? s : nullptr; a.scale = scale;
  a.ngroups = cdiv(desc->E, GDR_QUANT_GROUP_SIZE);
  cudaStream_t st = (cudaStream_t)stream;
  if (desc->dtype == GDR_F32)
    return residual ? launch_fwd<float, float, true>(a, st) : launch_fwd<float, float, false>(a, st);
  if (!residual) return launch_fwd<__nv_bfloat16, float, false>(a, st);
  if (desc->res_dtype == GDR_F32) return launch_fwd<__nv_bfloat16, float, true>(a, st);
  return launch_fwd<__nv_bfloat16, __nv_bfloat16, true>(a, st);
}

int gdr_norm_bwd(const gdr_norm_desc *desc, const void *dy, const void *s, const void *ds, const void *weight,
                 void *dx, void *dres, float *dweight, void *stream) {
  int rc = validate(desc);
  if (rc != GDR_OK) return rc;
  if (desc->quant != GDR_QUANT_NONE) return set_error(GDR_ERR_UNSUPPORTED, "the backward has no 8-bit form");
  cudaStream_t st = (cudaStream_t)stream;
  if (desc->M == 0) {
    if (!dweight) return GDR_OK;
    const cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)desc->E, st);
    return e == cudaSuccess ? GDR_OK : cuda_error(e, "clearing dweight");
  }
  if (!dy || !s || !weight) return set_error(GDR_ERR_NULLPTR, "dy, s and weight must be non-NULL");
  NormArgs a{};
  a.d = *desc;
  a.x = dy; a.res = s; a.ds = ds; a.weight = weight; a.y = dx; a.s = dres;
  if (desc->dtype == GDR_F32) return launch_bwd<float, float>(a, dweight, st);
  if (desc->res_dtype == GDR_F32) return launch_bwd<__nv_bfloat16, float>(a, dweight, st);
  return launch_bwd<__nv_bfloat16, __nv_bfloat16>(a, dweight, st);
}

}  // extern "C"
