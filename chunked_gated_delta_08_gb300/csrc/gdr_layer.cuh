// gdr_layer.cuh -- device helpers of the operators around the recurrence: the
// norm, the short convolution and the selective state space scan.
//
// Rows.  These operators take [tokens, channels] inputs whose rows may lie
// further apart than their length (a slice of a wider projection output): a row
// index is multiplied by a 64-bit leading dimension.  Loads go eight elements at
// a time where every base and leading dimension allows 16-byte accesses
// (the host decides, per call), else one at a time.
#pragma once

#include "gdr_device.cuh"
#include "gdr_internal.h"

namespace gdr {

typedef unsigned long long f2;  // two fp32 values for the packed instructions
__device__ __forceinline__ f2 f2_pack(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_split(f2 v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f2 f2_ex2(f2 v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return f2_pack(ex2(lo), ex2(hi));
}
__device__ __forceinline__ f2 f2_rcp(f2 v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return f2_pack(rcp(lo), rcp(hi));
}
__device__ __forceinline__ f2 f2_both(float x) { return f2_pack(x, x); }

// 1 / (1 + e^-x), to a few units in the last place; 0 and 1 at the ends, NaN for NaN.
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp(1.f + ex2(x * -kLog2e)); }
__device__ __forceinline__ f2 f2_sigmoid(f2 v) {
  return f2_rcp(f2_add(f2_both(1.f), f2_ex2(f2_mul(v, f2_both(-kLog2e)))));
}
// x sigmoid(x) and its derivative s + x s (1 - s).
__device__ __forceinline__ f2 f2_silu(f2 v) { return f2_mul(v, f2_sigmoid(v)); }
__device__ __forceinline__ f2 f2_silu_grad(f2 v) {
  const f2 s = f2_sigmoid(v);
  return f2_fma(f2_mul(v, s), f2_fma(s, f2_both(-1.f), f2_both(1.f)), s);
}

// Eight consecutive elements as fp32; p is 16-byte aligned (32 for fp32 is not needed: two loads).
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void unpack8(const uint4 &u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4 *>(p), v);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&t);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                             pack_bf16(v[6], v[7]));
}

// Four elements; p is aligned to all four.
__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&v)[4]) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&v)[4]) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// VEC elements (8, 4 or 1) at p.
template <int VEC, typename T>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[VEC]) {
  if constexpr (VEC == 8) load8(p, v);
  else if constexpr (VEC == 4) load4(p, v);
  else v[0] = to_f32(p[0]);
}
template <int VEC, typename T>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) store8(p, v);
  else if constexpr (VEC == 4) store4(p, v);
  else p[0] = from_f32<T>(v[0]);
}

// Asynchronous copy of 16 or 8 bytes into shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *smem, const void *global) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(smem);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(global) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of the thread's committed groups are under way.
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// An element of a parameter vector that is fp32 or of the input dtype.
template <typename T>
__device__ __forceinline__ float param(const void *p, bool f32, int64_t i) {
  return f32 ? static_cast<const float *>(p)[i] : to_f32(static_cast<const T *>(p)[i]);
}

// max that keeps NaN: a row or group that holds one must not hide it in its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Whether cu_seqlens is non-decreasing from 0 to T.  Every thread of the block
// calls it and gets the same answer; the first violation seen is recorded.
__device__ __forceinline__ bool seqlens_ok(const int64_t *cu, int64_t N, int64_t T, int *status) {
  if (!cu) return true;
  bool bad = threadIdx.x == 0 && (cu[0] != 0 || cu[N] != T);
  for (int64_t n = threadIdx.x; n < N; n += blockDim.x) bad |= cu[n + 1] < cu[n];
  if (!__syncthreads_or(bad)) return true;
  if (threadIdx.x == 0) raise_status(status, GDR_ERR_SEQLENS);
  return false;
}

__device__ __forceinline__ bool seqlens_ok(const SeqCheck &s) { return seqlens_ok(s.cu, s.N, s.T, s.status); }

// The sequence of flat token t (the last n with first token <= t: empty ones
// are passed over).  Dense layout: sequences of T tokens each.
__device__ __forceinline__ int64_t seq_of_token(const int64_t *cu, int64_t N, int64_t T, int64_t t) {
  if (!cu) return t / T;
  int64_t lo = 0, hi = N;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Column sums of part [rows, cols], rows ld apart, by a block of 32 SETS threads:
// columns 32 block and on, SETS interleaved sets of rows, each added in order,
// then the sets in order.  Columns come in groups of `width`, of which the first
// `keep` go to the output, close together; columns from `split` on to the second.
struct ColSum {
  const float *part;
  int64_t rows, ld, cols, width, keep;
  float *out;
  int64_t split;
  float *out2;
};
template <int SETS>
__device__ __forceinline__ void col_sum_block(const ColSum &q, int64_t block, float (&sm)[SETS][33]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t c = block * 32 + lane;
  float acc = 0.f;
  if (c < q.cols) {
#pragma unroll 4
    for (int64_t r = w; r < q.rows; r += SETS) acc += q.part[r * q.ld + c];
  }
  sm[w][lane] = acc;
  __syncthreads();
  if (w == 0 && c < q.cols && c % q.width < q.keep) {
#pragma unroll
    for (int i = 1; i < SETS; ++i) acc += sm[i][lane];
    float *to = q.out;
    if (c >= q.split) {
      c -= q.split;
      to = q.out2;
    }
    if (to) to[c / q.width * q.keep + c % q.width] = acc;
  }
}

}  // namespace gdr
