// gdr_ssm.cuh -- what the selective scan's kernels share: arguments, the layout
// of channels and states over a block's threads, and the staging of a tile of
// tokens in shared memory.
//
//   h_t = exp(delta_t a) h_{t-1} + (delta_t x_t) b_t      per channel e and state s
//   y_t = (sum_s c_t h_t + d x_t) silu(z_t)
//
// Layout.  A thread owns four neighbouring channels and four neighbouring
// states, 16 recurrences in registers; SL lanes (4, 8 or 16: up to 16, 32 or 64
// states) cover a channel's states.  Per token it reads four deltas, four
// inputs, four b and four c from shared memory, 16-byte loads that broadcast,
// for 16 states; sums over states cross SL lanes, sums over channels cross the
// others.  One channel per thread would need no exchange over states but eight
// 16-byte loads of b and c for the same work.
//
// Time.  The flat token axis is cut into chunks of L tokens.  A sequence's first
// token replaces the state by h0, wherever in a chunk it falls, so chunks need
// not follow the sequences' borders.  A chunk maps the state that enters it to
// P h + h_local with P = exp(a sum(delta)), P = 0 once a sequence started in it.
#pragma once

#include <math_constants.h>

#include "gdr_layer.cuh"

namespace gdr {

struct SsmArgs {
  gdr_ssm_desc d;
  const void *x, *dt, *b, *c, *z, *dy;
  const float *a, *dskip, *dt_bias, *h0, *dht;
  const int64_t *cu;
  void *y, *dx, *ddt, *dz;
  float *ht, *dh0;
  // scratch: states per chunk [chunks, E, SP] and sums of delta [chunks, E]
  float *hloc, *sumd, *gloc;
  // backward: partials of db and dc [ctiles, M, 2 SP]; of dd and ddt_bias [chunks, 2, E] (da's reuse hloc)
  float *part_bc, *part_e;
  int vec;       // backward: 16-byte loads of x, dt, z, dy
  int64_t M, chunks;
  int64_t L;
  int tpg;       // blocks across the channels of a group
  int ctiles;    // blocks across all channels: G * tpg
  int s4;        // state rows may be read and written 16 bytes at a time
  int *status;
};

constexpr int kSsmThreads = 128;
constexpr int kTile = 16;  // tokens staged together

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

constexpr float kLog2e = 1.4426950408889634f;

// delta from the raw dt (bias added): softplus, its large arguments returned as they are.
__device__ __forceinline__ float ssm_delta(float v, int softplus) {
  if (!softplus) return v;
  return v > 20.f ? v : log1pf(expf(v));
}

// Four states from s0 of a row of S (zero past its end).
__device__ __forceinline__ void load_states(const float *row, int s0, int S, int s4, float (&v)[4]) {
  if (s4) {
    if (s0 < S) load4(row + s0, v);
    else v[0] = v[1] = v[2] = v[3] = 0.f;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = s0 + i < S ? row[s0 + i] : 0.f;
}
__device__ __forceinline__ void store_states(float *row, int s0, int S, int s4, const float (&v)[4]) {
  if (s4) {
    if (s0 < S) store4(row + s0, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (s0 + i < S) row[s0 + i] = v[i];
}

// Sums of v[0..3] over the SL lanes of a channel group; lane sl returns that of
// channel sl & 3.  Halves of the values are exchanged, so that three shuffles
// serve four channels; lanes past the first four first fold onto them.
template <int SL>
__device__ __forceinline__ float sum_over_states(float (&v)[4], int sl) {
#pragma unroll
  for (int o = SL / 2; o >= 4; o >>= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
  const bool b1 = sl & 2, b0 = sl & 1;
  float k0 = b1 ? v[2] : v[0], k1 = b1 ? v[3] : v[1];
  const float g0 = b1 ? v[0] : v[2], g1 = b1 ? v[1] : v[3];
  k0 += __shfl_xor_sync(0xffffffffu, g0, 2);
  k1 += __shfl_xor_sync(0xffffffffu, g1, 2);
  const float k = b0 ? k1 : k0, g = b0 ? k0 : k1;
  return k + __shfl_xor_sync(0xffffffffu, g, 1);
}

// Where a block and its threads stand.
template <int SL>
struct Place {
  static constexpr int CPW = 128 / SL;  // channels of a warp
  static constexpr int CB = 4 * CPW;    // of a block
  static constexpr int SP = 4 * SL;     // states, padded
  int lane, warp, sl, cl;
  int64_t chunk, e0, e_end;  // first channel of the block; end of its group
  int64_t g;
  int col;                   // the thread's first channel within the block
  __device__ __forceinline__ explicit Place(const SsmArgs &a) {
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    sl = lane % SL;
    cl = lane / SL;
    chunk = blockIdx.x / (unsigned)a.ctiles;
    const int ct = blockIdx.x % (unsigned)a.ctiles;
    const int64_t eg = a.d.E / a.d.G;
    g = ct / a.tpg;
    e0 = g * eg + (int64_t)(ct % a.tpg) * CB;
    e_end = (g + 1) * eg;
    col = warp * CPW + cl * 4;
  }
};

// For each token of a tile: the sequence that starts there, and the one that
// ends there, or -1.
template <int TT>
struct Borders {
  int first[TT], last[TT];
};
template <int TT>
__device__ __forceinline__ void stage_borders(const SsmArgs &a, int64_t t0, int nt, Borders<TT> &bd) {
  if (threadIdx.x < nt) {
    const int64_t t = t0 + threadIdx.x, n = seq_of_token(a.cu, a.d.N, a.d.T, t);
    const SeqRange r = seq_range(a.cu, n, a.d.T);
    bd.first[threadIdx.x] = t == r.bos ? (int)n : -1;
    bd.last[threadIdx.x] = t + 1 == r.eos ? (int)n : -1;
  }
}

// Runs f(t, column, in range) over a tile of [TT, CB] elements, VEC columns at a time.
template <int TT, int SL, int VEC, typename F>
__device__ __forceinline__ void for_tile(const Place<SL> &p, int nt, F &&f) {
  constexpr int CB = Place<SL>::CB, N = TT * CB / VEC;
#pragma unroll
  for (int i0 = 0; i0 < N; i0 += kSsmThreads) {
    const int i = i0 + threadIdx.x;
    if (N % kSsmThreads != 0 && i >= N) break;
    const int t = i / (CB / VEC), c = (i % (CB / VEC)) * VEC;
    f(t, c, t < nt && p.e0 + c < p.e_end);
  }
}

// b or c of a tile as fp32 [TT][SP], zero past S and past the tokens.
template <typename T, int SL, int TT>
__device__ __forceinline__ void stage_states(const SsmArgs &a, const Place<SL> &p, const void *src, int64_t ld,
                                             int64_t t0, int nt, float *dst) {
  constexpr int SP = Place<SL>::SP;
  const T *row = static_cast<const T *>(src) + p.g * a.d.S;
#pragma unroll
  for (int i0 = 0; i0 < TT * SP; i0 += kSsmThreads) {
    const int i = i0 + threadIdx.x, t = i / SP, s = i % SP;
    dst[i] = t < nt && s < a.d.S ? to_f32(row[(t0 + t) * ld + s]) : 0.f;
  }
}

// The state h0 of sequence n (zero where there is none) for a thread's channels.
template <int SL>
__device__ __forceinline__ void load_h0(const SsmArgs &a, const Place<SL> &p, const float *h0, int64_t n,
                                        f2 (&h)[4][2]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t e = p.e0 + p.col + j;
    float v[4] = {};
    if (h0 && e < p.e_end) load_states(h0 + (n * a.d.E + e) * a.d.S, p.sl * 4, (int)a.d.S, a.s4, v);
    h[j][0] = f2_pack(v[0], v[1]);
    h[j][1] = f2_pack(v[2], v[3]);
  }
}
template <int SL>
__device__ __forceinline__ void store_final(const SsmArgs &a, const Place<SL> &p, float *ht, int64_t n,
                                            const f2 (&h)[4][2]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t e = p.e0 + p.col + j;
    float v[4];
    f2_split(h[j][0], v[0], v[1]);
    f2_split(h[j][1], v[2], v[3]);
    if (e < p.e_end) store_states(ht + (n * a.d.E + e) * a.d.S, p.sl * 4, (int)a.d.S, a.s4, v);
  }
}
// Chunk states [chunks, E, SP]: always whole 16-byte groups.
template <int SL>
__device__ __forceinline__ void load_chunk(const SsmArgs &a, const Place<SL> &p, const float *src, int64_t chunk,
                                           f2 (&h)[4][2]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t e = p.e0 + p.col + j;
    float v[4] = {};
    if (src && e < p.e_end) load4(src + (chunk * a.d.E + e) * Place<SL>::SP + p.sl * 4, v);
    h[j][0] = f2_pack(v[0], v[1]);
    h[j][1] = f2_pack(v[2], v[3]);
  }
}
template <int SL>
__device__ __forceinline__ void store_chunk(const SsmArgs &a, const Place<SL> &p, float *dst, int64_t chunk,
                                            const f2 (&h)[4][2]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t e = p.e0 + p.col + j;
    float v[4];
    f2_split(h[j][0], v[0], v[1]);
    f2_split(h[j][1], v[2], v[3]);
    if (e < p.e_end) store4(dst + (chunk * a.d.E + e) * Place<SL>::SP + p.sl * 4, v);
  }
}

// a[e, s] log2(e) of a thread's channels and states (zero outside: such states stay zero).
template <int SL>
__device__ __forceinline__ void load_a(const SsmArgs &a, const Place<SL> &p, f2 (&A)[4][2]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t e = p.e0 + p.col + j;
    float v[4] = {};
    if (e < p.e_end) load_states(a.a + e * a.d.S, p.sl * 4, (int)a.d.S, a.s4, v);
    A[j][0] = f2_pack(v[0] * kLog2e, v[1] * kLog2e);
    A[j][1] = f2_pack(v[2] * kLog2e, v[3] * kLog2e);
  }
}

// States of sequences without tokens: `to` = `from` (zero where null).
template <int SL>
__device__ __forceinline__ void copy_empty_states(const SsmArgs &a, const Place<SL> &p, const float *from, float *to) {
  if (!to) return;
  for (int64_t n = 0; n < a.d.N; ++n) {
    const SeqRange r = seq_range(a.cu, n, a.d.T);
    if (r.eos > r.bos) continue;
    f2 h[4][2];
    load_h0<SL>(a, p, from, n, h);
    store_final<SL>(a, p, to, n, h);
  }
}

// Host side, shared by the forward and the backward.
int ssm_validate(const gdr_ssm_desc *d, const int64_t *cu);
int ssm_prepare(SsmArgs &a, bool backward, int *sl, bool *vec);

}  // namespace gdr
