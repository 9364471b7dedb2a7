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
// 16-byte loads of b and c for the same work.  The packed fp32 instructions take
// channels two by two: delta, x and the gradients come from shared memory as
// pairs, and b and c are staged twice over, (b, b), so that no pair is ever
// assembled in the loop.
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

// delta from the raw dt (bias added): softplus(v) = max(v, 0) + log1p(u), u = e^-|v|,
// with log1p(u) = 2 atanh(r), r = u / (2 + u) <= 1/3, by its series in r^2.  Nine
// terms leave 1e-9 of the value; log(1 + u) would lose a small u against the 1, and
// small deltas are the ones a state remembers longest.  `slope`: ddelta/dv.
__device__ __forceinline__ float ssm_delta(float v, int softplus, float *slope = nullptr) {
  if (!softplus) {
    if (slope) *slope = 1.f;
    return v;
  }
  const float u = ex2(-fabsf(v) * kLog2e);
  const float r = __fdividef(u, 2.f + u), q = r * r;
  float w = 1.f / 17.f;
  w = fmaf(w, q, 1.f / 15.f);
  w = fmaf(w, q, 1.f / 13.f);
  w = fmaf(w, q, 1.f / 11.f);
  w = fmaf(w, q, 1.f / 9.f);
  w = fmaf(w, q, 1.f / 7.f);
  w = fmaf(w, q, 1.f / 5.f);
  w = fmaf(w, q, 1.f / 3.f);
  w = fmaf(w, q, 1.f);
  if (slope) {
    const float k = __fdividef(1.f, 1.f + u);
    *slope = v >= 0.f ? k : u * k;
  }
  return fmaf(r + r, w, fmaxf(v, 0.f));  // a NaN comes through u
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
// True in threads whose token is a border.
template <int TT>
__device__ __forceinline__ bool stage_borders(const SsmArgs &a, int64_t t0, int nt, Borders<TT> &bd) {
  bool border = false;
  if (threadIdx.x < nt) {
    const int64_t t = t0 + threadIdx.x, n = seq_of_token(a.cu, a.d.N, a.d.T, t);
    const SeqRange r = seq_range(a.cu, n, a.d.T);
    bd.first[threadIdx.x] = t == r.bos ? (int)n : -1;
    bd.last[threadIdx.x] = t + 1 == r.eos ? (int)n : -1;
    border = t == r.bos || t + 1 == r.eos;
  }
  return border;
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

// b or c of a tile as fp32 [TT][SP], each twice, zero past S and past the tokens.
template <typename T, int SL, int TT>
__device__ __forceinline__ void stage_states(const SsmArgs &a, const Place<SL> &p, const void *src, int64_t ld,
                                             int64_t t0, int nt, float2 *dst) {
  constexpr int SP = Place<SL>::SP;
  const T *row = static_cast<const T *>(src) + p.g * a.d.S;
#pragma unroll
  for (int i0 = 0; i0 < TT * SP; i0 += kSsmThreads) {
    const int i = i0 + threadIdx.x, t = i / SP, s = i % SP;
    const float v = t < nt && s < a.d.S ? to_f32(row[(t0 + t) * ld + s]) : 0.f;
    dst[i] = make_float2(v, v);
  }
}

// A thread's 16 states: pair i holds channels 2 i and 2 i + 1, for each of the
// four states.
typedef f2 States[2][4];

template <int SL, typename F>
__device__ __forceinline__ void read_states(const Place<SL> &p, States &h, F &&row) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float v[4] = {}, w[4] = {};
    const int64_t e = p.e0 + p.col + 2 * i;
    if (e < p.e_end) row(e, v);
    if (e + 1 < p.e_end) row(e + 1, w);
#pragma unroll
    for (int s = 0; s < 4; ++s) h[i][s] = f2_pack(v[s], w[s]);
  }
}
template <int SL, typename F>
__device__ __forceinline__ void write_states(const Place<SL> &p, const States &h, F &&row) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float v[4], w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) f2_split(h[i][s], v[s], w[s]);
    const int64_t e = p.e0 + p.col + 2 * i;
    if (e < p.e_end) row(e, v);
    if (e + 1 < p.e_end) row(e + 1, w);
  }
}
// The state h0 of sequence n (zero where there is none).
template <int SL>
__device__ __forceinline__ void load_h0(const SsmArgs &a, const Place<SL> &p, const float *h0, int64_t n, States &h) {
  read_states(p, h, [&](int64_t e, float (&v)[4]) {
    if (h0) load_states(h0 + (n * a.d.E + e) * a.d.S, p.sl * 4, (int)a.d.S, a.s4, v);
  });
}
template <int SL>
__device__ __forceinline__ void store_final(const SsmArgs &a, const Place<SL> &p, float *ht, int64_t n,
                                            const States &h) {
  write_states(p, h, [&](int64_t e, const float (&v)[4]) {
    store_states(ht + (n * a.d.E + e) * a.d.S, p.sl * 4, (int)a.d.S, a.s4, v);
  });
}
// Chunk states [chunks, E, SP]: always whole 16-byte groups.
template <int SL>
__device__ __forceinline__ void load_chunk(const SsmArgs &a, const Place<SL> &p, const float *src, int64_t chunk,
                                           States &h) {
  read_states(p, h, [&](int64_t e, float (&v)[4]) {
    if (src) load4(src + (chunk * a.d.E + e) * Place<SL>::SP + p.sl * 4, v);
  });
}
template <int SL>
__device__ __forceinline__ void store_chunk(const SsmArgs &a, const Place<SL> &p, float *dst, int64_t chunk,
                                            const States &h) {
  write_states(p, h, [&](int64_t e, const float (&v)[4]) {
    store4(dst + (chunk * a.d.E + e) * Place<SL>::SP + p.sl * 4, v);
  });
}

// a[e, s] log2(e) of a thread's channels and states (zero outside: such states stay zero).
template <int SL>
__device__ __forceinline__ void load_a(const SsmArgs &a, const Place<SL> &p, States &A) {
  read_states(p, A, [&](int64_t e, float (&v)[4]) {
    load_states(a.a + e * a.d.S, p.sl * 4, (int)a.d.S, a.s4, v);
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] *= kLog2e;
  });
}

// Four values of a staged row: the thread's channels, as two pairs.
struct Pairs {
  f2 v[2];
  __device__ __forceinline__ explicit Pairs(const float *row) {
    const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(row);
    v[0] = u.x;
    v[1] = u.y;
  }
};
// Four values of a staged row of b or c: the thread's states, each twice.
struct Twice {
  f2 v[4];
  __device__ __forceinline__ explicit Twice(const float2 *row) {
    const ulonglong2 *u = reinterpret_cast<const ulonglong2 *>(row);
    v[0] = u[0].x;
    v[1] = u[0].y;
    v[2] = u[1].x;
    v[3] = u[1].y;
  }
};

// One token of the recurrence.
__device__ __forceinline__ void advance(States &h, const States &A, const Pairs &delta, const Pairs &x,
                                        const Twice &b) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f2 u = f2_mul(delta.v[i], x.v[i]);
#pragma unroll
    for (int s = 0; s < 4; ++s) h[i][s] = f2_fma(f2_ex2(f2_mul(A[i][s], delta.v[i])), h[i][s], f2_mul(u, b.v[s]));
  }
}

// States of sequences without tokens: `to` = `from` (zero where null).
template <int SL>
__device__ __forceinline__ void copy_empty_states(const SsmArgs &a, const Place<SL> &p, const float *from, float *to) {
  if (!to) return;
  for (int64_t n = 0; n < a.d.N; ++n) {
    const SeqRange r = seq_range(a.cu, n, a.d.T);
    if (r.eos > r.bos) continue;
    States h;
    load_h0<SL>(a, p, from, n, h);
    store_final<SL>(a, p, to, n, h);
  }
}

// Host side, shared by the forward and the backward.
int ssm_validate(const gdr_ssm_desc *d, const int64_t *cu);
int ssm_prepare(SsmArgs &a, bool backward, int *sl, bool *vec);

}  // namespace gdr
