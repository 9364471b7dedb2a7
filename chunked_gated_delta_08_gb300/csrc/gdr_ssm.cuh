// gdr_ssm.cuh -- what the selective scan's kernels share: arguments, the layout
// of channels and states over a block's threads, and the staging of a tile of
// tokens in shared memory.
//
//   h_t = exp(delta_t a) h_{t-1} + (delta_t x_t) b_t      per channel e and state s
//   y_t = (sum_s c_t h_t + d x_t) silu(z_t)
//
// Layout.  A thread owns four neighbouring channels (the backward's last kernel:
// two) and four neighbouring states, 16 recurrences in registers; SL lanes (4, 8
// or 16: up to 16, 32 or 64 states) cover a channel's states.  Per token it reads
// four deltas, four inputs, four b and four c from shared memory, 16-byte loads
// that broadcast, for 16 states; sums over states cross SL lanes, sums over
// channels cross the others.  One channel per thread would need no exchange over
// states but eight 16-byte loads of b and c for the same work.  The packed fp32
// instructions take channels two by two: delta, x and the gradients come from
// shared memory as pairs; b and c are doubled in registers (staged as (b, b) they
// cost twice the shared-memory reads: 633 us against 603 on 16384 x 4096 x 16).
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
  // backward: partials of db and dc [ctiles, M, 2 SP]; of ddt_bias and dd [chunks, 2, E] (da's reuse hloc)
  float *part_bc, *part_e;
  int vec;       // backward: 16-byte loads of x, dt, z, dy
  int64_t M, chunks;
  int64_t L;
  int tpg;       // blocks across the channels of a group
  int ctiles;    // blocks across all channels: G * tpg
  int bc4;       // step: four elements of b and c at a time
  int s4;        // state rows may be read and written 16 bytes at a time
  int *status;
};

constexpr int kSsmThreads = 128;
constexpr int kTile = 16;  // tokens staged together

// delta from the raw dt (bias added): softplus(v) = max(v, 0) + log1p(u), u = e^-|v|,
// with log1p(u) = 2 atanh(r), r = u / (2 + u) <= 1/3, by its series in r^2.  Seven
// terms leave 9^-7 / 15 = 1.4e-8 of the value, a quarter of an fp32 rounding.
// log(1 + u) would lose a small u against the 1, and small deltas are the ones a
// state remembers longest.  `slope`: ddelta/dv.
template <bool SLOPE = false>
__device__ __forceinline__ f2 f2_delta(f2 v, int softplus, f2 *slope = nullptr) {
  if (!softplus) {
    if (SLOPE) *slope = f2_both(1.f);
    return v;
  }
  float lo, hi;
  f2_split(v, lo, hi);
  const f2 u = f2_ex2(f2_pack(-fabsf(lo) * kLog2e, -fabsf(hi) * kLog2e));
  const f2 r = f2_mul(u, f2_rcp(f2_add(u, f2_both(2.f)))), q = f2_mul(r, r);
  f2 w = f2_both(1.f / 13.f);
  w = f2_fma(w, q, f2_both(1.f / 11.f));
  w = f2_fma(w, q, f2_both(1.f / 9.f));
  w = f2_fma(w, q, f2_both(1.f / 7.f));
  w = f2_fma(w, q, f2_both(1.f / 5.f));
  w = f2_fma(w, q, f2_both(1.f / 3.f));
  w = f2_fma(w, q, f2_both(1.f));
  if (SLOPE) {  // 1 / (1 + u), or u / (1 + u) where v < 0
    const f2 k = f2_rcp(f2_add(u, f2_both(1.f)));
    float k0, k1, m0, m1;
    f2_split(k, k0, k1);
    f2_split(f2_mul(u, k), m0, m1);
    *slope = f2_pack(lo >= 0.f ? k0 : m0, hi >= 0.f ? k1 : m1);
  }
  return f2_fma(f2_add(r, r), w, f2_pack(fmaxf(lo, 0.f), fmaxf(hi, 0.f)));  // a NaN comes through u
}
__device__ __forceinline__ float ssm_delta(float v, int softplus) {
  float lo, hi;
  f2_split(f2_delta(f2_both(v), softplus), lo, hi);
  return lo;
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

// Sums of v[0..NV) over the SL lanes of a channel group, NV 4 or 2; lane sl
// returns that of v[sl & (NV - 1)].  Halves of the values are exchanged, so that
// three shuffles serve four values; lanes past the first NV first fold onto them.
template <int SL, int NV>
__device__ __forceinline__ float sum_over_states(float (&v)[NV], int sl) {
#pragma unroll
  for (int o = SL / 2; o >= NV; o >>= 1)
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
  const bool b0 = sl & 1;
  float k0 = v[0], k1 = v[1];
  if constexpr (NV == 4) {
    const bool b1 = sl & 2;
    k0 = b1 ? v[2] : v[0];
    k1 = b1 ? v[3] : v[1];
    k0 += __shfl_xor_sync(0xffffffffu, b1 ? v[0] : v[2], 2);
    k1 += __shfl_xor_sync(0xffffffffu, b1 ? v[1] : v[3], 2);
  }
  return (b0 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, b0 ? k0 : k1, 1);
}

// Where a block and its threads stand.
template <int SL_, int NP_ = 2, int WARPS = 4>
struct Place {
  static constexpr int SL = SL_, NP = NP_;
  static constexpr int CPW = 32 / SL * 2 * NP;  // channels of a warp
  static constexpr int CB = WARPS * CPW;        // of a block
  static constexpr int SP = 4 * SL;             // states, padded
  static constexpr int kThreads = 32 * WARPS;
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
    col = warp * CPW + cl * 2 * NP;
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

// Eight neighbouring columns of one token, in pairs: how a thread stages a tile.
typedef f2 Eight[4];
__device__ __forceinline__ void put8(float *p, const Eight &v) {
  reinterpret_cast<ulonglong2 *>(p)[0] = make_ulonglong2(v[0], v[1]);
  reinterpret_cast<ulonglong2 *>(p)[1] = make_ulonglong2(v[2], v[3]);
}
__device__ __forceinline__ void get8(const float *p, Eight &v) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(p)[0], b = reinterpret_cast<const ulonglong2 *>(p)[1];
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}
// Eight elements as they lie in memory, those of the first n columns (zero past
// them).  VEC: by 16-byte accesses, which the host allows where groups of
// channels are a multiple of the 8 (bf16) or 4 (fp32) elements of one; else one by
// one.
template <typename T, bool VEC>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16, true> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, int n) {
    u = n > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void expand(Eight &v) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <>
struct Raw8<float, true> {  // n is 0, 4 or 8
  ulonglong2 u[2];
  __device__ __forceinline__ void load(const float *p, int n) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      u[i] = n > 4 * i ? reinterpret_cast<const ulonglong2 *>(p)[i] : make_ulonglong2(0, 0);
  }
  __device__ __forceinline__ void expand(Eight &v) const {
    v[0] = u[0].x;
    v[1] = u[0].y;
    v[2] = u[1].x;
    v[3] = u[1].y;
  }
};
template <typename T>
struct Raw8<T, false> {
  T u[8];
  __device__ __forceinline__ void load(const T *p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = i < n ? p[i] : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void expand(Eight &v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_pack(to_f32(u[2 * i]), to_f32(u[2 * i + 1]));
  }
};

// A block's threads over a tile of [TT, CB] elements, eight columns each: the
// k-th of a thread's kCount is token `token(k)`, columns `col` and on, the same
// columns for every k.
template <int TT, int CB, int THREADS>
struct Stager {
  static constexpr int kRow = CB / 8, kCount = (TT * kRow + THREADS - 1) / THREADS;
  static_assert(THREADS % kRow == 0, "a thread keeps its columns");
  int row, col, n;  // n: columns inside the group
  template <typename P>
  __device__ __forceinline__ explicit Stager(const P &p) {
    row = threadIdx.x / kRow;
    col = (threadIdx.x % kRow) * 8;
    const int64_t left = p.e_end - p.e0 - col;
    n = left < 0 ? 0 : left < 8 ? (int)left : 8;
  }
  __device__ __forceinline__ int token(int k) const { return row + k * (THREADS / kRow); }
  // Whether token(k) is in the tile at all: not where the block has more threads than the tile.
  __device__ __forceinline__ bool has(int k) const { return TT * kRow >= THREADS * (k + 1) || token(k) < TT; }
};

// A thread's part of the next tile on its way into shared memory while this one
// is computed: bf16 with 16-byte accesses (fp32 tiles would take twice the room,
// and are loaded when they are staged).  A thread reads only what it copied, so
// its own wait is enough.
template <typename T, int ARRAYS, int COUNT, int THREADS>
struct Ahead {
  static constexpr bool kUse = sizeof(T) == 2;
  uint4 v[kUse ? ARRAYS : 1][kUse ? COUNT : 1][kUse ? THREADS : 1];
  __device__ __forceinline__ void fetch(int array, int k, const T *p, int n) {
    uint4 *to = &v[array][k][threadIdx.x];
    if (n > 0) copy_async<16>(to, p);
    else *to = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(int array, int k, Eight &o) const {
    Raw8<__nv_bfloat16, true> r;
    r.u = v[array][k][threadIdx.x];
    r.expand(o);
  }
};

// The block's columns of a row of E values (dt_bias, d): zero past the group, and where null.
template <int CB, int THREADS, typename P>
__device__ __forceinline__ void stage_row(const P &p, const float *src, float *dst) {
  for (int i = threadIdx.x; i < CB; i += THREADS) dst[i] = src && p.e0 + i < p.e_end ? src[p.e0 + i] : 0.f;
}

// b or c of a tile as fp32 [TT][SP], zero past S and past the tokens.
template <typename T, int TT, int THREADS, typename P>
__device__ __forceinline__ void stage_states(const SsmArgs &a, const P &p, const void *src, int64_t ld, int64_t t0,
                                             int nt, float *dst) {
  constexpr int SP = P::SP;
  const T *row = static_cast<const T *>(src) + p.g * a.d.S;
#pragma unroll
  for (int i0 = 0; i0 < TT * SP; i0 += THREADS) {
    const int i = i0 + threadIdx.x, t = i / SP, s = i % SP;
    if (TT * SP % THREADS != 0 && i >= TT * SP) break;
    const float v = t < nt && s < a.d.S ? to_f32(row[(t0 + t) * ld + s]) : 0.f;
    dst[i] = v;
  }
}

// A thread's states: pair i holds channels 2 i and 2 i + 1, for each of the four
// states.
template <int NP>
using StatesOf = f2[NP][4];
typedef StatesOf<2> States;

template <typename P, int NP, typename F>
__device__ __forceinline__ void read_states(const P &p, f2 (&h)[NP][4], F &&row) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    float v[4] = {}, w[4] = {};
    const int64_t e = p.e0 + p.col + 2 * i;
    if (e < p.e_end) row(e, v);
    if (e + 1 < p.e_end) row(e + 1, w);
#pragma unroll
    for (int s = 0; s < 4; ++s) h[i][s] = f2_pack(v[s], w[s]);
  }
}
template <typename P, int NP, typename F>
__device__ __forceinline__ void write_states(const P &p, const f2 (&h)[NP][4], F &&row) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    float v[4], w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) f2_split(h[i][s], v[s], w[s]);
    const int64_t e = p.e0 + p.col + 2 * i;
    if (e < p.e_end) row(e, v);
    if (e + 1 < p.e_end) row(e + 1, w);
  }
}
// The state h0 of sequence n (zero where there is none).
template <typename P, int NP>
__device__ __forceinline__ void load_h0(const SsmArgs &a, const P &p, const float *h0, int64_t n, f2 (&h)[NP][4]) {
  read_states(p, h, [&](int64_t e, float (&v)[4]) {
    if (h0) load_states(h0 + (n * a.d.E + e) * a.d.S, p.sl * 4, (int)a.d.S, a.s4, v);
  });
}
template <typename P, int NP>
__device__ __forceinline__ void store_final(const SsmArgs &a, const P &p, float *ht, int64_t n,
                                            const f2 (&h)[NP][4]) {
  write_states(p, h, [&](int64_t e, const float (&v)[4]) {
    store_states(ht + (n * a.d.E + e) * a.d.S, p.sl * 4, (int)a.d.S, a.s4, v);
  });
}
// Chunk states [chunks, E, SP]: always whole 16-byte groups.
template <typename P, int NP>
__device__ __forceinline__ void load_chunk(const SsmArgs &a, const P &p, const float *src, int64_t chunk,
                                           f2 (&h)[NP][4]) {
  read_states(p, h, [&](int64_t e, float (&v)[4]) {
    if (src) load4(src + (chunk * a.d.E + e) * P::SP + p.sl * 4, v);
  });
}
template <typename P, int NP>
__device__ __forceinline__ void store_chunk(const SsmArgs &a, const P &p, float *dst, int64_t chunk,
                                            const f2 (&h)[NP][4]) {
  write_states(p, h, [&](int64_t e, const float (&v)[4]) {
    store4(dst + (chunk * a.d.E + e) * P::SP + p.sl * 4, v);
  });
}

// a[e, s] log2(e) of a thread's channels and states (zero outside: such states stay zero).
template <typename P, int NP>
__device__ __forceinline__ void load_a(const SsmArgs &a, const P &p, f2 (&A)[NP][4]) {
  read_states(p, A, [&](int64_t e, float (&v)[4]) {
    load_states(a.a + e * a.d.S, p.sl * 4, (int)a.d.S, a.s4, v);
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] *= kLog2e;
  });
}

// A staged row's values of the thread's channels, in pairs.
template <int NP>
struct Pairs {
  f2 v[NP];
  __device__ __forceinline__ explicit Pairs(const float *row) {
    if constexpr (NP == 2) {
      const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(row);
      v[0] = u.x;
      v[1] = u.y;
    } else {
      v[0] = *reinterpret_cast<const f2 *>(row);
    }
  }
};
// Four values of a staged row of b or c: the thread's states, each twice.
struct Twice {
  f2 v[4];
  __device__ __forceinline__ explicit Twice(const float *row) {
    const float4 u = *reinterpret_cast<const float4 *>(row);
    v[0] = f2_both(u.x);
    v[1] = f2_both(u.y);
    v[2] = f2_both(u.z);
    v[3] = f2_both(u.w);
  }
};

// One token of the recurrence.
template <int NP>
__device__ __forceinline__ void advance(f2 (&h)[NP][4], const f2 (&A)[NP][4], const Pairs<NP> &delta,
                                        const Pairs<NP> &x, const Twice &b) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const f2 u = f2_mul(delta.v[i], x.v[i]);
#pragma unroll
    for (int s = 0; s < 4; ++s) h[i][s] = f2_fma(f2_ex2(f2_mul(A[i][s], delta.v[i])), h[i][s], f2_mul(u, b.v[s]));
  }
}

// States of sequences without tokens: `to` = `from` (zero where null).  Chunk c
// looks after sequences c, c + chunks, ...
template <typename P>
__device__ __forceinline__ void copy_empty_states(const SsmArgs &a, const P &p, const float *from, float *to) {
  if (!to) return;
  for (int64_t n = p.chunk; n < a.d.N; n += a.chunks) {
    const SeqRange r = seq_range(a.cu, n, a.d.T);
    if (r.eos > r.bos) continue;
    StatesOf<P::NP> h;
    load_h0(a, p, from, n, h);
    store_final(a, p, to, n, h);
  }
}

// What a chunk makes of the value v that enters it: 2^e v + loc.  Where a state
// grows (a > 0, or a negative delta) the factor may leave fp32's range and the
// product not, zero above all: such a factor is multiplied in three parts, each in
// range, of which more than 2^381 in all take any v but zero past the range as well.
// Selects, as lanes of a warp have near and far factors: a branch took 4 us more in
// the backward of 16384 x 2048 x 16.
__device__ __forceinline__ float carry_over(float e, float v, float loc) {
  const bool far = !(fabsf(e) <= 126.f);
  const float third = e * (1.f / 3.f), r = ex2(far ? (third > 127.f ? 127.f : third) : e), m = far ? r : 1.f;
  return fmaf(r, (m * v) * m, loc);
}

// Host side, shared by the forward and the backward.
int ssm_validate(const gdr_ssm_desc *d, const int64_t *cu);
int ssm_prepare(SsmArgs &a, bool backward, int *sl, bool *vec);

}  // namespace gdr
