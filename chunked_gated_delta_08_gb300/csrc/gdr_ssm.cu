// gdr_ssm.cu -- the selective state space scan: forward and single-token step.
// gdr_ssm.cuh has the formulas, the layout and the cut of the time axis.
//
// Forward, three launches:
//   local   per (chunk, channels): the chunk's state from zero, and sum(delta)
//   carry   per (channel, state): the state that enters each chunk, in order
//   main    per (chunk, channels): the recurrence again from there, y and ht
// The recurrence runs twice so that chunks run at once; where one chunk covers
// a sequence (short ones, or enough sequences to fill the GPU) main runs alone.
// The work is arithmetic: per channel, state and token one exponential and
// four fp32 operations in each pass, against 8 bytes of HBM traffic per channel
// and token in bf16.  16384 tokens x 4096 channels x 16 states take 577 us, where one
// exponential each would take 115 us and the bytes 81.  Nothing is full: local and
// main issue on 60 % of cycles, the fp32 pipe is 50 to 58 % and the exponential unit
// 39 to 55 % busy; the 14 warps of a multiprocessor wait about as often for a value
// just computed as for a pipe.  Four blocks of 128 registers on a multiprocessor are the best
// of four, five (+2 %) and six (+17 %, spilling); eight channels to a thread, which
// halve the reads of b and c, took 5 % longer.
#include <algorithm>

#include "gdr_ssm.cuh"

namespace gdr {
namespace {

template <typename T, typename P, bool VEC, bool MAIN>
struct __align__(16) FwdShared {
  Ahead<T, VEC ? (MAIN ? 3 : 2) : 1, VEC ? Stager<kTile, P::CB, kSsmThreads>::kCount : 1, VEC ? kSsmThreads : 1> ahead;
  float delta[kTile][P::CB], x[kTile][P::CB], gate[MAIN ? kTile : 1][P::CB];
  float bias[P::CB];
  float b[kTile * P::SP], c[kTile * P::SP];
  Borders<kTile> bd;
};

// MAIN: y and ht from the states that enter the chunks (a.hloc, zero where
// null).  Else: the chunk's own state and sum of delta.
template <typename T, int SL, bool VEC, bool MAIN>
__global__ void __launch_bounds__(kSsmThreads, 4) ssm_fwd_kernel(SsmArgs a) {
  using P = Place<SL>;
  constexpr int NB = kTile * P::SP / kSsmThreads;
  constexpr bool kAhead = VEC && sizeof(T) == 2;
  __shared__ FwdShared<T, P, VEC, MAIN> sm;
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  const P p(a);
  if (MAIN) copy_empty_states(a, p, a.h0, a.ht);
  const Stager<kTile, P::CB, kSsmThreads> st(p);
  States A, h;
  T next_b[NB], next_c[MAIN ? NB : 1];
  const int64_t begin = p.chunk * a.L, end = begin + a.L < a.M ? begin + a.L : a.M;
  auto columns = [&](int64_t t0, int k) {  // of the thread's k-th token of a tile: columns to load
    return st.has(k) && st.token(k) < end - t0 ? st.n : 0;
  };
  auto source = [&](const void *p0, int64_t ld, int64_t t0, int k) {
    return static_cast<const T *>(p0) + (t0 + st.token(k)) * ld + p.e0 + st.col;
  };
  auto fetch_ahead = [&](int64_t t0) {
#pragma unroll
    for (int k = 0; k < st.kCount; ++k) {
      const int n = columns(t0, k);
      sm.ahead.fetch(0, k, source(a.x, a.d.ld_x, t0, k), n);
      sm.ahead.fetch(1, k, source(a.dt, a.d.ld_dt, t0, k), n);
      if (MAIN && a.z) sm.ahead.fetch(2, k, source(a.z, a.d.ld_z, t0, k), n);
    }
    copy_commit();
  };
  auto fetch_states = [&](int64_t t0) {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = k * kSsmThreads + threadIdx.x, t = i / P::SP, s = i % P::SP;
      const bool in = t < end - t0 && s < a.d.S;
      const int64_t at = p.g * a.d.S + s;
      next_b[k] = in ? static_cast<const T *>(a.b)[(t0 + t) * a.d.ld_b + at] : from_f32<T>(0.f);
      if (MAIN) next_c[k] = in ? static_cast<const T *>(a.c)[(t0 + t) * a.d.ld_c + at] : from_f32<T>(0.f);
    }
  };
  if constexpr (kAhead) {
    if (begin < end) {
      fetch_ahead(begin);
      fetch_states(begin);
    }
  }
  stage_row<P::CB, kSsmThreads>(p, a.dt_bias, sm.bias);
  load_a(a, p, A);
  load_chunk(a, p, MAIN ? a.hloc : nullptr, p.chunk, h);
  const int mine = p.sl & 3;  // of the thread's four channels, the one whose output it finishes
  const int64_t e_mine = p.e0 + p.col + mine;
  const bool owner = p.sl < 4 && e_mine < p.e_end;
  const float skip = MAIN && a.dskip && owner ? a.dskip[e_mine] : 0.f;
  T *y = static_cast<T *>(a.y) + begin * a.d.E + e_mine;
  f2 sum[2] = {0, 0};
  bool started = false;  // a sequence starts in this chunk

  auto token = [&](int t) {
    const Pairs<2> delta(&sm.delta[t][p.col]);
    advance(h, A, delta, Pairs<2>(&sm.x[t][p.col]), Twice(&sm.b[t * P::SP + p.sl * 4]));
    if (MAIN) {
      const Twice c(&sm.c[t * P::SP + p.sl * 4]);
      float v[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f2 o = f2_mul(c.v[0], h[i][0]);
#pragma unroll
        for (int s = 1; s < 4; ++s) o = f2_fma(c.v[s], h[i][s], o);
        f2_split(o, v[2 * i], v[2 * i + 1]);
      }
      const float o = sum_over_states<SL>(v, p.sl);
      if (owner) *y = from_f32<T>(fmaf(skip, sm.x[t][p.col + mine], o) * sm.gate[t][p.col + mine]);
      y += a.d.E;
    } else {
      sum[0] = f2_add(sum[0], delta.v[0]);
      sum[1] = f2_add(sum[1], delta.v[1]);
    }
  };

  int64_t bos = -1, eos = -1;  // of the sequence that the tile begins in
  for (int64_t t0 = begin; t0 < end; t0 += kTile) {
    const int nt = end - t0 < kTile ? (int)(end - t0) : kTile;
    if (!kAhead) fetch_states(t0);
    if (t0 >= eos) {
      const SeqRange r = seq_range(a.cu, seq_of_token(a.cu, a.d.N, a.d.T, t0), a.d.T);
      bos = r.bos;
      eos = r.eos;
    }
    const bool borders = bos >= t0 || eos <= t0 + nt;  // a sequence starts or ends in the tile
    __syncthreads();                                   // the previous tile is consumed
    if (borders) stage_borders(a, t0, nt, sm.bd);
    Eight bias;
    get8(&sm.bias[st.col], bias);
    if (kAhead) copy_wait<0>();
    auto get = [&](int array, const void *src, int64_t ld, int k, Eight &v) {
      if constexpr (kAhead) {
        sm.ahead.get(array, k, v);
      } else {
        Raw8<T, VEC> r;
        r.load(source(src, ld, t0, k), columns(t0, k));
        r.expand(v);
      }
    };
#pragma unroll
    for (int k = 0; k < st.kCount; ++k) {
      if (!st.has(k)) continue;
      const int t = st.token(k);
      Eight v;
      get(0, a.x, a.d.ld_x, k, v);
      put8(&sm.x[t][st.col], v);
      get(1, a.dt, a.d.ld_dt, k, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2_delta(f2_add(v[i], bias[i]), a.d.flags & GDR_SSM_SOFTPLUS);
      put8(&sm.delta[t][st.col], v);
      if (MAIN) {
        if (a.z) get(2, a.z, a.d.ld_z, k, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a.z ? f2_silu(v[i]) : f2_both(1.f);
        put8(&sm.gate[t][st.col], v);
      }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const float bv = to_f32(next_b[k]);
      sm.b[k * kSsmThreads + threadIdx.x] = bv;
      if (MAIN) {
        const float cv = to_f32(next_c[k]);
        sm.c[k * kSsmThreads + threadIdx.x] = cv;
      }
    }
    if constexpr (kAhead) {
      if (t0 + kTile < end) {
        fetch_ahead(t0 + kTile);
        fetch_states(t0 + kTile);
      }
    }
    __syncthreads();
    if (!borders && nt == kTile) {
#pragma unroll 4
      for (int t = 0; t < kTile; ++t) token(t);
    } else {
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        if (borders && sm.bd.first[t] >= 0) {
          load_h0(a, p, a.h0, sm.bd.first[t], h);
          started = true;
        }
        token(t);
        if (MAIN && a.ht && borders && sm.bd.last[t] >= 0) store_final(a, p, a.ht, sm.bd.last[t], h);
      }
    }
  }
  if (!MAIN) {
    store_chunk(a, p, a.hloc, p.chunk, h);
    if (owner) {
      float s[4];
      f2_split(sum[0], s[0], s[1]);
      f2_split(sum[1], s[2], s[3]);
      const float mine_sum = mine == 0 ? s[0] : mine == 1 ? s[1] : mine == 2 ? s[2] : s[3];
      a.sumd[p.chunk * a.d.E + e_mine] = started ? CUDART_NAN_F : mine_sum;  // NaN: nothing passes through
    }
  }
}

// In place, per (channel, state): hloc[c] becomes the state that enters chunk c.
// A batch of chunks is loaded at once; the additions run in order.
constexpr int kCarryBatch = 16;
__global__ void __launch_bounds__(128) ssm_carry_kernel(SsmArgs a, int SP) {
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (i >= a.d.E * SP) return;
  const int64_t e = i / SP, row = a.d.E * SP;
  const int s = (int)(i % SP);
  const float A = s < a.d.S ? a.a[e * a.d.S + s] * kLog2e : 0.f;
  float h = 0.f;
  for (int64_t c0 = 0; c0 < a.chunks; c0 += kCarryBatch) {
    float loc[kCarryBatch], sum[kCarryBatch];
#pragma unroll
    for (int k = 0; k < kCarryBatch; ++k) {
      const int64_t c = c0 + k;
      loc[k] = c < a.chunks ? a.hloc[c * row + i] : 0.f;
      sum[k] = c < a.chunks ? a.sumd[c * a.d.E + e] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kCarryBatch; ++k) {
      const int64_t c = c0 + k;
      if (c < a.chunks) {
        a.hloc[c * row + i] = h;
        h = isnan(sum[k]) ? loc[k] : carry_over(A * sum[k], h, loc[k]);
      }
    }
  }
}

// One token per row.  A block takes 256 / SL channels and goes through rows, four
// at a time; SL lanes share a channel, four states each, so that a warp's states
// are consecutive 16-byte groups.  The states of the next four rows are on their
// way into shared memory (a thread copies what it alone reads) while these are
// computed.  Of a channel's first four lanes, lane k works out delta, delta x and
// the gate of row k for all (they cost more than the four recurrences of a lane),
// and finishes that row's output.  The bound is HBM: each state is read and
// written once, 256 rows of 4096 x 16 in 31 us, 69 % of the copy rate.  One row
// group to a block took 37 us, and 66 us at 92 registers.  With fp32 inputs, whose b
// and c take twice the registers and spill 16 to 28 bytes, 42 us against 33 with cold caches.
constexpr int kStepRows = 4;

// Four states of a thread, in pairs, and four elements of b or c as they lie in
// memory.  AL: by 16-byte (bf16: 8-byte) accesses, all four or none inside S;
// else one by one.
template <bool AL>
__device__ __forceinline__ void load_quad(const float *p, int s0, int S, f2 (&v)[2]) {
  float f[4] = {};
  if (AL) {
    if (s0 < S) load4(p, f);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (s0 + q < S) f[q] = p[q];
  }
  v[0] = f2_pack(f[0], f[1]);
  v[1] = f2_pack(f[2], f[3]);
}
template <bool AL>
__device__ __forceinline__ void store_quad(float *p, int s0, int S, const f2 (&v)[2]) {
  float f[4];
  f2_split(v[0], f[0], f[1]);
  f2_split(v[1], f[2], f[3]);
  if (AL) {
    if (s0 < S) store4(p, f);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (s0 + q < S) p[q] = f[q];
  }
}
template <typename T, bool AL>
struct Quad;
template <bool AL>
struct Quad<__nv_bfloat16, AL> {
  uint2 u = {0, 0};
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, int s0, int S) {
    if (AL) {
      if (s0 < S) u = *reinterpret_cast<const uint2 *>(p);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = s0 + q < S ? __bfloat16_as_ushort(p[q]) : 0;
      u = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
  }
  __device__ __forceinline__ void expand(f2 (&v)[2]) const {
    v[0] = f2_pack(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    v[1] = f2_pack(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  }
};
template <bool AL>
struct Quad<float, AL> {
  f2 u[2] = {0, 0};
  __device__ __forceinline__ void load(const float *p, int s0, int S) { load_quad<AL>(p, s0, S, u); }
  __device__ __forceinline__ void expand(f2 (&v)[2]) const {
    v[0] = u[0];
    v[1] = u[1];
  }
};

// AL: states, a, b and c allow their whole accesses.
template <typename T, int SL, bool AL>
__global__ void __launch_bounds__(256, 4) ssm_step_kernel(SsmArgs a, const int32_t *slots, float *state,
                                                          unsigned tiles, int groups) {
  __shared__ __align__(16) float ahead[2][kStepRows][256][4];
  // rows, channels and leading dimensions are below 2^31; products of two are 64-bit
  const int rows = (int)a.d.B, E = (int)a.d.E, S = (int)a.d.S;
  const int i = (int)(blockIdx.x % tiles) * 256 + threadIdx.x;
  const int e = i / SL, sl = i % SL, s0 = sl * 4;
  const bool in = e < E;
  const int es = E * S, mine_s = e * S + s0;  // at most 2^30
  const int at = (in ? (unsigned)e / (unsigned)(a.d.E / a.d.G) : 0) * S + s0;
  auto slot_of = [&](int g, int k) {  // negative: nothing to do
    const int r = g * kStepRows + k;
    int slot = g < groups && r < rows && in ? (slots ? slots[r] : r) : -1;
    if (slot >= a.d.N) {
      raise_status(a.status, GDR_ERR_SLOTS);
      slot = -1;
    }
    return slot;
  };
  auto fetch = [&](int slot, int buf, int k) {
    float *to = ahead[buf][k][threadIdx.x];
    const float *from = state + (int64_t)slot * es + mine_s;
    if (AL) {
      if (slot >= 0 && s0 < S) copy_async<16>(to, from);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (slot >= 0 && s0 + q < S) to[q] = from[q];
    }
  };
  int g = (int)(blockIdx.x / tiles);
  const int stride = (int)(gridDim.x / tiles);
  int slot[kStepRows];
#pragma unroll
  for (int k = 0; k < kStepRows; ++k) {
    *reinterpret_cast<float4 *>(ahead[0][k][threadIdx.x]) = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4 *>(ahead[1][k][threadIdx.x]) = make_float4(0.f, 0.f, 0.f, 0.f);
    slot[k] = slot_of(g, k);
    fetch(slot[k], 0, k);
  }
  copy_commit();
  f2 A[2] = {0, 0};
  float bias = 0.f, skip = 0.f;
  if (in) {
    load_quad<AL>(a.a + mine_s, s0, S, A);
    if (a.dt_bias) bias = a.dt_bias[e];
    if (a.dskip) skip = a.dskip[e];
  }
  A[0] = f2_mul(A[0], f2_both(kLog2e));
  A[1] = f2_mul(A[1], f2_both(kLog2e));

  int buf = 0;
  for (; g < groups; g += stride, buf ^= 1) {
    int next[kStepRows];
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) next[k] = slot_of(g + stride, k);
    Quad<T, AL> b[kStepRows], c[kStepRows];
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) {
      if (slot[k] >= 0) {
        const int64_t r = g * kStepRows + k;
        b[k].load(static_cast<const T *>(a.b) + r * (int)a.d.ld_b + at, s0, S);
        c[k].load(static_cast<const T *>(a.c) + r * (int)a.d.ld_c + at, s0, S);
      }
    }
    const int r = g * kStepRows + sl;  // the row this lane prepares and finishes
    const bool owner = sl < kStepRows && in && r < rows;
    float x = 0.f, delta = 0.f, gate = 1.f;
    if (owner) {
      x = to_f32(static_cast<const T *>(a.x)[(int64_t)r * (int)a.d.ld_x + e]);
      delta = to_f32(static_cast<const T *>(a.dt)[(int64_t)r * (int)a.d.ld_dt + e]) + bias;
      if (a.z) gate = to_f32(static_cast<const T *>(a.z)[(int64_t)r * (int)a.d.ld_z + e]);
    }
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) fetch(next[k], buf ^ 1, k);
    copy_commit();
    if (owner) {
      delta = ssm_delta(delta, a.d.flags & GDR_SSM_SOFTPLUS);
      if (a.z) gate *= sigmoid_fast(gate);
    }
    const float u = delta * x;
    copy_wait<1>();  // these rows' states are here
    float out[kStepRows];
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) {
      const f2 dk = f2_both(__shfl_sync(0xffffffffu, delta, k, SL)), uk = f2_both(__shfl_sync(0xffffffffu, u, k, SL));
      const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(ahead[buf][k][threadIdx.x]);
      f2 h[2] = {v.x, v.y}, bk[2], ck[2];
      b[k].expand(bk);
      c[k].expand(ck);
#pragma unroll
      for (int q = 0; q < 2; ++q) h[q] = f2_fma(f2_ex2(f2_mul(dk, A[q])), h[q], f2_mul(uk, bk[q]));
      float lo, hi;
      f2_split(f2_fma(ck[1], h[1], f2_mul(ck[0], h[0])), lo, hi);
      out[k] = lo + hi;
      if (slot[k] >= 0) store_quad<AL>(state + (int64_t)slot[k] * es + mine_s, s0, S, h);
    }
    const float y = sum_over_states<SL>(out, sl);
    if (owner) {
      const int mine = sl == 0 ? slot[0] : sl == 1 ? slot[1] : sl == 2 ? slot[2] : slot[3];
      static_cast<T *>(a.y)[(int64_t)r * E + e] = from_f32<T>(mine >= 0 ? fmaf(skip, x, y) * gate : 0.f);
    }
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) slot[k] = next[k];
  }
}

template <typename T, bool MAIN>
int launch_fwd(const SsmArgs &a, int sl, bool vec, cudaStream_t st) {
  const unsigned grid = (unsigned)(a.chunks * a.ctiles);
  auto go = [&](auto SL) {
    if (vec) ssm_fwd_kernel<T, decltype(SL)::value, true, MAIN><<<grid, kSsmThreads, 0, st>>>(a);
    else ssm_fwd_kernel<T, decltype(SL)::value, false, MAIN><<<grid, kSsmThreads, 0, st>>>(a);
    return launched(MAIN ? "ssm_fwd_kernel" : "ssm_local_kernel");
  };
  if (sl == 4) return go(std::integral_constant<int, 4>{});
  if (sl == 8) return go(std::integral_constant<int, 8>{});
  return go(std::integral_constant<int, 16>{});
}

template <bool MAIN>
int launch_fwd(const SsmArgs &a, int sl, bool vec, cudaStream_t st) {
  return a.d.dtype == GDR_BF16 ? launch_fwd<__nv_bfloat16, MAIN>(a, sl, vec, st)
                               : launch_fwd<float, MAIN>(a, sl, vec, st);
}

int lanes_of(int64_t S) { return S <= 16 ? 4 : S <= 32 ? 8 : 16; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

template <typename T>
int launch_step(const SsmArgs &a, const int32_t *slots, float *state, cudaStream_t st) {
  auto go = [&](auto SL) {
    const int64_t tiles = cdiv(a.d.E * decltype(SL)::value, 256), groups = cdiv(a.d.B, kStepRows);
    // one wave of blocks, each through its share of the rows
    const int64_t across = std::min(groups, std::max<int64_t>(1, 4 * kSMs / tiles));
    auto *kernel = a.s4 && a.bc4 ? ssm_step_kernel<T, decltype(SL)::value, true> : ssm_step_kernel<T, decltype(SL)::value, false>;
    kernel<<<(unsigned)(tiles * across), 256, 0, st>>>(a, slots, state, (unsigned)tiles, (int)groups);
    return launched("ssm_step_kernel");
  };
  const int sl = lanes_of(a.d.S);
  if (sl == 4) return go(std::integral_constant<int, 4>{});
  if (sl == 8) return go(std::integral_constant<int, 8>{});
  return go(std::integral_constant<int, 16>{});
}

int validate(const gdr_ssm_desc *d, const int64_t *cu, bool step) {
  if (!d) return set_error(GDR_ERR_NULLPTR, "desc is NULL");
  if (d->dtype != GDR_F32 && d->dtype != GDR_BF16) return set_error(GDR_ERR_DTYPE, "dtype must be GDR_F32 or GDR_BF16");
  if (d->flags & ~GDR_SSM_SOFTPLUS) return set_error(GDR_ERR_DTYPE, "unknown bits in flags");
  if (d->B < 0 || d->T < 0 || d->N < 0 || d->N > 0x7fffffff)
    return set_error(GDR_ERR_SHAPE, "B, T and N must be >= 0 (N below 2^31)");
  if (d->S < 1 || d->S > 64) return set_error(GDR_ERR_SHAPE, "S must be in [1, 64]");
  if (d->E < 1 || d->E > (1 << 24)) return set_error(GDR_ERR_SHAPE, "E must be in [1, 2^24]");
  if (d->G < 1 || d->E % d->G != 0) return set_error(GDR_ERR_SHAPE, "E must be a multiple of G");
  if (d->ld_x < d->E || d->ld_dt < d->E || d->ld_z < d->E || d->ld_dy < d->E || d->ld_b < d->G * d->S ||
      d->ld_c < d->G * d->S)
    return set_error(GDR_ERR_SHAPE, "leading dimensions must be at least E, or G * S");
  constexpr int64_t kMost = 0x7fffffff;
  if (d->ld_x > kMost || d->ld_dt > kMost || d->ld_z > kMost || d->ld_b > kMost || d->ld_c > kMost || d->ld_dy > kMost)
    return set_error(GDR_ERR_SHAPE, "leading dimensions must be below 2^31");
  if (step && d->B > kMost - 4) return set_error(GDR_ERR_SHAPE, "too many rows for one launch");
  if (step) return d->T == 1 ? GDR_OK : set_error(GDR_ERR_SHAPE, "a step takes one token per row: T must be 1");
  if (cu) {
    if (d->B != 1) return set_error(GDR_ERR_SHAPE, "cu_seqlens requires B == 1");
  } else if (d->N != d->B) {
    return set_error(GDR_ERR_SHAPE, "N must equal B when cu_seqlens is NULL");
  }
  return GDR_OK;
}

// Chunk length, in whole tiles.  The grid runs in waves of four blocks on each
// multiprocessor; in units of a quarter of a token's time in one wave, a wave of
// local and main takes 4 (L + 8), the chunk's start included, and the carry about
// one per chunk (measured: 0.7 us a token, 0.2 us a chunk).  The last wave is
// what matters: 16384 x 4096 channels in chunks of 256 tokens leave it a third
// full and take 593 us, against 580 us with the length chosen here; 32768 x 1024
// take 321 and 301 us.
constexpr int kWave = 4 * kSMs;
int64_t chunk_cost(const SsmArgs &a, int64_t L) {
  const int64_t chunks = cdiv(a.M, L);
  return 4 * cdiv(chunks * a.ctiles, kWave) * (L + 8) + chunks;
}
int64_t chunk_length(const SsmArgs &a) {
  int64_t best = kTile, least = chunk_cost(a, kTile);
  for (int64_t L = 2 * kTile; L <= 512; L += kTile) {
    const int64_t cost = chunk_cost(a, L);
    if (cost < least) {
      least = cost;
      best = L;
    }
  }
  return best;
}

int run_fwd(SsmArgs a, cudaStream_t st) {
  int sl, rc;
  bool vec;
  if ((rc = ssm_prepare(a, false, &sl, &vec)) != GDR_OK) return rc;
  // A dense batch may take each sequence as one chunk: main alone, three fifths of the work per token.
  a.L = chunk_length(a);
  const bool whole =
      !a.cu && (a.d.T <= 2 * kTile || 12 * cdiv(a.d.B * a.ctiles, kWave) * (a.d.T + 8) <= 5 * chunk_cost(a, a.L));
  if (whole) a.L = std::max<int64_t>(1, a.d.T);
  else if (a.M <= 4 * kTile) a.L = 4 * kTile;  // so few tokens take less than the launches that would share them out
  a.chunks = std::max<int64_t>(1, cdiv(a.M, a.L));
  if (a.chunks * a.ctiles > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many tokens and channels for one launch");
  if (whole || a.chunks == 1) return launch_fwd<true>(a, sl, vec, st);
  const size_t hb = align256(sizeof(float) * (size_t)(a.chunks * a.d.E * 4 * sl));
  char *base = nullptr;
  rc = scratch_begin(hb + sizeof(float) * (size_t)(a.chunks * a.d.E), st, "scan scratch", &base);
  if (rc != GDR_OK) return rc;
  a.hloc = (float *)base;
  a.sumd = (float *)(base + hb);
  rc = launch_fwd<false>(a, sl, vec, st);
  if (rc == GDR_OK) {
    ssm_carry_kernel<<<(unsigned)cdiv(a.d.E * 4 * sl, 128), 128, 0, st>>>(a, 4 * sl);
    rc = launched("ssm_carry_kernel");
  }
  if (rc == GDR_OK) rc = launch_fwd<true>(a, sl, vec, st);
  return scratch_end(base, st, "scan scratch", rc);
}

}  // namespace

int ssm_validate(const gdr_ssm_desc *d, const int64_t *cu) { return validate(d, cu, false); }

int ssm_prepare(SsmArgs &a, bool backward, int *sl, bool *vec) {
  int rc;
  a.M = a.d.B * a.d.T;
  a.status = current_status_word(&rc);
  if (!a.status) return rc;
  *sl = lanes_of(a.d.S);
  a.tpg = (int)cdiv(a.d.E / a.d.G, 512 / *sl);
  a.ctiles = (int)(a.d.G * a.tpg);
  const int64_t unit = a.d.dtype == GDR_BF16 ? 8 : 4;  // elements of a 16-byte access
  *vec = (a.d.E / a.d.G) % unit == 0 && a.d.ld_x % unit == 0 && a.d.ld_dt % unit == 0 && (!a.z || a.d.ld_z % unit == 0) &&
         is_aligned16(a.x) && is_aligned16(a.dt) && is_aligned16(a.z);
  a.s4 = a.d.S % 4 == 0 && is_aligned16(a.a) && is_aligned16(a.h0) && is_aligned16(a.ht) && is_aligned16(a.dht) && is_aligned16(a.dh0);
  if (backward) *vec = *vec && a.d.ld_dy % unit == 0 && is_aligned16(a.dy);
  return GDR_OK;
}

}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_ssm_fwd(const gdr_ssm_desc *desc, const void *x, const void *dt, const float *a, const void *b,
                const void *c, const float *d, const void *z, const float *dt_bias, const float *h0,
                const int64_t *cu_seqlens, void *y, float *ht, void *stream) {
  int rc = validate(desc, cu_seqlens, false);
  if (rc != GDR_OK) return rc;
  if (desc->N == 0 && !cu_seqlens) return GDR_OK;
  if (!a || (desc->B * desc->T > 0 && (!x || !dt || !b || !c || !y)))
    return set_error(GDR_ERR_NULLPTR, "x, dt, a, b, c and y must be non-NULL");
  SsmArgs s{};
  s.d = *desc;
  s.x = x; s.dt = dt; s.a = a; s.b = b; s.c = c; s.dskip = d; s.z = z; s.dt_bias = dt_bias; s.h0 = h0;
  s.cu = cu_seqlens; s.y = y; s.ht = ht;
  return run_fwd(s, (cudaStream_t)stream);
}

int gdr_ssm_step(const gdr_ssm_desc *desc, const void *x, const void *dt, const float *a, const void *b,
                 const void *c, const float *d, const void *z, const float *dt_bias, const int32_t *slots,
                 float *state, void *y, void *stream) {
  int rc = validate(desc, nullptr, true);
  if (rc != GDR_OK) return rc;
  if (desc->B == 0) return GDR_OK;
  if (!x || !dt || !a || !b || !c || !state || !y)
    return set_error(GDR_ERR_NULLPTR, "x, dt, a, b, c, state and y must be non-NULL");
  SsmArgs s{};
  s.d = *desc;
  s.x = x; s.dt = dt; s.a = a; s.b = b; s.c = c; s.dskip = d; s.z = z; s.dt_bias = dt_bias; s.y = y;
  s.s4 = desc->S % 4 == 0 && is_aligned16(a) && is_aligned16(state);
  s.bc4 = desc->S % 4 == 0 && desc->ld_b % 4 == 0 && desc->ld_c % 4 == 0 && is_aligned16(b) && is_aligned16(c);
  s.status = current_status_word(&rc);
  if (!s.status) return rc;
  return desc->dtype == GDR_BF16 ? launch_step<__nv_bfloat16>(s, slots, state, (cudaStream_t)stream)
                                 : launch_step<float>(s, slots, state, (cudaStream_t)stream);
}

}  // extern "C"
