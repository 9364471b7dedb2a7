// gdr_conv.cu -- short causal convolution per channel: forward, backward, and
// the single-token step with states in a pool of slots.
//
//   p_t = bias + sum_j w_j x_{t - W + 1 + j};  y_t = act(p_t)
//   backward, g_t = dy_t act'(p_t):  dx_t = sum_i w_{W-1-i} g_{t+i},  dw_j = sum_t g_t x_{t-W+1+j}
// with x_{-1}, .. x_{-W+1} taken from the sequence's state, and the last W - 1
// inputs of each sequence left as its new state.
//
// A thread owns two or four neighbouring channels, in pairs for the packed fp32
// instructions, and walks a run of tokens with the W - 1 inputs before in
// registers, so every input is read from HBM once (the W - 1 tokens around a run
// come from L2 again).  The next batch of tokens is loaded while one is computed.
// Runs are cut from the flat token axis; a sequence's border inside one reloads
// the window.  The bound is HBM: 16384 x 4096 bf16 take 51.5 us, 78 % of the copy
// rate, where eight channels to a thread, at 155 registers, took 104.  The
// backward takes 98 us, 61 %, and issues on 53 % of the cycles: neither is full.  A
// thread has four tokens of two arrays under way, 20 KB a multiprocessor, half of what
// the forward has (41 KB), and its warps wait for loads more than for anything else.
#include <algorithm>

#include "gdr_layer.cuh"

namespace gdr {
namespace {

struct ConvArgs {
  gdr_conv_desc d;
  const void *x, *weight, *bias, *s0, *dy, *dst;
  const int64_t *cu;
  const int32_t *slots;
  void *y, *st;  // backward: dx, ds0; step: st is the pool
  float *part;   // backward: [runs, W + 1, E]
  float *dweight, *dbias;
  int64_t M, runs;
  int L, cx;     // tokens in a run; threads across channels in a block
  unsigned tiles;  // blocks across channels
  int *status;
};

constexpr int kThreads = 128;

// The sequence under the cursor.
struct Seq {
  int64_t n, bos, eos;
};

__device__ __forceinline__ Seq seq_at(const ConvArgs &a, int64_t t) {
  const int64_t n = seq_of_token(a.cu, a.d.N, a.d.T, t);
  const SeqRange r = seq_range(a.cu, n, a.d.T);
  return {n, r.bos, r.eos};
}

// A thread's NP pairs of channels in memory.  AL: one aligned access holds them
// all (the host checks); else element by element, the first `n` of them.
template <typename T, int NP, bool AL>
struct Io {
  struct Raw {
    f2 v[NP];
  };
  static __device__ __forceinline__ Raw load(const T *p, int n) {
    Raw r;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      r.v[i] = f2_pack(2 * i < n ? to_f32(p[2 * i]) : 0.f, 2 * i + 1 < n ? to_f32(p[2 * i + 1]) : 0.f);
    return r;
  }
  static __device__ __forceinline__ void expand(const Raw &r, f2 (&v)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) v[i] = r.v[i];
  }
  static __device__ __forceinline__ void store(T *p, int n, const f2 (&v)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float lo, hi;
      f2_split(v[i], lo, hi);
      if (2 * i < n) p[2 * i] = from_f32<T>(lo);
      if (2 * i + 1 < n) p[2 * i + 1] = from_f32<T>(hi);
    }
  }
};
template <int NP>
struct Io<__nv_bfloat16, NP, true> {
  struct __align__(4 * NP) Raw {
    uint32_t u[NP];
  };
  static __device__ __forceinline__ Raw load(const __nv_bfloat16 *p, int) { return *reinterpret_cast<const Raw *>(p); }
  static __device__ __forceinline__ void expand(const Raw &r, f2 (&v)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) v[i] = f2_pack(__uint_as_float(r.u[i] << 16), __uint_as_float(r.u[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, int, const f2 (&v)[NP]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float lo, hi;
      f2_split(v[i], lo, hi);
      r.u[i] = pack_bf16(lo, hi);
    }
    *reinterpret_cast<Raw *>(p) = r;
  }
};
template <int NP>
struct Io<float, NP, true> {
  struct __align__(8 * NP) Raw {
    f2 v[NP];
  };
  static __device__ __forceinline__ Raw load(const float *p, int) { return *reinterpret_cast<const Raw *>(p); }
  static __device__ __forceinline__ void expand(const Raw &r, f2 (&v)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) v[i] = r.v[i];
  }
  static __device__ __forceinline__ void store(float *p, int, const f2 (&v)[NP]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < NP; ++i) r.v[i] = v[i];
    *reinterpret_cast<Raw *>(p) = r;
  }
};

template <typename T, int NP, int W>
struct Taps {
  f2 w[W][NP], bias[NP];
  __device__ __forceinline__ void load(const ConvArgs &a, int64_t e, int n) {
    const bool f32 = a.d.weight_dtype == GDR_F32;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int64_t e0 = e + 2 * i;
      const bool in0 = 2 * i < n, in1 = 2 * i + 1 < n;
#pragma unroll
      for (int j = 0; j < W; ++j)
        w[j][i] = f2_pack(in0 ? param<T>(a.weight, f32, e0 * W + j) : 0.f,
                          in1 ? param<T>(a.weight, f32, (e0 + 1) * W + j) : 0.f);
      bias[i] = f2_pack(in0 && a.bias ? param<T>(a.bias, f32, e0) : 0.f,
                        in1 && a.bias ? param<T>(a.bias, f32, e0 + 1) : 0.f);
    }
  }
  // The filter at the window's last token.
  __device__ __forceinline__ f2 at(const f2 (&win)[W][NP], int i) const {
    f2 v = bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) v = f2_fma(w[j][i], win[j][i], v);
    return v;
  }
};

// The W - 1 inputs before token t of sequence s (x rows, or rows of the state).
template <typename T, int NP, bool AL, int W>
__device__ __forceinline__ void load_window(const ConvArgs &a, const Seq &s, int64_t t, int64_t e, int n,
                                            f2 (&win)[W][NP]) {
  using I = Io<T, NP, AL>;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t u = t - (W - 1) + j;
    if (u >= s.bos) {
      I::expand(I::load(static_cast<const T *>(a.x) + u * a.d.ld_x + e, n), win[j]);
    } else if (a.s0) {
      I::expand(I::load(static_cast<const T *>(a.s0) + (s.n * (W - 1) + (u - s.bos + W - 1)) * a.d.E + e, n), win[j]);
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) win[j][i] = 0;
    }
  }
}

// States of sequences without tokens: `to` = `from` (zero where null).  Run r
// looks after sequences r, r + runs, ...
template <typename T, int NP, bool AL, int W>
__device__ __forceinline__ void copy_empty(const ConvArgs &a, int64_t run, int64_t e, int n, const void *from,
                                           void *to) {
  using I = Io<T, NP, AL>;
  if (!to) return;
  for (int64_t q = run; q < a.d.N; q += a.runs) {
    const SeqRange r = seq_range(a.cu, q, a.d.T);
    if (r.eos > r.bos) continue;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      f2 v[NP] = {};
      const int64_t at = (q * (W - 1) + j) * a.d.E + e;
      if (from) I::expand(I::load(static_cast<const T *>(from) + at, n), v);
      I::store(static_cast<T *>(to) + at, n, v);
    }
  }
}

template <int NP, int W>
__device__ __forceinline__ void shift(f2 (&win)[W][NP]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < NP; ++i) win[j][i] = win[j + 1][i];
}

// Where a thread stands: its first channel, how many it has, its run (or row).
struct Place {
  int64_t e, run;
  int n;
  __device__ __forceinline__ Place(const ConvArgs &a, int vec) {
    e = (int64_t)((blockIdx.x % a.tiles) * a.cx + threadIdx.x % a.cx) * vec;
    run = (int64_t)(blockIdx.x / a.tiles) * (kThreads / a.cx) + threadIdx.x / a.cx;
    n = a.d.E - e < vec ? (int)(a.d.E - e) : vec;
  }
};

template <typename T, int NP, bool AL, int W>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a) {
  using I = Io<T, NP, AL>;
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  const Place p(a, 2 * NP);
  if (p.n <= 0 || p.run >= a.runs) return;
  copy_empty<T, NP, AL, W>(a, p.run, p.e, p.n, a.s0, a.st);
  int64_t t = p.run * a.L;
  const int64_t end = t + a.L < a.M ? t + a.L : a.M;
  if (t >= end) return;
  const bool silu = a.d.activation == GDR_ACT_SILU;
  constexpr int U = 8;  // tokens of a batch
  // counted from the run's first token, in 32 bits; pointers move along
  const int len = (int)(end - t);
  const T *x = static_cast<const T *>(a.x) + t * a.d.ld_x + p.e;
  T *y = static_cast<T *>(a.y) + t * a.d.E + p.e;
  typename I::Raw next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u < len) next[u] = I::load(x, p.n);
    x += a.d.ld_x;
  }
  Taps<T, NP, W> taps;
  taps.load(a, p.e, p.n);
  Seq s = seq_at(a, t);
  int border = s.eos - t <= len ? (int)(s.eos - t) : len + 1;  // where the sequence ends, if it does here
  f2 win[W][NP];
  load_window<T, NP, AL, W>(a, s, t, p.e, p.n, win);
  auto token = [&](const typename I::Raw &in) {
    I::expand(in, win[W - 1]);
    f2 o[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      o[i] = taps.at(win, i);
      if (silu) o[i] = f2_silu(o[i]);
    }
    I::store(y, p.n, o);
    y += a.d.E;
    shift<NP, W>(win);
  };
  for (int q = 0; q < len; q += U) {
    typename I::Raw in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      in[u] = next[u];
      if (q + U + u < len) next[u] = I::load(x, p.n);
      x += a.d.ld_x;
    }
    if (q + U <= len && q + U < border) {  // a whole batch inside one sequence
#pragma unroll
      for (int u = 0; u < U; ++u) token(in[u]);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (q + u < len) {
          if (q + u == border) {  // the next sequence that has tokens starts here
            s = seq_at(a, t + q + u);
            border = s.eos - t <= len ? (int)(s.eos - t) : len + 1;
            load_window<T, NP, AL, W>(a, s, t + q + u, p.e, p.n, win);
          }
          token(in[u]);
          if (a.st && q + u + 1 == border) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
              I::store(static_cast<T *>(a.st) + (s.n * (W - 1) + j) * a.d.E + p.e, p.n, win[j]);
          }
        }
      }
    }
  }
}

// Backward.  A run is taken sequence by sequence; for its tokens [ta, tb) the
// walk goes W - 1 further, because dx_t needs g up to token t + W - 1 (zero past
// the sequence).  At step u the gradient of token u - W + 1 is complete; where
// that is before the sequence it is the gradient of a row of the state.
template <typename T, int NP, bool AL, int W>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvArgs a) {
  using I = Io<T, NP, AL>;
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  const Place p(a, 2 * NP);
  if (p.n <= 0 || p.run >= a.runs) return;
  copy_empty<T, NP, AL, W>(a, p.run, p.e, p.n, a.dst, a.st);
  const int64_t t0 = p.run * a.L, end = t0 + a.L < a.M ? t0 + a.L : a.M;
  const bool silu = a.d.activation == GDR_ACT_SILU;
  Taps<T, NP, W> taps;
  taps.load(a, p.e, p.n);
  f2 dw[W][NP], db[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    db[i] = 0;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0;
  }
  const T *dst = a.dst ? static_cast<const T *>(a.dst) + p.e : nullptr;
  T *ds0 = a.st ? static_cast<T *>(a.st) + p.e : nullptr;
  constexpr int U = 4;
  for (int64_t ta = t0; ta < end;) {
    const Seq s = seq_at(a, ta);
    const int64_t tb = s.eos < end ? s.eos : end;
    // counted from ta, in 32 bits; pointers move along
    const int own = (int)(tb - ta), last = own + W - 1;       // the run's own tokens; one past the last step
    const int eos = s.eos - ta < last ? (int)(s.eos - ta) : last;  // one past the last token read
    const int tail = s.eos - ta - (W - 1) < last ? (int)(s.eos - ta) - (W - 1) : last;  // tokens from here are in st
    const bool begins = ta == s.bos && ds0;
    const T *x = static_cast<const T *>(a.x) + ta * a.d.ld_x + p.e;
    const T *dy = static_cast<const T *>(a.dy) + ta * a.d.ld_dy + p.e;
    T *dx = static_cast<T *>(a.y) + (ta - (W - 1)) * a.d.E + p.e;  // row of the token that step 0 completes
    f2 win[W][NP], g[W][NP];
    typename I::Raw nx[U], ny[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < eos) {
        nx[u] = I::load(x, p.n);
        ny[u] = I::load(dy, p.n);
      }
      x += a.d.ld_x;
      dy += a.d.ld_dy;
    }
    load_window<T, NP, AL, W>(a, s, ta, p.e, p.n, win);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < NP; ++i) g[j][i] = 0;
    // g at a token, from its input and upstream gradient; dw and db where it is one of the run's own
    auto grad = [&](const typename I::Raw &rx, const typename I::Raw &ry, bool mine) {
      I::expand(rx, win[W - 1]);
      I::expand(ry, g[W - 1]);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (silu) g[W - 1][i] = f2_mul(g[W - 1][i], f2_silu_grad(taps.at(win, i)));
        if (mine) {
          db[i] = f2_add(db[i], g[W - 1][i]);
#pragma unroll
          for (int j = 0; j < W; ++j) dw[j][i] = f2_fma(g[W - 1][i], win[j][i], dw[j][i]);
        }
      }
    };
    auto complete = [&](f2 (&o)[NP]) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        o[i] = f2_mul(taps.w[W - 1][i], g[0][i]);
#pragma unroll
        for (int j = 1; j < W; ++j) o[i] = f2_fma(taps.w[W - 1 - j][i], g[j][i], o[i]);
      }
    };
    for (int q0 = 0; q0 < last; q0 += U) {
      typename I::Raw cx[U], cy[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        cx[u] = nx[u];
        cy[u] = ny[u];
        if (q0 + U + u < eos) {
          nx[u] = I::load(x, p.n);
          ny[u] = I::load(dy, p.n);
        }
        x += a.d.ld_x;
        dy += a.d.ld_dy;
      }
      // a whole batch of the run's own tokens that completes none before ta and none of st's
      if (q0 >= W - 1 && q0 + U <= own && q0 + U - (W - 1) <= tail) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          grad(cx[u], cy[u], true);
          f2 o[NP];
          complete(o);
          I::store(dx, p.n, o);
          dx += a.d.E;
          shift<NP, W>(win);
          shift<NP, W>(g);
        }
        continue;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u, to = q - (W - 1);  // `to` is complete now
        if (q >= last) continue;
        if (q < eos) {
          grad(cx[u], cy[u], q < own);
        } else {
#pragma unroll
          for (int i = 0; i < NP; ++i) g[W - 1][i] = 0;
        }
        if (to >= 0 || begins) {
          f2 o[NP];
          complete(o);
          if (dst && to >= tail) {
            f2 v[NP];
            I::expand(I::load(dst + (s.n * (W - 1) + (to - tail)) * a.d.E, p.n), v);
#pragma unroll
            for (int i = 0; i < NP; ++i) o[i] = f2_add(o[i], v[i]);
          }
          if (to >= 0) I::store(dx, p.n, o);
          else I::store(ds0 + (s.n * (W - 1) + (to + W - 1)) * a.d.E, p.n, o);
        }
        dx += a.d.E;
        shift<NP, W>(win);
        shift<NP, W>(g);
      }
    }
    ta = tb;
  }
  if (a.runs == 1) {  // nothing to add up
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float lo, hi;
      const int64_t e = p.e + 2 * i;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        f2_split(dw[j][i], lo, hi);
        if (2 * i < p.n) a.dweight[e * W + j] = lo;
        if (2 * i + 1 < p.n) a.dweight[(e + 1) * W + j] = hi;
      }
      f2_split(db[i], lo, hi);
      if (a.dbias && 2 * i < p.n) a.dbias[e] = lo;
      if (a.dbias && 2 * i + 1 < p.n) a.dbias[e + 1] = hi;
    }
    return;
  }
  using O = Io<float, NP, AL>;
  float *part = a.part + p.run * (W + 1) * a.d.E + p.e;
#pragma unroll
  for (int j = 0; j < W; ++j) O::store(part + j * a.d.E, p.n, dw[j]);
  O::store(part + W * a.d.E, p.n, db);
}

// dweight [E, W] and dbias [E] from the runs' partials: 32 columns a block, SETS
// interleaved sets of runs, each added in order, then the sets in order.
template <int SETS>
__global__ void __launch_bounds__(32 * SETS) conv_sum_kernel(const float *__restrict__ part, int64_t runs, int64_t E,
                                                             int W, float *__restrict__ dweight,
                                                             float *__restrict__ dbias, SeqCheck seqs) {
  __shared__ float sm[SETS][33];
  if (!seqlens_ok(seqs)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (c < E) {
#pragma unroll 4
    for (int64_t r = w; r < runs; r += SETS) acc += part[(r * (W + 1) + j) * E + c];
  }
  sm[w][lane] = acc;
  __syncthreads();
  if (w == 0 && c < E) {
#pragma unroll
    for (int i = 1; i < SETS; ++i) acc += sm[i][lane];
    if (j < W) dweight[c * W + j] = acc;
    else if (dbias) dbias[c] = acc;
  }
}

// One token per row: window from the slot, shifted back with the new input.
template <typename T, int NP, bool AL, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvArgs a) {
  using I = Io<T, NP, AL>;
  const Place p(a, 2 * NP);
  if (p.n <= 0 || p.run >= a.d.B) return;
  int64_t slot = a.slots ? a.slots[p.run] : p.run;
  if (slot >= a.d.N) {
    raise_status(a.status, GDR_ERR_SLOTS);
    slot = -1;
  }
  T *y = static_cast<T *>(a.y) + p.run * a.d.E + p.e;
  f2 o[NP] = {};
  if (slot < 0) {
    I::store(y, p.n, o);
    return;
  }
  T *st = static_cast<T *>(a.st) + slot * (W - 1) * a.d.E + p.e;
  f2 win[W][NP];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) I::expand(I::load(st + j * a.d.E, p.n), win[j]);
  I::expand(I::load(static_cast<const T *>(a.x) + p.run * a.d.ld_x + p.e, p.n), win[W - 1]);
  Taps<T, NP, W> taps;
  taps.load(a, p.e, p.n);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) I::store(st + j * a.d.E, p.n, win[j + 1]);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    o[i] = taps.at(win, i);
    if (a.d.activation == GDR_ACT_SILU) o[i] = f2_silu(o[i]);
  }
  I::store(y, p.n, o);
}

// Threads across channels: a power of two that covers E, a block at most.
int channel_threads(int64_t E, int vec) {
  int cx = 1;
  while (cx < kThreads && (int64_t)cx * vec < E) cx *= 2;
  return cx;
}

template <typename F>
int with_taps(int64_t W, F &&f) {
  if (W == 2) return f(std::integral_constant<int, 2>{});
  if (W == 3) return f(std::integral_constant<int, 3>{});
  return f(std::integral_constant<int, 4>{});
}

enum Dir { kFwd, kBwd, kStep };

// Tokens in a run.  A run reads W - 1 tokens again, loads its weights and leaves
// partials, so it is long; and the grid is whole waves of the blocks that the
// multiprocessors hold at once, as few as keep runs within `hi`.
int64_t run_length(int64_t M, int64_t tiles, int64_t per, int64_t resident, int64_t lo, int64_t hi) {
  const int64_t wave = std::max<int64_t>(1, resident * kSMs / tiles) * per;  // runs at once
  return std::max(lo, cdiv(M, wave * std::max<int64_t>(1, cdiv(M, wave * hi))));
}

// Four channels of a thread in the forward and the step.  The backward keeps
// taps, windows, gradients and their sums of its channels: two of them.
template <typename T, bool AL>
int launch(ConvArgs a, Dir dir, float *dweight, float *dbias, cudaStream_t st) {
  const gdr_conv_desc &d = a.d;
  const int vec = dir == kBwd ? 2 : 4;
  a.cx = channel_threads(d.E, vec);
  const int64_t tiles = cdiv(d.E, (int64_t)vec * a.cx), per = kThreads / a.cx;
  a.tiles = (unsigned)tiles;
  if (dir == kStep) {
    const int64_t blocks = tiles * cdiv(d.B, per);
    if (blocks > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many rows for one launch");
    return with_taps(d.W, [&](auto w) {
      conv_step_kernel<T, 2, AL, decltype(w)::value><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      return launched("conv_step_kernel");
    });
  }
  // blocks on a multiprocessor, by registers: bf16 in whole accesses 96, else up to 117 backward and 154 forward
  constexpr bool kLean = AL && sizeof(T) == 2;
  a.L = (int)(dir == kFwd ? run_length(a.M, tiles, per, kLean ? 5 : 3, 8, 96)
                          : run_length(a.M, tiles, per, kLean ? 5 : 4, 16, 384));
  if (dir == kBwd && a.M <= 64) a.L = 64;  // one run: a second launch and scratch take longer than 64 tokens in a row
  a.runs = std::max<int64_t>(1, cdiv(a.M, a.L));
  const int64_t blocks = tiles * cdiv(a.runs, per);
  if (blocks > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many tokens for one launch");
  if (dir == kFwd) {
    return with_taps(d.W, [&](auto w) {
      conv_fwd_kernel<T, 2, AL, decltype(w)::value><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      return launched("conv_fwd_kernel");
    });
  }
  a.dweight = dweight;
  a.dbias = dbias;
  auto go = [&] {
    return with_taps(d.W, [&](auto w) {
      conv_bwd_kernel<T, 1, AL, decltype(w)::value><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      return launched("conv_bwd_kernel");
    });
  };
  if (a.runs == 1) return go();
  char *base = nullptr;
  int rc = scratch_begin(sizeof(float) * (size_t)(a.runs * (d.W + 1) * d.E), st, "convolution backward scratch", &base);
  if (rc != GDR_OK) return rc;
  a.part = (float *)base;
  rc = go();
  if (rc == GDR_OK) {
    const dim3 grid((unsigned)cdiv(d.E, 32), (unsigned)(d.W + (dbias ? 1 : 0)));
    const SeqCheck seqs{a.cu, d.N, a.M, a.status};
    // small blocks where the columns fill the GPU, else the runs further apart
    if ((int64_t)grid.x * grid.y >= 4 * kSMs)
      conv_sum_kernel<8><<<grid, 256, 0, st>>>(a.part, a.runs, d.E, (int)d.W, dweight, dbias, seqs);
    else
      conv_sum_kernel<32><<<grid, 1024, 0, st>>>(a.part, a.runs, d.E, (int)d.W, dweight, dbias, seqs);
    rc = launched("conv_sum_kernel");
  }
  return scratch_end(base, st, "convolution backward scratch", rc);
}

int validate(const gdr_conv_desc *d, const int64_t *cu, bool step) {
  if (!d) return set_error(GDR_ERR_NULLPTR, "desc is NULL");
  if (d->dtype != GDR_F32 && d->dtype != GDR_BF16) return set_error(GDR_ERR_DTYPE, "dtype must be GDR_F32 or GDR_BF16");
  if (d->weight_dtype != d->dtype && d->weight_dtype != GDR_F32)
    return set_error(GDR_ERR_DTYPE, "weight and bias must be of the input dtype or fp32");
  if (d->activation != GDR_ACT_NONE && d->activation != GDR_ACT_SILU)
    return set_error(GDR_ERR_DTYPE, "unknown activation");
  if (d->flags) return set_error(GDR_ERR_DTYPE, "unknown bits in flags");
  if (d->W < 2 || d->W > 4) return set_error(GDR_ERR_SHAPE, "W must be in [2, 4]");
  if (d->B < 0 || d->T < 0 || d->N < 0) return set_error(GDR_ERR_SHAPE, "B, T and N must be >= 0");
  if (d->E < 1 || d->E > (1 << 24)) return set_error(GDR_ERR_SHAPE, "E must be in [1, 2^24]");
  if (d->ld_x < d->E || d->ld_dy < d->E) return set_error(GDR_ERR_SHAPE, "leading dimensions must be at least E");
  if (step) return d->T == 1 ? GDR_OK : set_error(GDR_ERR_SHAPE, "a step takes one token per row: T must be 1");
  if (cu) {
    if (d->B != 1) return set_error(GDR_ERR_SHAPE, "cu_seqlens requires B == 1");
  } else if (d->N != d->B) {
    return set_error(GDR_ERR_SHAPE, "N must equal B when cu_seqlens is NULL");
  }
  return GDR_OK;
}

int run(ConvArgs a, Dir dir, float *dweight, float *dbias, void *stream) {
  int rc;
  a.M = a.d.B * a.d.T;
  a.status = current_status_word(&rc);
  if (!a.status) return rc;
  const bool al = a.d.E % 4 == 0 && a.d.ld_x % 4 == 0 && a.d.ld_dy % 4 == 0 && is_aligned16(a.x) &&
                  is_aligned16(a.s0) && is_aligned16(a.dy) && is_aligned16(a.dst) && is_aligned16(a.y) &&
                  is_aligned16(a.st);
  cudaStream_t st = (cudaStream_t)stream;
  if (a.d.dtype == GDR_BF16)
    return al ? launch<__nv_bfloat16, true>(a, dir, dweight, dbias, st)
              : launch<__nv_bfloat16, false>(a, dir, dweight, dbias, st);
  return al ? launch<float, true>(a, dir, dweight, dbias, st) : launch<float, false>(a, dir, dweight, dbias, st);
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_conv_fwd(const gdr_conv_desc *desc, const void *x, const void *weight, const void *bias, const void *s0,
                 const int64_t *cu_seqlens, void *y, void *st, void *stream) {
  int rc = validate(desc, cu_seqlens, false);
  if (rc != GDR_OK) return rc;
  if (desc->N == 0 && !cu_seqlens) return GDR_OK;
  if (!weight || (desc->B * desc->T > 0 && (!x || !y)))
    return set_error(GDR_ERR_NULLPTR, "x, weight and y must be non-NULL");
  ConvArgs a{};
  a.d = *desc;
  a.x = x; a.weight = weight; a.bias = bias; a.s0 = s0; a.cu = cu_seqlens; a.y = y; a.st = st;
  return run(a, kFwd, nullptr, nullptr, stream);
}

int gdr_conv_bwd(const gdr_conv_desc *desc, const void *x, const void *weight, const void *bias, const void *s0,
                 const int64_t *cu_seqlens, const void *dy, const void *dst, void *dx, float *dweight, float *dbias,
                 void *ds0, void *stream) {
  int rc = validate(desc, cu_seqlens, false);
  if (rc != GDR_OK) return rc;
  if (!weight || !dweight || (desc->B * desc->T > 0 && (!x || !dy || !dx)))
    return set_error(GDR_ERR_NULLPTR, "x, weight, dy, dx and dweight must be non-NULL");
  ConvArgs a{};
  a.d = *desc;
  a.x = x; a.weight = weight; a.bias = bias; a.s0 = s0; a.cu = cu_seqlens; a.dy = dy; a.dst = dst; a.y = dx; a.st = ds0;
  return run(a, kBwd, dweight, dbias, stream);
}

int gdr_conv_step(const gdr_conv_desc *desc, const void *x, const void *weight, const void *bias,
                  const int32_t *slots, void *state, void *y, void *stream) {
  int rc = validate(desc, nullptr, true);
  if (rc != GDR_OK) return rc;
  if (desc->B == 0) return GDR_OK;
  if (!x || !weight || !state || !y) return set_error(GDR_ERR_NULLPTR, "x, weight, state and y must be non-NULL");
  ConvArgs a{};
  a.d = *desc;
  a.x = x; a.weight = weight; a.bias = bias; a.slots = slots; a.st = state; a.y = y;
  return run(a, kStep, nullptr, nullptr, stream);
}

}  // extern "C"
