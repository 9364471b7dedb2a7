// gdr_ssm_bwd.cu -- backward of the selective state space scan.
//
// With up_t = dy_t silu(z_t), a_t = exp(delta_t a) and g_t = dL/dh_t,
//   g_t = c_t up_t + a_{t+1} g_{t+1}        (g of the last token also takes dht)
//   dc_t = sum_e up_t h_t                    db_t = sum_e g_t delta_t x_t
//   q_t = g_t a_t h_{t-1}                    da = sum_t q_t delta_t
//   dx_t = d up_t + delta_t sum_s g_t b_t    ddelta_t = sum_s q_t a + x_t sum_s g_t b_t
//   dz_t = dy_t silu'(z_t) (sum_s c_t h_t + d x_t),  dh0 = a_0 g_0
//
// Launches (chunks of L <= 64 tokens, gdr_ssm.cuh):
//   local   per (chunk, channels): the chunk's state from zero, and what its own
//           tokens give to the gradient of the state entering it (forwards, times the
//           product of decays; backwards where that leaves fp32's range)
//   carry   per (channel, state): the state entering each chunk (forwards) and the
//           gradient reaching its end from later chunks (backwards), in order
//   main    per (chunk, channels): the states again, kept every 8 tokens in shared
//           memory; then 8 tokens at a time from the last: the states once more,
//           in registers, and the reverse recurrence with all products
//   sums    the partials of db and dc over channels, of da, dd and ddt_bias over chunks
// (one chunk needs no local and carry).
// States are recomputed, never inverted: h_{t-1} = (h_t - ..) / a_t loses what a
// small a_t has forgotten.  The work is arithmetic: four exponentials and about
// 25 fp32 operations per channel, state and token, some 250 instructions per
// token of a thread's eight states.  16384 tokens x 2048 channels x 16 states take
// 1129 us, four fifths of it main, which issues on 49 % of cycles with the fp32 pipe
// 36 % and the exponential unit 20 % busy: its 12 warps a multiprocessor wait for
// shared memory, shuffles and values just computed.
#include <algorithm>

#include "gdr_ssm.cuh"

namespace gdr {
namespace {

constexpr int kSub = 8;      // tokens whose states a thread holds in registers
constexpr int kMaxL = 64;    // tokens of a chunk
constexpr int kSubs = kMaxL / kSub;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T, typename P, bool VEC>
struct __align__(16) LocalShared {
  Ahead<T, VEC ? 4 : 1, VEC ? Stager<kTile, P::CB, P::kThreads>::kCount : 1, VEC ? P::kThreads : 1> ahead;
  float delta[kTile][P::CB], x[kTile][P::CB], up[kTile][P::CB];
  float bias[P::CB];
  float b[kTile * P::SP], c[kTile * P::SP];
  Borders<kTile> bd;
  unsigned signs;  // of the deltas, where they come without softplus: 1 some are negative, 2 some positive
};

// Keeps the signs of eight deltas.
__device__ __forceinline__ void note_signs(const Eight &v, unsigned *signs) {
  unsigned found = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x, y;
    f2_split(v[i], x, y);
    found |= (x < 0.f || y < 0.f ? 1u : 0u) | (x > 0.f || y > 0.f ? 2u : 0u);
  }
  atomicOr(signs, found);
}

// Eight columns of token t, n of them inside the group.
template <typename T, bool VEC>
__device__ __forceinline__ void fetch8(const void *src, int64_t ld, int64_t t, int64_t e, int n, Eight &v) {
  Raw8<T, VEC> r;
  r.load(static_cast<const T *>(src) + t * ld + e, n);
  r.expand(v);
}

// The sequence that enters a chunk, and its tokens [begin, stop) there (none where a
// sequence starts with the chunk).
struct Entering {
  int64_t n, begin, stop;
  bool ends;  // in the chunk
  __device__ __forceinline__ Entering(const SsmArgs &a, int64_t chunk) {
    begin = chunk * a.L;
    const int64_t end = begin + a.L < a.M ? begin + a.L : a.M;
    n = seq_of_token(a.cu, a.d.N, a.d.T, begin);
    const SeqRange r = seq_range(a.cu, n, a.d.T);
    stop = r.bos == begin ? begin : r.eos < end ? r.eos : end;
    ends = r.bos < begin && r.eos <= end;
  }
};

// The local pass sums the gradient entering a chunk forwards, each token's part times
// the product of the decays so far.  Where a state grows, that product can leave
// fp32's range and the gradient not.  Such gradients of a thread's channels and states
// are worked out again from the last token back, one decay at a time, as main does it:
// all of them where one is not finite (`all`); else, of raw deltas with both signs,
// those whose product may have been below fp32's range and come back with what was left
// of it.  A call that finds its place again, so that local holds no registers for it.
template <typename T, int SL>
__device__ __noinline__ void redo_entering(const SsmArgs &a, bool all) {
  const Place<SL> p(a);
  const Entering in(a, p.chunk);
  const int s0 = p.sl * 4;
  const T *c = static_cast<const T *>(a.c) + p.g * a.d.S + s0;
  for (int64_t e = p.e0 + p.col; e < p.e0 + p.col + 4 && e < p.e_end; ++e) {
    const float bias = a.dt_bias ? a.dt_bias[e] : 0.f;
    auto raw = [&](int64_t t) { return to_f32(static_cast<const T *>(a.dt)[t * a.d.ld_dt + e]) + bias; };
    float reach = CUDART_INF_F;
    if (!all) {  // the furthest from zero that the sums of delta come
      float sum = 0.f, far = 0.f, low = 0.f, high = 0.f;
#pragma unroll 4
      for (int64_t t = in.begin; t < in.stop; ++t) {
        const float v = raw(t);
        low = fminf(low, v);
        high = fmaxf(high, v);
        sum += v;
        far = fmaxf(far, fabsf(sum));
      }
      reach = low < 0.f && high > 0.f ? far : 0.f;
    }
    float A[4], g[4] = {};
    bool some = false;
    load_states(a.a + e * a.d.S, s0, (int)a.d.S, 0, A);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      A[s] *= kLog2e;
      some |= !(fabsf(A[s]) * reach < 126.f);
    }
    if (!some) continue;
    if (a.dht && in.ends) load_states(a.dht + (in.n * a.d.E + e) * a.d.S, s0, (int)a.d.S, 0, g);
    for (int64_t t = in.stop - 1; t >= in.begin; --t) {
      const float delta = ssm_delta(raw(t), a.d.flags & GDR_SSM_SOFTPLUS);
      float up = to_f32(static_cast<const T *>(a.dy)[t * a.d.ld_dy + e]);
      if (a.z) {
        const float z = to_f32(static_cast<const T *>(a.z)[t * a.d.ld_z + e]);
        up *= z * sigmoid_fast(z);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (s0 + s < a.d.S) g[s] = ex2(A[s] * delta) * fmaf(to_f32(c[t * a.d.ld_c + s]), up, g[s]);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (!(fabsf(A[s]) * reach < 126.f)) a.gloc[(p.chunk * a.d.E + e) * p.SP + s0 + s] = g[s];
  }
}

template <typename T, int SL, bool VEC>
__global__ void __launch_bounds__(kSsmThreads, 4) ssm_bwd_local_kernel(const __grid_constant__ SsmArgs a) {
  using P = Place<SL>;
  constexpr bool kAhead = VEC && sizeof(T) == 2;
  __shared__ LocalShared<T, P, VEC> sm;
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  const P p(a);
  const Stager<kTile, P::CB, P::kThreads> st(p);
  const int64_t begin = p.chunk * a.L, end = begin + a.L < a.M ? begin + a.L : a.M;
  const void *const src[4] = {a.x, a.dt, a.dy, a.z};
  const int64_t lds[4] = {a.d.ld_x, a.d.ld_dt, a.d.ld_dy, a.d.ld_z};
  auto columns = [&](int64_t t0, int k) { return st.has(k) && st.token(k) < end - t0 ? st.n : 0; };
  auto fetch_ahead = [&](int64_t t0) {
#pragma unroll
    for (int k = 0; k < st.kCount; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (src[i])
          sm.ahead.fetch(i, k, static_cast<const T *>(src[i]) + (t0 + st.token(k)) * lds[i] + p.e0 + st.col,
                         columns(t0, k));
    copy_commit();
  };
  if constexpr (kAhead) {
    if (begin < end) fetch_ahead(begin);
  }
  stage_row<P::CB, P::kThreads>(p, a.dt_bias, sm.bias);
  if (threadIdx.x == 0) sm.signs = 0;
  __syncthreads();
  // pass: product of the decays since the chunk began.  What a sequence that starts
  // in the chunk holds is no part of the gradient entering it, and is left out, not
  // multiplied by zero: it need not be finite.
  States A, h, g, pass;
  load_a(a, p, A);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      h[i][s] = g[i][s] = 0;
      pass[i][s] = f2_pack(1.f, 1.f);
    }
  f2 sum[2] = {0, 0};
  bool started = false;
  auto token = [&](int t) {  // before a sequence has started
    const Pairs<2> delta(&sm.delta[t][p.col]), x(&sm.x[t][p.col]), up(&sm.up[t][p.col]);
    const Twice b(&sm.b[t * P::SP + p.sl * 4]), c(&sm.c[t * P::SP + p.sl * 4]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f2 u = f2_mul(delta.v[i], x.v[i]);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const f2 at = f2_ex2(f2_mul(A[i][s], delta.v[i]));
        h[i][s] = f2_fma(at, h[i][s], f2_mul(u, b.v[s]));
        pass[i][s] = f2_mul(pass[i][s], at);
        g[i][s] = f2_fma(pass[i][s], f2_mul(up.v[i], c.v[s]), g[i][s]);
      }
      sum[i] = f2_add(sum[i], delta.v[i]);
    }
  };
  auto state_only = [&](int t) {
    advance(h, A, Pairs<2>(&sm.delta[t][p.col]), Pairs<2>(&sm.x[t][p.col]), Twice(&sm.b[t * P::SP + p.sl * 4]));
  };
  int64_t bos = -1, eos = -1;  // of the sequence that the tile begins in
  for (int64_t t0 = begin; t0 < end; t0 += kTile) {
    const int nt = end - t0 < kTile ? (int)(end - t0) : kTile;
    if (t0 >= eos) {
      const SeqRange r = seq_range(a.cu, seq_of_token(a.cu, a.d.N, a.d.T, t0), a.d.T);
      bos = r.bos;
      eos = r.eos;
    }
    const bool borders = bos >= t0 || eos <= t0 + nt;  // a sequence starts or ends in the tile
    __syncthreads();                                   // the previous tile is consumed
    if (borders) stage_borders(a, t0, nt, sm.bd);
    if (kAhead) copy_wait<0>();
    auto get = [&](int i, int k, Eight &v) {
      if constexpr (kAhead) sm.ahead.get(i, k, v);
      else fetch8<T, VEC>(src[i], lds[i], t0 + st.token(k), p.e0 + st.col, columns(t0, k), v);
    };
#pragma unroll
    for (int k = 0; k < st.kCount; ++k) {
      if (!st.has(k)) continue;
      const int t = st.token(k);
      Eight v, w;
      get(0, k, v);
      put8(&sm.x[t][st.col], v);
      get(1, k, v);
      get8(&sm.bias[st.col], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2_delta(f2_add(v[i], w[i]), a.d.flags & GDR_SSM_SOFTPLUS);
      put8(&sm.delta[t][st.col], v);
      if (!(a.d.flags & GDR_SSM_SOFTPLUS)) note_signs(v, &sm.signs);
      get(2, k, v);
      if (a.z) {
        get(3, k, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f2_mul(v[i], f2_silu(w[i]));
      }
      put8(&sm.up[t][st.col], v);
    }
    stage_states<T, kTile, P::kThreads>(a, p, a.b, a.d.ld_b, t0, nt, sm.b);
    stage_states<T, kTile, P::kThreads>(a, p, a.c, a.d.ld_c, t0, nt, sm.c);
    if constexpr (kAhead) {
      if (t0 + kTile < end) fetch_ahead(t0 + kTile);
    }
    __syncthreads();
    if (!borders && nt == kTile && !started) {
#pragma unroll 4
      for (int t = 0; t < kTile; ++t) token(t);
    } else {
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        if (borders && sm.bd.first[t] >= 0) {
          load_h0(a, p, a.h0, sm.bd.first[t], h);
          started = true;
        }
        if (started) state_only(t);
        else token(t);
        if (a.dht && !started && borders && sm.bd.last[t] >= 0) {
          States dh;
          load_h0(a, p, a.dht, sm.bd.last[t], dh);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) g[i][s] = f2_fma(pass[i][s], dh[i][s], g[i][s]);
        }
      }
    }
  }
  store_chunk(a, p, a.hloc, p.chunk, h);
  store_chunk(a, p, a.gloc, p.chunk, g);
  f2 zero = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) zero = f2_fma(g[i][s], 0, zero);
  float lo, hi;
  f2_split(zero, lo, hi);
  const bool all = !(lo == 0.f && hi == 0.f);  // some g is not finite
  const int mine = p.sl & 3;
  const int64_t e_mine = p.e0 + p.col + mine;
  if (p.sl < 4 && e_mine < p.e_end) {
    float s[4];
    f2_split(sum[0], s[0], s[1]);
    f2_split(sum[1], s[2], s[3]);
    const float mine_sum = mine == 0 ? s[0] : mine == 1 ? s[1] : mine == 2 ? s[2] : s[3];
    a.sumd[p.chunk * a.d.E + e_mine] = started ? CUDART_NAN_F : mine_sum;  // NaN: nothing passes through
  }
  if (all || sm.signs == 3) redo_entering<T, SL>(a, all);
}

// In place: blockIdx.y 0 turns hloc[c] into the state entering chunk c, 1 turns
// gloc[c] into the gradient that reaches the end of chunk c from later chunks.
constexpr int kCarryBatch = 16;
__global__ void __launch_bounds__(128) ssm_bwd_carry_kernel(SsmArgs a, int SP) {
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (i >= a.d.E * SP) return;
  const int64_t e = i / SP, row = a.d.E * SP;
  const int s = (int)(i % SP);
  const bool back = blockIdx.y == 1;
  float *v = (back ? a.gloc : a.hloc) + i;
  const float A = s < a.d.S ? a.a[e * a.d.S + s] * kLog2e : 0.f;
  float acc = 0.f;
  for (int64_t c0 = 0; c0 < a.chunks; c0 += kCarryBatch) {
    float loc[kCarryBatch], sum[kCarryBatch];
#pragma unroll
    for (int k = 0; k < kCarryBatch; ++k) {
      const int64_t c = back ? a.chunks - 1 - (c0 + k) : c0 + k;
      const bool in = c0 + k < a.chunks;
      loc[k] = in ? v[c * row] : 0.f;
      sum[k] = in ? a.sumd[c * a.d.E + e] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kCarryBatch; ++k) {
      const int64_t c = back ? a.chunks - 1 - (c0 + k) : c0 + k;
      if (c0 + k < a.chunks) {
        v[c * row] = acc;
        acc = isnan(sum[k]) ? loc[k] : carry_over(A * sum[k], acc, loc[k]);
      }
    }
  }
}

// Main: two channels to a thread, where the other kernels have four: the states
// of eight tokens held back take half the registers and the unrolled code half
// the instructions.  Blocks of four warps, three on a multiprocessor at 168
// registers, were the best of three on 16384 tokens of 2048 channels, before rows were
// copied ahead: the whole backward took 1178 us, with four at 128, which spill, 1198 us,
// with two of eight warps 1219 us.
constexpr int kMainWarps = 4;
template <int SL>
using MainPlace = Place<SL, 1, kMainWarps>;

template <typename T, typename P, bool VEC>
struct MainShared {
  // x and dt, or dy and z, of the thread's eight columns in the next run
  Ahead<T, VEC ? 2 : 1, 1, VEC ? P::kThreads : 1> ahead;
  ulonglong2 ckpt[kSubs - 1][2][P::kThreads];  // a thread's states before each run of kSub tokens but the first
  union {
    struct {
      float delta[kTile][P::CB], x[kTile][P::CB];
      float b[kTile * P::SP];
    } f;
    struct {
      float delta[kSub][P::CB], x[kSub][P::CB], up[kSub][P::CB], slope[kSub][P::CB], zf[kSub][P::CB];
      float b[kSub * P::SP], c[kSub * P::SP];
    } r;
  };
  float sums[3][kSub][P::CB];  // per channel and token, over the states: c . h, b . g, a . q
  float bias[P::CB], skip[P::CB];
  float total[2][kSub][P::CB];  // ddt and up x over the chunk, by column and thread row
  float red[kSub][kMainWarps][2 * P::SP];  // db, dc of a token by warp
  Borders<kMaxL> bd;
  unsigned border_mask[kMaxL / 32];
};

// A thread's token and eight columns of a run or tile, and their loads: two
// arrays p0 and p1, ahead of their use where that is worth it (gdr_ssm.cuh).
template <typename T, typename P, bool VEC>
struct MainLoads {
  static constexpr bool kAhead = VEC && sizeof(T) == 2;
  const SsmArgs &a;
  const P &p;
  MainShared<T, P, VEC> &sm;
  int t, col;
  __device__ __forceinline__ int columns(int nt) const {
    const int64_t left = p.e_end - p.e0 - col;
    return t >= nt || left < 0 ? 0 : left < 8 ? (int)left : 8;
  }
  __device__ __forceinline__ const T *at(const void *src, int64_t ld, int64_t t0) const {
    return static_cast<const T *>(src) + (t0 + t) * ld + p.e0 + col;
  }
  __device__ __forceinline__ void fetch(const void *p0, int64_t ld0, const void *p1, int64_t ld1, int64_t t0,
                                        int nt) const {
    if constexpr (kAhead) {
      const int n = columns(nt);
      sm.ahead.fetch(0, 0, at(p0, ld0, t0), n);
      if (p1) sm.ahead.fetch(1, 0, at(p1, ld1, t0), n);
      copy_commit();
    }
  }
  __device__ __forceinline__ void get(int which, const void *src, int64_t ld, int64_t t0, int nt, Eight &v) const {
    if constexpr (kAhead) sm.ahead.get(which, 0, v);
    else fetch8<T, VEC>(src, ld, t0 + t, p.e0 + col, columns(nt), v);
  }
};

// dt as it is read becomes delta, and where asked its slope.
template <bool SLOPE, typename P>
__device__ __forceinline__ void to_delta(const SsmArgs &a, const float *bias, Eight &v, Eight &slope) {
  Eight w;
  get8(bias, w);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = f2_delta<SLOPE>(f2_add(v[i], w[i]), a.d.flags & GDR_SSM_SOFTPLUS, &slope[i]);
}

// Eight columns to memory, n of them inside the group.
template <typename T, bool VEC>
__device__ __forceinline__ void store_columns(T *p, int n, const Eight &v) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_split(v[i], f[2 * i], f[2 * i + 1]);
  if (VEC && sizeof(T) == 4) {
    const float lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
    if (n > 0) store4(p, lo);
    if (n > 4) store4(p + 4, hi);
  } else if (VEC) {
    if (n > 0) store8(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(f[i]);
  }
}

// The gradients of a run's tokens from the sums over states, by the threads that
// staged them: dx and ddt by the first half of the block, dz by the second.
template <typename T, typename P, bool VEC>
__device__ __forceinline__ void finish(const SsmArgs &a, const P &p, int64_t t0, int nt, MainShared<T, P, VEC> &sm) {
  constexpr int kHalf = P::kThreads / 2, kRow = P::CB / 8;
  const int half = threadIdx.x / kHalf, i0 = threadIdx.x % kHalf, t = i0 / kRow, col = i0 % kRow * 8;
  if (t >= nt) return;
  const int64_t e = p.e0 + col, left = p.e_end - e, at = (t0 + t) * a.d.E + e;
  const int n = left < 0 ? 0 : left < 8 ? (int)left : 8;
  Eight x, up, o, v, w, skip, total;
  get8(&sm.r.x[t][col], x);
  get8(&sm.r.up[t][col], up);
  get8(&sm.skip[col], skip);
  get8(&sm.total[half][t][col], total);
  if (half == 0) {
    get8(&sm.r.delta[t][col], v);
    get8(&sm.sums[1][t][col], w);  // b . g
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f2_fma(skip[i], up[i], f2_mul(v[i], w[i]));
    store_columns<T, VEC>(static_cast<T *>(a.dx) + at, n, o);
    get8(&sm.sums[2][t][col], v);  // a . q, where a carries log2(e)
    get8(&sm.r.slope[t][col], o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = f2_mul(o[i], f2_fma(x[i], w[i], f2_mul(v[i], f2_both(kLn2))));
      total[i] = f2_add(total[i], o[i]);
    }
    store_columns<T, VEC>(static_cast<T *>(a.ddt) + at, n, o);
  } else {
    if (a.dz) {
      get8(&sm.sums[0][t][col], v);  // c . h
      get8(&sm.r.zf[t][col], o);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = f2_mul(o[i], f2_fma(skip[i], x[i], v[i]));
      store_columns<T, VEC>(static_cast<T *>(a.dz) + at, n, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) total[i] = f2_fma(up[i], x[i], total[i]);
  }
  put8(&sm.total[half][t][col], total);
}

// Sums v[0..7] (db of the thread's four states, then dc) over the channel lanes
// of a warp, halving the values a lane holds at each step, and leaves them in
// out[2 * SP] (db, then dc).
template <typename P>
__device__ __forceinline__ void sum_over_channels(float (&v)[8], const P &p, float *out) {
  constexpr int SP = P::SP, CL = 32 / P::SL;
  int base = 0;  // which of the eight the lane holds first
  int n = 8;
#pragma unroll
  for (int o = CL / 2; o > 0; o >>= 1) {
    n /= 2;
    const bool up = p.cl & o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < n) {
        const float keep = up ? v[n + i] : v[i], give = up ? v[i] : v[n + i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o * P::SL);
      }
    }
    base += up ? n : 0;
  }
#pragma unroll
  for (int i = 0; i < 8 / CL; ++i) {
    const int k = base + i;
    out[(k >> 2) * SP + p.sl * 4 + (k & 3)] = v[i];
  }
}

template <typename T, int SL, bool VEC>
__global__ void __launch_bounds__(32 * kMainWarps, 3) ssm_bwd_main_kernel(SsmArgs a) {
  using P = MainPlace<SL>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  MainShared<T, P, VEC> &sm = *reinterpret_cast<MainShared<T, P, VEC> *>(smem_raw);
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  const P p(a);
  const int tid = threadIdx.x;
  copy_empty_states(a, p, a.dht, a.dh0);
  {  // The runs below wait for their rows one after the other: ask L2 for all of them now.
    constexpr int kLine = 128 / sizeof(T), kLines = (P::CB + kLine - 1) / kLine;
    const int64_t t0 = p.chunk * a.L, left = a.M - t0;
    const int tokens = left < a.L ? (left > 0 ? (int)left : 0) : (int)a.L;
    for (int i = tid; i < tokens * kLines; i += P::kThreads) {
      const int64_t t = t0 + i / kLines, e = p.e0 + i % kLines * kLine;
      if (e >= p.e_end) continue;
      prefetch_l2(static_cast<const T *>(a.x) + t * a.d.ld_x + e);
      prefetch_l2(static_cast<const T *>(a.dt) + t * a.d.ld_dt + e);
      prefetch_l2(static_cast<const T *>(a.dy) + t * a.d.ld_dy + e);
      if (a.z) prefetch_l2(static_cast<const T *>(a.z) + t * a.d.ld_z + e);
    }
  }
  StatesOf<1> A, h, g, dA;
  load_a(a, p, A);
  const float *entering = a.chunks > 1 ? a.hloc : nullptr;
  load_chunk(a, p, entering, p.chunk, h);
  load_chunk(a, p, a.chunks > 1 ? a.gloc : nullptr, p.chunk, g);
#pragma unroll
  for (int s = 0; s < 4; ++s) dA[0][s] = 0;
  const int64_t begin = p.chunk * a.L, end = begin + a.L < a.M ? begin + a.L : a.M;
  const int len = end > begin ? (int)(end - begin) : 0;
  const int subs = (len + kSub - 1) / kSub;
  stage_row<P::CB, P::kThreads>(p, a.dt_bias, sm.bias);
  stage_row<P::CB, P::kThreads>(p, a.dskip, sm.skip);
  for (int i = tid; i < 2 * kSub * P::CB; i += P::kThreads) (&sm.total[0][0][0])[i] = 0.f;
  const bool borders = stage_borders(a, begin, len, sm.bd);
  if (tid < 2) sm.border_mask[tid] = 0;
  __syncthreads();
  if (borders) atomicOr(&sm.border_mask[tid >> 5], 1u << (tid & 31));  // tokens that start or end a sequence

  auto keep = [&](int sub) {
    sm.ckpt[sub - 1][0][tid] = make_ulonglong2(h[0][0], h[0][1]);
    sm.ckpt[sub - 1][1][tid] = make_ulonglong2(h[0][2], h[0][3]);
  };
  auto back_to = [&](int sub, StatesOf<1> &to) {
    if (sub == 0) {
      load_chunk(a, p, entering, p.chunk, to);
      return;
    }
    const ulonglong2 u = sm.ckpt[sub - 1][0][tid], v = sm.ckpt[sub - 1][1][tid];
    to[0][0] = u.x;
    to[0][1] = u.y;
    to[0][2] = v.x;
    to[0][3] = v.y;
  };

  // States at the start of every run of kSub tokens; the last run needs only its start.
  const int flen = subs > 0 ? (subs - 1) * kSub : 0;
  constexpr int kRow = P::CB / 8, kHalf = P::kThreads / 2;
  {
    const MainLoads<T, P, VEC> ld{a, p, sm, tid / kRow, tid % kRow * 8};
    if (flen > 0) ld.fetch(a.x, a.d.ld_x, a.dt, a.d.ld_dt, begin, flen < kTile ? flen : kTile);
    for (int f0 = 0; f0 < flen; f0 += kTile) {
      const int nt = flen - f0 < kTile ? flen - f0 : kTile;
      __syncthreads();
      if (ld.kAhead) copy_wait<0>();
      if (ld.t < kTile) {
        Eight v, none;
        ld.get(0, a.x, a.d.ld_x, begin + f0, nt, v);
        put8(&sm.f.x[ld.t][ld.col], v);
        ld.get(1, a.dt, a.d.ld_dt, begin + f0, nt, v);
        to_delta<false, P>(a, &sm.bias[ld.col], v, none);
        put8(&sm.f.delta[ld.t][ld.col], v);
      }
      stage_states<T, kTile, P::kThreads>(a, p, a.b, a.d.ld_b, begin + f0, nt, sm.f.b);
      const int rest = flen - f0 - kTile;
      if (rest > 0) ld.fetch(a.x, a.d.ld_x, a.dt, a.d.ld_dt, begin + f0 + kTile, rest < kTile ? rest : kTile);
      __syncthreads();
#pragma unroll 1
      for (int t1 = 0; t1 < nt; t1 += kSub) {
#pragma unroll 4
        for (int t = t1; t < t1 + kSub; ++t) {
          if (sm.bd.first[f0 + t] >= 0) load_h0(a, p, a.h0, sm.bd.first[f0 + t], h);
          advance(h, A, Pairs<1>(&sm.f.delta[t][p.col]), Pairs<1>(&sm.f.x[t][p.col]),
                  Twice(&sm.f.b[t * P::SP + p.sl * 4]));
        }
        keep((f0 + t1) / kSub + 1);
      }
    }
  }

  // The first half of the block stages x and dt of a run, the second dy and z.
  const int half = tid / kHalf;
  const MainLoads<T, P, VEC> ld{a, p, sm, tid % kHalf / kRow, tid % kHalf % kRow * 8};
  auto fetch = [&](int sub) {
    const int nt = len - sub * kSub < kSub ? len - sub * kSub : kSub;
    if (half == 0) ld.fetch(a.x, a.d.ld_x, a.dt, a.d.ld_dt, begin + sub * kSub, nt);
    else ld.fetch(a.dy, a.d.ld_dy, a.z, a.d.ld_z, begin + sub * kSub, nt);
  };
  if (subs > 0) fetch(subs - 1);
#pragma unroll 1
  for (int sub = subs - 1; sub >= 0; --sub) {
    const int64_t t0 = begin + sub * kSub;
    const int nt = len - sub * kSub < kSub ? len - sub * kSub : kSub;
    __syncthreads();  // the previous run's staging and partials are consumed
    if (ld.kAhead) copy_wait<0>();
    if (ld.t < kSub) {
      Eight v, w, o;
      if (half == 0) {
        ld.get(0, a.x, a.d.ld_x, t0, nt, v);
        put8(&sm.r.x[ld.t][ld.col], v);
        ld.get(1, a.dt, a.d.ld_dt, t0, nt, v);
        to_delta<true, P>(a, &sm.bias[ld.col], v, w);
        put8(&sm.r.delta[ld.t][ld.col], v);
        put8(&sm.r.slope[ld.t][ld.col], w);
      } else {
        ld.get(0, a.dy, a.d.ld_dy, t0, nt, v);
        if (a.z) {
          ld.get(1, a.z, a.d.ld_z, t0, nt, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = f2_mul(v[i], f2_silu_grad(w[i]));
          put8(&sm.r.zf[ld.t][ld.col], o);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = f2_mul(v[i], f2_silu(w[i]));
        }
        put8(&sm.r.up[ld.t][ld.col], v);
      }
    }
    stage_states<T, kSub, P::kThreads>(a, p, a.b, a.d.ld_b, t0, nt, sm.r.b);
    stage_states<T, kSub, P::kThreads>(a, p, a.c, a.d.ld_c, t0, nt, sm.r.c);
    if (sub > 0) fetch(sub - 1);
    __syncthreads();
    // the reverse recurrence at token k, from the states before and after it
    auto reverse = [&](int k, const StatesOf<1> &prev, const StatesOf<1> &after) {
      asm volatile("" ::: "memory");  // one token's values at a time: loads moved up from later ones spill
      const f2 delta = Pairs<1>(&sm.r.delta[k][p.col]).v[0], up = Pairs<1>(&sm.r.up[k][p.col]).v[0];
      const f2 u = f2_mul(delta, Pairs<1>(&sm.r.x[k][p.col]).v[0]);
      const Twice b(&sm.r.b[k * P::SP + p.sl * 4]), c(&sm.r.c[k * P::SP + p.sl * 4]);
      f2 sy = 0, sb = 0, sq = 0;
      float v[8];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float lo, hi;
        g[0][s] = f2_fma(c.v[s], up, g[0][s]);
        f2_split(f2_mul(u, g[0][s]), lo, hi);
        v[s] = lo + hi;  // db
        f2_split(f2_mul(up, after[0][s]), lo, hi);
        v[4 + s] = lo + hi;  // dc
        sy = s ? f2_fma(c.v[s], after[0][s], sy) : f2_mul(c.v[s], after[0][s]);
        sb = s ? f2_fma(b.v[s], g[0][s], sb) : f2_mul(b.v[s], g[0][s]);
        g[0][s] = f2_mul(g[0][s], f2_ex2(f2_mul(A[0][s], delta)));
        const f2 q = f2_mul(g[0][s], prev[0][s]);
        dA[0][s] = f2_fma(q, delta, dA[0][s]);
        sq = s ? f2_fma(q, A[0][s], sq) : f2_mul(q, A[0][s]);
      }
      float yg[4], qa[2];
      f2_split(sy, yg[0], yg[1]);
      f2_split(sb, yg[2], yg[3]);
      f2_split(sq, qa[0], qa[1]);
      const float ygsum = sum_over_states<SL>(yg, p.sl);  // lanes 0, 1: c . h of the two channels; 2, 3: b . g
      const float qsum = sum_over_states<SL>(qa, p.sl);
      if (p.sl < 4) sm.sums[p.sl >> 1][k][p.col + (p.sl & 1)] = ygsum;
      if (p.sl < 2) sm.sums[2][k][p.col + p.sl] = qsum;
      sum_over_channels(v, p, sm.red[k][p.warp]);
    };
    auto forward = [&](int k) {
      asm volatile("" ::: "memory");
      advance(h, A, Pairs<1>(&sm.r.delta[k][p.col]), Pairs<1>(&sm.r.x[k][p.col]),
              Twice(&sm.r.b[k * P::SP + p.sl * 4]));
    };
    const int first_token = sub * kSub;
    back_to(sub, h);
    if (nt == kSub && !(sm.border_mask[first_token >> 5] >> (first_token & 31) & ((1u << kSub) - 1))) {
      StatesOf<1> before[kSub];  // before[k]: the state before token k
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
#pragma unroll
        for (int s = 0; s < 4; ++s) before[k][0][s] = h[0][s];
        forward(k);
      }
#pragma unroll
      for (int k = kSub - 1; k >= 0; --k) reverse(k, before[k], k == kSub - 1 ? h : before[k < kSub - 1 ? k + 1 : k]);
    } else {
      // A run that a sequence starts or ends in, or of fewer tokens: the states of each token over again.
#pragma unroll 1
      for (int k = nt - 1; k >= 0; --k) {
        StatesOf<1> prev;
        back_to(sub, h);
#pragma unroll 1
        for (int q = 0; q <= k; ++q) {
          const int first = sm.bd.first[first_token + q];
          if (first >= 0) load_h0(a, p, a.h0, first, h);
          if (q == k) {
#pragma unroll
            for (int s = 0; s < 4; ++s) prev[0][s] = h[0][s];
          }
          forward(q);
        }
        const int first = sm.bd.first[first_token + k], last = sm.bd.last[first_token + k];
        if (last >= 0) load_h0(a, p, a.dht, last, g);
        reverse(k, prev, h);
        if (first >= 0 && a.dh0) store_final(a, p, a.dh0, first, g);
      }
    }
    __syncthreads();
    // db and dc of these tokens over the block's channels
    float *out = a.part_bc + ((int64_t)(blockIdx.x % (unsigned)a.ctiles) * a.M + t0) * (2 * P::SP);
    for (int i = tid; i < nt * 2 * P::SP; i += P::kThreads) {
      const int k = i / (2 * P::SP), s = i % (2 * P::SP);
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kMainWarps; ++w) o += sm.red[k][w][s];
      out[i] = o;
    }
    finish<T, P, VEC>(a, p, t0, nt, sm);
  }
  // ddt_bias and dd of the chunk
  __syncthreads();
  for (int i = tid; i < 2 * P::CB; i += P::kThreads) {
    const int which = i / P::CB, c = i % P::CB;
    float o = 0.f;
#pragma unroll
    for (int k = 0; k < kSub; ++k) o += sm.total[which][k][c];
    if (p.e0 + c < p.e_end) a.part_e[(p.chunk * 2 + which) * a.d.E + p.e0 + c] = o;
  }
  store_chunk(a, p, a.hloc, p.chunk, dA);  // this block's states there have been read
}

// All sums over blocks in one launch: db and dc [M, G, S] from the partials of the
// channel blocks of each group, da and (ddt_bias, dd) from those of the chunks.
template <typename T>
__global__ void __launch_bounds__(256) ssm_sums_kernel(SsmArgs a, int SP, T *db, T *dc, unsigned bc_blocks, ColSum da,
                                                       unsigned da_blocks, ColSum per_channel) {
  __shared__ float sm[8][33];
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  if (blockIdx.x >= bc_blocks) {
    const unsigned block = blockIdx.x - bc_blocks;
    if (block < da_blocks) col_sum_block<8>(da, block, sm);
    else col_sum_block<8>(per_channel, block - da_blocks, sm);
    return;
  }
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = a.d.G * a.d.S;
  if (i >= a.M * per) return;
  const int64_t m = i / per, g = i % per / a.d.S;
  const int s = (int)(i % a.d.S);
  float b = 0.f, c = 0.f;
#pragma unroll 4
  for (int k = 0; k < a.tpg; ++k) {
    const float *row = a.part_bc + ((g * a.tpg + k) * a.M + m) * (2 * SP);
    b += row[s];
    c += row[SP + s];
  }
  db[i] = from_f32<T>(b);
  dc[i] = from_f32<T>(c);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Sums {
  void *db, *dc;
  float *da, *dd, *ddt_bias;
};

template <typename T, int SL>
int launch_sl(const SsmArgs &a, const Sums &out, cudaStream_t st) {
  const unsigned grid = (unsigned)(a.chunks * a.ctiles);
  SsmArgs m = a;  // main's blocks have half the channels
  m.tpg = (int)cdiv(a.d.E / a.d.G, MainPlace<SL>::CB);
  m.ctiles = (int)(a.d.G * m.tpg);
  auto launch_main = [&](auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    constexpr int smem = sizeof(MainShared<T, MainPlace<SL>, VEC>);
    const cudaError_t e =
        cudaFuncSetAttribute(ssm_bwd_main_kernel<T, SL, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_error(e, "ssm_bwd_main_kernel shared memory");
    ssm_bwd_main_kernel<T, SL, VEC><<<(unsigned)(m.chunks * m.ctiles), 32 * kMainWarps, smem, st>>>(m);
    return launched("ssm_bwd_main_kernel");
  };
  int rc = GDR_OK;
  if (a.chunks > 1) {  // else nothing enters or leaves but by the sequences' borders
    if (a.vec) ssm_bwd_local_kernel<T, SL, true><<<grid, kSsmThreads, 0, st>>>(a);
    else ssm_bwd_local_kernel<T, SL, false><<<grid, kSsmThreads, 0, st>>>(a);
    if ((rc = launched("ssm_bwd_local_kernel")) != GDR_OK) return rc;
    ssm_bwd_carry_kernel<<<dim3((unsigned)cdiv(a.d.E * 4 * SL, 128), 2), 128, 0, st>>>(a, 4 * SL);
    if ((rc = launched("ssm_bwd_carry_kernel")) != GDR_OK) return rc;
  }
  rc = a.vec ? launch_main(std::true_type{}) : launch_main(std::false_type{});
  if (rc != GDR_OK) return rc;
  const int64_t E = a.d.E, SP = 4 * SL;
  const unsigned bc_blocks = (unsigned)cdiv(a.M * a.d.G * a.d.S, 256), da_blocks = (unsigned)cdiv(E * SP, 32);
  const ColSum da{a.hloc, a.chunks, E * SP, E * SP, SP, a.d.S, out.da, E * SP, nullptr};
  const ColSum per_channel{a.part_e, a.chunks, 2 * E, 2 * E, E, E, out.ddt_bias, E, out.dd};
  const unsigned blocks = bc_blocks + da_blocks + (unsigned)cdiv(2 * E, 32);
  ssm_sums_kernel<T><<<blocks, 256, 0, st>>>(m, 4 * SL, (T *)out.db, (T *)out.dc, bc_blocks, da, da_blocks, per_channel);
  return launched("ssm_sums_kernel");
}

template <typename T>
int launch_t(const SsmArgs &a, int sl, const Sums &out, cudaStream_t st) {
  if (sl == 4) return launch_sl<T, 4>(a, out, st);
  if (sl == 8) return launch_sl<T, 8>(a, out, st);
  return launch_sl<T, 16>(a, out, st);
}

int run_bwd(SsmArgs a, const Sums &out, cudaStream_t st) {
  int sl, rc;
  bool vec;
  if ((rc = ssm_prepare(a, true, &sl, &vec)) != GDR_OK) return rc;
  // the outputs' rows are E long: 16-byte stores where E and the pointers allow them
  a.vec = vec && is_aligned16(a.dx) && is_aligned16(a.ddt) && is_aligned16(a.dz);
  // A few tokens are one chunk: two launches fewer than they would save.  Else
  // chunks of up to kMaxL tokens such that main's waves, of three blocks on each
  // multiprocessor, are few: a chunk costs its tokens and some eight more to begin.
  int64_t least = 0;
  for (int64_t L = kTile; L <= kMaxL; L += kTile) {
    const int64_t cost = cdiv(cdiv(a.M, L) * 2 * a.ctiles, 3 * kSMs) * (L + 8);
    if (L == kTile || cost <= least || a.M <= kMaxL) {
      least = cost;
      a.L = L;
    }
  }
  a.chunks = std::max<int64_t>(1, cdiv(a.M, a.L));
  const int64_t SP = 4 * sl, E = a.d.E;
  if (2 * a.chunks * a.ctiles > 0x7fffffff || cdiv(a.M * a.d.G * a.d.S, 256) > 0x3fffffff)
    return set_error(GDR_ERR_SHAPE, "too many tokens and channels for one launch");
  const size_t states = align256(sizeof(float) * (size_t)(a.chunks * E * SP));
  const size_t sums = align256(sizeof(float) * (size_t)(a.chunks * E));
  const size_t bc = align256(sizeof(float) * (size_t)(2 * a.ctiles * a.M * 2 * SP));
  char *base = nullptr;
  rc = scratch_begin(2 * states + 3 * sums + bc, st, "scan backward scratch", &base);
  if (rc != GDR_OK) return rc;
  a.hloc = (float *)base;
  a.gloc = (float *)(base + states);
  a.sumd = (float *)(base + 2 * states);
  a.part_e = (float *)(base + 2 * states + sums);
  a.part_bc = (float *)(base + 2 * states + 3 * sums);
  rc = a.d.dtype == GDR_BF16 ? launch_t<__nv_bfloat16>(a, sl, out, st) : launch_t<float>(a, sl, out, st);
  return scratch_end(base, st, "scan backward scratch", rc);
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" int gdr_ssm_bwd(const gdr_ssm_desc *desc, const void *x, const void *dt, const float *a, const void *b,
                           const void *c, const float *d, const void *z, const float *dt_bias, const float *h0,
                           const int64_t *cu_seqlens, const void *dy, const float *dht, void *dx, void *ddt, float *da,
                           void *db, void *dc, float *dd, void *dz, float *ddt_bias, float *dh0, void *stream) {
  int rc = ssm_validate(desc, cu_seqlens);
  if (rc != GDR_OK) return rc;
  if (!a || !da || (desc->B * desc->T > 0 && (!x || !dt || !b || !c || !dy || !dx || !ddt || !db || !dc)))
    return set_error(GDR_ERR_NULLPTR, "x, dt, a, b, c, dy, dx, ddt, da, db and dc must be non-NULL");
  if (dz && !z) return set_error(GDR_ERR_NULLPTR, "dz needs z");
  SsmArgs s{};
  s.d = *desc;
  s.x = x; s.dt = dt; s.a = a; s.b = b; s.c = c; s.dskip = d; s.z = z; s.dt_bias = dt_bias; s.h0 = h0;
  s.cu = cu_seqlens; s.dy = dy; s.dht = dht; s.dx = dx; s.ddt = ddt; s.dz = dz; s.dh0 = dh0;
  return run_bwd(s, Sums{db, dc, da, dd, ddt_bias}, (cudaStream_t)stream);
}
