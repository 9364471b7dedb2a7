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
//           tokens give to the gradient of the state entering it
//   carry   per (channel, state): the state entering each chunk (forwards) and the
//           gradient reaching its end from later chunks (backwards), in order
//   main    per (chunk, channels): the states again, kept every 8 tokens in shared
//           memory; then 8 tokens at a time from the last: the states once more,
//           in registers, and the reverse recurrence with all products
//   sums    the partials of db and dc over channels, of da, dd and ddt_bias over chunks
// States are recomputed, never inverted: h_{t-1} = (h_t - ..) / a_t loses what a
// small a_t has forgotten.  The bound is arithmetic: four exponentials and about
// 25 fp32 operations per channel, state and token.
#include <algorithm>

#include "gdr_ssm.cuh"

namespace gdr {
namespace {

constexpr int kSub = 8;      // tokens whose states a thread holds in registers
constexpr int kMaxL = 64;    // tokens of a chunk
constexpr int kSubs = kMaxL / kSub;
constexpr float kLn2 = 0.6931471805599453f;

template <int SL>
struct __align__(16) LocalShared {
  float delta[kTile][Place<SL>::CB], x[kTile][Place<SL>::CB], up[kTile][Place<SL>::CB];
  float2 b[kTile * Place<SL>::SP], c[kTile * Place<SL>::SP];
  Borders<kTile> bd;
};

template <typename T, int SL, int VEC>
__device__ __forceinline__ void stage_local(const SsmArgs &a, const Place<SL> &p, int64_t t0, int nt,
                                            LocalShared<SL> &sm) {
  for_tile<kTile, SL, VEC>(p, nt, [&](int t, int c, bool in) {
    const int64_t e = p.e0 + c;
    float xv[VEC] = {}, dv[VEC] = {}, zv[VEC] = {}, gv[VEC] = {};
    if (in) {
      load_vec<VEC>(static_cast<const T *>(a.x) + (t0 + t) * a.d.ld_x + e, xv);
      load_vec<VEC>(static_cast<const T *>(a.dt) + (t0 + t) * a.d.ld_dt + e, dv);
      load_vec<VEC>(static_cast<const T *>(a.dy) + (t0 + t) * a.d.ld_dy + e, gv);
      if (a.z) load_vec<VEC>(static_cast<const T *>(a.z) + (t0 + t) * a.d.ld_z + e, zv);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float raw = dv[i] + (a.dt_bias && in ? a.dt_bias[e + i] : 0.f);
      dv[i] = in ? ssm_delta(raw, a.d.flags & GDR_SSM_SOFTPLUS) : 0.f;
      gv[i] *= a.z ? zv[i] * sigmoid_fast(zv[i]) : 1.f;
    }
    store_vec<VEC>(&sm.delta[t][c], dv);
    store_vec<VEC>(&sm.x[t][c], xv);
    store_vec<VEC>(&sm.up[t][c], gv);
  });
}

template <typename T, int SL>
__global__ void __launch_bounds__(kSsmThreads) ssm_bwd_local_kernel(SsmArgs a) {
  using P = Place<SL>;
  __shared__ LocalShared<SL> sm;
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  const P p(a);
  States A, h, g, pass;  // pass: product of the decays since the chunk began; zero once a sequence started
  load_a<SL>(a, p, A);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      h[i][s] = g[i][s] = 0;
      pass[i][s] = f2_pack(1.f, 1.f);
    }
  const int64_t begin = p.chunk * a.L, end = begin + a.L < a.M ? begin + a.L : a.M;
  f2 sum[2] = {0, 0};
  bool started = false;
  auto token = [&](int t) {
    const Pairs delta(&sm.delta[t][p.col]), x(&sm.x[t][p.col]), up(&sm.up[t][p.col]);
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
  for (int64_t t0 = begin; t0 < end; t0 += kTile) {
    const int nt = end - t0 < kTile ? (int)(end - t0) : kTile;
    __syncthreads();
    const bool borders = stage_borders(a, t0, nt, sm.bd);
    if (a.vec) stage_local<T, SL, 8>(a, p, t0, nt, sm);
    else stage_local<T, SL, 1>(a, p, t0, nt, sm);
    stage_states<T, SL, kTile>(a, p, a.b, a.d.ld_b, t0, nt, sm.b);
    stage_states<T, SL, kTile>(a, p, a.c, a.d.ld_c, t0, nt, sm.c);
    if (!__syncthreads_or(borders) && nt == kTile) {
#pragma unroll 4
      for (int t = 0; t < kTile; ++t) token(t);
    } else {
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        if (sm.bd.first[t] >= 0) {
          load_h0<SL>(a, p, a.h0, sm.bd.first[t], h);
          started = true;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) pass[i][s] = 0;
        }
        token(t);
        if (a.dht && !started && sm.bd.last[t] >= 0) {
          States dh;
          load_h0<SL>(a, p, a.dht, sm.bd.last[t], dh);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) g[i][s] = f2_fma(pass[i][s], dh[i][s], g[i][s]);
        }
      }
    }
  }
  store_chunk<SL>(a, p, a.hloc, p.chunk, h);
  store_chunk<SL>(a, p, a.gloc, p.chunk, g);
  const int mine = p.sl & 3;
  const int64_t e_mine = p.e0 + p.col + mine;
  if (p.sl < 4 && e_mine < p.e_end) {
    float s[4];
    f2_split(sum[0], s[0], s[1]);
    f2_split(sum[1], s[2], s[3]);
    const float mine_sum = mine == 0 ? s[0] : mine == 1 ? s[1] : mine == 2 ? s[2] : s[3];
    a.sumd[p.chunk * a.d.E + e_mine] = started ? CUDART_NAN_F : mine_sum;  // NaN: nothing passes through
  }
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
        acc = isnan(sum[k]) ? loc[k] : fmaf(ex2(A * sum[k]), acc, loc[k]);
      }
    }
  }
}

template <int SL>
struct MainShared {
  using P = Place<SL>;
  ulonglong2 ckpt[kSubs][4][kSsmThreads];  // a thread's states before each run of kSub tokens
  union {
    struct {
      float delta[kTile][P::CB], x[kTile][P::CB];
      float2 b[kTile * P::SP];
    } f;
    struct {
      float delta[kSub][P::CB], x[kSub][P::CB], up[kSub][P::CB], slope[kSub][P::CB], zf[kSub][P::CB];
      float2 b[kSub * P::SP], c[kSub * P::SP];
    } r;
  };
  float red[kSub][4][2 * P::SP];  // db, dc of a token by warp
  Borders<kMaxL> bd;
};

template <typename T, int SL, int VEC>
__device__ __forceinline__ void stage_forward(const SsmArgs &a, const Place<SL> &p, int64_t t0, int nt,
                                              MainShared<SL> &sm) {
  for_tile<kTile, SL, VEC>(p, nt, [&](int t, int c, bool in) {
    const int64_t e = p.e0 + c;
    float xv[VEC] = {}, dv[VEC] = {};
    if (in) {
      load_vec<VEC>(static_cast<const T *>(a.x) + (t0 + t) * a.d.ld_x + e, xv);
      load_vec<VEC>(static_cast<const T *>(a.dt) + (t0 + t) * a.d.ld_dt + e, dv);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float raw = dv[i] + (a.dt_bias && in ? a.dt_bias[e + i] : 0.f);
      dv[i] = in ? ssm_delta(raw, a.d.flags & GDR_SSM_SOFTPLUS) : 0.f;
    }
    store_vec<VEC>(&sm.f.delta[t][c], dv);
    store_vec<VEC>(&sm.f.x[t][c], xv);
  });
}

template <typename T, int SL, int VEC>
__device__ __forceinline__ void stage_reverse(const SsmArgs &a, const Place<SL> &p, int64_t t0, int nt,
                                              MainShared<SL> &sm) {
  for_tile<kSub, SL, VEC>(p, nt, [&](int t, int c, bool in) {
    const int64_t e = p.e0 + c;
    float xv[VEC] = {}, dv[VEC] = {}, zv[VEC] = {}, gv[VEC] = {};
    if (in) {
      load_vec<VEC>(static_cast<const T *>(a.x) + (t0 + t) * a.d.ld_x + e, xv);
      load_vec<VEC>(static_cast<const T *>(a.dt) + (t0 + t) * a.d.ld_dt + e, dv);
      load_vec<VEC>(static_cast<const T *>(a.dy) + (t0 + t) * a.d.ld_dy + e, gv);
      if (a.z) load_vec<VEC>(static_cast<const T *>(a.z) + (t0 + t) * a.d.ld_z + e, zv);
    }
    float slope[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float raw = dv[i] + (a.dt_bias && in ? a.dt_bias[e + i] : 0.f);
      const float sg = sigmoid_fast(zv[i]), dy = gv[i];
      dv[i] = ssm_delta(raw, a.d.flags & GDR_SSM_SOFTPLUS, &slope[i]);
      if (!in) dv[i] = 0.f;
      gv[i] = dy * (a.z ? zv[i] * sg : 1.f);
      zv[i] = dy * sg * fmaf(zv[i], 1.f - sg, 1.f);
    }
    store_vec<VEC>(&sm.r.delta[t][c], dv);
    store_vec<VEC>(&sm.r.x[t][c], xv);
    store_vec<VEC>(&sm.r.up[t][c], gv);
    store_vec<VEC>(&sm.r.slope[t][c], slope);
    store_vec<VEC>(&sm.r.zf[t][c], zv);
  });
}

// Sums v[0..7] (db of the thread's four states, then dc) over the channel lanes
// of a warp, halving the values a lane holds at each step, and leaves them in
// out[2 * SP] (db, then dc).
template <int SL>
__device__ __forceinline__ void sum_over_channels(float (&v)[8], const Place<SL> &p, float *out) {
  constexpr int SP = Place<SL>::SP, CL = 32 / SL;
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
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o * SL);
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

template <typename T, int SL>
__global__ void __launch_bounds__(kSsmThreads, 2) ssm_bwd_main_kernel(SsmArgs a) {
  using P = Place<SL>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  MainShared<SL> &sm = *reinterpret_cast<MainShared<SL> *>(smem_raw);
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  const P p(a);
  const int tid = threadIdx.x;
  if (p.chunk == 0) copy_empty_states<SL>(a, p, a.dht, a.dh0);
  States A, h, g, dA;
  load_a<SL>(a, p, A);
  load_chunk<SL>(a, p, a.hloc, p.chunk, h);
  load_chunk<SL>(a, p, a.gloc, p.chunk, g);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) dA[i][s] = 0;
  const int64_t begin = p.chunk * a.L, end = begin + a.L < a.M ? begin + a.L : a.M;
  const int len = end > begin ? (int)(end - begin) : 0;
  const int subs = (len + kSub - 1) / kSub;
  const int mine = p.sl & 3;
  const int64_t e_mine = p.e0 + p.col + mine;
  const bool owner = p.sl < 4 && e_mine < p.e_end;
  const float skip = a.dskip && owner ? a.dskip[e_mine] : 0.f;
  float dd = 0.f, dbias = 0.f;
  stage_borders(a, begin, len, sm.bd);

  auto keep = [&](int sub) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sm.ckpt[sub][i][tid] = make_ulonglong2(h[i >> 1][2 * (i & 1)], h[i >> 1][2 * (i & 1) + 1]);
  };
  auto back_to = [&](int sub, States &to) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ulonglong2 v = sm.ckpt[sub][i][tid];
      to[i >> 1][2 * (i & 1)] = v.x;
      to[i >> 1][2 * (i & 1) + 1] = v.y;
    }
  };

  // States at the start of every run of kSub tokens; the last run needs only its start.
  keep(0);
  const int flen = subs > 0 ? (subs - 1) * kSub : 0;
  for (int f0 = 0; f0 < flen; f0 += kTile) {
    const int nt = flen - f0 < kTile ? flen - f0 : kTile;
    __syncthreads();
    if (a.vec) stage_forward<T, SL, 8>(a, p, begin + f0, nt, sm);
    else stage_forward<T, SL, 1>(a, p, begin + f0, nt, sm);
    stage_states<T, SL, kTile>(a, p, a.b, a.d.ld_b, begin + f0, nt, sm.f.b);
    __syncthreads();
    for (int t1 = 0; t1 < nt; t1 += kSub) {
#pragma unroll 4
      for (int t = t1; t < t1 + kSub; ++t) {
        if (sm.bd.first[f0 + t] >= 0) load_h0<SL>(a, p, a.h0, sm.bd.first[f0 + t], h);
        advance(h, A, Pairs(&sm.f.delta[t][p.col]), Pairs(&sm.f.x[t][p.col]), Twice(&sm.f.b[t * P::SP + p.sl * 4]));
      }
      keep((f0 + t1) / kSub + 1);
    }
  }

  for (int sub = subs - 1; sub >= 0; --sub) {
    const int64_t t0 = begin + sub * kSub;
    const int nt = len - sub * kSub < kSub ? len - sub * kSub : kSub;
    __syncthreads();  // the previous run's staging and partials are consumed
    if (a.vec) stage_reverse<T, SL, 8>(a, p, t0, nt, sm);
    else stage_reverse<T, SL, 1>(a, p, t0, nt, sm);
    stage_states<T, SL, kSub>(a, p, a.b, a.d.ld_b, t0, nt, sm.r.b);
    stage_states<T, SL, kSub>(a, p, a.c, a.d.ld_c, t0, nt, sm.r.c);
    __syncthreads();
    States after[kSub];  // after[k]: the state after token k (past the end: never read)
    back_to(sub, h);
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      if (k < nt) {
        if (sm.bd.first[sub * kSub + k] >= 0) load_h0<SL>(a, p, a.h0, sm.bd.first[sub * kSub + k], h);
        advance(h, A, Pairs(&sm.r.delta[k][p.col]), Pairs(&sm.r.x[k][p.col]), Twice(&sm.r.b[k * P::SP + p.sl * 4]));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) after[k][i][s] = h[i][s];
    }
#pragma unroll
    for (int k = kSub - 1; k >= 0; --k) {
      if (k >= nt) continue;
      const int first = sm.bd.first[sub * kSub + k], last = sm.bd.last[sub * kSub + k];
      if (last >= 0) load_h0<SL>(a, p, a.dht, last, g);
      States prev;
      if (first >= 0) {
        load_h0<SL>(a, p, a.h0, first, prev);
      } else if (k == 0) {
        back_to(sub, prev);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int s = 0; s < 4; ++s) prev[i][s] = after[k > 0 ? k - 1 : 0][i][s];
      }
      const Pairs delta(&sm.r.delta[k][p.col]), x(&sm.r.x[k][p.col]), up(&sm.r.up[k][p.col]);
      const Twice b(&sm.r.b[k * P::SP + p.sl * 4]), c(&sm.r.c[k * P::SP + p.sl * 4]);
      f2 db[4], dc[4];
      float ys[4], gb[4], qa[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f2 u = f2_mul(delta.v[i], x.v[i]);
        f2 sy = 0, sb = 0, sq = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          g[i][s] = f2_fma(c.v[s], up.v[i], g[i][s]);
          dc[s] = i ? f2_fma(up.v[i], after[k][i][s], dc[s]) : f2_mul(up.v[i], after[k][i][s]);
          sy = s ? f2_fma(c.v[s], after[k][i][s], sy) : f2_mul(c.v[s], after[k][i][s]);
          db[s] = i ? f2_fma(u, g[i][s], db[s]) : f2_mul(u, g[i][s]);
          sb = s ? f2_fma(b.v[s], g[i][s], sb) : f2_mul(b.v[s], g[i][s]);
          g[i][s] = f2_mul(g[i][s], f2_ex2(f2_mul(A[i][s], delta.v[i])));
          const f2 q = f2_mul(g[i][s], prev[i][s]);
          dA[i][s] = f2_fma(q, delta.v[i], dA[i][s]);
          sq = s ? f2_fma(q, A[i][s], sq) : f2_mul(q, A[i][s]);
        }
        f2_split(sy, ys[2 * i], ys[2 * i + 1]);
        f2_split(sb, gb[2 * i], gb[2 * i + 1]);
        f2_split(sq, qa[2 * i], qa[2 * i + 1]);
      }
      const float ysum = sum_over_states<SL>(ys, p.sl), gsum = sum_over_states<SL>(gb, p.sl),
                  qsum = sum_over_states<SL>(qa, p.sl) * kLn2;  // A carries log2(e)
      if (owner) {
        const int col = p.col + mine;
        const float xo = sm.r.x[k][col], uo = sm.r.up[k][col];
        const float ddt = fmaf(xo, gsum, qsum) * sm.r.slope[k][col];
        const int64_t at = (t0 + k) * a.d.E + e_mine;
        static_cast<T *>(a.dx)[at] = from_f32<T>(fmaf(skip, uo, sm.r.delta[k][col] * gsum));
        static_cast<T *>(a.ddt)[at] = from_f32<T>(ddt);
        if (a.dz) static_cast<T *>(a.dz)[at] = from_f32<T>(sm.r.zf[k][col] * fmaf(skip, xo, ysum));
        dd = fmaf(uo, xo, dd);
        dbias += ddt;
      }
      float v[8];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float lo, hi;
        f2_split(db[s], lo, hi);
        v[s] = lo + hi;
        f2_split(dc[s], lo, hi);
        v[4 + s] = lo + hi;
      }
      sum_over_channels<SL>(v, p, sm.red[k][p.warp]);
      if (first >= 0 && a.dh0) store_final<SL>(a, p, a.dh0, first, g);
    }
    __syncthreads();
    // db and dc of these tokens over the block's channels
    float *out = a.part_bc + ((int64_t)(blockIdx.x % (unsigned)a.ctiles) * a.M + t0) * (2 * P::SP);
    for (int i = tid; i < nt * 2 * P::SP; i += kSsmThreads) {
      const int k = i / (2 * P::SP), s = i % (2 * P::SP);
      out[i] = (sm.red[k][0][s] + sm.red[k][1][s]) + (sm.red[k][2][s] + sm.red[k][3][s]);
    }
  }
  store_chunk<SL>(a, p, a.hloc, p.chunk, dA);  // this block's states there have been read
  if (owner) {
    a.part_e[p.chunk * 2 * a.d.E + e_mine] = dd;
    a.part_e[(p.chunk * 2 + 1) * a.d.E + e_mine] = dbias;
  }
}

// db and dc [M, G, S] from the partials of the channel blocks of each group.
template <typename T>
__global__ void __launch_bounds__(256) ssm_sum_bc_kernel(SsmArgs a, int SP, T *db, T *dc) {
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
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

template <typename T, int SL>
int launch_sl(const SsmArgs &a, void *db, void *dc, cudaStream_t st) {
  const unsigned grid = (unsigned)(a.chunks * a.ctiles);
  constexpr int smem = sizeof(MainShared<SL>);
  const cudaError_t e =
      cudaFuncSetAttribute(ssm_bwd_main_kernel<T, SL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_error(e, "ssm_bwd_main_kernel shared memory");
  ssm_bwd_local_kernel<T, SL><<<grid, kSsmThreads, 0, st>>>(a);
  int rc = launched("ssm_bwd_local_kernel");
  if (rc != GDR_OK) return rc;
  ssm_bwd_carry_kernel<<<dim3((unsigned)cdiv(a.d.E * 4 * SL, 128), 2), 128, 0, st>>>(a, 4 * SL);
  if ((rc = launched("ssm_bwd_carry_kernel")) != GDR_OK) return rc;
  ssm_bwd_main_kernel<T, SL><<<grid, kSsmThreads, smem, st>>>(a);
  if ((rc = launched("ssm_bwd_main_kernel")) != GDR_OK) return rc;
  if (a.M > 0) {
    ssm_sum_bc_kernel<T><<<(unsigned)cdiv(a.M * a.d.G * a.d.S, 256), 256, 0, st>>>(a, 4 * SL, (T *)db, (T *)dc);
    rc = launched("ssm_sum_bc_kernel");
  }
  return rc;
}

template <typename T>
int launch_t(const SsmArgs &a, int sl, void *db, void *dc, cudaStream_t st) {
  if (sl == 4) return launch_sl<T, 4>(a, db, dc, st);
  if (sl == 8) return launch_sl<T, 8>(a, db, dc, st);
  return launch_sl<T, 16>(a, db, dc, st);
}

int run_bwd(SsmArgs a, float *da, void *db, void *dc, float *dd, float *ddt_bias, cudaStream_t st) {
  int sl, rc;
  bool vec;
  if ((rc = ssm_prepare(a, true, &sl, &vec)) != GDR_OK) return rc;
  a.vec = vec;
  a.L = kMaxL;
  while (a.L > 2 * kSub && cdiv(a.M, a.L) * a.ctiles < 2 * kSMs) a.L /= 2;
  a.chunks = std::max<int64_t>(1, cdiv(a.M, a.L));
  const int64_t SP = 4 * sl, E = a.d.E;
  if (a.chunks * a.ctiles > 0x7fffffff || cdiv(a.M * a.d.G * a.d.S, 256) > 0x7fffffff)
    return set_error(GDR_ERR_SHAPE, "too many tokens and channels for one launch");
  const size_t states = align256(sizeof(float) * (size_t)(a.chunks * E * SP));
  const size_t sums = align256(sizeof(float) * (size_t)(a.chunks * E));
  const size_t bc = align256(sizeof(float) * (size_t)(a.ctiles * a.M * 2 * SP));
  char *base = nullptr;
  rc = scratch_begin(2 * states + 3 * sums + bc, st, "scan backward scratch", &base);
  if (rc != GDR_OK) return rc;
  a.hloc = (float *)base;
  a.gloc = (float *)(base + states);
  a.sumd = (float *)(base + 2 * states);
  a.part_e = (float *)(base + 2 * states + sums);
  a.part_bc = (float *)(base + 2 * states + 3 * sums);
  rc = a.d.dtype == GDR_BF16 ? launch_t<__nv_bfloat16>(a, sl, db, dc, st) : launch_t<float>(a, sl, db, dc, st);
  const SeqCheck seqs{a.cu, a.d.N, a.M, a.status};
  if (rc == GDR_OK) rc = launch_col_sum(a.hloc, a.chunks, E * SP, E * SP, SP, a.d.S, da, seqs, st);
  if (rc == GDR_OK && dd) rc = launch_col_sum(a.part_e, a.chunks, 2 * E, E, E, E, dd, seqs, st);
  if (rc == GDR_OK && ddt_bias) rc = launch_col_sum(a.part_e + E, a.chunks, 2 * E, E, E, E, ddt_bias, seqs, st);
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
  return run_bwd(s, da, db, dc, dd, ddt_bias, (cudaStream_t)stream);
}
