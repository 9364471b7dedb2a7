// gdr_heads.cu -- root-mean-square norm of queries and keys for each head, with
// the position rotation in the same pass, and the backward.
//
//   n = x rho w,  rho = 1 / sqrt(mean(x^2) + eps)     over the D channels of one head
//   y: pairs (a, b) of n turned by the token's angles,  a cos - b sin,  b cos + a sin;  channels past 2 R as they are
//   backward: dn = dy turned back,  p = w dn,  dx = rho (p - x rho^2 mean(p x)),  dw = sum over rows of dn x rho
//
// One pass over memory: a head's row is held in fp32 registers between its sum and
// its output, queries and keys in one launch.  The bound is HBM.
#include <algorithm>
#include <type_traits>

#include "gdr_layer.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;

struct HeadArgs {
  gdr_qk_norm_desc d;
  const void *q, *k, *wq, *wk, *dyq, *dyk;
  const float *cos, *sin;
  const int64_t *pos;
  void *yq, *yk;  // backward: dq, dk
  float *part;    // backward: [blocks, D] sums of dw, the blocks of q before those of k
  int *status;
  int64_t bq;     // blocks of q; the others take k
};

// One of the two tensors.
template <typename T>
struct Side {
  const T *x, *dy;
  T *y;
  const void *w;
  int64_t ld, ld_dy, heads;
};
template <typename T>
__device__ __forceinline__ Side<T> side_of(const HeadArgs &p, bool query) {
  const gdr_qk_norm_desc &d = p.d;
  if (query) return {(const T *)p.q, (const T *)p.dyq, (T *)p.yq, p.wq, d.ld_q, d.ld_dyq, d.H};
  return {(const T *)p.k, (const T *)p.dyk, (T *)p.yk, p.wk, d.ld_k, d.ld_dyk, d.HK};
}

// Channels of thread t of a row: two runs of RUN (16 bytes of fp32 or of bf16, or 8 of bf16).  Where
// halves are paired, the runs are the a and the b of RUN pairs; neighbours' pairs lie
// within each run, and a row's threads take runs side by side.  R % RUN == 0, D % (2 RUN) == 0.
template <int RUN, bool NEAR>
struct Place {
  int c0, c1;
  bool on, turned0, turned1;
  __device__ __forceinline__ Place(const HeadArgs &p, int t) {
    const int R = (int)p.d.R, D = (int)p.d.D;
    on = 2 * RUN * t < D;
    if constexpr (NEAR) {
      c0 = RUN * t;
      c1 = D / 2 + c0;
      turned0 = on && c0 < 2 * R;
      turned1 = on && c1 < 2 * R;
    } else {
      turned0 = turned1 = on && RUN * t < R;
      c0 = turned0 ? RUN * t : 2 * RUN * t;
      c1 = turned0 ? R + RUN * t : c0 + RUN;
    }
  }
};

// A thread's 2 RUN channels in packed pairs: those of the first run, then of the second.  (Single fp32 operations
// and selects made 267 instructions of four rows of 128, and issue the bound: 51 %.)
//
// Cosines and sines of a thread's RUN pairs; BACK turns back.  A padding token (pos < 0) has no place in the table:
// nothing is loaded, and nothing may be applied.
template <int RUN, bool NEAR, bool BACK>
struct Turn {
  float c[RUN], s[RUN];
  __device__ __forceinline__ void load_run(const HeadArgs &p, int64_t pos, int first, int at, int n) {
    const float *pc = p.cos + pos * p.d.R + first, *ps = p.sin + pos * p.d.R + first;
#pragma unroll
    for (int i = 0; i < RUN; i += 2) {
      if (i < n) {
        const float2 u = *reinterpret_cast<const float2 *>(pc + i), v = *reinterpret_cast<const float2 *>(ps + i);
        c[at + i] = u.x;
        c[at + i + 1] = u.y;
        s[at + i] = BACK ? -v.x : v.x;
        s[at + i + 1] = BACK ? -v.y : v.y;
      }
    }
  }
  __device__ __forceinline__ Turn(const HeadArgs &p, const Place<RUN, NEAR> &l, int64_t pos) {
    if (pos < 0) return;
    if constexpr (NEAR) {
      if (l.turned0) load_run(p, pos, l.c0 / 2, 0, RUN / 2);
      if (l.turned1) load_run(p, pos, l.c1 / 2, RUN / 2, RUN / 2);
    } else if (l.turned0) {
      load_run(p, pos, l.c0, 0, RUN);
    }
  }
  // Channels that are not turned are not touched.
  __device__ __forceinline__ void apply(f2 (&v)[RUN], const Place<RUN, NEAR> &l) const {
    if constexpr (NEAR) {
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        if (i < RUN / 2 ? l.turned0 : l.turned1) {
          float a, b;
          f2_split(v[i], a, b);
          v[i] = f2_pack(fmaf(a, c[i], -(b * s[i])), fmaf(b, c[i], a * s[i]));
        }
      }
    } else if (l.turned0) {
#pragma unroll
      for (int i = 0; i < RUN / 2; ++i) {
        const f2 cc = f2_pack(c[2 * i], c[2 * i + 1]), ss = f2_pack(s[2 * i], s[2 * i + 1]);
        const f2 a = v[i], b = v[RUN / 2 + i];
        v[i] = f2_fma(f2_mul(b, ss), f2_both(-1.f), f2_mul(a, cc));
        v[RUN / 2 + i] = f2_fma(b, cc, f2_mul(a, ss));
      }
    }
  }
};

template <int TPR>
__device__ __forceinline__ float row_sum(f2 v) {
  float x, y;
  f2_split(v, x, y);
  x += y;
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Both runs of a thread as they lie in memory (half the registers of bf16 until they are used); zeros where `on` is
// false.
template <typename T, int RUN>
struct Raw {
  static constexpr int kWords = RUN * sizeof(T) / 4;
  uint32_t a[kWords], b[kWords];
  static __device__ __forceinline__ void load_run(const T *p, uint32_t (&r)[kWords]) {
    if constexpr (kWords == 4) {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      r[0] = u.x;
      r[1] = u.y;
      r[2] = u.z;
      r[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2 *>(p);
      r[0] = u.x;
      r[1] = u.y;
    }
  }
  __device__ __forceinline__ void load(const T *p, int c0, int c1, bool on) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) a[i] = b[i] = 0;
    if (on) {
      load_run(p + c0, a);
      load_run(p + c1, b);
    }
  }
  static __device__ __forceinline__ f2 pair(const uint32_t (&r)[kWords], int i) {
    if constexpr (sizeof(T) == 4) return f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    else return f2_pack(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void get(f2 (&v)[RUN]) const {
#pragma unroll
    for (int i = 0; i < RUN / 2; ++i) {
      v[i] = pair(a, i);
      v[RUN / 2 + i] = pair(b, i);
    }
  }
};
template <int RUN, typename T>
__device__ __forceinline__ void store_two(T *p, int c0, int c1, const f2 (&v)[RUN]) {
  float a[RUN], b[RUN];
#pragma unroll
  for (int i = 0; i < RUN / 2; ++i) {
    f2_split(v[i], a[2 * i], a[2 * i + 1]);
    f2_split(v[RUN / 2 + i], b[2 * i], b[2 * i + 1]);
  }
  store_vec<RUN>(p + c0, a);
  store_vec<RUN>(p + c1, b);
}
template <typename T, int RUN, bool NEAR>
__device__ __forceinline__ void load_weight(const HeadArgs &p, const void *w, const Place<RUN, NEAR> &l, f2 (&v)[RUN]) {
  float a[RUN] = {}, b[RUN] = {};
  if (l.on) {
    if (p.d.weight_dtype == GDR_F32) {
      load_vec<RUN>(static_cast<const float *>(w) + l.c0, a);
      load_vec<RUN>(static_cast<const float *>(w) + l.c1, b);
    } else {
      load_vec<RUN>(static_cast<const T *>(w) + l.c0, a);
      load_vec<RUN>(static_cast<const T *>(w) + l.c1, b);
    }
  }
#pragma unroll
  for (int i = 0; i < RUN / 2; ++i) {
    v[i] = f2_pack(a[2 * i], a[2 * i + 1]);
    v[RUN / 2 + i] = f2_pack(b[2 * i], b[2 * i + 1]);
  }
}

// A token's position: -1 (or one past the table, which is reported) makes a padding row of zeros.  The load
// and the check are apart, so that the rows' loads are on their way before the position has come.
__device__ __forceinline__ int64_t load_position(const HeadArgs &p, int64_t m) { return p.d.R ? p.pos[m] : 0; }
__device__ __forceinline__ int64_t checked(const HeadArgs &p, int64_t pos) {
  if (!p.d.R || pos < p.d.P) return pos < 0 ? -1 : pos;
  raise_status(p.status, GDR_ERR_POSITION);
  return -1;
}

// A warp's items (token, run of heads): every `step`-th of its tensor, without a division on the way.
struct Walk {
  int64_t m, dm;
  int run, dr, runs;
  __device__ __forceinline__ Walk(int64_t first, int64_t step, int64_t heads, int per) {
    runs = (int)((heads + per - 1) / per);
    m = first / runs;
    run = (int)(first - m * runs);
    dm = step / runs;
    dr = (int)(step - dm * runs);
  }
  __device__ __forceinline__ void next() {
    m += dm;
    run += dr;
    if (run >= runs) {
      run -= runs;
      ++m;
    }
  }
};

// TPR threads to a row (a power of two, at least D / (2 RUN)), so 32 / TPR rows to a warp at once; U such
// sets of one token's heads to a warp.  A block belongs to q or to k: its weights stay in registers.
// Warps go through the items (token, run of heads) of their tensor, the next one's rows on their way:
// 16384 x 40 x 128 bf16 in 64 us, 80 % of the copy rate (79 us with one item to a warp, 3 blocks at 80
// registers 82).
template <typename T, int RUN, int TPR, int U, bool NEAR>
__global__ void __launch_bounds__(kThreads, 2) head_fwd_kernel(const __grid_constant__ HeadArgs p) {
  constexpr int G = 32 / TPR, HI = G * U, kWarps = kThreads / 32;
  const bool query = blockIdx.x < p.bq;
  const Side<T> sd = side_of<T>(p, query);
  const int64_t block = query ? blockIdx.x : blockIdx.x - p.bq, blocks = query ? p.bq : gridDim.x - p.bq;
  const int lane = threadIdx.x & 31, D = (int)p.d.D, grp = lane / TPR;
  const Place<RUN, NEAR> l(p, lane % TPR);
  f2 w[RUN];
  load_weight<T>(p, sd.w, l, w);
  Walk it(block * kWarps + (threadIdx.x >> 5), blocks * kWarps, sd.heads, HI);
  Raw<T, RUN> rx[U], nx[U];
  int64_t at = 0, nat = 0;
  const auto fetch = [&](Raw<T, RUN> (&r)[U], int64_t &pos) {
    if (it.m >= p.d.M) return;
    const int64_t h = (int64_t)it.run * HI + grp;
    pos = load_position(p, it.m);
    const T *x = sd.x + it.m * sd.ld + h * D;
#pragma unroll
    for (int u = 0; u < U; ++u) r[u].load(x + u * G * D, l.c0, l.c1, l.on && h + u * G < sd.heads);
  };
  fetch(nx, nat);
  while (it.m < p.d.M) {
    const int64_t m = it.m, h0 = (int64_t)it.run * HI + grp;
    at = nat;
#pragma unroll
    for (int u = 0; u < U; ++u) rx[u] = nx[u];
    it.next();
    const int64_t pos = checked(p, at);  // one token to a warp
    const Turn<RUN, NEAR, false> a(p, l, pos);
    fetch(nx, nat);  // the next item's rows are on their way while this one is worked on
    T *y = sd.y + (m * sd.heads + h0) * D;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f2 v[RUN], ss = f2_both(0.f);
      rx[u].get(v);
#pragma unroll
      for (int i = 0; i < RUN; ++i) ss = f2_fma(v[i], v[i], ss);
      const f2 rho = f2_both(rsqrtf(row_sum<TPR>(ss) / (float)D + p.d.eps));
      if (l.on && h0 + u * G < sd.heads) {
#pragma unroll
        for (int i = 0; i < RUN; ++i) v[i] = pos < 0 ? f2_both(0.f) : f2_mul(f2_mul(v[i], rho), w[i]);
        if (pos >= 0) a.apply(v, l);
        store_two(y + u * G * D, l.c0, l.c1, v);
      }
    }
  }
}

// The same with dy beside x; a thread sums dw of its channels over its items, a block's
// warps and rows meet in shared memory, the blocks in a second launch.  x and dy of the next
// item are copied into the thread's own part of shared memory meanwhile (in registers they spilled:
// 16384 x 40 x 128 bf16 took 145 us, and 112-120 without any rows ahead; so it takes 95, 80 % of the copy
// rate, and with one row to a thread 110).
template <typename T, int RUN, int U>
struct Ahead {
  static constexpr int kBytes = RUN * sizeof(T);
  struct __align__(16) Part {
    unsigned char b[kThreads][kBytes];  // a run of every thread
  };
  Part part[2][U][2][2];  // buffer, row, x or dy, run
};
template <int TPR, int RUN>
struct Sums {
  float of[kThreads / TPR][2 * RUN * TPR + 1];
};
template <typename T, int RUN, int TPR, int U>
constexpr size_t bwd_smem() {
  return std::max(sizeof(Ahead<T, RUN, U>), sizeof(Sums<TPR, RUN>));
}
template <typename T, int RUN, int TPR, int U, bool NEAR>
__global__ void __launch_bounds__(kThreads, 2) head_bwd_kernel(const __grid_constant__ HeadArgs p) {
  constexpr int G = 32 / TPR, HI = G * U, kWarps = kThreads / 32;
  extern __shared__ __align__(16) unsigned char shared[];
  const auto get_two = [](const unsigned char *a, const unsigned char *b, bool on, f2 (&v)[RUN]) {
    Raw<T, RUN> r;
    r.load(reinterpret_cast<const T *>(a), 0, (int)((b - a) / (int64_t)sizeof(T)), on);
    r.get(v);
  };
  auto &ahead = *reinterpret_cast<Ahead<T, RUN, U> *>(shared);
  auto &red = reinterpret_cast<Sums<TPR, RUN> *>(shared)->of;
  const bool query = blockIdx.x < p.bq;
  const Side<T> sd = side_of<T>(p, query);
  const int64_t block = query ? blockIdx.x : blockIdx.x - p.bq, blocks = query ? p.bq : gridDim.x - p.bq;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = (int)p.d.D, grp = lane / TPR;
  const Place<RUN, NEAR> l(p, lane % TPR);
  f2 w[RUN], sum[RUN];
#pragma unroll
  for (int i = 0; i < RUN; ++i) sum[i] = f2_both(0.f);
  load_weight<T>(p, sd.w, l, w);
  Walk it(block * kWarps + warp, blocks * kWarps, sd.heads, HI);
  int64_t at = 0, nat = 0;
  int buf = 0;
  const auto fetch = [&](int to) {
    if (it.m < p.d.M) {
      const int64_t h = (int64_t)it.run * HI + grp;
      nat = load_position(p, it.m);
      const T *x = sd.x + it.m * sd.ld + h * D, *dy = sd.dy + it.m * sd.ld_dy + h * D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (l.on && h + u * G < sd.heads) {
          auto &part = ahead.part[to][u];
          copy_async<Ahead<T, RUN, U>::kBytes>(part[0][0].b[threadIdx.x], x + u * G * D + l.c0);
          copy_async<Ahead<T, RUN, U>::kBytes>(part[0][1].b[threadIdx.x], x + u * G * D + l.c1);
          copy_async<Ahead<T, RUN, U>::kBytes>(part[1][0].b[threadIdx.x], dy + u * G * D + l.c0);
          copy_async<Ahead<T, RUN, U>::kBytes>(part[1][1].b[threadIdx.x], dy + u * G * D + l.c1);
        }
      }
    }
    copy_commit();
  };
  fetch(0);
  while (it.m < p.d.M) {
    const int64_t m = it.m, h0 = (int64_t)it.run * HI + grp;
    at = nat;
    it.next();
    fetch(buf ^ 1);
    const int64_t pos = checked(p, at);  // one token to a warp
    const Turn<RUN, NEAR, true> a(p, l, pos);
    copy_wait<1>();  // this item is here, the next one on its way
    T *dx = sd.y + (m * sd.heads + h0) * D;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f2 v[RUN], g[RUN], ss = f2_both(0.f), px = ss;
      const bool on = l.on && h0 + u * G < sd.heads;
      const auto &part = ahead.part[buf][u];
      get_two(part[0][0].b[threadIdx.x], part[0][1].b[threadIdx.x], on, v);
      get_two(part[1][0].b[threadIdx.x], part[1][1].b[threadIdx.x], on, g);
      if (pos >= 0) a.apply(g, l);
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        ss = f2_fma(v[i], v[i], ss);
        px = f2_fma(f2_mul(w[i], g[i]), v[i], px);
      }
      const float r = rsqrtf(row_sum<TPR>(ss) / (float)D + p.d.eps);
      const f2 rho = f2_both(r), mean = f2_both(-(row_sum<TPR>(px) / (float)D * r * r));
      if (on) {
        f2 o[RUN];
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
          o[i] = pos < 0 ? f2_both(0.f) : f2_mul(rho, f2_fma(v[i], mean, f2_mul(w[i], g[i])));
          if (pos >= 0) sum[i] = f2_fma(g[i], f2_mul(v[i], rho), sum[i]);
        }
        store_two(dx + u * G * D, l.c0, l.c1, o);
      }
    }
    buf ^= 1;
  }
  copy_wait<0>();
  __syncthreads();  // the copies' memory holds the sums from here on
  if (l.on) {
#pragma unroll
    for (int i = 0; i < RUN / 2; ++i) {
      float *const to = red[warp * G + grp];
      f2_split(sum[i], to[l.c0 + 2 * i], to[l.c0 + 2 * i + 1]);
      f2_split(sum[RUN / 2 + i], to[l.c1 + 2 * i], to[l.c1 + 2 * i + 1]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float s = 0.f;
#pragma unroll 4
    for (int j = 0; j < kWarps * G; ++j) s += red[j][i];
    p.part[(int64_t)blockIdx.x * D + i] = s;
  }
}

// Odd widths, pairs that no run divides, or bases off the vectors' alignment: a warp to
// a row, a lane to every 32nd pair (or channel past the pairs).
constexpr int kMostUnits = 8;  // units of a lane: D <= 256
__device__ __forceinline__ void unit_of(const HeadArgs &p, int u, int &ca, int &cb) {  // cb < 0: one channel
  const int R = (int)p.d.R;
  ca = u >= R ? u + R : p.d.interleaved ? 2 * u : u;
  cb = u >= R ? -1 : p.d.interleaved ? 2 * u + 1 : u + R;
}
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) head_odd_kernel(const __grid_constant__ HeadArgs p) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float red[BWD ? kWarps : 1][256];
  const bool query = blockIdx.x < p.bq;
  const Side<T> sd = side_of<T>(p, query);
  const int64_t block = query ? blockIdx.x : blockIdx.x - p.bq, blocks = query ? p.bq : gridDim.x - p.bq;
  const int D = (int)p.d.D, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units = D - (int)p.d.R;
  const int64_t rows = p.d.M * sd.heads;
  const bool f32 = p.d.weight_dtype == GDR_F32;
  float sums[2][BWD ? kMostUnits : 1] = {};
  for (int64_t row = block * kWarps + warp; row < rows; row += blocks * kWarps) {
    const int64_t m = row / sd.heads, h = row - m * sd.heads;
    const T *x = sd.x + m * sd.ld + h * D, *dy = sd.dy + (BWD ? m * sd.ld_dy + h * D : 0);
    T *y = sd.y + row * D;
    const int64_t pos = checked(p, load_position(p, m));
    float va[kMostUnits], vb[kMostUnits], ga[kMostUnits], gb[kMostUnits], ss = 0.f, px = 0.f;
#pragma unroll
    for (int i = 0; i < kMostUnits; ++i) {
      const int u = lane + 32 * i;
      va[i] = vb[i] = ga[i] = gb[i] = 0.f;
      if (u >= units) continue;
      int ca, cb;
      unit_of(p, u, ca, cb);
      va[i] = to_f32(x[ca]);
      if (cb >= 0) vb[i] = to_f32(x[cb]);
      ss = fmaf(va[i], va[i], fmaf(vb[i], vb[i], ss));
      if constexpr (BWD) {
        ga[i] = to_f32(dy[ca]);
        if (cb >= 0 && pos >= 0) {
          gb[i] = to_f32(dy[cb]);
          const float c = p.cos[pos * p.d.R + u], s = p.sin[pos * p.d.R + u], g0 = ga[i], g1 = gb[i];
          ga[i] = fmaf(g0, c, g1 * s);
          gb[i] = fmaf(g1, c, -(g0 * s));
        }
        px = fmaf(param<T>(sd.w, f32, ca) * ga[i], va[i], px);
        if (cb >= 0) px = fmaf(param<T>(sd.w, f32, cb) * gb[i], vb[i], px);
      }
    }
    const float rho = rsqrtf(warp_sum(ss) / (float)D + p.d.eps);
    const float mean = BWD ? warp_sum(px) / (float)D * rho * rho : 0.f;
#pragma unroll
    for (int i = 0; i < kMostUnits; ++i) {
      const int u = lane + 32 * i;
      if (u >= units) continue;
      int ca, cb;
      unit_of(p, u, ca, cb);
      float a, b = 0.f;
      if constexpr (BWD) {
        a = rho * (param<T>(sd.w, f32, ca) * ga[i] - va[i] * mean);
        if (cb >= 0) b = rho * (param<T>(sd.w, f32, cb) * gb[i] - vb[i] * mean);
        if (pos >= 0) {
          sums[0][i] += ga[i] * (va[i] * rho);
          sums[1][i] += gb[i] * (vb[i] * rho);
        }
      } else {
        a = va[i] * rho * param<T>(sd.w, f32, ca);
        if (cb >= 0 && pos >= 0) {
          b = vb[i] * rho * param<T>(sd.w, f32, cb);
          const float c = p.cos[pos * p.d.R + u], s = p.sin[pos * p.d.R + u], n0 = a, n1 = b;
          a = fmaf(n0, c, -(n1 * s));
          b = fmaf(n1, c, n0 * s);
        }
      }
      y[ca] = from_f32<T>(pos < 0 ? 0.f : a);
      if (cb >= 0) y[cb] = from_f32<T>(pos < 0 ? 0.f : b);
    }
  }
  if constexpr (BWD) {
#pragma unroll
    for (int i = 0; i < kMostUnits; ++i) {
      const int u = lane + 32 * i;
      if (u >= units) continue;
      int ca, cb;
      unit_of(p, u, ca, cb);
      red[warp][ca] = sums[0][i];
      if (cb >= 0) red[warp][cb] = sums[1][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
      float s = 0.f;
      for (int j = 0; j < kWarps; ++j) s += red[j][i];
      p.part[(int64_t)blockIdx.x * D + i] = s;
    }
  }
}

// dw of q and of k from the blocks' sums.
__global__ void __launch_bounds__(1024) head_sum_kernel(ColSum q, ColSum k) {
  __shared__ float sm[32][33];
  col_sum_block<32>(blockIdx.y ? k : q, blockIdx.x, sm);
}

// Whether every row can be read in runs of `run` elements.
bool runs_ok(const HeadArgs &a, int run, bool bwd) {
  const gdr_qk_norm_desc &d = a.d;
  const uintptr_t bytes = (d.dtype == GDR_BF16 ? 2 : 4) * run, wb = d.weight_dtype == GDR_F32 ? 16 : bytes;
  const auto on = [&](const void *p, int64_t ld, uintptr_t n) { return (uintptr_t)p % n == 0 && ld % run == 0; };
  bool ok = d.D % (2 * run) == 0 && d.R % run == 0 && on(a.q, d.ld_q, bytes) && on(a.k, d.ld_k, bytes) &&
            on(a.wq, 0, wb) && on(a.wk, 0, wb) && on(a.yq, 0, bytes) && on(a.yk, 0, bytes) && on(a.cos, 0, 8) &&
            on(a.sin, 0, 8);
  if (bwd) ok = ok && on(a.dyq, d.ld_dyq, bytes) && on(a.dyk, d.ld_dyk, bytes);
  return ok;
}

// A launch's blocks: as many as its items fill, at most `most`; those of q and of k go by their items.
struct Blocks {
  int64_t q, all;
};
Blocks blocks_of(const gdr_qk_norm_desc &d, int heads_per_item, int64_t most) {
  constexpr int kWarps = kThreads / 32;
  const int64_t q = cdiv(d.M * cdiv(d.H, heads_per_item), kWarps), k = cdiv(d.M * cdiv(d.HK, heads_per_item), kWarps);
  if (q + k <= most) return {q, q + k};
  const int64_t bk = d.HK ? std::max<int64_t>(1, most * k / (q + k)) : 0;
  return {most - bk, most};
}

template <typename T, int RUN, int TPR, int U>
int launch_vec(const HeadArgs &a, bool bwd, int64_t blocks, cudaStream_t st) {
  const bool near = a.d.interleaved;
  if (bwd) {
    const auto kernel = near ? head_bwd_kernel<T, RUN, TPR, U, true> : head_bwd_kernel<T, RUN, TPR, U, false>;
    constexpr size_t smem = bwd_smem<T, RUN, TPR, U>();
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(head_bwd_kernel)");
    kernel<<<(unsigned)blocks, kThreads, smem, st>>>(a);
    return launched("head_bwd_kernel");
  }
  const auto kernel = near ? head_fwd_kernel<T, RUN, TPR, U, true> : head_fwd_kernel<T, RUN, TPR, U, false>;
  kernel<<<(unsigned)blocks, kThreads, 0, st>>>(a);
  return launched("head_fwd_kernel");
}

// Rows of a thread (U), while as many of the next item are on their way.
constexpr int kRowsFwd = 2, kRowsBwd = 2;
template <typename T, int RUN>
int launch_runs(const HeadArgs &a, bool bwd, int tpr, int64_t blocks, cudaStream_t st) {
  const auto go = [&](auto t) {
    constexpr int TPR = decltype(t)::value;
    return bwd ? launch_vec<T, RUN, TPR, kRowsBwd>(a, bwd, blocks, st)
               : launch_vec<T, RUN, TPR, kRowsFwd>(a, bwd, blocks, st);
  };
  if (tpr == 4) return go(std::integral_constant<int, 4>{});
  if (tpr == 8) return go(std::integral_constant<int, 8>{});
  if constexpr (RUN == 8) return go(std::integral_constant<int, 16>{});  // D <= 256
  if (tpr == 16) return go(std::integral_constant<int, 16>{});
  return go(std::integral_constant<int, 32>{});
}

template <typename T>
int launch(HeadArgs a, bool bwd, float *dwq, float *dwk, cudaStream_t st) {
  const gdr_qk_norm_desc &d = a.d;
  constexpr int kWide = sizeof(T) == 2 ? 8 : 4;
  const int run = runs_ok(a, kWide, bwd) ? kWide : runs_ok(a, 4, bwd) ? 4 : 1;
  int tpr = run > 1 ? 4 : 32;
  while (2 * run * tpr < d.D && run > 1) tpr *= 2;
  // blocks stay, two to a multiprocessor (four of the warp-to-a-row form)
  const Blocks n = blocks_of(d, run > 1 ? 32 / tpr * (bwd ? kRowsBwd : kRowsFwd) : 1, (run > 1 ? 2 : 4) * kSMs);
  if (n.all > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many rows for one launch");
  a.bq = n.q;
  char *base = nullptr;
  int rc = GDR_OK;
  if (bwd) {
    rc = scratch_begin(sizeof(float) * (size_t)(std::max<int64_t>(1, n.all) * d.D), st, "head norm scratch", &base);
    if (rc != GDR_OK) return rc;
    a.part = (float *)base;
  }
  if (n.all > 0) {
    if (run == 1) {
      if (bwd) head_odd_kernel<T, true><<<(unsigned)n.all, kThreads, 0, st>>>(a);
      else head_odd_kernel<T, false><<<(unsigned)n.all, kThreads, 0, st>>>(a);
      rc = launched("head_odd_kernel");
    } else if (run == 8) {
      if constexpr (sizeof(T) == 2) rc = launch_runs<T, 8>(a, bwd, tpr, n.all, st);
    } else {
      rc = launch_runs<T, 4>(a, bwd, tpr, n.all, st);
    }
  }
  if (!bwd) return rc;
  if (rc == GDR_OK) {
    const auto sum = [&](int64_t first, int64_t rows, float *out) {
      return ColSum{a.part + first * d.D, rows, d.D, d.D, d.D, d.D, out, d.D, nullptr};
    };
    head_sum_kernel<<<dim3((unsigned)cdiv(d.D, 32), dwk ? 2 : 1), 1024, 0, st>>>(sum(0, n.q, dwq),
                                                                                sum(n.q, n.all - n.q, dwk));
    rc = launched("head_sum_kernel");
  }
  return scratch_end(base, st, "head norm scratch", rc);
}

int validate(const gdr_qk_norm_desc *d) {
  if (!d) return set_error(GDR_ERR_NULLPTR, "desc is NULL");
  if (d->dtype != GDR_F32 && d->dtype != GDR_BF16) return set_error(GDR_ERR_DTYPE, "dtype must be GDR_F32 or GDR_BF16");
  if (d->weight_dtype != d->dtype && d->weight_dtype != GDR_F32)
    return set_error(GDR_ERR_DTYPE, "weight_dtype must be dtype or GDR_F32");
  if (d->flags) return set_error(GDR_ERR_DTYPE, "unknown bits in flags");
  if (d->interleaved != 0 && d->interleaved != 1) return set_error(GDR_ERR_DTYPE, "interleaved must be 0 or 1");
  constexpr int64_t kMost = 0x7fffffff;
  if (d->M < 0 || d->M > kMost) return set_error(GDR_ERR_SHAPE, "M must be in [0, 2^31)");
  if (d->H < 1 || d->HK < 0 || d->H > 65535 || d->HK > 65535)
    return set_error(GDR_ERR_SHAPE, "H must be in [1, 65535] and HK in [0, 65535]");
  if (d->D < 1 || d->D > 256) return set_error(GDR_ERR_SHAPE, "D must be in [1, 256]");
  if (d->R < 0 || 2 * d->R > d->D)
    return set_error(GDR_ERR_SHAPE, "the rotation must not be wider than a head: 2 R <= D");
  if (d->P < 0 || d->P > kMost) return set_error(GDR_ERR_SHAPE, "P must be in [0, 2^31)");
  if (d->ld_q < d->H * d->D || d->ld_k < d->HK * d->D || d->ld_dyq < d->H * d->D || d->ld_dyk < d->HK * d->D)
    return set_error(GDR_ERR_SHAPE, "leading dimensions must be at least H * D, or HK * D");
  if (d->ld_q > kMost || d->ld_k > kMost || d->ld_dyq > kMost || d->ld_dyk > kMost)
    return set_error(GDR_ERR_SHAPE, "leading dimensions must be below 2^31");
  if (!(d->eps >= 0.f)) return set_error(GDR_ERR_SHAPE, "eps must be >= 0");
  return GDR_OK;
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

int gdr_qk_norm_fwd(const gdr_qk_norm_desc *desc, const void *q, const void *k, const void *wq, const void *wk,
                    const float *cos, const float *sin, const int64_t *positions, void *yq, void *yk, void *stream) {
  int rc = validate(desc);
  if (rc != GDR_OK) return rc;
  if (desc->M == 0) return GDR_OK;
  if (!q || !wq || !yq || (desc->HK > 0 && (!k || !wk || !yk)))
    return set_error(GDR_ERR_NULLPTR, "q, k, wq, wk, yq and yk must be non-NULL");
  if (desc->R > 0 && (!cos || !sin || !positions))
    return set_error(GDR_ERR_NULLPTR, "a rotation needs cos, sin and positions");
  if (desc->R > 0 && desc->P == 0) return set_error(GDR_ERR_SHAPE, "the rotation's table has no positions");
  HeadArgs a{};
  a.d = *desc;
  a.q = q; a.k = k; a.wq = wq; a.wk = wk; a.cos = cos; a.sin = sin; a.pos = positions; a.yq = yq; a.yk = yk;
  a.status = current_status_word(&rc);
  if (!a.status) return rc;
  return desc->dtype == GDR_BF16 ? launch<__nv_bfloat16>(a, false, nullptr, nullptr, (cudaStream_t)stream)
                                 : launch<float>(a, false, nullptr, nullptr, (cudaStream_t)stream);
}

int gdr_qk_norm_bwd(const gdr_qk_norm_desc *desc, const void *dyq, const void *dyk, const void *q, const void *k,
                    const void *wq, const void *wk, const float *cos, const float *sin, const int64_t *positions,
                    void *dq, void *dk, float *dwq, float *dwk, void *stream) {
  int rc = validate(desc);
  if (rc != GDR_OK) return rc;
  if (!wq || !dwq || (desc->HK > 0 && (!wk || !dwk)))
    return set_error(GDR_ERR_NULLPTR, "wq, wk, dwq and dwk must be non-NULL");
  if (desc->M > 0 && (!dyq || !q || !dq || (desc->HK > 0 && (!dyk || !k || !dk))))
    return set_error(GDR_ERR_NULLPTR, "dyq, dyk, q, k, dq and dk must be non-NULL");
  if (desc->M > 0 && desc->R > 0 && (!cos || !sin || !positions))
    return set_error(GDR_ERR_NULLPTR, "a rotation needs cos, sin and positions");
  if (desc->M > 0 && desc->R > 0 && desc->P == 0) return set_error(GDR_ERR_SHAPE, "the rotation's table has no positions");
  HeadArgs a{};
  a.d = *desc;
  a.q = q; a.k = k; a.wq = wq; a.wk = wk; a.dyq = dyq; a.dyk = dyk; a.cos = cos; a.sin = sin; a.pos = positions;
  a.yq = dq; a.yk = dk;
  a.status = current_status_word(&rc);
  if (!a.status) return rc;
  return desc->dtype == GDR_BF16 ? launch<__nv_bfloat16>(a, true, dwq, dwk, (cudaStream_t)stream)
                                 : launch<float>(a, true, dwq, dwk, (cudaStream_t)stream);
}

}  // extern "C"
