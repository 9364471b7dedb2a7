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

#include "gdr_layer.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;

struct HeadArgs {
  gdr_qk_norm_desc d;
  const void *q, *k, *wq, *wk, *dyq, *dyk;
  const float *cos, *sin;
  const int64_t *pos;
  void *yq, *yk;   // backward: dq, dk
  float *part;     // backward: [blocks, 2, D] sums of dw
  int *status;
  int64_t cq, ck;  // runs of heads of a token: of queries, of keys
};

// Eight channels of a thread, as two runs of four: the a and the b of four pairs
// where halves are paired, neighbours otherwise; and the pairs' first index.
// Thread t of a row; R % 4 == 0, D % 8 == 0.
__device__ __forceinline__ void channels_of(const HeadArgs &p, int t, int &c0, int &c1, bool &turned) {
  const int R = (int)p.d.R;
  turned = 4 * t < R;
  if (turned && !p.d.interleaved) {
    c0 = 4 * t;
    c1 = R + 4 * t;
  } else {
    c0 = 8 * t;
    c1 = c0 + 4;
  }
}

// The four cosines and sines of a thread's pairs.  `sign` -1 turns back.
struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ Turn turn_of(const HeadArgs &p, int64_t pos, int t, bool turned, float sign) {
  Turn u;
  if (turned) {
    load4(p.cos + pos * p.d.R + 4 * t, u.c);
    load4(p.sin + pos * p.d.R + 4 * t, u.s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u.c[i] = turned ? u.c[i] : 1.f;
    u.s[i] = turned ? u.s[i] * sign : 0.f;
  }
  return u;
}
// v[0..3] and v[4..7] are the two runs.
__device__ __forceinline__ void turn(float (&v)[8], const Turn &u, bool turned, bool interleaved) {
  if (!turned) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float &a = interleaved ? v[2 * i] : v[i], &b = interleaved ? v[2 * i + 1] : v[i + 4];
    const float x = a, y = b;
    a = fmaf(x, u.c[i], -(y * u.s[i]));
    b = fmaf(y, u.c[i], x * u.s[i]);
  }
}

template <int TPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ void load_weight(const void *w, bool f32, int c0, int c1, float (&v)[8]) {
  float a[4], b[4];
  if (f32) {
    load4(static_cast<const float *>(w) + c0, a);
    load4(static_cast<const float *>(w) + c1, b);
  } else {
    load4(static_cast<const T *>(w) + c0, a);
    load4(static_cast<const T *>(w) + c1, b);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
template <typename T>
__device__ __forceinline__ void load_two(const T *p, int c0, int c1, float (&v)[8]) {
  float a[4], b[4];
  load4(p + c0, a);
  load4(p + c1, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
template <typename T>
__device__ __forceinline__ void store_two(T *p, int c0, int c1, const float (&v)[8]) {
  const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
  store4(p + c0, a);
  store4(p + c1, b);
}

// The rows of one run of up to U heads of a token.
struct Run {
  int64_t m, h0;  // token, first head of the run
  int heads;
  bool query;
};
template <int U>
__device__ __forceinline__ Run run_of(const HeadArgs &p, int64_t item) {
  Run r;
  r.m = item / (p.cq + p.ck);
  int64_t c = item - r.m * (p.cq + p.ck);
  r.query = c < p.cq;
  if (!r.query) c -= p.cq;
  r.h0 = c * U;
  r.heads = (int)min((int64_t)U, (r.query ? p.d.H : p.d.HK) - r.h0);
  return r;
}

// A token's position: -1 (or one past the table, which is reported) makes a padding row of zeros.
__device__ __forceinline__ int64_t position_of(const HeadArgs &p, int64_t m) {
  if (!p.d.R) return 0;
  const int64_t pos = p.pos[m];
  if (pos < p.d.P) return pos < 0 ? -1 : pos;
  raise_status(p.status, GDR_ERR_POSITION);
  return -1;
}

// TPR threads to a row (a power of two, at least D / 8 and 4), U heads of a token to
// each such group, all of whose rows are asked for before the first is used.
template <typename T, int TPR, int U>
__global__ void __launch_bounds__(kThreads) head_fwd_kernel(const __grid_constant__ HeadArgs p) {
  const int D = (int)p.d.D, t = threadIdx.x % TPR;
  const int64_t items = p.d.M * (p.cq + p.ck);
  const int64_t item = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  const Run r = run_of<U>(p, item < items ? item : items - 1);  // the last warp's spare groups: a copy of the last run
  const bool on = 8 * t < D;
  int c0, c1;
  bool turned;
  channels_of(p, t, c0, c1, turned);
  const int64_t ld = r.query ? p.d.ld_q : p.d.ld_k, heads = r.query ? p.d.H : p.d.HK;
  const T *x = static_cast<const T *>(r.query ? p.q : p.k) + r.m * ld + r.h0 * D;
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (on && u < r.heads) load_two(x + u * D, c0, c1, v[u]);
    else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
    }
  }
  const int64_t pos = position_of(p, r.m);
  const Turn a = turn_of(p, max(pos, (int64_t)0), t, turned && on && pos >= 0, 1.f);
  float w[8];
  if (on) load_weight<T>(r.query ? p.wq : p.wk, p.d.weight_dtype == GDR_F32, c0, c1, w);
  T *y = static_cast<T *>(r.query ? p.yq : p.yk) + (r.m * heads + r.h0) * D;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[u][i], v[u][i], ss);
    const float rho = rsqrtf(row_sum<TPR>(ss) / (float)D + p.d.eps);
    if (on && u < r.heads && item < items) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = pos < 0 ? 0.f : v[u][i] * rho * w[i];
      turn(v[u], a, turned, p.d.interleaved);
      store_two(y + u * D, c0, c1, v[u]);
    }
  }
}

// Blocks go through the runs; a thread sums its channels' dw of queries and of keys
// over its runs, the block's groups meet in shared memory, the blocks in a second launch.
template <typename T, int TPR, int U>
__global__ void __launch_bounds__(kThreads) head_bwd_kernel(const __grid_constant__ HeadArgs p) {
  __shared__ float red[kThreads / TPR][2][TPR * 8 + 1];
  const int D = (int)p.d.D, t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int64_t items = p.d.M * (p.cq + p.ck), step = (int64_t)gridDim.x * (kThreads / TPR);
  const bool on = 8 * t < D, f32 = p.d.weight_dtype == GDR_F32;
  int c0, c1;
  bool turned;
  channels_of(p, t, c0, c1, turned);
  float sq[8] = {}, sk[8] = {};
  for (int64_t first = (int64_t)blockIdx.x * (kThreads / TPR); first < items; first += step) {  // all threads stay for the shuffles
    const int64_t item = first + grp;
    const bool real = item < items;
    const Run r = run_of<U>(p, real ? item : items - 1);
    const int64_t ld = r.query ? p.d.ld_q : p.d.ld_k, ldy = r.query ? p.d.ld_dyq : p.d.ld_dyk,
                  heads = r.query ? p.d.H : p.d.HK;
    const T *x = static_cast<const T *>(r.query ? p.q : p.k) + r.m * ld + r.h0 * D;
    const T *dy = static_cast<const T *>(r.query ? p.dyq : p.dyk) + r.m * ldy + r.h0 * D;
    float v[U][8], g[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (on && u < r.heads) {
        load_two(x + u * D, c0, c1, v[u]);
        load_two(dy + u * D, c0, c1, g[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = g[u][i] = 0.f;
      }
    }
    const int64_t pos = position_of(p, r.m);
    const Turn a = turn_of(p, max(pos, (int64_t)0), t, turned && on && pos >= 0, -1.f);
    float w[8];
    if (on) load_weight<T>(r.query ? p.wq : p.wk, f32, c0, c1, w);
    else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0.f;
    }
    T *dx = static_cast<T *>(r.query ? p.yq : p.yk) + (r.m * heads + r.h0) * D;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      turn(g[u], a, turned, p.d.interleaved);
      float ss = 0.f, px = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(v[u][i], v[u][i], ss);
        px = fmaf(w[i] * g[u][i], v[u][i], px);
      }
      ss = row_sum<TPR>(ss) / (float)D + p.d.eps;
      const float rho = rsqrtf(ss), m = row_sum<TPR>(px) / (float)D * rho * rho;
      if (on && u < r.heads && real) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = pos < 0 ? 0.f : rho * (w[i] * g[u][i] - v[u][i] * m);
        store_two(dx + u * D, c0, c1, o);
        if (pos >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float dw = g[u][i] * (v[u][i] * rho);
            if (r.query) sq[i] += dw;
            else sk[i] += dw;
          }
        }
      }
    }
  }
  if (on) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i < 4 ? c0 + i : c1 + i - 4;
      red[grp][0][c] = sq[i];
      red[grp][1][c] = sk[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float s = 0.f;
#pragma unroll 4
    for (int j = 0; j < kThreads / TPR; ++j) s += red[j][i / D][i % D];
    p.part[(int64_t)blockIdx.x * 2 * D + i] = s;
  }
}

// Odd widths, pairs that four do not divide, or bases off the vectors' alignment: a
// warp to a row, a lane to every 32nd pair (or channel past the pairs).
constexpr int kMostUnits = 8;  // units of a lane: D <= 256
__device__ __forceinline__ void unit_of(const HeadArgs &p, int u, int &ca, int &cb) {  // cb < 0: one channel
  const int R = (int)p.d.R;
  ca = u >= R ? u + R : p.d.interleaved ? 2 * u : u;
  cb = u >= R ? -1 : p.d.interleaved ? 2 * u + 1 : u + R;
}
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) head_odd_kernel(const __grid_constant__ HeadArgs p) {
  __shared__ float red[BWD ? kThreads / 32 : 1][2][256];
  const int D = (int)p.d.D, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units = D - (int)p.d.R;
  const int64_t rows = p.d.M * (p.d.H + p.d.HK);
  const bool f32 = p.d.weight_dtype == GDR_F32;
  float sums[2][2][BWD ? kMostUnits : 1] = {};
  for (int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + warp; row < rows; row += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t m = row / (p.d.H + p.d.HK);
    int64_t h = row - m * (p.d.H + p.d.HK);
    const bool query = h < p.d.H;
    if (!query) h -= p.d.H;
    const T *x = static_cast<const T *>(query ? p.q : p.k) + m * (query ? p.d.ld_q : p.d.ld_k) + h * D;
    const T *dy = BWD ? static_cast<const T *>(query ? p.dyq : p.dyk) + m * (query ? p.d.ld_dyq : p.d.ld_dyk) + h * D : x;
    const void *w = query ? p.wq : p.wk;
    T *y = static_cast<T *>(query ? p.yq : p.yk) + (m * (query ? p.d.H : p.d.HK) + h) * D;
    const int64_t pos = position_of(p, m);
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
        px = fmaf(param<T>(w, f32, ca) * ga[i], va[i], px);
        if (cb >= 0) px = fmaf(param<T>(w, f32, cb) * gb[i], vb[i], px);
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
        a = rho * (param<T>(w, f32, ca) * ga[i] - va[i] * mean);
        if (cb >= 0) b = rho * (param<T>(w, f32, cb) * gb[i] - vb[i] * mean);
        if (pos >= 0) {
          if (query) {
            sums[0][0][i] += ga[i] * (va[i] * rho);
            sums[0][1][i] += gb[i] * (vb[i] * rho);
          } else {
            sums[1][0][i] += ga[i] * (va[i] * rho);
            sums[1][1][i] += gb[i] * (vb[i] * rho);
          }
        }
      } else {
        a = va[i] * rho * param<T>(w, f32, ca);
        if (cb >= 0 && pos >= 0) {
          b = vb[i] * rho * param<T>(w, f32, cb);
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
      for (int z = 0; z < 2; ++z) {
        red[warp][z][ca] = sums[z][0][i];
        if (cb >= 0) red[warp][z][cb] = sums[z][1][i];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      float s = 0.f;
      for (int j = 0; j < kThreads / 32; ++j) s += red[j][i / D][i % D];
      p.part[(int64_t)blockIdx.x * 2 * D + i] = s;
    }
  }
}

__global__ void __launch_bounds__(1024) head_sum_kernel(ColSum q) {
  __shared__ float sm[32][33];
  col_sum_block<32>(q, blockIdx.x, sm);
}

bool vec_ok(const HeadArgs &a, bool bwd) {
  const gdr_qk_norm_desc &d = a.d;
  const uintptr_t bytes = d.dtype == GDR_BF16 ? 8 : 16;  // of four elements
  const auto on = [&](const void *p, int64_t ld, uintptr_t n) { return (uintptr_t)p % n == 0 && ld % 4 == 0; };
  const uintptr_t wb = d.weight_dtype == GDR_F32 ? 16 : bytes;
  bool ok = d.D % 8 == 0 && d.R % 4 == 0 && on(a.q, d.ld_q, bytes) && on(a.k, d.ld_k, bytes) && on(a.wq, 0, wb) &&
            on(a.wk, 0, wb) && on(a.yq, 0, bytes) && on(a.yk, 0, bytes) && on(a.cos, 0, 16) && on(a.sin, 0, 16);
  if (bwd) ok = ok && on(a.dyq, d.ld_dyq, bytes) && on(a.dyk, d.ld_dyk, bytes);
  return ok;
}

constexpr int kHeads = 4;     // heads of a run
constexpr int kWaveBlocks = 4 * kSMs;  // blocks of the backward's grid

template <typename T, int TPR>
int launch_vec(const HeadArgs &a, bool bwd, int64_t blocks, cudaStream_t st) {
  if (bwd) head_bwd_kernel<T, TPR, kHeads><<<(unsigned)blocks, kThreads, 0, st>>>(a);
  else head_fwd_kernel<T, TPR, kHeads><<<(unsigned)blocks, kThreads, 0, st>>>(a);
  return launched(bwd ? "head_bwd_kernel" : "head_fwd_kernel");
}

template <typename T>
int launch(HeadArgs a, bool bwd, float *dwq, float *dwk, cudaStream_t st) {
  const gdr_qk_norm_desc &d = a.d;
  const bool vec = vec_ok(a, bwd);
  int tpr = 4;
  while (8 * tpr < d.D) tpr *= 2;
  if (!vec) tpr = 32;
  a.cq = vec ? cdiv(d.H, kHeads) : d.H;
  a.ck = vec ? cdiv(d.HK, kHeads) : d.HK;
  int64_t blocks = cdiv(d.M * (a.cq + a.ck), kThreads / tpr);
  if (bwd || !vec) blocks = std::min<int64_t>(blocks, kWaveBlocks);
  if (blocks > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many rows for one launch");
  char *base = nullptr;
  int rc;
  if (bwd) {
    rc = scratch_begin(sizeof(float) * (size_t)(std::max<int64_t>(1, blocks) * 2 * d.D), st, "head norm scratch", &base);
    if (rc != GDR_OK) return rc;
    a.part = (float *)base;
  }
  rc = GDR_OK;
  if (blocks > 0) {
    if (!vec) {
      if (bwd) head_odd_kernel<T, true><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      else head_odd_kernel<T, false><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      rc = launched("head_odd_kernel");
    } else if (tpr == 4) rc = launch_vec<T, 4>(a, bwd, blocks, st);
    else if (tpr == 8) rc = launch_vec<T, 8>(a, bwd, blocks, st);
    else if (tpr == 16) rc = launch_vec<T, 16>(a, bwd, blocks, st);
    else rc = launch_vec<T, 32>(a, bwd, blocks, st);
  }
  if (!bwd) return rc;
  if (rc == GDR_OK) {
    const ColSum s{a.part, blocks, 2 * d.D, 2 * d.D, 2 * d.D, 2 * d.D, dwq, d.D, dwk};
    head_sum_kernel<<<(unsigned)cdiv(2 * d.D, 32), 1024, 0, st>>>(s);
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
  if (d->R < 0 || 2 * d->R > d->D) return set_error(GDR_ERR_SHAPE, "the rotation must not be wider than a head: 2 R <= D");
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
